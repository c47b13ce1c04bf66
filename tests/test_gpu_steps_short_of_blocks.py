"""Steps over a block-scaled cache in which some sequences are not served: nothing of theirs changes."""
import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from oracle import block_scaled as S
from tests import block_scaled_helpers as K
from tests import sparse_helpers as H
from tests.test_gpu_block_scaled import BF, Server, i32

pytestmark = pytest.mark.gpu


def host(s):
    return [[x.cpu().clone() for x in c] for c in s.caches], s.table.cpu(), s.lens.cpu()


def same_tokens(before, after, table, b, n, bs):
    """Codes of sequence b's n tokens and the scales of their blocks, bit for bit."""
    for t in range(n):
        i = int(table[b, t // bs])
        for x, y in zip(before, after):
            if x.dim() == 4:
                assert torch.equal(x[i, :, t % bs], y[i, :, t % bs]), (b, t)
            else:
                assert torch.equal(x[i].view(torch.int32), y[i].view(torch.int32)), (b, t)


@pytest.mark.parametrize("captured", [False, True])
def test_one_token_each_until_the_blocks_run_out(captured):
    g, B, hq, hkv, d, bs = H.gen(31), 7, 8, 2, 128, 16
    s = Server(B, 11, hkv, d, bs, 8, layers=1)  # 11 blocks: 7 for the prompts, 4 to grow into
    x = s.buffers(100, hq)
    x["new"].copy_(i32([16, 15, 9, 16, 16, 14, 14]))
    x["key"].copy_(H.randn(g, *x["key"].shape, dtype=BF))
    s.step(x, 0.06, decode=False)
    y = s.buffers(B, hq)
    y["new"].copy_(i32([1, 1, 0, 1, 1, 1, 1]))  # sequence 2 asks for nothing
    if captured:
        keep = [t.clone() for t in (s.table, s.lens, s.free, s.count, *s.caches[0])]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step(y, 0.06, decode=False)
        torch.cuda.synchronize()
        for t, was in zip((s.table, s.lens, s.free, s.count, *s.caches[0]), keep):
            t.copy_(was)
    idle = 0
    for step in range(20):
        caches, _, lens = host(s)
        y["q"].copy_(H.randn(g, *y["q"].shape, dtype=BF))
        y["key"].copy_(H.randn(g, *y["key"].shape, dtype=BF) * 2.0 ** (step % 5))  # scales rise
        y["out"].fill_(9.0)
        graph.replay() if captured else s.step(y, 0.06, decode=False)
        after, table, now = host(s)
        starts, rows = y["starts"].cpu(), int(y["starts"][-1])
        served = (now - lens).tolist()
        assert served == (starts[1:] - starts[:-1]).tolist() and served[2] == 0
        idle += served.count(0) - 1
        ref = [t.clone() for t in caches[0]]
        S.append(y["key"].cpu(), y["key"].cpu(), *ref, table, now, starts)
        for a, b in zip(after[0], ref):
            assert torch.equal(a, b)
        for b, n in enumerate(served):
            if n == 0:
                same_tokens(caches[0], after[0], table, b, int(lens[b]), bs)
        out = y["out"].cpu()
        want, mag, size, least = S.attention(y["q"].cpu(), *after[0], table, now, 0.06, starts)
        K.assert_attention(out[:rows], want[:rows], mag[:rows], size[:rows], least[:rows], BF, f"step {step}")
        assert (out[rows:] == 9.0).all()
    assert idle > 10 and wllm.device_errors() == 0
