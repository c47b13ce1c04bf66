"""What is asked of a device once and kept is kept for each device by itself."""
import glob
import os
import re

from paged_kv_cache_185_gb300 import build


def sources():
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*"))):
        if path.endswith((".cu", ".cuh", ".h", ".cpp")):
            yield os.path.basename(path), re.sub(r"//.*", "", open(path).read())


def test_records_have_a_place_for_each_device():
    seen = 0
    for name, code in sources():
        for names in re.findall(r"static std::atomic<[\w ]+> ([^;]+);", code):
            for record in names.split(","):
                seen += 1
                assert re.fullmatch(r"\w+\[64\]", record.strip()), f"{name}: {record}"
    assert seen >= 6


def test_occupancy_is_asked_where_the_device_is_known():
    asking = {name for name, code in sources() if "cudaOccupancyMaxActiveBlocksPerMultiprocessor" in code}
    assert asking == {"launch.h", "decode_persistent.cuh"}
    for name, code in sources():
        if name in asking:
            before = code[:code.index("cudaOccupancyMaxActiveBlocksPerMultiprocessor")]
            assert "cudaGetDevice(&dev)" in before[-1800:]
