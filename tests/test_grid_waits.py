"""What came before a kernel on its stream is visible to it from griddepcontrol.wait
on: in the sources every kernel that may start early waits in all its threads, at
the top level of its body, before it lets the next one start."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_224_gb300", "csrc")


def test_every_wait_is_unconditional():
    waits = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        if path.endswith("pa_device.cuh"):
            continue
        for line in re.sub(r"//.*", "", open(path).read()).split("\n"):
            if "pdl_wait()" in line:
                waits += 1
                assert re.fullmatch(r"    pdl_wait\(\);\s*", line), (os.path.basename(path), line.strip())
    assert waits >= 8
