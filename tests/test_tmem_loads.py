"""A value that tcgen05.ld loads may be used only after the wait for it, which the
compiler does not know: in the sources every load has its wait in the same statement."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_224_gb300", "csrc")


def test_every_tensor_memory_load_and_its_wait_are_one_statement():
    loads = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//.*", "", open(path).read())
        for m in re.finditer(r"asm volatile\((.*?)\);", text, re.S):
            body = m.group(1)
            if "tcgen05.ld" in body or "wait::ld" in body:
                loads += 1
                assert "tcgen05.ld" in body and body.rindex("tcgen05.wait::ld") > body.rindex("tcgen05.ld"), (path, body[:80])
    assert loads >= 4
