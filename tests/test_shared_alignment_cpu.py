"""A kernel that moves 16 bytes at once may do so in its dynamic shared memory, which is only as aligned as its declaration
says (the static objects in front of it may end anywhere): the declaration asks for 16 bytes, or the kernel rounds the
address up itself."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_eviction_decode_gb300", "csrc")
DECLARATION = re.compile(r"extern __shared__ (.*?)(\w+)\[\];")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = f.read()
        found = list(DECLARATION.finditer(text))
        for i, m in enumerate(found):
            ends = [text.find("__global__", m.end()), found[i + 1].start() if i + 1 < len(found) else -1]
            yield pytest.param(m.group(1), m.group(2), text[m.end():min([e for e in ends if e >= 0], default=len(text))],
                               id=f"{os.path.basename(path)}:{text.count(chr(10), 0, m.start()) + 1}")


@pytest.mark.parametrize("kind,name,body", list(kernels()))
def test_wide_accesses_have_their_alignment(kind, name, body):
    if not re.search(r"\b(u?int4|float4)\b", body):
        return
    rounded = re.search(rf"reinterpret_cast<uintptr_t>\({name}\) \+", body)
    stated = re.search(r"__align__\((\d+)\)", kind)
    assert rounded or (stated and int(stated.group(1)) >= 16), f"{kind}{name}: 16-byte accesses, alignment not stated"
