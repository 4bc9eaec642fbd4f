"""The order of steps that chained launches rely on, read from the kernels'
sources: a wrong one shows on a device only as a hang, and only beside other
kernels."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemm_w4_b200", "csrc")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        for part in text.split("__global__")[1:]:
            body = part[:part.index("\n}\n")]
            yield os.path.basename(path), re.search(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\([^)]*\)", "", body)).group(1), body


@pytest.mark.parametrize("file,name,body", [k for k in kernels() if re.search(r"\balloc<|tmem_alloc\(", k[2])],
                         ids=lambda v: v if len(v) < 40 else "")
def test_tensor_memory_comes_before_the_next_launch(file, name, body):
    # A launch that starts early may take all of an SM's tensor memory and
    # then wait for this one: each CTA has to hold its own by then.
    if "pdl_launch_dependents" not in body:
        return
    assert re.search(r"\balloc<|tmem_alloc\(", body).start() < body.index("pdl_launch_dependents"), (file, name)


def test_kernels_with_tensor_memory_are_found():
    names = {name for _, name, body in kernels() if re.search(r"\balloc<|tmem_alloc\(", body)}
    assert {"fp4_narrow_kernel", "fp4_wide_kernel", "prefill_kernel"} <= names
