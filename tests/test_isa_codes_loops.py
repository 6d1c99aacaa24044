"""The step loops of the products of codes (gfx950 assembly from hipcc, no GPU
needed), kernel by kernel: how many there are, how many products a step has, and
that each waits for its ring only."""
import os
import re

import pytest

from tests import isa_check as ic
from tests.test_isa_products import kernel_bodies

pytestmark = pytest.mark.skipif(not os.path.exists(ic.HIPCC), reason="hipcc not installed")

# products of each step loop: of the large tiles one for 4, 3, 2 and 1 blocks of 32
# rows a wave; of the others one
LOOPS = {"codes_run_kernelILb1ELb0E": [32, 24, 16, 8], "codes_run_kernelILb0ELb1E": [32, 24, 16, 8],
         "codes_run_kernelILb0ELb0E": [32, 24, 16, 8], "CodesTileILi1ELi128ELi256E": [8],
         "CodesTileILi1ELi64ELi64E": [2], "CodesTileILi2ELi128ELi256E": [32],
         "CodesTileILi2ELi64ELi64E": [8]}


@pytest.fixture(scope="module")
def bodies(tmp_path_factory):
    out = tmp_path_factory.mktemp("isa") / "products_fp8.s"
    return kernel_bodies(ic.compile_asm("products_fp8.hip", str(out)))


@pytest.mark.parametrize("kernel", LOOPS)
def test_step_loops(bodies, kernel):
    (body,) = [b for name, b in bodies.items() if kernel in name]
    found = []
    for header, loop in ic.loops(body).items():
        ins = loop["instrs"]
        products = sum(i.startswith("v_mfma") for i in ins)
        if not products:
            continue
        assert any(i.startswith("buffer_load") and " lds" in i for i in ins), header
        waits = [i for i in ins if i.startswith("s_waitcnt") and "vmcnt" in i]
        assert waits and not any(re.search(r"vmcnt\(0\)", i) for i in waits), (header, waits)
        assert not any(i.startswith(("scratch_", "global_store", "flat_")) for i in ins), header
        found.append(products)
    assert sorted(found, reverse=True) == LOOPS[kernel]


def test_every_kernel_of_codes_is_listed(bodies):
    """Beside them only the kernel for few rows, which has no ring, multiplies."""
    for name, body in bodies.items():
        if any(i.strip().startswith("v_mfma") for i in body):
            assert sum(k in name for k in LOOPS) == (0 if "product_thin" in name else 1), name
