"""Compiled-code properties of the products of codes and of the kernels that move
and quantise rows (gfx950 assembly from hipcc, no GPU needed): no barrier in a
loop that part of a wave can keep running; k loops that wait on vector memory for
their rings only; no accumulators in scratch memory."""
import concurrent.futures
import os
import re

import pytest

from tests import isa_check as ic
from tests.test_isa_products import kernel_bodies, ring_loops

pytestmark = pytest.mark.skipif(not os.path.exists(ic.HIPCC), reason="hipcc not installed")

SOURCES = ["products_fp8.hip", "rows.hip", "quantize.hip"]


@pytest.fixture(scope="module")
def asms(tmp_path_factory):
    d = tmp_path_factory.mktemp("isa")
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(lambda s: ic.compile_asm(s, str(d / (s + ".s"))), SOURCES)))


@pytest.mark.parametrize("src", SOURCES)
def test_no_barrier_in_divergent_loop(asms, src):
    bodies = kernel_bodies(asms[src])
    assert bodies
    bad = {k[:90]: ic.barrier_loops_with_exec_exits(v) for k, v in bodies.items()}
    assert not {k: v for k, v in bad.items() if v}


def test_k_loops_wait_only_for_their_rings(asms):
    """A steady-state loop leaves later stages in flight: it never waits for all
    of its loads, but for the row scales that the large tiles fetch a step ahead
    and use at the step's start."""
    found = 0
    for name, body in kernel_bodies(asms["products_fp8.hip"]).items():
        for header, ins in ring_loops(body).items():
            waits = [i for i in ins if i.startswith("s_waitcnt") and "vmcnt" in i]
            found += 1
            assert waits, (name[:90], header)
            assert not any(re.search(r"vmcnt\(0\)", i) for i in waits), (name[:90], header, waits)
            assert not any(i.startswith(("scratch_", "global_store", "flat_")) for i in ins), \
                (name[:90], header)
    assert found >= 4 + 3 * 3  # codes_kernel: two shapes, two kinds; codes_run_kernel


@pytest.mark.parametrize("src", SOURCES)
def test_accumulators_stay_in_registers(asms, src):
    """No vector register is spilled; of the large tiles' gathered form a few are,
    once a tile: its loops over steps touch no scratch memory (above)."""
    meta = asms[src][asms[src].index("amdhsa.kernels"):]
    seen = 0
    for block in re.split(r"\n  - \.agpr_count", meta)[1:]:
        name = re.search(r"\.name:\s+(\S+)", block).group(1)
        scratch = int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", block).group(1))
        spills = int(re.search(r"\.vgpr_spill_count:\s+(\d+)", block).group(1))
        most = 16 if "codes_run_kernelILb1E" in name else 0
        assert scratch <= 64 and spills <= most, (name, scratch, spills)
        seen += 1
    assert seen >= 3


def test_products_take_the_8_bit_matrix_instructions(asms):
    """bf16 results on f8f6f4 products without block scales; fp32 results, and few
    rows, on bf16 ones."""
    for name, body in kernel_bodies(asms["products_fp8.hip"]).items():
        f8 = sum("f8f6f4" in i for i in body)
        bf = sum("v_mfma" in i and "_bf16" in i for i in body)
        if "codes_run_kernel" in name or "CodesTileILi1E" in name:
            assert f8 and not bf, name
        elif "CodesTileILi2E" in name or "product_thin" in name:
            assert bf and not f8, name
        else:
            assert not f8 and not bf, name
        assert not any("v_mfma_scale" in i for i in body), name
