"""Compiled-code properties of the linear and grouped products (gfx950
assembly from hipcc, no GPU needed): no barrier in a loop that part of a wave
can keep running; k loops that wait on vector memory only for their rings; no
accumulators in scratch memory."""
import concurrent.futures
import os
import re

import pytest

from tests import isa_check as ic

pytestmark = pytest.mark.skipif(not os.path.exists(ic.HIPCC), reason="hipcc not installed")


SOURCES = ["products.hip", "product_grads.hip", "product_pairs.hip"]


@pytest.fixture(scope="module")
def asms(tmp_path_factory):
    d = tmp_path_factory.mktemp("isa")
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(lambda s: ic.compile_asm(s, str(d / (s + ".s"))), SOURCES)))


def kernel_bodies(asm):
    """{kernel symbol: its lines}, up to the kernel's descriptor (a kernel of
    several tile bodies ends in more than one place)."""
    lines, out, name = asm.split("\n"), {}, None
    for line in lines:
        m = re.match(r"^(_Z\w+):", line)
        if m:
            name, out[m.group(1)] = m.group(1), []
        if name:
            if line.strip().startswith(".amdhsa_kernel"):
                name = None
            else:
                out[name].append(line)
    return out


def ring_loops(body):
    """{loop header: instructions} of the innermost loops that multiply and
    load into LDS."""
    return {h: d["instrs"] for h, d in ic.loops(body).items()
            if sum(i.startswith("v_mfma") for i in d["instrs"]) >= 4
            and any(i.startswith("buffer_load") and " lds" in i for i in d["instrs"])}


@pytest.mark.parametrize("src", SOURCES)
def test_no_barrier_in_divergent_loop(asms, src):
    bodies = kernel_bodies(asms[src])
    assert any("product_kernel" in k or "gradients_kernel" in k for k in bodies)
    bad = {k[:90]: ic.barrier_loops_with_exec_exits(v) for k, v in bodies.items()}
    assert not {k: v for k, v in bad.items() if v}


@pytest.mark.parametrize("src", SOURCES)
def test_k_loops_wait_only_for_their_rings(asms, src):
    """The steady-state loop (which refills its rings) holds one vector-memory
    wait that leaves later stages in flight; transposing LDS reads must not
    make the compiler add waits for all of them (the gathered weight
    gradient's loads of row sources may add waits of their own)."""
    found = 0
    for name, body in kernel_bodies(asms[src]).items():
        gather = "Lb1E" in name
        for header, ins in ring_loops(body).items():
            waits = [i for i in ins if i.startswith("s_waitcnt") and "vmcnt" in i]
            full = [i for i in waits if re.search(r"vmcnt\(0\)", i)]
            found += 1
            # one ring wait; the loop over the last steps has its other form too
            assert len(full) <= 1, (name[:90], header, waits)
            if not gather:
                assert len(waits) <= 2, (name[:90], header, waits)
    assert found >= 8


@pytest.mark.parametrize("src", SOURCES)
def test_accumulators_stay_in_registers(asms, src):
    """No vector register is spilled, no ring loop touches scratch memory, and
    no kernel has more of it than a reserve for scalar registers."""
    meta = asms[src][asms[src].index("amdhsa.kernels"):]
    seen = 0
    for block in re.split(r"\n  - \.agpr_count", meta)[1:]:
        name = re.search(r"\.name:\s+(\S+)", block).group(1)
        scratch = int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", block).group(1))
        spills = int(re.search(r"\.vgpr_spill_count:\s+(\d+)", block).group(1))
        assert scratch <= 64 and spills == 0, (name, scratch, spills)
        seen += 1
    assert seen >= 8
    for name, body in kernel_bodies(asms[src]).items():
        for header, ins in ring_loops(body).items():
            assert not any(i.startswith("scratch_") for i in ins), (name[:90], header)
