"""The C entry points of the linear and grouped products and SwiGLU on the
host: struct layouts, workspace sizes, and bad arguments refused before
anything touches the GPU (none of these calls launch anything)."""
import ctypes

import pytest

import sparse_moe_layer_fp32_amd as moe

INVALID, UNSUPPORTED, WORKSPACE = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED,
                                   moe.MOE_ERR_WORKSPACE)
FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
MISALIGNED = ctypes.c_void_p((1 << 20) + 8)


def linear(**kw):
    return moe.make_linear_config(**{**dict(tokens=64, in_features=512, out_features=256), **kw})


def grouped(**kw):
    return moe.make_grouped_config(**{**dict(rows=64, num_groups=4, in_features=512,
                                             out_features=256), **kw})


def swiglu(**kw):
    return moe.make_swiglu_config(**{**dict(rows=64, inter=256), **kw})


def test_struct_layouts():
    assert ctypes.sizeof(moe.moe_linear_config) == 32
    assert ctypes.sizeof(moe.moe_grouped_config) == 48
    assert ctypes.sizeof(moe.moe_swiglu_config) == 24
    assert moe.moe_grouped_config.row_div.offset == 28
    assert moe.moe_swiglu_config.limit.offset == 16


def test_names_of_activations_and_dtypes():
    assert [linear(activation=a).activation for a in moe.ACTIVATIONS] == list(range(5))
    assert linear(y_dtype="f32").y_dtype == 1 and linear(dw_dtype="bf16").dw_dtype == 0
    for kw in (dict(activation="swish"), dict(y_dtype="f16"), dict(dw_dtype="fp32")):
        with pytest.raises(ValueError, match="is none of"):
            linear(**kw)


SIZES = [
    (dict(in_features=0), INVALID), (dict(out_features=-8), INVALID),
    (dict(in_features=12), UNSUPPORTED), (dict(out_features=255), UNSUPPORTED),
    (dict(in_features=65544), UNSUPPORTED), (dict(out_features=65544), UNSUPPORTED),
]


def set_rows(cfg, n):
    setattr(cfg, "tokens" if hasattr(cfg, "tokens") else "rows", n)
    return cfg


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(tokens=-1), INVALID), (dict(tokens=2 ** 26 + 1), UNSUPPORTED),
    (dict(tokens=2 ** 26, in_features=512), UNSUPPORTED)])
def test_linear_refuses_sizes(kw, status):
    cfg, lib = linear(**kw), moe.load_library()
    assert lib.moe_linear_workspace_size(ctypes.byref(cfg)) == 0
    assert lib.moe_linear_forward(ctypes.byref(cfg), *[FAKE] * 7, 1 << 40, None) == status
    assert lib.moe_linear_backward(ctypes.byref(cfg), *[FAKE] * 9, 1 << 40, None) == status
    assert moe.moe_last_error()
    with pytest.raises(moe.MoeError):
        moe.moe_linear_workspace_size(cfg)


@pytest.mark.parametrize("field,value", [("activation", 5), ("activation", -1), ("y_dtype", 2),
                                         ("dw_dtype", -1)])
def test_linear_refuses_unknown_choices(field, value):
    cfg, lib = linear(), moe.load_library()
    setattr(cfg, field, value)
    assert lib.moe_linear_forward(ctypes.byref(cfg), *[FAKE] * 7, 1 << 40, None) == INVALID
    assert "unknown" in moe.moe_last_error()


def test_linear_refuses_pointers_and_workspaces():
    cfg, lib = linear(activation="gelu"), moe.load_library()
    need = moe.moe_linear_workspace_size(cfg)
    fwd = [FAKE] * 7  # x w bias residual y z ws
    for i in (0, 1, 4, 6):
        a = list(fwd)
        a[i] = None
        assert lib.moe_linear_forward(ctypes.byref(cfg), *a, need, None) == INVALID, i
    for i in range(7):
        a = list(fwd)
        a[i] = MISALIGNED
        assert lib.moe_linear_forward(ctypes.byref(cfg), *a, need, None) == UNSUPPORTED, i
    assert lib.moe_linear_forward(ctypes.byref(cfg), *fwd, need - 1, None) == WORKSPACE
    bwd = [FAKE] * 9  # dy z x w dz dx dw dbias ws
    for i in (0, 1, 2, 3, 4, 8):
        a = list(bwd)
        a[i] = None
        assert lib.moe_linear_backward(ctypes.byref(cfg), *a, need, None) == INVALID, i
    for i in range(9):
        a = list(bwd)
        a[i] = MISALIGNED
        assert lib.moe_linear_backward(ctypes.byref(cfg), *a, need, None) == UNSUPPORTED, i
    assert lib.moe_linear_backward(ctypes.byref(cfg), *bwd, need - 1, None) == WORKSPACE
    assert lib.moe_linear_forward(None, *fwd, need, None) == INVALID


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(rows=-1), INVALID), (dict(rows=2 ** 26 + 1), UNSUPPORTED),
    (dict(num_groups=0), INVALID), (dict(num_groups=1025), UNSUPPORTED),
    (dict(row_div=0), INVALID), (dict(x_rows=-1), INVALID),
    (dict(num_groups=1024, in_features=65536, out_features=512), UNSUPPORTED)])
def test_grouped_refuses_sizes(kw, status):
    cfg, lib = grouped(**kw), moe.load_library()
    assert lib.moe_grouped_workspace_size(ctypes.byref(cfg)) == 0
    assert lib.moe_grouped_forward(ctypes.byref(cfg), *[FAKE] * 7, 1 << 40, None) == status
    assert lib.moe_grouped_backward(ctypes.byref(cfg), *[FAKE] * 9, 1 << 40, None) == status


def test_grouped_refuses_pointers_and_workspaces():
    cfg, lib = grouped(x_rows=16, row_div=4), moe.load_library()
    need = moe.moe_grouped_workspace_size(cfg)
    fwd = [FAKE] * 7  # x row_ids offsets w bias y ws
    for i in (0, 2, 3, 5, 6):
        a = list(fwd)
        a[i] = None
        assert lib.moe_grouped_forward(ctypes.byref(cfg), *a, need, None) == INVALID, i
    a = list(fwd)
    a[1] = None  # no row_ids, but x has another number of rows
    assert lib.moe_grouped_forward(ctypes.byref(cfg), *a, need, None) == INVALID
    assert "row_ids" in moe.moe_last_error()
    for i in range(7):
        a = list(fwd)
        a[i] = MISALIGNED
        assert lib.moe_grouped_forward(ctypes.byref(cfg), *a, need, None) == UNSUPPORTED, i
    assert lib.moe_grouped_forward(ctypes.byref(cfg), *fwd, need - 1, None) == WORKSPACE
    bwd = [FAKE] * 9  # dy x row_ids offsets w dx dw dbias ws
    for i in (0, 1, 2, 3, 4, 8):
        a = list(bwd)
        a[i] = None
        assert lib.moe_grouped_backward(ctypes.byref(cfg), *a, need, None) == INVALID, i
    for i in range(9):
        a = list(bwd)
        a[i] = MISALIGNED
        assert lib.moe_grouped_backward(ctypes.byref(cfg), *a, need, None) == UNSUPPORTED, i
    assert lib.moe_grouped_backward(ctypes.byref(cfg), *bwd, need - 1, None) == WORKSPACE
    cfg.reserved = 1
    assert lib.moe_grouped_forward(ctypes.byref(cfg), *fwd, need, None) == INVALID


def test_grouped_refuses_a_gathered_x_beyond_its_offsets():
    lib = moe.load_library()
    cfg = grouped(x_rows=(0xF0000000 // 1024) - 1)
    need = moe.moe_grouped_workspace_size(cfg)
    assert need
    cfg.x_rows += 1
    assert lib.moe_grouped_forward(ctypes.byref(cfg), *[FAKE] * 7, need, None) == UNSUPPORTED
    assert lib.moe_grouped_backward(ctypes.byref(cfg), *[FAKE] * 9, need, None) == UNSUPPORTED
    assert "row_ids" in moe.moe_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(inter=0), INVALID), (dict(inter=252), UNSUPPORTED),
    (dict(ld=248), INVALID), (dict(ld=260), UNSUPPORTED), (dict(rows=2 ** 62), UNSUPPORTED),
    (dict(rows=2 ** 27), UNSUPPORTED)])
def test_swiglu_refuses_sizes(kw, status):
    cfg, lib = swiglu(**kw), moe.load_library()
    assert lib.moe_swiglu_forward(ctypes.byref(cfg), FAKE, FAKE, FAKE, None) == status
    assert lib.moe_swiglu_backward(ctypes.byref(cfg), *[FAKE] * 6, None) == status


@pytest.mark.parametrize("rows,inter,ld", [
    (2 ** 32 - 1, 8, 0), (2 ** 32 - 255, 8, 0), (2 ** 27 - 7, 256, 0), (2 ** 26 - 3, 256, 512)])
def test_swiglu_refuses_more_threads_than_a_launch_holds(rows, inter, ld):
    cfg, lib = swiglu(rows=rows, inter=inter, ld=ld), moe.load_library()
    assert lib.moe_swiglu_forward(ctypes.byref(cfg), FAKE, FAKE, FAKE, None) == UNSUPPORTED
    assert lib.moe_swiglu_backward(ctypes.byref(cfg), *[FAKE] * 6, None) == UNSUPPORTED


def test_swiglu_refuses_pointers():
    cfg, lib = swiglu(), moe.load_library()
    for i in range(3):
        a = [FAKE] * 3
        a[i] = None
        assert lib.moe_swiglu_forward(ctypes.byref(cfg), *a, None) == INVALID
        a[i] = MISALIGNED
        assert lib.moe_swiglu_forward(ctypes.byref(cfg), *a, None) == UNSUPPORTED
    for i in range(6):
        a = [FAKE] * 6
        a[i] = MISALIGNED
        assert lib.moe_swiglu_backward(ctypes.byref(cfg), *a, None) == UNSUPPORTED
        if i < 5:
            a[i] = None
            assert lib.moe_swiglu_backward(ctypes.byref(cfg), *a, None) == INVALID
    cfg.reserved = 2
    assert lib.moe_swiglu_forward(ctypes.byref(cfg), *[FAKE] * 3, None) == INVALID


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    cfg = linear()
    t = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d)  # noqa: E731
    with pytest.raises(ValueError, match="on the GPU"):
        moe.moe_linear_forward(cfg, t(64, 512), t(256, 512), None, None, t(64, 256), None, t(1))
    with pytest.raises(ValueError, match="required"):
        moe.moe_linear_forward(cfg, None, t(256, 512), None, None, t(64, 256), None, t(1))
    with pytest.raises(TypeError):
        moe.moe_swiglu_forward(swiglu(), 3, t(64, 256), t(64, 256))
    with pytest.raises(ValueError, match="on the GPU"):
        moe.moe_swiglu_forward(swiglu(), t(64, 256), t(64, 256), t(64, 256))


def test_workspace_sizes_cover_the_source_rows():
    for rows in (0, 1, 1000, 65536):
        assert moe.moe_grouped_workspace_size(grouped(rows=rows)) >= 4 * rows
        assert moe.moe_linear_workspace_size(linear(tokens=rows)) > 0
