"""The C entry points of dispatch, combine, quantisation and the products of
codes on the host: struct layouts, workspace sizes, and bad arguments refused
before anything touches the GPU (none of these calls launch anything)."""
import ctypes

import pytest

import sparse_moe_layer_fp32_amd as moe

INVALID, UNSUPPORTED, WORKSPACE = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED,
                                   moe.MOE_ERR_WORKSPACE)
FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
MISALIGNED = ctypes.c_void_p((1 << 20) + 8)
ROW_CALLS = {  # pointers: which are required
    "moe_dispatch_forward": (1, 1, 1),
    "moe_dispatch_backward": (1, 1, 0, 1),
    "moe_combine_forward": (1, 1, 0, 0, 1),
    "moe_combine_backward": (1, 1, 1, 0, 0, 0),
}


def dispatch(**kw):
    return moe.make_dispatch_config(**{**dict(tokens=64, rows=128, top_k=2, hidden=256), **kw})


def quantize(**kw):
    return moe.make_quantize_config(**{**dict(tokens=64, features=256), **kw})


def linear(**kw):
    return moe.make_linear_config(**{**dict(tokens=64, in_features=512, out_features=256), **kw})


def grouped(**kw):
    return moe.make_grouped_config(**{**dict(rows=64, num_groups=4, in_features=512,
                                             out_features=256), **kw})


def test_struct_layouts():
    assert ctypes.sizeof(moe.moe_dispatch_config) == 32
    assert moe.moe_dispatch_config.row_dtype.offset == 28
    assert ctypes.sizeof(moe.moe_quantize_config) == 24
    assert moe.moe_quantize_config.features.offset == 20


@pytest.mark.parametrize("name", list(ROW_CALLS))
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), INVALID), (dict(rows=-1), INVALID), (dict(top_k=0), INVALID),
    (dict(hidden=0), INVALID), (dict(hidden=12), UNSUPPORTED), (dict(hidden=65544), UNSUPPORTED),
    (dict(top_k=33), UNSUPPORTED), (dict(tokens=2 ** 25 + 1, hidden=8), UNSUPPORTED),
    (dict(rows=2 ** 26 + 1, hidden=8), UNSUPPORTED), (dict(tokens=2 ** 25, hidden=264), UNSUPPORTED),
    (dict(rows=2 ** 26, hidden=136), UNSUPPORTED)])
def test_rows_refuse_sizes(name, kw, status):
    fn = getattr(moe.load_library(), name)
    cfg = dispatch(**kw)
    assert fn(ctypes.byref(cfg), *[FAKE] * len(ROW_CALLS[name]), None) == status
    assert moe.moe_last_error()


@pytest.mark.parametrize("name", list(ROW_CALLS))
def test_rows_refuse_pointers_and_types(name):
    fn, need = getattr(moe.load_library(), name), ROW_CALLS[name]
    for i, required in enumerate(need):
        args = [FAKE] * len(need)
        args[i] = MISALIGNED
        assert fn(ctypes.byref(dispatch()), *args, None) == UNSUPPORTED, i
        if required:
            args[i] = None
            assert fn(ctypes.byref(dispatch()), *args, None) == INVALID, i
    assert fn(None, *[FAKE] * len(need), None) == INVALID
    for field in ("token_dtype", "row_dtype"):
        cfg = dispatch()
        setattr(cfg, field, 2)
        assert fn(ctypes.byref(cfg), *[FAKE] * len(need), None) == INVALID
    with pytest.raises(ValueError, match="is none of"):
        dispatch(row_dtype="f16")


def test_nothing_to_do_is_valid():
    lib = moe.load_library()
    empty = dispatch(tokens=0, rows=0)
    for name, need in ROW_CALLS.items():
        assert getattr(lib, name)(ctypes.byref(empty), *[None] * len(need), None) == moe.MOE_OK
    # no gradient wanted, and no rows to send anything to
    assert lib.moe_combine_backward(ctypes.byref(dispatch()), FAKE, None, FAKE, None, None, None,
                                    None) == moe.MOE_OK
    assert lib.moe_dispatch_forward(ctypes.byref(dispatch(rows=0)), FAKE, FAKE, None,
                                    None) == moe.MOE_OK
    assert lib.moe_quantize_rows(ctypes.byref(quantize(tokens=0)), *[None] * 5) == moe.MOE_OK


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), INVALID), (dict(features=0), INVALID), (dict(features=24), UNSUPPORTED),
    (dict(features=65552), UNSUPPORTED), (dict(top_k=0), INVALID),
    (dict(tokens=2 ** 25, features=272), UNSUPPORTED)])
def test_quantize_refuses_sizes(kw, status):
    lib = moe.load_library()
    assert lib.moe_quantize_rows(ctypes.byref(quantize(**kw)), *[FAKE] * 4, None) == status


def test_quantize_refuses_arguments():
    lib = moe.load_library()
    for i in (0, 2, 3):
        args = [FAKE] * 4
        args[i] = None
        assert lib.moe_quantize_rows(ctypes.byref(quantize()), *args, None) == INVALID
    for i in range(4):
        args = [FAKE] * 4
        args[i] = MISALIGNED
        assert lib.moe_quantize_rows(ctypes.byref(quantize()), *args, None) == UNSUPPORTED
    # rows of codes that do not match, without positions to say which is which
    for kw in (dict(rows=65), dict(top_k=2)):
        assert lib.moe_quantize_rows(ctypes.byref(quantize(**kw)), FAKE, None, FAKE, FAKE,
                                     None) == INVALID
    assert lib.moe_quantize_rows(None, *[FAKE] * 4, None) == INVALID
    for sizes, status in (((0, 64, 64), INVALID), ((1, 64, 24), UNSUPPORTED),
                          ((1, 0, 64), INVALID), ((1, 65537, 64), UNSUPPORTED),
                          ((2 ** 22, 1, 16), UNSUPPORTED), ((2 ** 31 - 1, 65536, 65536), UNSUPPORTED)):
        assert lib.moe_quantize_weight(*sizes, FAKE, FAKE, FAKE, None) == status, sizes
    for i in range(3):
        args = [FAKE] * 3
        args[i] = None
        assert lib.moe_quantize_weight(1, 64, 64, *args, None) == INVALID
        args[i] = MISALIGNED
        assert lib.moe_quantize_weight(1, 64, 64, *args, None) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(in_features=0), INVALID), (dict(in_features=24), UNSUPPORTED),
    (dict(out_features=12), UNSUPPORTED), (dict(in_features=65552), UNSUPPORTED),
    (dict(y_dtype=2), INVALID)])
def test_products_refuse_sizes(kw, status):
    lib = moe.load_library()
    for make, size, call, n in ((linear, "linear", lib.moe_linear_forward_fp8, 8),
                                (grouped, "grouped", lib.moe_grouped_forward_fp8, 8)):
        cfg = make(**{k: v for k, v in kw.items() if k != "y_dtype"})
        if "y_dtype" in kw:
            cfg.y_dtype = kw["y_dtype"]
        assert getattr(lib, f"moe_{size}_fp8_workspace_size")(ctypes.byref(cfg)) == 0
        assert call(ctypes.byref(cfg), *[FAKE] * (n + 1), 1 << 40, None) == status
        with pytest.raises(moe.MoeError):
            getattr(moe, f"moe_{size}_fp8_workspace_size")(cfg)


def test_products_refuse_pointers_and_workspaces():
    lib = moe.load_library()
    cfg = linear()
    need = moe.moe_linear_fp8_workspace_size(cfg)
    args = [FAKE] * 9  # x xs w ws bias residual y z work
    for i in (0, 1, 2, 3, 6, 8):
        a = list(args)
        a[i] = None
        assert lib.moe_linear_forward_fp8(ctypes.byref(cfg), *a, need, None) == INVALID, i
    for i in range(9):
        a = list(args)
        a[i] = MISALIGNED
        assert lib.moe_linear_forward_fp8(ctypes.byref(cfg), *a, need, None) == UNSUPPORTED, i
    assert lib.moe_linear_forward_fp8(ctypes.byref(cfg), *args, need - 1, None) == WORKSPACE
    assert lib.moe_linear_forward_fp8(None, *args, need, None) == INVALID
    cfg = grouped(x_rows=16, row_div=4)
    need = moe.moe_grouped_fp8_workspace_size(cfg)
    args = [FAKE] * 9  # x xs ids offsets w ws bias y work
    for i in (0, 1, 3, 4, 5, 7, 8):
        a = list(args)
        a[i] = None
        assert lib.moe_grouped_forward_fp8(ctypes.byref(cfg), *a, need, None) == INVALID, i
    a = list(args)
    a[2] = None  # x_rows differs from rows
    assert lib.moe_grouped_forward_fp8(ctypes.byref(cfg), *a, need, None) == INVALID
    for i in range(9):
        a = list(args)
        a[i] = MISALIGNED
        assert lib.moe_grouped_forward_fp8(ctypes.byref(cfg), *a, need, None) == UNSUPPORTED, i
    assert lib.moe_grouped_forward_fp8(ctypes.byref(cfg), *args, need - 1, None) == WORKSPACE


def test_no_rows_need_no_x():
    lib = moe.load_library()
    cfg = linear(tokens=0)
    need = moe.moe_linear_fp8_workspace_size(cfg)
    assert lib.moe_linear_forward_fp8(ctypes.byref(cfg), None, None, FAKE, FAKE, None, None, None,
                                      None, FAKE, need, None) == moe.MOE_OK
    cfg = grouped(rows=0)
    need = moe.moe_grouped_fp8_workspace_size(cfg)
    assert lib.moe_grouped_forward_fp8(ctypes.byref(cfg), None, None, None, FAKE, FAKE, FAKE, None,
                                       None, FAKE, need, None) == moe.MOE_OK
