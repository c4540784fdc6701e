"""Refusals of the mixture-of-experts block's entry points (no GPU: every call here returns
before a launch): one changed argument at a time against arguments that are in order."""
import ctypes
import os

import pytest

from conftest import ROOT

A = 1 << 32  # addresses that nothing follows: 16 MiB apart, never read


@pytest.fixture(scope="module")
def plr():
    if not os.path.exists(os.path.join(ROOT, "reduce_atom_amd", "libplr.so")):
        import __graft_entry__

        __graft_entry__._load_builder().build()
    import reduce_atom_amd

    return reduce_atom_amd


def _at(i):
    return A + (i << 24)


def _srcs(*addresses):
    return (ctypes.c_void_p * max(1, len(addresses)))(*addresses)


BF16, F16, F32, F8 = range(4)

NORM = dict(dtype=BF16, out_dtype=BF16, world=2, rows=4, cols=64, srcs=_srcs(_at(1), _at(2)), src_pitch=128,
            residual=_at(3), residual_pitch=128, gamma=_at(4), eps=1e-6, sum_out=_at(5), sum_pitch=128, out=_at(6),
            out_pitch=128, out_scale=None, rstd=_at(8), stream=None)
NORM_BACK = dict(dtype=BF16, rows=4, cols=64, dout=_at(1), dout_pitch=128, h=_at(2), h_pitch=128, gamma=_at(3),
                 rstd=_at(4), dsum=_at(5), dsum_pitch=128, dx=_at(6), dx_pitch=128, dgamma=_at(7), workspace=_at(8),
                 stream=None)
ROUTE = dict(dtype=F32, tokens=4, experts=8, k=2, logits=_at(1), logits_pitch=32, ids=_at(2), weights=_at(3),
             positions=_at(4), row_token=_at(5), offsets=_at(6), workspace=_at(7), stream=None)
ROUTE_BACK = dict(dtype=F32, tokens=4, experts=8, k=2, ids=_at(1), weights=_at(2), dweights=_at(3), dlogits=_at(4),
                  dlogits_pitch=32, stream=None)
GROUP = dict(dtype=BF16, out_dtype=F32, groups=2, rows=4, n=16, k=32, x=_at(1), x_pitch=64, x_rows=4, row_of=_at(2),
             w=_at(3), offsets=_at(4), x_scale=None, w_scale=None, y=_at(5), y_pitch=64, stream=None)
GROUP_DX = dict(dtype=BF16, out_dtype=BF16, groups=2, rows=4, n=16, k=32, dy=_at(1), dy_pitch=32, w=_at(2),
                offsets=_at(3), dx=_at(4), dx_pitch=64, stream=None)
GROUP_DW = dict(dtype=BF16, out_dtype=F32, groups=2, rows=4, n=16, k=32, dy=_at(1), dy_pitch=32, x=_at(2), x_pitch=64,
                x_rows=4, row_of=_at(3), offsets=_at(4), dw=_at(5), stream=None)
COMBINE = dict(dtype=F16, tokens=4, k=2, cols=64, y=_at(1), y_pitch=128, y_rows=8, positions=_at(2), weights=_at(3),
               out=_at(4), out_pitch=128, stream=None)
COMBINE_BACK = dict(dtype=F16, tokens=4, k=2, cols=64, dout=_at(1), dout_pitch=128, y=_at(2), y_pitch=128, y_rows=8,
                    positions=_at(3), weights=_at(4), dy=_at(5), dy_pitch=128, dweights=_at(6), stream=None)
CALLS = dict(plr_rmsnorm=NORM, plr_rmsnorm_backward=NORM_BACK, plr_route=ROUTE, plr_route_backward=ROUTE_BACK,
             plr_group_matmul=GROUP, plr_group_matmul_dx=GROUP_DX, plr_group_matmul_dw=GROUP_DW, plr_combine=COMBINE,
             plr_combine_backward=COMBINE_BACK)

INVAL, ALIGN, UNSUPPORTED = 1, 2, 3
MANY = 1 << 40

REFUSED = [
    # types
    ("plr_rmsnorm", dict(dtype=F8), INVAL), ("plr_rmsnorm", dict(dtype=4), INVAL),
    ("plr_rmsnorm", dict(out_dtype=F16), INVAL), ("plr_rmsnorm_backward", dict(dtype=F8), INVAL),
    ("plr_route", dict(dtype=F8), INVAL), ("plr_route_backward", dict(dtype=-1), INVAL),
    ("plr_group_matmul", dict(dtype=F32), UNSUPPORTED), ("plr_group_matmul", dict(dtype=9), INVAL),
    ("plr_group_matmul", dict(out_dtype=F16), INVAL), ("plr_group_matmul", dict(out_dtype=F8), INVAL),
    ("plr_group_matmul_dx", dict(dtype=F8), UNSUPPORTED), ("plr_group_matmul_dw", dict(dtype=F8), UNSUPPORTED),
    ("plr_combine", dict(dtype=F8), INVAL), ("plr_combine_backward", dict(dtype=7), INVAL),
    # sizes
    ("plr_rmsnorm", dict(world=0), INVAL), ("plr_rmsnorm", dict(world=17), UNSUPPORTED),
    ("plr_rmsnorm", dict(rows=-1), INVAL), ("plr_rmsnorm", dict(cols=0), INVAL),
    ("plr_rmsnorm", dict(cols=60), ALIGN), ("plr_rmsnorm", dict(rows=MANY), UNSUPPORTED),
    ("plr_rmsnorm", dict(cols=32776, src_pitch=65552), UNSUPPORTED),
    ("plr_rmsnorm", dict(out_dtype=F8, out_scale=_at(7), cols=56), ALIGN),
    ("plr_rmsnorm", dict(out_dtype=F8), INVAL), ("plr_rmsnorm", dict(eps=-1.0), INVAL),
    ("plr_rmsnorm", dict(eps=float("nan")), INVAL),
    ("plr_rmsnorm_backward", dict(cols=12), ALIGN), ("plr_rmsnorm_backward", dict(cols=1 << 20), UNSUPPORTED),
    ("plr_route", dict(experts=0), INVAL), ("plr_route", dict(experts=1025), UNSUPPORTED),
    ("plr_route", dict(k=0), INVAL), ("plr_route", dict(k=17), UNSUPPORTED), ("plr_route", dict(tokens=-1), INVAL),
    ("plr_route", dict(tokens=1 << 25), UNSUPPORTED), ("plr_route_backward", dict(k=17), UNSUPPORTED),
    ("plr_group_matmul", dict(groups=0), INVAL), ("plr_group_matmul", dict(groups=4097), UNSUPPORTED),
    ("plr_group_matmul", dict(rows=-1), INVAL), ("plr_group_matmul", dict(n=12), ALIGN),
    ("plr_group_matmul", dict(k=36), ALIGN), ("plr_group_matmul", dict(n=0), INVAL),
    ("plr_group_matmul", dict(n=(1 << 20) + 8), UNSUPPORTED), ("plr_group_matmul", dict(rows=MANY), UNSUPPORTED),
    ("plr_group_matmul", dict(dtype=F8, x_scale=_at(6), w_scale=_at(7), k=24), ALIGN),
    ("plr_group_matmul", dict(dtype=F8), INVAL), ("plr_group_matmul", dict(dtype=F8, x_scale=_at(6)), INVAL),
    ("plr_group_matmul", dict(x_scale=_at(6), w_scale=_at(7)), INVAL),
    ("plr_group_matmul", dict(row_of=None, x_rows=3), INVAL), ("plr_group_matmul", dict(x_rows=-1), INVAL),
    ("plr_group_matmul", dict(rows=1 << 30, x_rows=1 << 30, n=1 << 20, y_pitch=1 << 22), UNSUPPORTED),
    ("plr_group_matmul_dx", dict(rows=1 << 30, k=1 << 20, dx_pitch=1 << 21), UNSUPPORTED),
    ("plr_group_matmul_dw", dict(groups=4096, n=1 << 16, k=1 << 16), UNSUPPORTED),
    ("plr_group_matmul_dx", dict(n=4), ALIGN), ("plr_group_matmul_dw", dict(row_of=None, x_rows=2), INVAL),
    ("plr_group_matmul_dw", dict(k=4), ALIGN), ("plr_combine", dict(k=0), INVAL),
    ("plr_combine", dict(k=17), UNSUPPORTED), ("plr_combine", dict(cols=4), ALIGN),
    ("plr_combine", dict(y_rows=-1), INVAL), ("plr_combine", dict(tokens=1 << 25), UNSUPPORTED),
    ("plr_combine_backward", dict(cols=4), ALIGN), ("plr_combine_backward", dict(tokens=-1), INVAL),
    # pitches
    ("plr_rmsnorm", dict(src_pitch=112), INVAL), ("plr_rmsnorm", dict(src_pitch=136), ALIGN),
    ("plr_rmsnorm", dict(out_pitch=120), ALIGN), ("plr_rmsnorm", dict(residual_pitch=64), INVAL),
    ("plr_rmsnorm", dict(sum_pitch=0), INVAL), ("plr_rmsnorm", dict(out_pitch=1 << 62), UNSUPPORTED),
    ("plr_rmsnorm_backward", dict(dx_pitch=64), INVAL), ("plr_rmsnorm_backward", dict(h_pitch=130), ALIGN),
    ("plr_route", dict(logits_pitch=28), INVAL), ("plr_route", dict(logits_pitch=34), ALIGN),
    ("plr_route_backward", dict(dlogits_pitch=16), INVAL), ("plr_group_matmul", dict(x_pitch=48), INVAL),
    ("plr_group_matmul", dict(y_pitch=72), ALIGN), ("plr_group_matmul_dx", dict(dy_pitch=16), INVAL),
    ("plr_group_matmul_dw", dict(x_pitch=72), ALIGN), ("plr_combine", dict(y_pitch=64), INVAL),
    ("plr_combine", dict(out_pitch=136), ALIGN), ("plr_combine_backward", dict(dy_pitch=0), INVAL),
    # an output over an input, over part of it, or over another output
    ("plr_rmsnorm", dict(sum_out=_at(1) + 128), INVAL), ("plr_rmsnorm", dict(out=_at(4)), INVAL),
    ("plr_rmsnorm", dict(out=_at(5) + 16), INVAL), ("plr_rmsnorm", dict(rstd=_at(3)), INVAL),
    ("plr_rmsnorm", dict(sum_out=_at(1), sum_pitch=144), INVAL),
    ("plr_rmsnorm", dict(out=_at(1), out_dtype=F8, out_scale=_at(7)), INVAL),
    ("plr_rmsnorm_backward", dict(dx=_at(3)), INVAL), ("plr_rmsnorm_backward", dict(dgamma=_at(1)), INVAL),
    ("plr_rmsnorm_backward", dict(workspace=_at(2) + 64), INVAL), ("plr_rmsnorm_backward", dict(dx=_at(1) + 16), INVAL),
    ("plr_route", dict(ids=_at(1)), INVAL), ("plr_route", dict(positions=_at(2) + 4), INVAL),
    ("plr_route", dict(workspace=_at(6)), INVAL), ("plr_route_backward", dict(dlogits=_at(2)), INVAL),
    ("plr_group_matmul", dict(y=_at(1)), INVAL), ("plr_group_matmul", dict(y=_at(3) + 1024), INVAL),
    ("plr_group_matmul", dict(y=_at(4)), INVAL), ("plr_group_matmul_dx", dict(dx=_at(2)), INVAL),
    ("plr_group_matmul_dw", dict(dw=_at(2)), INVAL), ("plr_combine", dict(out=_at(1) + 256), INVAL),
    ("plr_combine_backward", dict(dy=_at(1)), INVAL), ("plr_combine_backward", dict(dweights=_at(4)), INVAL),
    ("plr_combine_backward", dict(dy=_at(2) + 16), INVAL),
]

OPTIONAL = {  # what may be NULL
    "plr_rmsnorm": {"residual", "sum_out", "rstd", "out_scale"}, "plr_rmsnorm_backward": {"dsum"}, "plr_route": set(),
    "plr_route_backward": set(), "plr_group_matmul": {"row_of", "x_scale", "w_scale"}, "plr_group_matmul_dx": set(),
    "plr_group_matmul_dw": {"row_of"}, "plr_combine": {"weights"}, "plr_combine_backward": {"weights", "dweights"},
}


def _call(plr, name, changed):
    args = dict(CALLS[name], **changed)
    assert list(args) == list(CALLS[name])
    return getattr(plr._lib, name)(*args.values())


@pytest.mark.parametrize("name,changed,code", REFUSED, ids=lambda v: str(v)[:60])
def test_refused(plr, name, changed, code):
    assert _call(plr, name, changed) == code


@pytest.mark.parametrize("name", CALLS)
def test_null_and_unaligned_addresses(plr, name):
    vectors = {"ids", "weights", "dweights", "positions", "row_token", "row_of", "x_scale", "w_scale", "rstd", "out_scale"}
    for field, v in CALLS[name].items():
        if not (isinstance(v, int) and v >= A):
            continue
        if field not in OPTIONAL[name]:
            assert _call(plr, name, {field: None}) == INVAL, field
        off = 2 if field in vectors or (name == "plr_route" and field == "logits") else 4 if field == "offsets" else 8
        assert _call(plr, name, {field: v + off}) == ALIGN, field
    if name == "plr_rmsnorm":
        assert _call(plr, name, dict(srcs=_srcs(_at(1), None))) == INVAL
        assert _call(plr, name, dict(srcs=_srcs(_at(1), _at(2) + 8))) == ALIGN
        assert _call(plr, name, dict(srcs=None)) == INVAL


def test_nothing_to_do_is_no_error(plr):
    assert _call(plr, "plr_rmsnorm", dict(rows=0)) == 0
    assert _call(plr, "plr_route_backward", dict(tokens=0)) == 0
    assert _call(plr, "plr_group_matmul", dict(rows=0)) == 0
    assert _call(plr, "plr_group_matmul_dx", dict(rows=0)) == 0
    assert _call(plr, "plr_combine", dict(tokens=0)) == 0
    assert _call(plr, "plr_combine_backward", dict(tokens=0)) == 0


def test_no_rows_in_8_bits_is_no_error(plr):
    # an empty tensor's address is NULL: out_scale has no entries then
    none = dict(rows=0, srcs=_srcs(None, None), residual=None, sum_out=None, out=None, rstd=None)
    for out_dtype, cols, code in ((BF16, 64, 0), (F8, 64, 0), (F8, 56, ALIGN)):
        assert _call(plr, "plr_rmsnorm", dict(none, out_dtype=out_dtype, cols=cols)) == code
    assert _call(plr, "plr_rmsnorm", dict(rows=1, out_dtype=F8, out_scale=None)) == INVAL


def test_products_of_no_rows_in_8_bits_are_no_error(plr):
    # x_scale has no entries where x has no rows; a scale for a 16-bit type stays refused
    none = dict(rows=0, x=None, x_rows=0, row_of=None, x_scale=None, y=None)
    f8 = dict(none, dtype=F8, w_scale=_at(7))
    assert _call(plr, "plr_group_matmul", none) == 0
    assert _call(plr, "plr_group_matmul", f8) == 0
    assert _call(plr, "plr_group_matmul", dict(f8, w_scale=None)) == INVAL
    assert _call(plr, "plr_group_matmul", dict(f8, x=_at(1), x_rows=4)) == INVAL
    assert _call(plr, "plr_group_matmul", dict(f8, x=_at(1), x_rows=4, x_scale=_at(6))) == 0
    assert _call(plr, "plr_group_matmul", dict(none, x_scale=_at(6))) == INVAL
    assert _call(plr, "plr_group_matmul", dict(none, w_scale=_at(7))) == INVAL


def test_workspace_sizes(plr):
    lib = plr._lib
    assert lib.plr_rmsnorm_backward_workspace_bytes(BF16, 1, 64) == 4 * 64
    n = lib.plr_rmsnorm_backward_workspace_bytes(BF16, 100000, 7168)
    assert n % (4 * 7168) == 0 and n <= 1024 * 4 * 7168
    assert plr.plr_rmsnorm_backward_workspace_bytes("bf16", 100000, 7168) == n
    for bad in ((F8, 1, 64), (BF16, -1, 64), (BF16, 1, 60), (BF16, 1, 1 << 20)):
        assert lib.plr_rmsnorm_backward_workspace_bytes(*bad) == 0
    assert lib.plr_route_workspace_bytes(64, 8) >= 2 * 8 * 4
    for bad in ((-1, 8), (4, 0), (4, 1025), (1 << 25, 8)):
        assert lib.plr_route_workspace_bytes(*bad) == 0


def test_layouts_take_no_8bit_type(plr):
    with pytest.raises(plr.PlrError) as e:
        plr.plr_layout_create("reduce", plr.PLR_F8, 2, 64, "packed", "packed")
    assert e.value.code == plr.PLR_EINVAL


def test_binding_refuses_host_tensors_and_wrong_shapes(plr):
    import torch

    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        plr.plr_rmsnorm([x], x[0], x)
    with pytest.raises(ValueError, match="at least one"):
        plr.plr_rmsnorm([], x[0], x)
    with pytest.raises(ValueError, match="groups, n, k"):
        plr.plr_group_matmul(x, x, None, x)
    with pytest.raises(ValueError, match="device tensor"):
        plr.plr_combine(x, torch.zeros(4, 2, dtype=torch.int32), None, x)
