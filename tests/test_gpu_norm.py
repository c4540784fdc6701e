"""plr_rmsnorm and its gradient against 64 bits: every type and output, row lengths on
both sides of each launch shape, one row to many, rows apart, outputs in an input's place,
rows of zeros, NaN and infinities; the gradient against the formula and differences."""
import math

import pytest
import torch

import blockref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def plr():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import reduce_atom_amd

    return reduce_atom_amd


def _rand(seed, shape, dt, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(dt).cuda()


def _run(plr, srcs, gamma, out_dt, residual=None, eps=EPS):
    R, C = srcs[0].shape
    s = torch.full((R, C), 7.0, device="cuda").to(srcs[0].dtype)
    out = torch.empty(R, C, dtype=out_dt, device="cuda")
    scale = torch.empty(R, device="cuda") if out_dt == ref.F8 else None
    rstd = torch.empty(R, device="cuda")
    plr.plr_rmsnorm(srcs, gamma, out, eps=eps, residual=residual, sum_out=s, out_scale=scale, rstd=rstd)
    torch.cuda.synchronize()
    return s, out, scale, rstd


# errors before the output's rounding: the sum has at most 16 + 1 terms; the mean's sum is
# at most 32 products per thread, 6 + 4 + 16 further additions; then a few operations
def _check(got, want, dt, out_dt):
    s, out, scale, rstd = got
    h, mag, r, y = want
    dh = 17 * ref.U32 * mag
    ref.assert_within(s, h, dh, dt, "sum")
    rel = 64 * ref.U32 + (dh * h.abs()).sum(-1) / (h * h).sum(-1).clamp_min(1e-300)
    ref.assert_within(rstd, r, rel * r, torch.float32, "rstd")
    slack = y.abs() * (rel[:, None] + 8 * ref.U32) + dh * (y / h.where(h != 0, torch.ones_like(h))).abs()
    if out_dt != ref.F8:
        ref.assert_within(out, y, slack, dt, "out")
        return
    m = y.abs().amax(-1).clamp_min(2.0 ** -100)
    ref.assert_within(scale, m / 448, slack.amax(-1) / 448 + 2 * ref.U32 * m / 448, torch.float32, "scale")
    back = out.float().cpu().double() * scale.cpu().double()[:, None]
    # e4m3: half a step is 2^-4 of the value, or 2^-10 of the scale below the normal range
    bound = torch.maximum(y.abs() * 2.0 ** -4, (m / 448 * 2.0 ** -10)[:, None]) * 1.001 + 2 * slack
    assert ((back - y).abs() <= bound).all()


SHAPES = [(1, 16), (3, 64), (5, 1008), (2, 7168), (1, 8192), (3, 8208), (2, 16384), (130, 272)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("dt", ref.DTYPES, ids=ref.ids)
def test_forward(plr, dt, f8, R, C):
    W = 1 + (R + C // 16) % 4
    srcs = [_rand(10 + w, (R, C), dt) for w in range(W)]
    res = _rand(5, (R, C), dt, 2.0) if C % 64 else None
    gamma = _rand(6, (C,), dt)
    out_dt = ref.F8 if f8 else dt
    _check(_run(plr, srcs, gamma, out_dt, res), ref.norm(srcs, res, gamma, EPS), dt, out_dt)


@pytest.mark.parametrize("W", [1, 2, 4, 5, 8, 9, 16])
def test_every_world(plr, W):
    srcs = [_rand(20 + w, (7, 7168), torch.bfloat16, 0.5) for w in range(W)]
    res, gamma = _rand(3, (7, 7168), torch.bfloat16), _rand(4, (7168,), torch.bfloat16)
    for out_dt in (torch.bfloat16, ref.F8):
        _check(_run(plr, srcs, gamma, out_dt, res), ref.norm(srcs, res, gamma, EPS), torch.bfloat16, out_dt)


def test_longest_rows(plr):
    for dt, C in ((torch.bfloat16, 32768), (torch.float32, 16384)):
        srcs = [_rand(30 + w, (2, C), dt) for w in range(16)]
        gamma = _rand(4, (C,), dt)
        _check(_run(plr, srcs, gamma, dt), ref.norm(srcs, None, gamma, EPS), dt, dt)


def test_sum_is_the_ordered_one(plr):
    # 2^24 + 1 + 1 in binary32: in source order the ones are lost one by one
    one = torch.ones(1, 16, device="cuda")
    big = torch.full((1, 16), 2.0 ** 24, device="cuda")
    s, *_ = _run(plr, [big, one, one], torch.ones(16, device="cuda"), torch.float32)
    assert (s == 2.0 ** 24).all()
    s, *_ = _run(plr, [one, one], torch.ones(16, device="cuda"), torch.float32, residual=big)
    assert (s == 2.0 ** 24 + 2).all()


def test_rows_apart_and_in_place(plr):
    wide = _rand(1, (9, 1024), torch.bfloat16)
    wide2 = _rand(2, (9, 1024), torch.bfloat16)
    gamma = _rand(3, (256,), torch.bfloat16)
    x, y = wide[:, 128:384], wide2[:, 128:384]
    res = wide[:, 512:768]
    want = ref.norm([x, y], res, gamma, EPS)
    keep = wide.clone()
    out = torch.empty(9, 256, dtype=torch.bfloat16, device="cuda")
    plr.plr_rmsnorm([x, y], gamma, out, eps=EPS, residual=res, sum_out=res)  # the residual stream in place
    torch.cuda.synchronize()
    ref.assert_within(res, want[0], 3 * ref.U32 * want[1], torch.bfloat16, "sum in place")
    keep[:, 512:768] = res
    assert torch.equal(keep, wide)  # nothing beside it was touched
    again = torch.empty_like(out)
    first = [x.clone(), y.clone()]
    plr.plr_rmsnorm(first, gamma, again, eps=EPS, residual=keep[:, 512:768].clone())
    z = first[0].clone()
    plr.plr_rmsnorm([z, first[1]], gamma, z, eps=EPS, residual=keep[:, 512:768].clone())
    torch.cuda.synchronize()
    assert torch.equal(z, again)


@pytest.mark.parametrize("out_dt", [torch.bfloat16, ref.F8], ids=ref.ids)
def test_rows_of_zeros_nan_and_infinity(plr, out_dt):
    x = _rand(1, (5, 512), torch.bfloat16)
    x[1] = 0
    x[2, 17] = math.nan
    x[3, 5] = math.inf
    x[4] = 2.0 ** -130  # subnormal
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    s, out, scale, rstd = _run(plr, [x], gamma, out_dt, eps=0.0 if out_dt == ref.F8 else EPS)
    o = out.float()
    assert o[0].isfinite().all() and o[2].isnan().all()
    if out_dt == ref.F8:  # eps 0: a row of zeros is 0 * inf
        assert scale[2].isnan() and o[3].isnan().all() and scale[3].isnan() and o[1].isnan().all()
        _, out, scale, _ = _run(plr, [x], gamma, out_dt)
        assert (out.float()[1] == 0).all() and scale[1].cpu() == torch.tensor(2.0 ** -100) / 448
    else:
        assert (o[1] == 0).all() and rstd[1] == torch.tensor(EPS).rsqrt()
        assert o[3, 5].isnan() and (o[3, :5] == 0).all()


def test_every_8bit_value(plr):
    # rows whose largest value is 448 and rstd 1 (eps makes up for the mean): each value is
    # rounded as torch rounds it, ties and the subnormal range among them
    v = torch.cat([torch.arange(0, 449 * 64) / 64.0, torch.arange(0, 2048) / 2.0 ** 16])
    v = torch.cat([v, -v])
    v = torch.nn.functional.pad(v, (0, -v.numel() % 4096)).view(-1, 4096).contiguous()
    v[:, 0] = 448.0
    x = v.cuda()
    out = torch.empty(x.shape, dtype=ref.F8, device="cuda")
    scale, rstd = torch.empty(x.shape[0], device="cuda"), torch.empty(x.shape[0], device="cuda")
    plr.plr_rmsnorm([x], torch.ones(4096, device="cuda"), out, out_scale=scale, rstd=rstd)
    y = x * rstd[:, None]
    m = y.abs().amax(-1)
    # a division (torch takes 448 / m as 448 times a rounded reciprocal)
    want = (y * torch.div(torch.full_like(m, 448.0), m)[:, None]).to(ref.F8)
    assert torch.equal(out.view(torch.uint8), want.view(torch.uint8))


def test_no_rows(plr):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    plr.plr_rmsnorm([x], g, torch.empty_like(x))
    dg = torch.full((64,), 3.0, device="cuda")
    ws = torch.empty(plr.plr_rmsnorm_backward_workspace_bytes("bf16", 0, 64), dtype=torch.uint8, device="cuda")
    plr.plr_rmsnorm_backward(x, x, g, torch.empty(0, device="cuda"), torch.empty_like(x), dg, ws)
    torch.cuda.synchronize()
    assert (dg == 0).all()


@pytest.mark.parametrize("dt", ref.DTYPES, ids=ref.ids)
def test_no_rows_in_8_bits(plr, dt):
    x = torch.empty(0, 64, dtype=dt, device="cuda")
    plr.plr_rmsnorm([x, x], torch.ones(64, dtype=dt, device="cuda"), torch.empty(0, 64, dtype=ref.F8, device="cuda"),
                    residual=x, sum_out=torch.empty_like(x), out_scale=torch.empty(0, device="cuda"),
                    rstd=torch.empty(0, device="cuda"))
    torch.cuda.synchronize()


def _backward(plr, dout, h, gamma, rstd, dsum, dx=None):
    R, C = h.shape
    dx = torch.empty(R, C, dtype=h.dtype, device="cuda") if dx is None else dx
    dg = torch.full((C,), 9.0, device="cuda")
    ws = torch.empty(plr.plr_rmsnorm_backward_workspace_bytes(h.dtype, R, C), dtype=torch.uint8, device="cuda")
    plr.plr_rmsnorm_backward(dout, h, gamma, rstd, dx, dg, ws, dsum=dsum)
    torch.cuda.synchronize()
    return dx, dg


def _check_backward(got, dout, h, gamma, rstd, dsum):
    dx, dg = got
    want, want_g = ref.norm_backward(dout, h, gamma, rstd, dsum)
    d, x, g, r = dout.cpu().double(), h.cpu().double(), gamma.cpu().double(), rstd.cpu().double()[:, None]
    # the row's sum is off by at most 64 roundings of its terms' magnitudes
    terms = r * ((d * g).abs() + (x * r).abs() * (d * g * x * r).abs().mean(-1, keepdim=True))
    slack = 64 * ref.U32 * terms + (2 * ref.U32 * dsum.cpu().double().abs() if dsum is not None else 0)
    ref.assert_within(dx, want, slack, h.dtype, "dx")
    n = min(h.shape[0], 64) + 24  # additions on the way to one of dgamma's sums: rows of a workgroup, then a run
    ref.assert_within(dg, want_g, n * ref.U32 * (d * x * r).abs().sum(0), torch.float32, "dgamma")


@pytest.mark.parametrize("R,C", [(1, 16), (2, 7168), (7, 1008), (3, 8208), (2, 16384), (1500, 272), (1025, 1024)])
@pytest.mark.parametrize("dt", ref.DTYPES, ids=ref.ids)
def test_backward(plr, dt, R, C):
    h, dout = _rand(1, (R, C), dt, 2.0), _rand(2, (R, C), dt)
    gamma = _rand(3, (C,), dt)
    dsum = _rand(4, (R, C), dt) if R % 2 else None
    rstd = torch.rsqrt(h.float().square().mean(-1) + EPS)
    _check_backward(_backward(plr, dout, h, gamma, rstd, dsum), dout, h, gamma, rstd, dsum)


def test_backward_in_place_and_repeatable(plr):
    h, dout, dsum = (_rand(s, (600, 512), torch.bfloat16) for s in (1, 2, 3))
    gamma = _rand(4, (512,), torch.bfloat16)
    rstd = torch.rsqrt(h.float().square().mean(-1) + EPS)
    dx, dg = _backward(plr, dout, h, gamma, rstd, dsum)
    own = dsum.clone()
    dx2, dg2 = _backward(plr, dout, h, gamma, rstd, own, dx=own)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)


def test_gradient_against_differences(plr):
    # loss = <dout, out> + <dsum, sum>: its slope along a direction, in binary32. The
    # difference quotient's own error: the curvature (of the order of the slope times step^2)
    # and binary32 rounding of the outputs over the step, 2^-23 * sqrt(terms) / 2^-7
    R, C, step = 4, 512, 2.0 ** -7
    srcs = [_rand(1 + w, (R, C), torch.float32) for w in range(2)]
    res, gamma = _rand(7, (R, C), torch.float32), _rand(8, (C,), torch.float32)
    dout, dsum = _rand(9, (R, C), torch.float32), _rand(10, (R, C), torch.float32)
    u, v = _rand(11, (R, C), torch.float32), _rand(12, (C,), torch.float32)

    def loss(x0, gm):
        s, out, _, _ = _run(plr, [x0, srcs[1]], gm, torch.float32, res)
        return float((dout.double() * out.double()).sum() + (dsum.double() * s.double()).sum())

    s, out, _, rstd = _run(plr, srcs, gamma, torch.float32, res)
    dx, dg = _backward(plr, dout, s, gamma, rstd, dsum)
    got = (loss(srcs[0] + step * u, gamma) - loss(srcs[0] - step * u, gamma)) / (2 * step)
    scale = float((dx.double() * u.double()).abs().sum())
    assert abs(got - float((dx.double() * u.double()).sum())) <= scale * (step ** 2 + 1e-5)
    got = (loss(srcs[0], gamma + step * v) - loss(srcs[0], gamma - step * v)) / (2 * step)
    scale = float((dg.double() * v.double()).abs().sum())
    assert abs(got - float((dg.double() * v.double()).sum())) <= scale * 1e-4


def test_on_another_stream(plr):
    s = torch.cuda.Stream()
    x, gamma = _rand(1, (64, 7168), torch.bfloat16), _rand(2, (7168,), torch.bfloat16)
    a, b = torch.empty_like(x), torch.empty_like(x)
    plr.plr_rmsnorm([x], gamma, a)
    s.wait_stream(torch.cuda.current_stream())
    plr.plr_rmsnorm([x], gamma, b, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("W", [1, 3, 8, 16])
def test_many_long_rows(plr, W, f8):
    # more rows than compute units and more than 128 vectors: two vectors a thread
    dt = ref.DTYPES[W % 3]
    srcs = [_rand(40 + w, (300, 4112), dt, 0.5) for w in range(W)]
    res, gamma = _rand(3, (300, 4112), dt), _rand(4, (4112,), dt)
    out_dt = ref.F8 if f8 else dt
    _check(_run(plr, srcs, gamma, out_dt, res), ref.norm(srcs, res, gamma, EPS), dt, out_dt)


@pytest.mark.parametrize("f8", [False, True])
def test_more_rows_than_workgroups(plr, f8):
    # 2^20 workgroups, one wave each: some take a second row; and two waves each, which share sums
    for R, C in (((1 << 20) + 5, 16), ((1 << 20) + 3, 528)):
        x, gamma = _rand(1, (R, 16), torch.bfloat16), _rand(2, (C,), torch.bfloat16)
        x = x.repeat(1, C // 16)
        out_dt = ref.F8 if f8 else torch.bfloat16
        got = _run(plr, [x], gamma, out_dt)
        for a in (0, R // 2, R - 4096):  # these rows in 64 bits, all rows against calls of fewer
            part = slice(a, a + 4096)
            _check([t if t is None else t[part] for t in got], ref.norm([x[part]], None, gamma, EPS), torch.bfloat16, out_dt)
        for a in range(0, R, 1 << 18):
            part = slice(a, a + (1 << 18))
            for t, u in zip(got, _run(plr, [x[part]], gamma, out_dt)):
                assert t is None and u is None or torch.equal(t[part].view(torch.uint8), u.view(torch.uint8))


@pytest.mark.parametrize("dt,C", [(torch.bfloat16, 32768), (torch.float16, 32768), (torch.float32, 16384)],
                         ids=lambda v: ref.ids(v) if isinstance(v, torch.dtype) else str(v))
def test_backward_of_the_longest_rows(plr, dt, C):
    h, dout, dsum = (_rand(s, (3, C), dt) for s in (1, 2, 4))
    gamma = _rand(3, (C,), dt)
    rstd = torch.rsqrt(h.float().square().mean(-1) + EPS)
    _check_backward(_backward(plr, dout, h, gamma, rstd, dsum), dout, h, gamma, rstd, dsum)
