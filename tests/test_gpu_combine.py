"""plr_combine and its gradient against 64 bits: every type, slot counts on both sides of
each launch shape, empty slots, tokens with none, rows apart, rows past the last."""
import math

import pytest
import torch

import blockref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def plr():
    assert torch.cuda.is_available(), "the GPU tests need a GPU"
    import reduce_atom_amd

    return reduce_atom_amd


def _case(seed, T, k, C, dt, drop=0.2):
    g = torch.Generator().manual_seed(seed)
    y = torch.randn(T * k, C, generator=g).to(dt)
    pos = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k)
    pos[torch.rand(T, k, generator=g) < drop] = -1
    w = torch.randn(T, k, generator=g)
    w[pos < 0] = math.nan  # an empty slot's weight is not looked at
    named = torch.zeros(T * k, dtype=torch.bool)
    named[pos[pos >= 0].long()] = True
    y[~named] = math.nan   # nor is a row that no slot names
    return y.cuda(), pos.cuda(), w.cuda(), named


SHAPES = [(1, 1, 8), (1, 2, 7168), (3, 3, 264), (17, 4, 2048), (9, 5, 2056), (40, 8, 7168), (5, 9, 136), (6, 16, 1000)]


@pytest.mark.parametrize("T,k,C", SHAPES)
@pytest.mark.parametrize("dt", ref.DTYPES, ids=ref.ids)
def test_forward(plr, dt, T, k, C):
    y, pos, w, _ = _case(T + k, T, k, C, dt)
    pos[0] = -1  # a token with no row at all
    out = torch.full((T, C), 3.0, device="cuda").to(dt)
    plr.plr_combine(y, pos, w, out)
    want, mag = ref.combine(y, pos, w, T)
    ref.assert_within(out, want, (k + 1) * ref.U32 * mag, dt, "out")
    assert (out[0] == 0).all()
    pos[0] = torch.arange(k) * 0 + T * k  # past the last row: empty too
    if T > 1:
        pos[1, 0] = -5
    plr.plr_combine(y, pos, None, out)
    want, mag = ref.combine(y, pos, None, T)
    ref.assert_within(out, want, (k + 1) * ref.U32 * mag, dt, "unweighted")


def test_sum_follows_the_slots(plr):
    y = torch.tensor([2.0 ** 24, 1.0, 1.0], device="cuda")[:, None].expand(3, 8).contiguous()
    out = torch.empty(2, 8, device="cuda")
    pos = torch.tensor([[0, 1, 2], [1, 2, 0]], dtype=torch.int32, device="cuda")
    plr.plr_combine(y, pos, None, out)
    assert (out[0] == 2.0 ** 24).all() and (out[1] == 2.0 ** 24 + 2).all()


@pytest.mark.parametrize("T,k,C", SHAPES)
@pytest.mark.parametrize("dt", ref.DTYPES, ids=ref.ids)
def test_backward(plr, dt, T, k, C):
    y, pos, w, named = _case(2 * T + k, T, k, C, dt)
    dout = torch.randn(T, C, generator=torch.Generator().manual_seed(5)).to(dt).cuda()
    dy = torch.full((T * k, C), 3.0, device="cuda").to(dt)
    dw = torch.full((T, k), math.nan, device="cuda")
    plr.plr_combine_backward(dout, y, pos, w, dy, dw)
    torch.cuda.synchronize()
    p, d = pos.cpu().long(), dout.cpu().double()
    want = torch.full((T * k, C), 3.0, dtype=torch.float64)
    want_w, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if p[t, j] >= 0:
                want[p[t, j]] = w[t, j].cpu().double() * d[t]
                prod = d[t] * y[p[t, j]].cpu().double()
                want_w[t, j], mag[t, j] = prod.sum(), prod.abs().sum()
    ref.assert_within(dy, want, ref.U32 * want.abs(), dt, "dy")
    assert (dy[~named.cuda()] == 3.0).all()
    # a thread adds C / 256 rounded up products of its vectors, then the wave and the waves
    n = (C // 256 + 8) + 16
    ref.assert_within(dw, want_w, n * ref.U32 * mag, torch.float32, "dweights")
    # without dweights, y is not needed; ones without weights; dy in y's place
    dy2 = torch.full_like(dy, 3.0)
    plr.plr_combine_backward(dout, None, pos, w, dy2, None)
    assert torch.equal(dy2, dy)
    own = torch.where(named.cuda()[:, None], y, torch.full_like(y, 3.0))
    dw2 = torch.empty_like(dw)
    plr.plr_combine_backward(dout, own, pos, w, own, dw2)
    assert torch.equal(own, dy) and torch.equal(dw2, dw)
    plr.plr_combine_backward(dout, None, pos, None, dy2, None)
    for t in range(min(T, 4)):
        for j in range(k):
            if p[t, j] >= 0:
                assert torch.equal(dy2[p[t, j]], dout[t])


def test_rows_apart(plr):
    y, pos, w, _ = _case(1, 12, 3, 512, torch.bfloat16, drop=0)
    wide = torch.full((36, 1024), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 256:768] = y
    dest = torch.full((12, 1024), 5.0, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(12, 512, dtype=torch.bfloat16, device="cuda")
    plr.plr_combine(y, pos, w, out)
    plr.plr_combine(wide[:, 256:768], pos, w, dest[:, 8:520])
    assert torch.equal(dest[:, 8:520], out)
    assert (dest[:, :8] == 5).all() and (dest[:, 520:] == 5).all()


def test_gradient_is_the_transpose(plr):
    # the forward is linear in y: <dout, combine(y)> = <dy, y>, and the slope in w is dweights
    y, pos, w, _ = _case(3, 10, 4, 256, torch.float32, drop=0)
    dout = torch.randn(10, 256, generator=torch.Generator().manual_seed(5)).cuda()
    out, dy, dw = torch.empty(10, 256, device="cuda"), torch.empty_like(y), torch.empty_like(w)
    plr.plr_combine(y, pos, w, out)
    plr.plr_combine_backward(dout, y, pos, w, dy, dw)
    lhs = (dout.double() * out.double()).sum()
    mag = (dy.double() * y.double()).abs().sum()
    assert abs(lhs - (dy.double() * y.double()).sum()) <= 16 * ref.U32 * mag
    v = torch.randn(10, 4, generator=torch.Generator().manual_seed(6)).cuda()
    hi, lo = torch.empty_like(out), torch.empty_like(out)
    plr.plr_combine(y, pos, w + v, hi)
    plr.plr_combine(y, pos, w - v, lo)
    got = (dout.double() * (hi.double() - lo.double())).sum() / 2
    assert abs(got - (dw.double() * v.double()).sum()) <= 16 * ref.U32 * (mag + (dw * v).double().abs().sum()) * 4


def test_no_tokens(plr):
    out = torch.empty(0, 64, device="cuda")
    plr.plr_combine(torch.ones(4, 64, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"), None, out)
    # no rows to take: every slot is empty
    out = torch.full((3, 64), 2.0, device="cuda")
    plr.plr_combine(torch.empty(0, 64, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), None, out)
    assert (out == 0).all()


@pytest.mark.parametrize("k,dt", [(2, torch.float32), (3, torch.bfloat16), (5, torch.float16), (9, torch.bfloat16)],
                         ids=str)
def test_more_tokens_than_workgroups(plr, k, dt):
    # some workgroups take a second token; one vector a row, so that the lanes that hold a token's slots
    # have, but for the first, no column of their own. Whole numbers: equal in any type
    T, C = (1 << 20) + 5, 16 // dt.itemsize
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randint(-3, 4, (T * k, C), generator=g, device="cuda").to(dt)
    pos = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    pos[torch.rand(T, k, generator=g, device="cuda") < 0.2] = -1
    w = torch.randint(-2, 3, (T, k), generator=g, device="cuda").float()
    kept = pos >= 0
    rows = torch.where(kept[..., None], y[pos.clamp_min(0).long()].float(), torch.zeros(1, device="cuda"))
    out = torch.full((T, C), 77.0, dtype=dt, device="cuda")
    plr.plr_combine(y, pos, w, out)
    assert torch.equal(out.float(), (rows * w[..., None]).sum(1))
    dout = torch.randint(-3, 4, (T, C), generator=g, device="cuda").to(dt)
    dy = torch.full((T * k, C), 77.0, dtype=dt, device="cuda")
    dw = torch.full((T, k), 77.0, device="cuda")
    plr.plr_combine_backward(dout, y, pos, w, dy, dw)
    want = torch.full((T * k, C), 77.0, device="cuda")
    want[pos[kept].long()] = (w[..., None] * dout.float()[:, None])[kept]
    assert torch.equal(dy.float(), want)
    assert torch.equal(dw, (rows * dout.float()[:, None]).sum(-1))


def test_more_parts_of_rows_than_workgroups(plr):
    # rows of two parts (128 vectors and one): 2^19 tokens at once
    T, C = (1 << 19) + 3, 1032
    y = torch.randint(-9, 10, (50, C), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    pos = torch.randint(-1, 50, (T, 1), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    out = torch.full((T, C), 77.0, dtype=torch.bfloat16, device="cuda")
    plr.plr_combine(y, pos, None, out)
    want = torch.cat([y, torch.zeros_like(y[:1])])[pos[:, 0].long()]  # -1: the row of zeros
    assert torch.equal(out, want)
