"""plr_route against plain loops (ids, positions, row_token and offsets exactly) at every
launch shape, with ties, masked experts, tokens without any, and its gradient."""
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


def _run(plr, logits, k):
    T, E = logits.shape
    i32 = {"dtype": torch.int32, "device": "cuda"}
    ids, pos = torch.full((T, k), -7, **i32), torch.full((T, k), -7, **i32)
    rt = torch.full((T * k,), -7, **i32)
    w = torch.full((T, k), math.nan, device="cuda")
    off = torch.full((E + 1,), -7, dtype=torch.int64, device="cuda")
    ws = torch.full((plr.plr_route_workspace_bytes(T, E),), 0x5A, dtype=torch.uint8, device="cuda")
    plr.plr_route(logits, ids, w, pos, rt, off, ws)
    torch.cuda.synchronize()
    return ids, w, pos, rt, off


def _check(plr, logits, k):
    got = _run(plr, logits, k)
    want = ref.route(logits, k)
    for name, g, r in zip(("ids", "weights", "positions", "row_token", "offsets"), got, want):
        if name != "weights":
            assert torch.equal(g.cpu(), r), name
    # expf and a division are good to a few units each, the sum of k <= 16 terms to 4 additions
    ref.assert_within(got[1], want[1], 16 * ref.U32 * want[1], torch.float32, "weights")
    return got


def _logits(seed, T, E, dt, step=None):
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(seed))
    if step:
        x = (x / step).round() * step  # many ties
    return x.to(dt).cuda()


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130, 1100])
@pytest.mark.parametrize("E,k", [(1, 1), (3, 4), (8, 2), (60, 6), (64, 4), (65, 8), (256, 8), (257, 3), (1000, 16), (1024, 1)])
def test_forward(plr, T, E, k):
    _check(plr, _logits(T + E, T, E, ref.DTYPES[(T + E) % 3]), k)


@pytest.mark.parametrize("dt", ref.DTYPES, ids=ref.ids)
def test_ties_take_the_lowest(plr, dt):
    for E in (48, 200, 700):
        _check(plr, _logits(1, 150, E, dt, step=1.0), 8)
    same = torch.zeros(70, 96, dtype=dt, device="cuda")
    same[::2] = -0.0
    ids = _check(plr, same, 5)[0]
    assert (ids.cpu() == torch.arange(5, dtype=torch.int32)).all()


def test_signed_zeros_are_equal(plr):
    x = torch.full((1, 8), -1.0, device="cuda")
    x[0, 2], x[0, 5] = -0.0, 0.0
    ids = _run(plr, x, 2)[0]
    assert ids.tolist() == [[2, 5]]


@pytest.mark.parametrize("T", [40, 200])
def test_masked_experts_and_tokens(plr, T):
    x = _logits(3, T, 32, torch.float32)
    x[::3, 4:] = -math.inf  # 4 experts left
    x[::7] = -math.inf      # none
    x[5, :30] = math.nan    # NaN is never chosen
    x[6] = -3.4e38          # the lowest value is still a value
    x[8] = torch.finfo(torch.float32).max
    _check(plr, x, 6)


def test_one_expert_takes_all(plr):
    x = _logits(5, 500, 64, torch.bfloat16)
    x[:, 37] = 100.0
    off = _check(plr, x, 1)[4]
    assert off[37] == 0 and off[38] == 500


def test_infinity_makes_nan_weights(plr):
    x = _logits(6, 3, 16, torch.float32)
    x[1, 9] = math.inf
    ids, w, *_ = _run(plr, x, 2)
    assert ids[1, 0] == 9 and w[1, 0].isnan() and w[0].isfinite().all() and w[2].isfinite().all()


def test_rows_apart_and_unaligned(plr):
    wide = _logits(7, 90, 101, torch.bfloat16)
    x = wide[:, 3:64]
    want = _check(plr, x.contiguous(), 4)
    for a, b in zip(_run(plr, x, 4), want):
        assert torch.equal(a, b)


def test_no_tokens(plr):
    off = _run(plr, torch.empty(0, 16, device="cuda"), 2)[4]
    assert (off == 0).all()


def test_many_tokens(plr):
    # 300 workgroups: positions against a stable sort
    x = _logits(8, 19200 - 5, 256, torch.bfloat16)
    k = 8
    ids, w, pos, rt, off = _run(plr, x, k)
    flat = ids.reshape(-1).long()
    by = torch.argsort(flat, stable=True)
    assert torch.equal(rt.long(), by // k)
    want = torch.empty_like(by)
    want[by] = torch.arange(by.numel(), device="cuda")
    assert torch.equal(pos.reshape(-1).long(), want)
    counts = torch.bincount(flat, minlength=256)
    assert torch.equal(off[1:], counts.cumsum(0))
    assert torch.equal(x.gather(1, ids.long()).float(), x.float().sort(-1, descending=True).values[:, :k])


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (33, 64, 4), (70, 250, 8), (3, 1024, 16)])
@pytest.mark.parametrize("dt", ref.DTYPES, ids=ref.ids)
def test_backward(plr, dt, T, E, k):
    x = _logits(T, T, E, torch.float32)
    x[0, E // 2:] = -math.inf
    ids, w, *_ = _run(plr, x, k)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    dw[ids < 0] = math.nan  # not looked at
    wide = torch.full((T, (E + 16) // 8 * 8), 5.0, device="cuda").to(dt)
    for dl in (torch.full((T, E), 3.0, device="cuda").to(dt), wide[:, :E]):
        plr.plr_route_backward(ids, w, dw, dl)
        torch.cuda.synchronize()
        want = ref.route_backward(ids, w, dw, E)
        mag = w.cpu().double().max() * torch.nan_to_num(dw.cpu().double()).abs().sum(-1, keepdim=True)
        ref.assert_within(dl, want, torch.where(want != 0, 8 * ref.U32 * mag, torch.zeros_like(want)), dt, "dlogits")
    assert (wide[:, E:] == 5.0).all()


def test_gradient_against_differences(plr):
    T, E, k, step = 6, 24, 4, 2.0 ** -8
    x = _logits(2, T, E, torch.float32)
    ids, w, *_ = _run(plr, x, k)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(3)).cuda()
    dl = torch.empty(T, E, device="cuda")
    plr.plr_route_backward(ids, w, dw, dl)
    u = torch.zeros(T, E, device="cuda")
    u.scatter_(1, ids.long(), torch.randn(T, k, generator=torch.Generator().manual_seed(4)).cuda())
    u.clamp_(-1, 1)

    def loss(z):
        i, p, *_ = _run(plr, z, k)
        at = torch.zeros(T, E, device="cuda", dtype=torch.float64)
        at.scatter_(1, i.long(), p.double())
        want = torch.zeros(T, E, device="cuda", dtype=torch.float64)
        want.scatter_(1, ids.long(), dw.double())
        assert torch.equal(i.sort(-1).values, ids.sort(-1).values)
        return float((at * want).sum())

    got = (loss(x + step * u) - loss(x - step * u)) / (2 * step)
    scale = float(dw.abs().sum())
    # a softmax's third derivative is below 1: step^2, and binary32 weights over the step
    assert abs(got - float((dl.double() * u.double()).sum())) <= scale * (step ** 2 + 2.0 ** -23 / step)


@pytest.mark.parametrize("E,k,dt", [(256, 8, torch.bfloat16), (60, 3, torch.float32)], ids=str)
def test_more_workgroups_than_counts_kept(plr, E, k, dt):
    # 1094 workgroups: 18 to a thread of the prefix sums, which keeps 8 counts in registers
    x = _logits(9, 70001, E, dt)
    x[::5] = -math.inf  # tokens without an expert
    ids, w, pos, rt, off = _run(plr, x, k)
    flat = torch.where(ids < 0, E, ids).reshape(-1).long()
    n = int((flat < E).sum())
    by = torch.argsort(flat, stable=True)
    want = torch.full_like(by, -1)
    want[by[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(pos.reshape(-1).long(), want)
    assert torch.equal(rt[:n].long(), by[:n] // k) and (rt[n:] == -1).all()
    assert off[0] == 0 and torch.equal(off[1:], torch.bincount(flat, minlength=E + 1)[:E].cumsum(0))
    assert torch.equal(ids[::5], torch.full_like(ids[::5], -1))
    live = torch.ones(len(x), dtype=torch.bool, device="cuda")
    live[::5] = False
    assert torch.equal(x[live].gather(1, ids[live].long()).float(), x[live].float().sort(-1, descending=True).values[:, :k])
