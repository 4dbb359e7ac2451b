"""GPU parity of the expert selection, counts, balance loss and gradient
against 64-bit definitions."""
import math

import pytest
import torch

import block_reference as ref
import vq_dequant_matmul_amd as vq
from block_reference import HALF_STEP, U, d

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def _logits(t, e, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((t, e), generator=g)).to(dtype)


def _mask(t, seed):
    return torch.rand((t,), generator=torch.Generator().manual_seed(seed)) < 0.7


def _c(t):
    return None if t is None else t.cuda()


def _weight_bound(logits, e, k):
    # exp's argument is off by half a step of up to the row's spread, exp and
    # the sums of up to E terms in lanes (E/64 + 6) by their roundings
    l = d(logits).masked_fill(~torch.isfinite(d(logits)), 0.0)
    spread = l.amax(1, keepdim=True) - l.amin(1, keepdim=True) + l.abs().amax(1, keepdim=True)
    return (spread + e / 64 + 6 + 10) * U


CASES = [  # tokens, experts, k
    (1, 1, 1), (1, 512, 10), (3, 8, 8), (5, 63, 4), (2, 64, 64), (130, 65, 7), (67, 128, 8),
    (257, 300, 1), (33, 512, 10), (9, 1024, 64), (4097, 16, 2), (1, 1000, 13),
]


@pytest.mark.parametrize("t,e,k", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid,renorm,biased", [(False, True, False), (False, False, True),
                                                   (True, True, True), (True, False, False)])
def test_route(t, e, k, dtype, sigmoid, renorm, biased):
    logits = _logits(t, e, dtype, t + e)
    bias = 0.1 * torch.randn((e,), generator=torch.Generator().manual_seed(2)) if biased else None
    mask = _mask(t, 5) if t > 1 else None
    if mask is not None:
        logits[~mask] = NAN
    kw = dict(score=int(sigmoid), renormalize=renorm, scale=2.5, bias=_c(bias), mask=_c(mask))
    ids, w, counts, loss = vq.vq_moe_route(logits.cuda(), k, balance=True, **kw)
    ids2, w2 = vq.vq_moe_route(logits.cuda(), k, **kw)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    ri, rw, rc, rl = ref.route(logits, k, sigmoid, renorm, 2.5, bias, mask)
    assert torch.equal(ids.cpu().long(), ri)
    assert torch.equal(counts.cpu().long(), rc)
    err = (d(w) - rw).abs()
    assert (err <= _weight_bound(logits, e, k) * rw + 1e-38).all(), (err / rw).max()
    # the loss: p's relative error, then sums of positive terms, at most
    # tokens/4 + 512 of them after one another
    rel = _weight_bound(logits, e, k).max() + (t / 4 + 512) * U
    assert abs(float(loss) - float(rl)) <= rel * float(rl)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_route_special_rows(sigmoid, biased):
    """Equal logits, -0 against 0, the type's lowest value, -inf, rows of -inf
    only, fewer live experts than slots, masked NaN and inf."""
    e, k = 70, 4
    low = torch.finfo(torch.float32).min
    rows = torch.zeros((12, e))
    rows[1, ::2] = -0.0
    rows[2] = -INF
    rows[3] = -INF
    rows[3, 69] = 1.0
    rows[4] = low
    rows[5] = low
    rows[5, [7, 66]] = 3.0
    rows[6] = 1e30
    rows[7] = NAN
    rows[8] = INF
    rows[9, 5:] = -INF
    rows[10, 3] = 1e4
    rows[11] = torch.linspace(-200, -150, e)
    mask = torch.ones(12, dtype=torch.uint8)
    mask[7] = mask[8] = 0
    bias = torch.zeros(e) if biased else None
    out = vq.vq_moe_route(rows.cuda(), k, score=int(sigmoid), bias=_c(bias), mask=mask.cuda(),
                          balance=True)
    ri, rw, rc, rl = ref.route(rows, k, sigmoid, True, 1.0, bias, mask)
    live = [0, 1, 2, 3, 5, 7, 8, 9, 10] if sigmoid and biased else range(12)
    # (scores that underflow to equal values differ in fp64's own range only)
    assert torch.equal(out[0].cpu().long()[live], ri[live])
    good = [i for i in live if not (sigmoid and i in (4, 11))]
    assert torch.allclose(d(out[1])[good], rw[good], rtol=2 ** -16, atol=2.0 ** -126)
    assert int(out[2].sum()) == int(rc.sum())
    assert torch.isfinite(out[3]).all()
    ids = out[0].cpu()
    assert all(len(set(r.tolist())) == k for r in ids) and ids.min() >= 0 and ids.max() < e


def test_route_nan_row_keeps_ids_in_range():
    rows = torch.zeros((3, 40))
    rows[1, 5:] = NAN
    rows[2] = NAN
    for biased in (None, torch.zeros(40).cuda()):
        ids, w = vq.vq_moe_route(rows.cuda(), 8, bias=biased, renormalize=False)
        ids = ids.cpu()
        assert all(len(set(r.tolist())) == 8 for r in ids) and ids.min() >= 0 and ids.max() < 40
        assert torch.isfinite(w[0]).all() and w[1].isnan().any() and w[2].isnan().all()


def test_route_near_ties_with_bias():
    """Keys a few 2^-40 apart: fp32 sums could not tell them apart."""
    e = 32
    logits = torch.zeros((64, e))
    bias = torch.zeros(e)
    g = torch.Generator().manual_seed(0)
    for t in range(64):
        logits[t] = torch.randperm(e, generator=g).float() * 2.0 ** -40 + (t % 3)
    for sigmoid in (False, True):
        ids, _ = vq.vq_moe_route(logits.cuda(), 6, score=int(sigmoid), bias=bias.cuda())
        assert torch.equal(ids.cpu().long(), ref.route(logits, 6, sigmoid, bias=bias)[0])


@pytest.mark.parametrize("n", [0, 3])
def test_route_nothing_counts(n):
    logits = torch.full((n, 20), NAN).cuda()
    mask = torch.zeros((n,), dtype=torch.bool).cuda()
    ids, w, counts, loss = vq.vq_moe_route(logits, 3, mask=mask, balance=True)
    assert (counts == 0).all() and float(loss) == 0.0 and (w == 0).all()
    assert ids.tolist() == [[0, 1, 2]] * n
    g = vq.vq_moe_route_grad(logits, ids, torch.ones_like(w), mask=mask, counts=counts,
                             d_loss=torch.ones(1).cuda())
    assert g.shape == (n, 20) and (g == 0).all()


@pytest.mark.parametrize("t,e,k", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid,renorm", [(False, True), (False, False), (True, True),
                                            (True, False)])
@pytest.mark.parametrize("parts", ["both", "weights", "loss"])
def test_route_grad(t, e, k, dtype, sigmoid, renorm, parts):
    logits = _logits(t, e, dtype, 3 * t + e)
    if e > k + 2:
        logits[:, e // 2] = -INF
    mask = _mask(t, 8) if t > 1 else None
    ids, _, counts, _ = ref.route(logits, k, sigmoid, renorm, 2.5, None, mask)
    g = torch.Generator().manual_seed(e)
    dw = torch.randn((t, k), generator=g) if parts != "loss" else None
    counts = counts if parts != "weights" else None
    dl = 0.3
    got = vq.vq_moe_route_grad(
        logits.cuda(), ids.int().cuda(), _c(dw), score=int(sigmoid), renormalize=renorm,
        scale=2.5, mask=_c(mask), counts=None if counts is None else counts.int().cuda(),
        d_loss=None if counts is None else torch.tensor([dl]).cuda())
    assert got.dtype == dtype and torch.isfinite(got).all()
    l = d(logits).requires_grad_()
    obj = ref.route_objective(l, ids, d(dw), counts, d(torch.tensor(dl)), sigmoid, renorm, 2.5,
                              mask)
    want = torch.zeros_like(l) if not obj.requires_grad else torch.autograd.grad(obj, l)[0]
    # magnitude of what is added and subtracted per element: the slot's own
    # gradient, p or w times the row's sum of |terms|
    with torch.no_grad():
        live = ref.live_rows(l, mask)[:, None]
        s, p = ref.scores(torch.where(live, l, torch.zeros_like(l)), sigmoid)
        mag = torch.zeros_like(l)
        if dw is not None:
            w = ref.weights(torch.where(live, l, torch.zeros_like(l)), ids, sigmoid, renorm, 2.5)
            a = (d(dw).abs() * w)
            mag.scatter_add_(1, ids, a + w / 2.5 * a.sum(1, keepdim=True))
            if not renorm and not sigmoid:
                mag += p * a.sum(1, keepdim=True)
        if counts is not None and counts.sum() > 0:
            f = dl * e * counts.double() / counts.sum() / (counts.sum() / k)
            mag += p * (f + (p * f).sum(1, keepdim=True))
        # 1 - s cancels near s = 1: its absolute error is a few half steps
        rel = (_weight_bound(logits, e, k) * 3 + 20 * U)
        bound = rel * mag + HALF_STEP[dtype] * want.abs() + 1e-38
    err = (d(got) - want).abs()
    assert (err <= bound).all(), (err / bound).max()
    dead = ~live.expand_as(l) | (l == -INF)
    assert (got.cpu()[dead] == 0).all()


def test_route_grad_against_differences():
    t, e, k = 24, 96, 6
    logits = _logits(t, e, torch.float32, 1, 1.0)
    ids, _, counts, _ = ref.route(logits, k)
    g = torch.Generator().manual_seed(2)
    dw = torch.randn((t, k), generator=g)
    got = d(vq.vq_moe_route_grad(logits.cuda(), ids.int().cuda(), dw.cuda(),
                                 counts=counts.int().cuda(), d_loss=torch.tensor([50.0]).cuda()))
    h = 1e-4
    for i in range(4):
        v = torch.randn((t, e), generator=g, dtype=torch.float64)

        def at(sign):
            return ref.route_objective(d(logits) + sign * h * v, ids, d(dw), counts, 50.0, False,
                                       True, 1.0, None)

        slope = float((at(1) - at(-1)) / (2 * h))
        size = float((got * v).abs().sum())
        # central differences: h^2 times third derivatives (below 1 each)
        assert abs(float((got * v).sum()) - slope) <= 2e-6 * size + 1e-6


def test_route_grad_repeated_and_bad_ids():
    """A repeated id adds up, an id out of range is left out."""
    logits = _logits(2, 10, torch.float32, 4).cuda()
    dw = torch.tensor([[1.0, 2.0, 0.5], [1.0, 2.0, 0.5]]).cuda()
    ids = torch.tensor([[3, 3, 1], [3, 10, -1]], dtype=torch.int32).cuda()
    got = vq.vq_moe_route_grad(logits, ids, dw, score=vq.VQ_SCORE_SIGMOID, renormalize=False)
    s = torch.sigmoid(d(logits))
    want = torch.zeros_like(s)
    want[0, 3], want[0, 1], want[1, 3] = 3.0, 0.5, 1.0
    want = want * s * (1 - s)
    assert torch.allclose(d(got), want, rtol=1e-6, atol=1e-12)


def test_route_repeats_and_graph():
    t, e, k = 700, 200, 6
    logits = _logits(t, e, torch.float32, 1).cuda()
    first = vq.vq_moe_route(logits, k, balance=True)
    for a, b in zip(first, vq.vq_moe_route(logits, k, balance=True)):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = vq.vq_moe_route(logits, k, balance=True)
        grad = vq.vq_moe_route_grad(logits, out[0], out[1], counts=out[2], d_loss=out[3])
    for i in range(3):
        logits.copy_(_logits(t, e, torch.float32, 20 + i))
        g.replay()
        want = vq.vq_moe_route(logits, k, balance=True)
        for a, b in zip(out, want):
            assert torch.equal(a, b), i
        assert torch.equal(grad, vq.vq_moe_route_grad(logits, want[0], want[1], counts=want[2],
                                                      d_loss=want[3]))


def test_route_binding_refuses():
    l = torch.zeros((4, 8)).cuda()
    with pytest.raises(vq.VQError, match="top_k"):
        vq.vq_moe_route(l, 9)
    with pytest.raises(ValueError, match="bias"):
        vq.vq_moe_route(l, 2, bias=torch.zeros(9).cuda())
    with pytest.raises(ValueError, match="mask"):
        vq.vq_moe_route(l, 2, mask=torch.ones(4).cuda())
    with pytest.raises(ValueError, match="contiguous"):
        vq.vq_moe_route(l[:, :6], 2)
    with pytest.raises(TypeError):
        vq.vq_moe_route(l.half(), 2)
    with pytest.raises(vq.VQError, match="workspace"):
        vq.vq_moe_route(l, 2, balance=True, workspace=torch.empty(16, dtype=torch.uint8).cuda())


@pytest.mark.parametrize("e,k", [(512, 10), (1000, 64), (128, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_route_keys_that_lie_close(e, k, sigmoid, biased):
    """More keys near the border than lanes: all equal, two values, a narrow
    band, a few large ones among equal ones."""
    g = torch.Generator().manual_seed(e)
    rows = torch.zeros((6, e))
    rows[1] = (torch.rand((e,), generator=g) < 0.5).float()
    rows[2] = 1.0 + 1e-6 * torch.randn((e,), generator=g)
    rows[3, ::7] = 2.0
    rows[4] = torch.randint(0, 3, (e,), generator=g).float()
    rows[5] = -60.0 + 2.0 * torch.randn((e,), generator=g)
    bias = (torch.randint(0, 2, (e,), generator=g).float() * 0.25) if biased else None
    ids, w = vq.vq_moe_route(rows.cuda(), k, score=int(sigmoid), bias=_c(bias))
    ri, rw, _, _ = ref.route(rows, k, sigmoid, bias=bias)
    assert torch.equal(ids.cpu().long(), ri)
    assert torch.allclose(d(w), rw, rtol=2 ** -16, atol=0)


def test_route_calls_on_two_streams():
    """Two calls at once, each with its own workspace."""
    logits = [_logits(3000, 256, torch.float32, i).cuda() for i in range(2)]
    want = [vq.vq_moe_route(l, 8, balance=True) for l in logits]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(vq.vq_moe_route(logits[i], 8, balance=True))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("base", [-20.0, -60.0, -84.0])
def test_route_small_scores_in_order(sigmoid, base):
    """A bias of zeros adds nothing to tell scores of 1e-9 to 1e-37 apart: logits
    one to a few fp32 steps from each other keep their order."""
    e, k, g = 96, 24, torch.Generator().manual_seed(int(-base))
    step = 2.0 ** -18 if base == -20.0 else 2.0 ** -17
    rows = torch.stack([base + step * torch.randperm(e, generator=g).float() for _ in range(32)])
    rows[:, 5] = 0.0
    rows[16:] += step * torch.randint(0, 2, (16, e), generator=g).float() * (rows[16:] < -1)
    ids, _ = vq.vq_moe_route(rows.cuda(), k, score=int(sigmoid), bias=torch.zeros(e).cuda())
    assert torch.equal(ids.cpu().long(), ref.route(rows, k, sigmoid, bias=torch.zeros(e))[0])


def test_route_of_the_most_tokens():
    """2^31 - 1 tokens of one expert: offsets past 32 bits, every element written."""
    n = 2 ** 31 - 1
    logits = torch.zeros((n, 1), dtype=torch.bfloat16, device="cuda")
    ids, w, counts, loss = vq.vq_moe_route(logits, 1, balance=True)
    # every p is 1: exact in a wave's and a workgroup's sum (below 2^24), then up to
    # 32 roundings where the workgroups' sums meet
    assert counts.tolist() == [n] and abs(float(loss) - 1.0) <= 32 * U
    for out, value in ((ids, 0), (w, 1.0)):
        assert all((part == value).all() for part in out.split(1 << 28))
    ids, w = vq.vq_moe_route(logits, 1, score=vq.VQ_SCORE_SIGMOID, renormalize=False)
    assert all((part == 0).all() for part in ids.split(1 << 28))
    assert all((part == 0.5).all() for part in w.split(1 << 28))
    got = vq.vq_moe_route_grad(logits, ids, w, score=vq.VQ_SCORE_SIGMOID, renormalize=False)
    assert all((part == 0.125).all() for part in got.split(1 << 28))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("parts", ["weights", "loss"])
def test_sigmoid_gradient_of_large_logits(dtype, renorm, parts):
    """Scores next to 1: the gradient's factor 1 - s is as exact as the rest, so
    the bound scales with it."""
    t, e, k, dl = 50, 72, 6, 40.0
    g = torch.Generator().manual_seed(12)
    logits = (10 + 20 * torch.rand((t, e), generator=g)).to(dtype)
    logits[::3, 1::2] *= -1
    ids, _, counts, _ = ref.route(logits, k, True, renorm)
    dw = torch.randn((t, k), generator=g) if parts == "weights" else None
    counts = counts if parts == "loss" else None
    got = vq.vq_moe_route_grad(
        logits.cuda(), ids.int().cuda(), _c(dw), score=vq.VQ_SCORE_SIGMOID, renormalize=renorm,
        counts=None if counts is None else counts.int().cuda(),
        d_loss=None if counts is None else torch.tensor([dl]).cuda())
    l = d(logits)
    s, rest = torch.sigmoid(l), torch.sigmoid(-l)     # rest = 1 - s
    if parts == "weights":
        w = ref.weights(l, ids, True, renorm, 1.0)
        a = d(dw) * w
        sub = w * a.sum(1, keepdim=True) if renorm else 0.0 * a
        want = torch.zeros_like(l).scatter_add(1, ids, a - sub) * rest
        mag = torch.zeros_like(l).scatter_add(1, ids, a.abs() + (
            w * a.abs().sum(1, keepdim=True) if renorm else 0.0)) * rest
    else:
        p = s / s.sum(1, keepdim=True)
        f = dl * e * counts.double() / counts.sum() / t
        want = p * (f - (p * f).sum(1, keepdim=True)) * rest
        mag = p * (f + (p * f).sum(1, keepdim=True)) * rest
    # two exponentials, each off by its argument's half step (|logit| <= 30) and
    # its own, twice as much for the fast ones; sums of e terms in lanes, products
    bound = (4 * (30 + 4) + e / 16 + 6 + 20) * U * mag + HALF_STEP[dtype] * want.abs() + 1e-37
    err = (d(got) - want).abs()
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("base", [-80.0, -40.0, 30.0])
def test_loss_of_sigmoid_scores_far_from_0(base):
    """One token, whose choice the bias makes: the loss is n_experts * p of that
    expert, and p is as exact far from a logit of 0 as near it."""
    e = 8
    bias = torch.zeros(e)
    bias[3] = 10.0
    for seed in range(48):
        logits = base + torch.randn((1, e), generator=torch.Generator().manual_seed(seed))
        loss = vq.vq_moe_route(logits.cuda(), 1, score=vq.VQ_SCORE_SIGMOID, bias=bias.cuda(),
                               balance=True)[3]
        want = float(ref.route(logits, 1, True, bias=bias)[3])
        # a score: exp 4, its sum with 1 and the reciprocal 3, own and in the sum; the
        # sum over 8 experts, its reciprocal, the product and the result, in half steps
        assert abs(float(loss) - want) <= (7 + 7 + 7 + 4) * U * want, seed


@pytest.mark.parametrize("t", [1 << 16, (1 << 24) + 5])
def test_loss_of_equal_tokens(t):
    """The same p of every token: a rounding of one addition repeats in all."""
    e, k = 3, 1
    logits = torch.zeros((t, e), device="cuda")
    ids, _, counts, loss = vq.vq_moe_route(logits, k, balance=True)
    assert counts.tolist() == [t, 0, 0]
    # loss = 3 * p[0]: p has 3 roundings, 16 tokens are added in fp32, a workgroup's
    # sum and the result are rounded once
    assert abs(float(loss) - 1.0) <= (3 + 16 + 2) * U


def test_loss_shows_a_nan():
    """A NaN logit of one token that counts, wherever it is, and of one that does not."""
    t, e = 5000, 130
    logits = _logits(t, e, torch.float32, 3)
    for sigmoid in (0, 1):
        for row in (0, 17, 4999):
            bad = logits.clone()
            bad[row, 77] = NAN
            mask = torch.ones(t, dtype=torch.bool)
            assert vq.vq_moe_route(bad.cuda(), 4, score=sigmoid, balance=True)[3].isnan().all()
            mask[row] = False
            loss = vq.vq_moe_route(bad.cuda(), 4, score=sigmoid, mask=mask.cuda(), balance=True)[3]
            assert torch.isfinite(loss).all()


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(37, 128, 6), (9, 512, 10), (21, 1000, 8), (5, 64, 4)])
def test_logits_at_any_address(off, dtype, t, e, k):
    """Logits and their gradient that start between two vectors."""
    logits = _logits(t, e, dtype, off + e).cuda()
    buf = torch.zeros(t * e + 16, dtype=dtype, device="cuda")
    view = buf[off:off + t * e].view(t, e)
    view.copy_(logits)
    want = vq.vq_moe_route(logits, k, balance=True)
    got = vq.vq_moe_route(view, k, balance=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dw, dl = torch.ones_like(want[1]), torch.ones(1, device="cuda")
    kw = dict(counts=want[2], d_loss=dl)
    g = vq.vq_moe_route_grad(logits, want[0], dw, **kw)
    out = torch.full((t * e + 16,), 3.0, dtype=dtype, device="cuda")
    vq.vq_moe_route_grad(view, want[0], dw, out=out[off:off + t * e].view(t, e), **kw)
    assert torch.equal(out[off:off + t * e].view(t, e), g)
    assert (out[:off] == 3).all() and (out[off + t * e:] == 3).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("e", [40, 70, 300])
def test_route_special_rows_in_full(sigmoid, biased, e):
    """Every row's ids and weights, those with scores of 0 or 1 everywhere too."""
    k, low = 4, torch.finfo(torch.float32).min
    rows = torch.zeros((9, e))
    rows[0] = low
    rows[1] = 1e30
    rows[2] = torch.linspace(-200, -150, e)
    rows[3, 1::2] = -0.0
    rows[4, :] = -INF
    rows[4, e - 1] = 1.0
    rows[5] = low
    rows[5, [7, e - 4]] = 3.0
    rows[6, 5:] = -INF
    rows[7, 3] = 1e4
    rows[8] = torch.linspace(20, 40, e)
    bias = torch.zeros(e) if biased else None
    ids, w = vq.vq_moe_route(rows.cuda(), k, score=int(sigmoid), bias=_c(bias))
    ri, rw, _, _ = ref.route(rows, k, sigmoid, bias=bias)
    assert torch.equal(ids.cpu().long(), ri)
    if sigmoid:
        rw[[0, 2]] = 0.0   # below -88 a score is 0, and weights of a sum of 0 are 0
    # exp's argument by half a step of the chosen logits' distances (0 where the
    # result is 0), exp 2, the sum with 1, division, sum of four, division
    sel = d(rows).gather(1, ri)
    far = (sel[:, :1] - sel).nan_to_num(0.0, 0.0, 0.0).clamp(max=100.0)
    err = (d(w) - rw).abs()
    assert (err <= (far + 12) * U * rw).all(), (err / rw).max()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_loss_of_a_long_batch_repeats(sigmoid):
    """More tokens than a wave's first sixteen: the same bits eagerly, again, and in
    a graph whose inputs change, and the loss of the definition."""
    t, e, k = 70001, 130, 5
    logits = _logits(t, e, torch.float32, 9).cuda()
    mask = _mask(t, 3).cuda()
    kw = dict(score=int(sigmoid), mask=mask, balance=True)
    first = vq.vq_moe_route(logits, k, **kw)
    _, _, counts, loss = ref.route(logits.cpu(), k, sigmoid, mask=mask.cpu())
    assert torch.equal(first[2].cpu().long(), counts)
    # p: its exponentials (4, and half a step of a distance of 20 at most), its sum and
    # product, a sum of 16; two roundings of the sums
    assert abs(float(first[3]) - float(loss)) <= (20 + 8 + e / 64 + 6 + 4 + 16 + 2) * U * float(loss)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = vq.vq_moe_route(logits, k, **kw)
    for i in range(3):
        logits.copy_(_logits(t, e, torch.float32, 30 + i))
        g.replay()
        for a, b in zip(out, vq.vq_moe_route(logits, k, **kw)):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [10, 72, 200, 519, 764])
def test_gradient_of_a_single_renormalised_choice(sigmoid, dtype, e):
    """One slot's renormalised weight is 1 whatever the logits: its gradient is 0, and
    with the loss the gradient is that of the loss alone."""
    t = 203
    logits = _logits(t, e, dtype, e).cuda()
    ids, w, counts, _ = vq.vq_moe_route(logits, 1, score=int(sigmoid), balance=True)
    assert (w == 1).all()
    dw = _logits(t, 1, torch.float32, 2).cuda()
    kw = dict(score=int(sigmoid), scale=2.5)
    assert (vq.vq_moe_route_grad(logits, ids, dw, **kw) == 0).all()
    loss = dict(counts=counts, d_loss=torch.tensor([0.3]).cuda())
    assert torch.equal(vq.vq_moe_route_grad(logits, ids, dw, **kw, **loss),
                       vq.vq_moe_route_grad(logits, ids, None, **kw, **loss))


@pytest.mark.parametrize("e", [5, 400, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_loss_of_a_long_batch_at_every_width(e, dtype, sigmoid):
    """Past a wave's first sixteen tokens, p summed in 64 bits on the device; a NaN of
    an early token that counts shows, of one that does not, not."""
    t, k = 131073, 3
    logits = _logits(t, e, dtype, e).cuda()
    mask = _mask(t, 4).cuda()
    mask[17] = True
    kw = dict(score=int(sigmoid), balance=True)
    _, _, counts, loss = vq.vq_moe_route(logits, k, mask=mask, **kw)
    total = torch.zeros(e, dtype=torch.float64, device="cuda")
    for part, live in zip(logits.split(8192), mask.split(8192)):
        total += ref.scores(part[live].double(), sigmoid)[1].sum(0)
    n = int(mask.sum())
    assert int(counts.sum()) == n * k
    want = e * float((counts.double() * total).sum()) / (n * k) / n
    # p: as exact as a weight, whose bound is the largest here; 16 additions, two roundings
    # of sums
    assert abs(float(loss) - want) <= (20 + 8 + e / 64 + 6 + 4 + 16 + 2) * U * want
    logits[17, 2] = NAN
    assert vq.vq_moe_route(logits, k, mask=mask, **kw)[3].isnan().all()
    mask[17] = False
    assert torch.isfinite(vq.vq_moe_route(logits, k, mask=mask, **kw)[3]).all()
