"""GPU parity of the fused block norms and their gradient against 64-bit
definitions.

Bounds: a row's mean square is summed in chains of at most hidden/256 + 16
additions, its root halves that; each product adds a rounding."""
import pytest
import torch

import block_reference as ref
import vq_dequant_matmul_amd as vq
from block_reference import HALF_STEP, U, d

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def _r(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _c(t):
    return None if t is None else t.cuda()


def _weights(n, t, dtype, gate, post, pre, offset):
    one = 1.0 - offset
    return dict(
        post_weight=(one + _r((n,), F, 11, 0.2)).to(dtype) if post else None,
        pre_weight=(one + _r((n,), F, 12, 0.2)).to(dtype) if pre else None,
        gate={"none": None, "token": _r((t, 1), dtype, 13), "channel": _r((n,), dtype, 14)}[gate])


def _terms(h, y, w, kw):
    """|skip h|, |block branch|, and the exact outputs."""
    o, x = ref.block_norm(d(h), d(y), d(w["post_weight"]), d(w["pre_weight"]), d(w["gate"]),
                          kw["eps"], kw["weight_offset"], kw["skip_scale"], kw["block_scale"])
    a = (kw["skip_scale"] * d(h)).abs()
    return a, (o - kw["skip_scale"] * d(h)).abs(), o, x


def _root_bound(n):
    return (n / 256 + 24) * U


CASES = [  # tokens, hidden
    (1, 8), (3, 64), (1, 4096), (5, 2048), (130, 704), (33, 2056), (7, 4104), (2, 8192), (3, 8200),
    (2, 16384), (1025, 256),
]
KINDS = [  # h, y, x, weights, gate, post, pre, offset, skip, block
    (F, F, BF, BF, "none", True, True, 0.0, 1.0, 1.0),
    (BF, BF, BF, BF, "channel", True, True, 1.0, 1.0, 0.22),
    (F, BF, F, F, "token", False, True, 0.0, 0.75, 1.0),
    (BF, F, F, F, "token", True, False, 0.0, 1.0, -2.0),
    (F, F, F, F, "channel", False, False, 0.0, 0.5, 1.0),
    (BF, None, BF, BF, "none", False, True, 1.0, 1.0, 1.0),
]


def _kw(kind):
    return dict(eps=1e-6, weight_offset=kind[7], skip_scale=kind[8], block_scale=kind[9])


def _make(t, n, kind):
    hd, yd, xd, wd, gate, post, pre, offset = kind[:8]
    h = _r((t, n), hd, t + n, 2.0)
    y = None if yd is None else _r((t, n), yd, t + n + 1, 0.3)
    return h, y, _weights(n, t, wd, gate, post, pre, offset)


def _check_forward(got, h, y, w, kw, n, what=""):
    a, b, o, x = _terms(h, y, w, kw)
    ho, xo = got
    fp = _root_bound(n) * (a + b)
    bound = fp + HALF_STEP[ho.dtype] * o.abs()
    err = (d(ho) - o).abs()
    assert (err <= bound + 1e-37).all(), (what, (err / bound).max())
    if xo is not None:
        # x comes from the unrounded sum; an error of it also moves the root
        r = 1 / torch.sqrt(o.square().mean(1, keepdim=True) + kw["eps"])
        wt = 1.0 if w["pre_weight"] is None else (d(w["pre_weight"]) + kw["weight_offset"]).abs()
        root = (fp * o.abs()).mean(1, keepdim=True) * r * r
        bound = wt * r * (fp + o.abs() * root) + (_root_bound(n) + HALF_STEP[xo.dtype]) * x.abs()
        err = (d(xo) - x).abs()
        assert (err <= bound + 1e-37).all(), (what, (err / bound).max())


@pytest.mark.parametrize("t,n", CASES)
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_block_norm(t, n, kind):
    kind = KINDS[kind]
    h, y, w = _make(t, n, kind)
    got = vq.vq_block_norm(h.cuda(), _c(y), x_dtype=kind[2], **{k: _c(v) for k, v in w.items()},
                           **_kw(kind))
    assert got[0].dtype == kind[0] and got[1].dtype == kind[2]
    _check_forward(got, h, y, w, _kw(kind), n)


def test_strided_in_place_and_the_rest_untouched():
    t, n = 9, 320
    big_h, big_y = _r((t, n + 72), F, 1).cuda(), _r((t, n + 8), BF, 2).cuda()
    h, y = big_h[:, 8:8 + n], big_y[:, :n]
    keep = big_h.clone()
    w = _weights(n, t, BF, "channel", True, True, 0.0)
    kw = dict(eps=1e-5, weight_offset=0.0, skip_scale=1.0, block_scale=1.0)
    big_x = torch.full((t + 2, n + 16), 9.0, dtype=BF, device="cuda")
    dev = {k: _c(v) for k, v in w.items()}
    plain = vq.vq_block_norm(h.contiguous(), y.contiguous(), **dev, **kw)
    h0 = h.cpu()
    out = vq.vq_block_norm(h, y, h_out=h, x_out=big_x[1:1 + t, :n], **dev, **kw)
    assert out[0].data_ptr() == h.data_ptr()
    assert torch.equal(h, plain[0]) and torch.equal(big_x[1:1 + t, :n], plain[1])
    _check_forward(out, h0, y.cpu(), w, kw, n)
    assert torch.equal(big_h[:, :8], keep[:, :8]) and torch.equal(big_h[:, 8 + n:],
                                                                  keep[:, 8 + n:])
    assert (big_x[0] == 9).all() and (big_x[-1] == 9).all() and (big_x[:, n:] == 9).all()


def test_rows_of_zeros_and_of_nan():
    """A row of zeros gives zeros; a bad row stays alone."""
    t, n = 6, 512
    h, y = _r((t, n), F, 3), _r((t, n), F, 4)
    h[2] = 0
    y[2] = 0
    y[4, 7] = float("nan")
    h[5, 1] = float("inf")
    w = {k: _c(v) for k, v in _weights(n, t, F, "none", True, True, 0.0).items()}
    ho, x = vq.vq_block_norm(h.cuda(), y.cuda(), x_dtype=F, **w)
    assert (ho[2] == 0).all() and (x[2] == 0).all()
    assert ho[4].isnan().all() and torch.isfinite(x[[0, 1, 3]]).all()
    y[4, 7] = 0
    h[5, 1] = 0
    ho2, x2 = vq.vq_block_norm(h.cuda(), y.cuda(), x_dtype=F, **w)
    assert torch.equal(x[:4], x2[:4])


@pytest.mark.parametrize("t,n", CASES)
@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("given", ["both", "h", "x"])
def test_block_norm_grad(t, n, kind, given):
    kind = KINDS[kind]
    h, y, w = _make(t, n, kind)          # h stands for the forward's output
    kw = _kw(kind)
    dh = _r((t, n), kind[0], 21) if given != "x" else None
    dx = _r((t, n), kind[2], 22) if given != "h" else None
    got = vq.vq_block_norm_grad(h.cuda(), _c(y), _c(dh), _c(dx), **{k: _c(v) for k, v in
                                                                    w.items()}, **kw)
    o, eps = kw["weight_offset"], kw["eps"]
    p = {k: None if v is None else d(v).requires_grad_() for k, v in w.items()}
    hv = d(h).requires_grad_()
    D = torch.zeros((t, n), dtype=torch.float64) if dh is None else d(dh)
    magD, d_pre, mag_pre = D.abs(), None, 0.0
    r = 1 / torch.sqrt(d(h).square().mean(1, keepdim=True) + eps)
    wt = 1.0 if w["pre_weight"] is None else d(w["pre_weight"]) + o
    if dx is not None:
        leaves = [hv] + ([p["pre_weight"]] if p["pre_weight"] is not None else [])
        g = torch.autograd.grad(ref.rms(hv, p["pre_weight"], eps, o), leaves, d(dx))
        D = D + g[0]
        d_pre = g[1] if len(g) > 1 else None
        u = (wt * d(dx)).abs()
        hh = (d(h) * r).abs()
        magD = magD + r * (u + hh * (u * hh).mean(1, keepdim=True))
        mag_pre = (d(dx) * d(h) * r).abs().sum(0)
    elif w["pre_weight"] is not None:
        d_pre = torch.zeros(n, dtype=torch.float64)
    rel = 3 * _root_bound(n)
    sums = rel + (t / min(t, 512) + 512 / 4 + 8) * U   # over tokens, then workgroups

    def near(a, want, bound, what):
        err = (d(a) - want).abs()
        bound = bound + 1e-37
        assert a.shape == want.shape and torch.isfinite(a).all(), what
        assert (err <= bound).all(), (what, (err / bound).max())

    near(got[0], kw["skip_scale"] * D, abs(kw["skip_scale"]) * (
        rel * magD + HALF_STEP[kind[0]] * D.abs()), "d_h")
    if d_pre is None:
        assert got[3] is None
    else:
        near(got[3], d_pre, sums * mag_pre, "d_pre")
    if y is None:
        assert got[1] is None and got[2] is None and got[4] is None
        return
    yv = d(y).requires_grad_()
    names = [k for k in ("post_weight", "gate") if p[k] is not None]
    g = torch.autograd.grad(ref.branch(yv, p["post_weight"], p["gate"], eps, o,
                                       kw["block_scale"]), [yv] + [p[k] for k in names], D)
    by = dict(zip(names, g[1:]))
    q = 1 / torch.sqrt(d(y).square().mean(1, keepdim=True) + eps) if p["post_weight"] is not None \
        else torch.ones((t, 1), dtype=torch.float64)
    po = (d(w["post_weight"]) + o).abs() if p["post_weight"] is not None else 1.0
    bD = abs(kw["block_scale"]) * magD
    z = q * po * d(y).abs()
    dz = bD * (1.0 if w["gate"] is None else d(w["gate"]).abs())
    v, yy = po * dz, (d(y) * q).abs()
    mag_y = v if p["post_weight"] is None else q * (v + yy * (v * yy).mean(1, keepdim=True))
    near(got[1], g[0], 2 * rel * mag_y + HALF_STEP[kind[1]] * g[0].abs(), "d_y")
    if "post_weight" in by:
        near(got[2], by["post_weight"], (rel + sums) * (dz * yy).sum(0), "d_post")
    else:
        assert got[2] is None
    if "gate" in by:
        mag = (z * bD).sum(0) if kind[4] == "channel" else (z * bD).sum(1, keepdim=True)
        near(got[4], by["gate"], (rel + sums) * mag, "d_gate")
    else:
        assert got[4] is None


def test_gradient_against_differences():
    t, n = 5, 96
    h, y = _r((t, n), F, 1), _r((t, n), F, 2)
    w = _weights(n, t, F, "channel", True, True, 0.0)
    kw = dict(eps=1e-6, weight_offset=0.0, skip_scale=0.8, block_scale=1.3)
    dev = {k: _c(v) for k, v in w.items()}
    ch, cx = _r((t, n), F, 5), _r((t, n), F, 6)
    ho, _ = vq.vq_block_norm(h.cuda(), y.cuda(), x_dtype=F, **dev, **kw)
    got = vq.vq_block_norm_grad(ho, y.cuda(), ch.cuda(), cx.cuda(), **dev, **kw)

    def objective(h, y, post, pre, gate):
        o, x = ref.block_norm(h, y, post, pre, gate, 1e-6, 0.0, 0.8, 1.3)
        return float((o * d(ch)).sum() + (x * d(cx)).sum())

    at = [d(h), d(y), d(w["post_weight"]), d(w["pre_weight"]), d(w["gate"])]
    for i, g in enumerate(got):
        v = d(_r(tuple(at[i].shape), F, 30 + i))
        step = 1e-5
        plus, minus = list(at), list(at)
        plus[i], minus[i] = at[i] + step * v, at[i] - step * v
        slope = (objective(*plus) - objective(*minus)) / (2 * step)
        # h_out enters the gradient rounded to fp32; step^2 of the differences
        assert abs(float((d(g) * v).sum()) - slope) <= 4e-6 * float((d(g) * v).abs().sum()) + 1e-7


def test_grad_of_no_tokens_and_strided_rows():
    n = 128
    w = {k: _c(v) for k, v in _weights(n, 0, F, "channel", True, True, 0.0).items()}
    e = torch.empty((0, n), device="cuda")
    got = vq.vq_block_norm_grad(e, e, e, e, **w)
    assert all((g == 0).all() for g in got[2:]) and got[0].shape == (0, n)
    t = 7
    big = [_r((t, n + 24), F, i).cuda() for i in range(4)]
    w = {k: _c(v) for k, v in _weights(n, t, F, "token", True, True, 0.0).items()}
    views = [b[:, 8:8 + n] for b in big]
    a = vq.vq_block_norm_grad(*views, **w)
    b = vq.vq_block_norm_grad(*(v.contiguous() for v in views), **w)
    for i, j in zip(a, b):
        assert torch.equal(i, j)


def test_repeats_streams_and_graph():
    t, n = 300, 1024
    h, y = _r((t, n), BF, 1).cuda(), _r((t, n), BF, 2).cuda()
    w = {k: _c(v) for k, v in _weights(n, t, BF, "channel", True, True, 0.0).items()}

    def both():
        ho, x = vq.vq_block_norm(h, y, **w)
        return [ho, x, *vq.vq_block_norm_grad(ho, y, ho, x, **w)]

    first = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for i in range(3):
        h.copy_(_r((t, n), BF, 50 + i))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, both())), i


def test_binding_refuses():
    h = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="y must"):
        vq.vq_block_norm(h, h[:, :32])
    with pytest.raises(ValueError, match="one type"):
        vq.vq_block_norm(h, h, post_weight=w, pre_weight=w.bfloat16())
    with pytest.raises(ValueError, match="gate"):
        vq.vq_block_norm(h, h, gate=torch.ones((3, 1), device="cuda"))
    with pytest.raises(vq.VQError, match="eps"):
        vq.vq_block_norm(h, h, eps=0.0)
    with pytest.raises(vq.VQError, match="need y"):
        vq.vq_block_norm(h, post_weight=w)
    with pytest.raises(vq.VQError, match="h_stride"):
        vq.vq_block_norm(h[:1].expand(4, 64))
    with pytest.raises(TypeError):
        vq.vq_block_norm_grad(h, h, h.bfloat16(), h)


@pytest.mark.parametrize("t,n", [((1 << 22) - 1, 8), (140001, 16384)])
def test_the_most_tokens_and_offsets_past_32_bits(t, n):
    """Every row equals the one it repeats, at the highest token counts and offsets."""
    h, y = _r((7, n), BF, 1).cuda(), _r((7, n), BF, 2).cuda()
    w = {k: _c(v) for k, v in _weights(n, t, BF, "channel", True, True, 0.0).items()}
    index = torch.arange(t, device="cuda") % 7
    big_h, big_y = h[index], y[index]
    want = vq.vq_block_norm(h, y, **w)
    got = vq.vq_block_norm(big_h, big_y, **w)
    wg = vq.vq_block_norm_grad(want[0], y, want[0], want[1], **w)
    gg = vq.vq_block_norm_grad(got[0], big_y, got[0], got[1], **w)
    for a, b in ((got[0], want[0]), (got[1], want[1]), (gg[0], wg[0]), (gg[1], wg[1])):
        whole = t // 7 * 7
        assert (a[:whole].view(-1, 7, n) == b).all() and torch.equal(a[whole:], b[:t - whole])


@pytest.mark.parametrize("hd", [F, BF])
@pytest.mark.parametrize("yd", [F, BF])
@pytest.mark.parametrize("xd", [F, BF])
@pytest.mark.parametrize("wd", [F, BF])
@pytest.mark.parametrize("t,n", [(5, 264), (3, 4104), (2, 8208)])
def test_every_choice_of_types(hd, yd, xd, wd, t, n, monkeypatch):
    kind = (hd, yd, xd, wd, "channel", True, True, 1.0, 0.9, 1.1)
    monkeypatch.setitem(globals(), "KINDS", [kind])
    test_block_norm(t, n, 0)
    test_block_norm_grad(t, n, 0, "both")


def test_gradients_on_two_streams():
    """Two calls at once, each with its own workspace."""
    t, n = 900, 2056
    ho, y = [_r((t, n), BF, i).cuda() for i in range(2)], _r((t, n), BF, 5).cuda()
    w = {k: _c(v) for k, v in _weights(n, t, BF, "channel", True, True, 0.0).items()}
    want = [vq.vq_block_norm_grad(h, y, h, h, **w) for h in ho]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(vq.vq_block_norm_grad(ho[i], y, ho[i], ho[i], **w))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
