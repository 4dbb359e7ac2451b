"""GPU tests of the operators around the routed experts run together: one MoE
block (norm, router, selection, routed and shared experts, norm) against its
own steps bit for bit and against 64-bit definitions with the CPU oracle's
experts, and a router's training step through selection and norm."""
import numpy as np
import pytest
import torch

import block_reference as ref
import oracle
import synth
import vq_dequant_matmul_amd as vq
from block_reference import d
from parity import REL_L2

pytestmark = pytest.mark.gpu
F, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _setup():
    oracle.build(force=False)
    vq.load_library()


def _r(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _block(seed, E, top_k, hidden, inter, shared_inter=0, wdt=F, **kw):
    host = [synth.make_tensor(seed, 1, rows=inter, cols=hidden, d=4, bits=9, n_experts=E),
            synth.make_tensor(seed, 2, rows=inter, cols=hidden, d=4, bits=9, n_experts=E),
            synth.make_tensor(seed, 3, rows=hidden, cols=inter, d=4, bits=9, n_experts=E)]
    shared = None
    if shared_inter:
        arrays = [ref.q4_make(shared_inter, hidden, 64, BF, True, seed + 4),
                  ref.q4_make(shared_inter, hidden, 64, BF, True, seed + 5),
                  ref.q4_make(hidden, shared_inter, 32, torch.float16, False, seed + 6)]
        shapes = [(shared_inter, hidden, 64), (shared_inter, hidden, 64), (hidden, shared_inter, 32)]
        shared = tuple(vq.VQQ4Tensor(*s, *(None if a is None else a.cuda() for a in arr))
                       for s, arr in zip(shapes, arrays))
        kw["_arrays"] = arrays
    arrays = kw.pop("_arrays", None)
    blk = vq.VQMoEBlock(*(vq.VQTensor.from_host(t) for t in host),
                        router=_r((E, hidden), BF, seed + 7, 2.0 / hidden ** 0.5).cuda(),
                        top_k=top_k, pre_weight=(1 + _r((hidden,), F, seed + 8, 0.1)).to(wdt).cuda(),
                        shared=shared, **{k: v.cuda() if isinstance(v, torch.Tensor) else v
                                          for k, v in kw.items()})
    return blk, host, arrays


def _by_steps(b, h, attn, attn_weight, next_weight):
    kw = dict(eps=b.eps, weight_offset=b.weight_offset)
    if attn is None:
        _, x = vq.vq_block_norm(h, pre_weight=b.pre_weight, x_dtype=b.x_dtype, **kw)
    else:
        h, x = vq.vq_block_norm(h, attn, post_weight=attn_weight, pre_weight=b.pre_weight,
                                x_dtype=b.x_dtype, skip_scale=b.skip_scale,
                                block_scale=b.block_scale, **kw)
    ids, w = vq.vq_moe_route(vq.vq_router_logits(b.router, x), b.top_k, score=b.score,
                             renormalize=b.renormalize, scale=b.route_scale, bias=b.route_bias)
    y = vq.vq_moe_ffn(b.gate, b.up, b.down, x, ids, w)
    if b.shared:
        vq.vq_q4_gemv(b.shared[2], vq.vq_q4_gate_up(b.shared[0], b.shared[1], x), out=y,
                      accumulate=True)
    out, x = vq.vq_block_norm(h, y, post_weight=b.post_weight, gate=b.channel_gate,
                              pre_weight=next_weight, x_dtype=b.x_dtype, skip_scale=b.skip_scale,
                              block_scale=b.block_scale, **kw)
    return out, x if next_weight is not None else None, ids


@pytest.mark.parametrize("n", [1, 5, 17, 64])
@pytest.mark.parametrize("kind", ["plain", "full"])
def test_block_equals_its_steps(n, kind):
    hidden = 512
    kw = {} if kind == "plain" else dict(
        shared_inter=320, post_weight=1 + _r((hidden,), F, 1, 0.1),
        channel_gate=_r((hidden,), F, 2), route_bias=_r((24,), F, 3, 0.1),
        score=vq.VQ_SCORE_SIGMOID, route_scale=2.5, skip_scale=0.9, block_scale=0.5, x_dtype=F)
    b, _, _ = _block(40 + n, 24, 4, hidden, 192, **kw)
    h = _r((n, hidden), F, n).cuda()
    attn = _r((n, hidden), F, n + 1).cuda() if kind == "full" else None
    aw = (1 + _r((hidden,), F, 5, 0.1)).cuda() if kind == "full" else None
    nw = (1 + _r((hidden,), F, 6, 0.1)).cuda() if kind == "full" or n == 5 else None
    want, want_x, _ = _by_steps(b, h, attn, aw, nw)
    work = h.clone()
    got, x = vq.vq_moe_block(b, work, attn, attn_weight=aw, next_weight=nw)
    assert got is work and torch.equal(got, want)
    assert (x is None) == (nw is None) and (x is None or torch.equal(x, want_x))


@pytest.mark.parametrize("n", [1, 7, 40])
def test_block_matches_definitions(n):
    hidden, E, k = 512, 16, 4
    b, host, arrays = _block(70, E, k, hidden, 192, shared_inter=256, x_dtype=F,
                             post_weight=1 + _r((hidden,), F, 1, 0.1))
    h = _r((n, hidden), F, 100 + n)
    got, _ = vq.vq_moe_block(b, h.cuda())
    _, x = ref.block_norm(d(h), None, None, d(b.pre_weight), None)
    ids, w, _, _ = ref.route(x @ d(b.router).T, k)
    y = d(torch.from_numpy(np.asarray(oracle.moe_ffn(
        *host, x.float().numpy(), ids.int().numpy(), w.float().numpy()))))
    s = [ref.q4_weights(*a, g) for a, g in zip(arrays, (64, 64, 32))]
    g, u = x @ s[0].T, x @ s[1].T
    y = y + (g * torch.sigmoid(g) * u) @ s[2].T
    branch = ref.rms(y, d(b.post_weight), 1e-6, 0.0)
    err = (d(got) - (d(h) + branch)).norm(dim=1) / branch.norm(dim=1)
    # the experts' own bar, and fp32's share of the other steps
    assert err.max() <= REL_L2 + 1e-4, err.max()


def test_block_in_a_graph_and_bounds():
    hidden, n = 512, 3
    b, _, _ = _block(90, 32, 8, hidden, 128, shared_inter=64)
    nw = torch.ones(hidden, device="cuda")
    buf = torch.full((n + 2, hidden), 5.0, device="cuda")
    h = buf[:n]
    h.copy_(_r((n, hidden), F, 1))
    ws = torch.empty(b.workspace_size(n), dtype=torch.uint8, device="cuda")
    x = torch.empty((n, hidden), dtype=BF, device="cuda")
    vq.vq_moe_block(b, h.clone(), next_weight=nw, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vq.vq_moe_block(b, h, next_weight=nw, x_out=x, workspace=ws)
    for i in range(3):
        h.copy_(_r((n, hidden), F, 10 + i))
        want, want_x, _ = _by_steps(b, h.clone(), None, None, nw)
        g.replay()
        assert torch.equal(h, want) and torch.equal(x, want_x), i
    assert (buf[n:] == 5.0).all()
    with pytest.raises(vq.VQError, match="workspace"):
        vq.vq_moe_block(b, h, workspace=ws[:-256])
    e = torch.empty((0, hidden), device="cuda")
    assert vq.vq_moe_block(b, e)[0].shape == (0, hidden)


def test_router_training_step():
    """Loss of a router: h -> norm -> logits -> weights and balance loss; its
    gradients by the norm's weight, the router and h against 64-bit autograd."""
    t, hidden, E, k = 130, 256, 20, 3
    h, y = _r((t, hidden), F, 1), _r((t, hidden), F, 2)
    pre, router = 1 + _r((hidden,), F, 3, 0.1), _r((E, hidden), F, 4, 0.1)
    c, dl = _r((t, k), F, 5), torch.tensor([3.0])
    dev = [v.cuda() for v in (h, y, pre, router, c, dl)]
    ho, x = vq.vq_block_norm(dev[0], dev[1], pre_weight=dev[2], x_dtype=F)
    logits = x @ dev[3].t()
    ids, w, counts, loss = vq.vq_moe_route(logits, k, balance=True)
    dlog = vq.vq_moe_route_grad(logits, ids, dev[4], counts=counts, d_loss=dev[5])
    d_router = dlog.t() @ x
    dh, dy, _, d_pre, _ = vq.vq_block_norm_grad(ho, dev[1], None, dlog @ dev[3],
                                                pre_weight=dev[2])
    H, Y, P, R = (d(v).requires_grad_() for v in (h, y, pre, router))
    _, X = ref.block_norm(H, Y, None, P, None)
    L = X @ R.T
    rid, rw, rc, rl = ref.route(L, k)
    assert torch.equal(ids.cpu().long(), rid) and torch.equal(counts.cpu().long(), rc)
    assert abs(float(loss) - float(rl)) <= 1e-5 * float(rl)
    obj = ref.route_objective(L, rid, d(c), rc, d(dl)[0], False, True, 1.0, None)
    for got, want in zip((dh, dy, d_pre, d_router), torch.autograd.grad(obj, (H, Y, P, R))):
        # fp32 products of up to 256 terms in a chain: 256 half steps of the
        # largest sums, with room for the two products in a row
        assert (d(got) - want).norm() <= 2 * 256 * ref.U * want.norm() + 1e-12


def test_block_refuses_tensors_that_need_a_history():
    hidden, n = 256, 2
    b, _, _ = _block(17, 8, 2, hidden, 64)
    h, nw = _r((n, hidden), F, 1).cuda(), torch.ones(hidden, device="cuda")
    keep = h.clone()
    for kw in (dict(h=torch.nn.Parameter(h)), dict(h=h, attn=torch.nn.Parameter(h)),
               dict(h=h, next_weight=torch.nn.Parameter(nw))):
        with pytest.raises(ValueError, match="history"):
            vq.vq_moe_block(b, **kw)
    assert torch.equal(h, keep)
    want = vq.vq_moe_block(b, h.clone(), next_weight=nw)
    with torch.no_grad():
        got = vq.vq_moe_block(b, h, next_weight=torch.nn.Parameter(nw))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hidden,inter,n", [(8256, 64, 17), (16384, 64, 20), (128, 8256, 33)])
def test_block_past_the_decode_kernels_columns(hidden, inter, n):
    """Sizes that only the grouped GEMM takes, up to the norms' widest row."""
    b, _, _ = _block(23, 4, 2, hidden, inter, shared_inter=64)
    h = _r((n, hidden), F, 3).cuda()
    want, _, _ = _by_steps(b, h.clone(), None, None, None)
    assert torch.equal(vq.vq_moe_block(b, h)[0], want)


def test_block_on_two_streams():
    """Two calls at once, each with its own workspace, on the same weights."""
    hidden, n = 512, 24
    b, _, _ = _block(29, 16, 4, hidden, 128, shared_inter=128)
    h = [_r((n, hidden), F, i).cuda() for i in range(2)]
    want = [vq.vq_moe_block(b, v.clone())[0] for v in h]
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [[v.clone() for _ in range(6)] for v in h]
    torch.cuda.synchronize()
    for k in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                vq.vq_moe_block(b, work[i][k])
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[i]) for i in range(2) for v in work[i])
