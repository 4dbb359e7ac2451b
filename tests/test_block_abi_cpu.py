"""Refusals of the operators around the routed experts, without a GPU: bad
host-visible arguments give the documented status and a message naming the
field (the pointers are never dereferenced), and the binding's own checks."""
import ctypes

import pytest
import torch

import vq_dequant_matmul_amd as vq

FAKE = 0x10000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return vq.load_library()


def _refused(lib, st, status, needle):
    assert st == status, lib.vq_last_error().decode()
    assert needle in lib.vq_last_error().decode()


def _q4(**kw):
    f = dict(rows=64, cols=128, group=64, scale_dtype=vq.VQ_F16, codes=FAKE, scales=FAKE,
             biases=FAKE)
    f.update(kw)
    return vq._CQ4(*(f[n] for n, _ in vq._CQ4._fields_))


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=0), 1, "rows"), (dict(cols=96), 1, "cols"), (dict(cols=0), 1, "cols"),
    (dict(cols=192, group=128), 1, "cols"), (dict(group=16), 2, "group"),
    (dict(scale_dtype=vq.VQ_F32), 1, "scale_dtype"), (dict(codes=None), 1, "non-NULL"),
    (dict(scales=None), 1, "non-NULL"), (dict(codes=FAKE + 4), 1, "aligned"),
    (dict(biases=FAKE + 2), 1, "aligned"), (dict(rows=2 ** 30, cols=2 ** 20), 2, "too large"),
])
def test_q4_descriptor(lib, kw, status, needle):
    t, good = _q4(**kw), _q4()
    _refused(lib, lib.vq_q4_gemv(ctypes.byref(t), 1, FAKE, 1, FAKE, 0, None), status, needle)
    _refused(lib, lib.vq_q4_gate_up(ctypes.byref(t), ctypes.byref(good), 1, FAKE, 1, FAKE, None),
             status, needle)
    _refused(lib, lib.vq_q4_gate_up(ctypes.byref(good), ctypes.byref(t), 1, FAKE, 1, FAKE, None),
             status, needle)


@pytest.mark.parametrize("n,x,dt,y,needle", [
    (-1, FAKE, 1, FAKE, "n_tokens"), (65, FAKE, 1, FAKE, "n_tokens"),
    (1, None, 1, FAKE, "x:"), (1, FAKE + 8, 1, FAKE, "x:"), (1, FAKE, 2, FAKE, "x_dtype"),
    (1, FAKE, 1, None, "y:"), (1, FAKE, 1, FAKE + 2, "y:"),
])
def test_q4_arguments(lib, n, x, dt, y, needle):
    t = _q4()
    _refused(lib, lib.vq_q4_gemv(ctypes.byref(t), n, x, dt, y, 0, None), 1, needle)
    st = lib.vq_router_logits(8, 64, FAKE, n, x, dt, y, None)
    _refused(lib, st, 1, "logits:" if needle == "y:" else needle)


def test_q4_null_and_mismatch(lib):
    t = _q4()
    _refused(lib, lib.vq_q4_gemv(None, 1, FAKE, 1, FAKE, 0, None), 1, "NULL")
    for kw, status in ((dict(rows=32), 1), (dict(cols=256), 1), (dict(group=32), 2),
                       (dict(biases=None), 2), (dict(scale_dtype=vq.VQ_BF16), 2)):
        u = _q4(**kw)
        _refused(lib, lib.vq_q4_gate_up(ctypes.byref(t), ctypes.byref(u), 1, FAKE, 1, FAKE, None),
                 status, "gate")
    assert lib.vq_q4_gemv(ctypes.byref(t), 0, None, 1, None, 0, None) == 0


def test_router_logits_sizes(lib):
    _refused(lib, lib.vq_router_logits(0, 64, FAKE, 1, FAKE, 1, FAKE, None), 1, "n_experts")
    _refused(lib, lib.vq_router_logits(8, 96, FAKE, 1, FAKE, 1, FAKE, None), 1, "hidden")
    _refused(lib, lib.vq_router_logits(8, 64, None, 1, FAKE, 1, FAKE, None), 1, "w:")
    _refused(lib, lib.vq_router_logits(8, 64, FAKE + 2, 1, FAKE, 1, FAKE, None), 1, "w:")


def _route(**kw):
    f = dict(n_experts=16, top_k=4, score=0, renormalize=1, scale=1.0)
    f.update(kw)
    return vq._CRoute(*(f[n] for n, _ in vq._CRoute._fields_))


@pytest.mark.parametrize("kw,status,needle", [
    (dict(n_experts=0), 1, "n_experts"), (dict(n_experts=1025), 2, "n_experts"),
    (dict(top_k=0), 1, "top_k"), (dict(top_k=17), 1, "top_k"),
    (dict(n_experts=128, top_k=65), 2, "top_k"), (dict(score=2), 1, "score"),
    (dict(scale=NAN), 1, "scale"), (dict(scale=INF), 1, "scale"),
])
def test_route_config(lib, kw, status, needle):
    c = ctypes.byref(_route(**kw))
    _refused(lib, lib.vq_moe_route(c, 1, FAKE, 0, None, None, FAKE, FAKE, None, None, None, 0,
                                   None), status, needle)
    _refused(lib, lib.vq_moe_route_grad(c, 1, FAKE, 0, None, FAKE, FAKE, None, None, FAKE, None),
             status, needle)
    assert lib.vq_moe_route_workspace_size(c, 1) == 0


def test_route_arguments(lib):
    c = ctypes.byref(_route())

    def call(n=1, logits=FAKE, dt=0, bias=None, ids=FAKE, w=FAKE, counts=None, loss=None, ws=None,
             size=0):
        return lib.vq_moe_route(c, n, logits, dt, bias, None, ids, w, counts, loss, ws, size, None)

    need = lib.vq_moe_route_workspace_size(c, 100)
    assert need > 0
    for kw, status, needle in (
            (dict(n=-1), 1, "n_tokens"), (dict(logits=None), 1, "logits"),
            (dict(logits=FAKE + 2), 1, "logits"), (dict(dt=2), 1, "logits_dtype"),
            (dict(ids=None), 1, "topk_ids"), (dict(w=FAKE + 1), 1, "topk_weights"),
            (dict(counts=FAKE), 1, "both"), (dict(loss=FAKE), 1, "both"),
            (dict(bias=FAKE + 1), 1, "bias"),
            (dict(n=100, counts=FAKE, loss=FAKE), 3, "workspace"),
            (dict(n=100, counts=FAKE, loss=FAKE, ws=FAKE, size=need - 1), 3, "workspace"),
            (dict(n=100, counts=FAKE, loss=FAKE, ws=FAKE + 16, size=need), 3, "workspace")):
        _refused(lib, call(**kw), status, needle)
    assert call(n=0) == 0


def test_route_grad_arguments(lib):
    c = ctypes.byref(_route())

    def call(n=1, logits=FAKE, dt=0, ids=FAKE, dw=FAKE, counts=None, dl=None, out=FAKE):
        return lib.vq_moe_route_grad(c, n, logits, dt, None, ids, dw, counts, dl, out, None)

    for kw, needle in ((dict(logits=None), "logits"), (dict(out=None), "d_logits"),
                       (dict(out=FAKE + 2), "d_logits"), (dict(ids=None), "topk_ids"),
                       (dict(counts=FAKE), "both"), (dict(dl=FAKE), "both"), (dict(n=-2), "n_tokens"),
                       (dict(counts=FAKE + 1, dl=FAKE), "counts")):
        _refused(lib, call(**kw), 1, needle)
    assert call(n=0, logits=None, out=None) == 0


def _norm(**kw):
    a = vq._CNorm(n_tokens=2, hidden=64, h_dtype=0, y_dtype=0, x_dtype=1, weight_dtype=0,
                  h_stride=64, y_stride=64, h_out_stride=64, x_stride=64, h=FAKE, y=FAKE,
                  post_weight=FAKE, pre_weight=FAKE, gate=None, gate_kind=0, eps=1e-6,
                  weight_offset=0.0, skip_scale=1.0, block_scale=1.0, h_out=FAKE, x=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status,needle", [
    (dict(n_tokens=-1), 1, "n_tokens"), (dict(hidden=0), 1, "hidden"),
    (dict(hidden=60), 1, "hidden"), (dict(hidden=16392, h_stride=16392), 2, "hidden"),
    (dict(h_dtype=2), 1, "h_dtype"), (dict(y_dtype=3), 1, "y_dtype"),
    (dict(x_dtype=2), 1, "x_dtype"), (dict(weight_dtype=2), 1, "weight_dtype"),
    (dict(h_stride=56), 1, "h_stride"), (dict(y_stride=68), 1, "y_stride"),
    (dict(h_out_stride=0), 1, "h_out_stride"), (dict(x_stride=-64), 1, "x_stride"),
    (dict(h=FAKE + 8), 1, "h:"), (dict(x=FAKE + 8), 1, "x:"), (dict(gate_kind=3), 1, "gate_kind"),
    (dict(gate_kind=1), 1, "gate"), (dict(gate=FAKE), 1, "gate"),
    (dict(y=None), 1, "need y"), (dict(eps=0.0), 1, "eps"), (dict(eps=NAN), 1, "eps"),
    (dict(eps=INF), 1, "eps"), (dict(skip_scale=INF), 1, "finite"),
    (dict(block_scale=NAN), 1, "finite"), (dict(weight_offset=INF), 1, "finite"),
    (dict(pre_weight=FAKE + 4), 1, "aligned"),
])
def test_norm_arguments(lib, kw, status, needle):
    a = _norm(**kw)
    _refused(lib, lib.vq_block_norm(ctypes.byref(a), None), status, needle)
    _refused(lib, lib.vq_block_norm_grad(ctypes.byref(a), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                         None, FAKE, 1 << 30, None), status, needle)


def test_norm_outputs(lib):
    a = _norm(h=None)
    _refused(lib, lib.vq_block_norm(ctypes.byref(a), None), 1, "h must")
    a = _norm(h_out=None, x=None)
    _refused(lib, lib.vq_block_norm(ctypes.byref(a), None), 1, "h_out or x")
    a = _norm(n_tokens=0)
    assert lib.vq_block_norm(ctypes.byref(a), None) == 0
    _refused(lib, lib.vq_block_norm(None, None), 1, "NULL")


def test_norm_grad_arguments(lib):
    def call(a=None, dh=FAKE, dx=FAKE, o=(FAKE, FAKE, FAKE, FAKE, None), ws=FAKE, size=1 << 30):
        return lib.vq_block_norm_grad(ctypes.byref(a or _norm()), dh, dx, *o, ws, size, None)

    need = lib.vq_block_norm_grad_workspace_size(ctypes.byref(_norm()))
    assert need > 0
    none = _norm(y=None, post_weight=None)
    for kw, status, needle in (
            (dict(dh=None, dx=None), 1, "d_h_out or d_x"), (dict(dh=FAKE + 4), 1, "d_h_out"),
            (dict(dx=FAKE + 4), 1, "d_x"), (dict(o=(FAKE + 4, None, None, None, None)), 1, "d_h"),
            (dict(o=(None, FAKE + 4, None, None, None)), 1, "d_y"),
            (dict(o=(None, None, None, None, FAKE)), 1, "d_gate"),
            (dict(o=(None, None, FAKE + 4, None, None)), 1, "aligned"),
            (dict(a=none, o=(None, FAKE, None, None, None)), 1, "need y"),
            (dict(a=_norm(post_weight=None), o=(None, None, FAKE, None, None)), 1, "post_weight"),
            (dict(a=_norm(pre_weight=None), o=(None, None, None, FAKE, None)), 1, "pre_weight"),
            (dict(a=_norm(h_out=None)), 1, "h_out"),
            (dict(ws=None), 3, "workspace"), (dict(size=need - 1), 3, "workspace"),
            (dict(ws=FAKE + 64), 3, "workspace")):
        _refused(lib, call(**kw), status, needle)


def test_binding_refuses_before_the_library():
    c, s = torch.zeros((4, 16), dtype=torch.int32), torch.zeros((4, 2), dtype=torch.float16)
    vq.VQQ4Tensor(4, 128, 64, c, s)
    with pytest.raises(ValueError, match="group"):
        vq.VQQ4Tensor(4, 128, 48, c, s)
    with pytest.raises(ValueError, match="codes"):
        vq.VQQ4Tensor(4, 256, 64, c, s)
    with pytest.raises(ValueError, match="scales"):
        vq.VQQ4Tensor(4, 128, 32, c, s)
    with pytest.raises(TypeError, match="scales"):
        vq.VQQ4Tensor(4, 128, 64, c, s.float())
    with pytest.raises(ValueError, match="biases"):
        vq.VQQ4Tensor(4, 128, 64, c, s, s[:2])
    with pytest.raises(ValueError, match="contiguous"):
        vq.VQQ4Tensor(4, 128, 64, c, s.t().contiguous().t())


def _block(**kw):
    t = [vq._CTensor(r, c, 4, 9, 512, 4, 4 * r, FAKE, FAKE, FAKE, None)
         for r, c in ((64, 128), (64, 128), (128, 64))]
    q = [_q4(rows=r, cols=c) for r, c in ((64, 128), (64, 128), (128, 64))]
    P = ctypes.pointer
    b = vq._CBlock(*(P(x) for x in t), *(P(x) for x in q), FAKE, None,
                   _route(n_experts=4, top_k=2), 1, 0, FAKE, None, None, 1e-6, 0.0, 1.0, 1.0)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


@pytest.mark.parametrize("kw,status,needle", [
    (dict(gate=None), 1, "gate"), (dict(down=None), 1, "down"), (dict(router=None), 1, "router"),
    (dict(router=FAKE + 2), 1, "router"), (dict(route=_route(n_experts=5, top_k=2)), 1, "experts"),
    (dict(route=_route(n_experts=4, top_k=5)), 1, "top_k"),
    (dict(route=_route(n_experts=4, top_k=2, score=3)), 1, "score"),
    (dict(x_dtype=2), 1, "x_dtype"), (dict(pre_weight=None), 1, "pre_weight"),
    (dict(shared_up=None), 1, "shared_up"),
    (dict(shared_down=ctypes.pointer(_q4(rows=64, cols=64))), 1, "shared expert"),
])
def test_block_arguments(lib, kw, status, needle):
    b = _block(**kw)
    _refused(lib, lib.vq_moe_block(ctypes.byref(b), 1, FAKE, None, None, None, None, FAKE, 1 << 30,
                                   None), status, needle)
    assert lib.vq_moe_block_workspace_size(ctypes.byref(b), 1) == 0


def test_block_calls(lib):
    ref = ctypes.byref

    def call(b=None, n=1, h=FAKE, attn=None, aw=None, nw=None, x=None, ws=FAKE, size=1 << 30):
        return lib.vq_moe_block(ref(b or _block()), n, h, attn, aw, nw, x, ws, size, None)

    need = lib.vq_moe_block_workspace_size(ref(_block()), 1)
    assert need > 0
    for kw, status, needle in (
            (dict(n=-1), 1, "n_tokens"), (dict(n=65), 1, "n_tokens"), (dict(h=None), 1, "h must"),
            (dict(aw=FAKE), 1, "attn"), (dict(nw=FAKE), 1, "both"), (dict(x=FAKE), 1, "both"),
            (dict(ws=None), 3, "workspace"), (dict(size=need - 1), 3, "workspace"),
            (dict(h=FAKE + 8), 1, "h:"), (dict(b=_block(eps=0.0)), 1, "eps"),
            (dict(b=_block(weight_dtype=2)), 1, "weight_dtype"),
            (dict(b=_block(shared_up=ctypes.pointer(_q4(rows=64, cols=128, biases=None)))), 1,
             "shared_up")):
        _refused(lib, call(**kw), status, needle)
    _refused(lib, lib.vq_moe_block(None, 1, FAKE, None, None, None, None, FAKE, 1 << 30, None), 1,
             "NULL")
    assert call(n=0, h=None, ws=None, size=0) == 0


def test_sizes_that_no_launch_holds(lib):
    for t in (_q4(rows=2 ** 27 + 1), _q4(rows=2 ** 30)):
        _refused(lib, lib.vq_q4_gemv(ctypes.byref(t), 1, FAKE, 1, FAKE, 0, None), 2, "too large")
    for e, hidden in ((2 ** 20 + 1, 64), (8, 2 ** 20 + 64)):
        _refused(lib, lib.vq_router_logits(e, hidden, FAKE, 1, FAKE, 1, FAKE, None), 2, "too large")
    a = _norm(n_tokens=2 ** 22)
    _refused(lib, lib.vq_block_norm(ctypes.byref(a), None), 2, "n_tokens")
    assert lib.vq_block_norm_grad_workspace_size(ctypes.byref(a)) == 0


def test_route_grad_binding_wants_a_matrix_of_ids():
    logits, ids = torch.zeros((2, 8)), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="topk_ids"):
        vq.vq_moe_route_grad(logits, ids, None)


@pytest.mark.parametrize("n", [0, 1, 2])
def test_norm_channel_gate_is_there_for_any_number_of_tokens(lib, n):
    """The gradient of the post weight multiplies by the gate, tokens or not."""
    a = _norm(n_tokens=n, gate_kind=vq.VQ_GATE_CHANNEL, gate=None)
    for o in ((None, None, FAKE, None, None), (None, None, None, None, FAKE),
              (None, None, None, FAKE, None)):
        _refused(lib, lib.vq_block_norm_grad(ctypes.byref(a), FAKE, FAKE, *o, FAKE, 1 << 30, None),
                 1, "gate")
    _refused(lib, lib.vq_block_norm(ctypes.byref(a), None), 1, "gate")
    assert lib.vq_block_norm_grad_workspace_size(ctypes.byref(a)) == 0
    a.gate_kind, a.gate = vq.VQ_GATE_NONE, FAKE
    _refused(lib, lib.vq_block_norm(ctypes.byref(a), None), 1, "gate")


def test_norm_token_gate_of_no_tokens(lib):
    """An array with a value per token may be NULL where there are no tokens."""
    a = _norm(n_tokens=0, gate_kind=vq.VQ_GATE_TOKEN, gate=None)
    assert lib.vq_block_norm(ctypes.byref(a), None) == 0
    assert lib.vq_block_norm_grad(ctypes.byref(a), None, None, None, None, None, None, None, None,
                                  0, None) == 0


def test_route_workspace_of_the_largest_batches(lib):
    """Partial sums are kept for a fixed number of workgroups at most, up to the last int32."""
    c = ctypes.byref(_route(n_experts=512))
    most = lib.vq_moe_route_workspace_size(c, 1 << 20)
    assert most > 512 * 512 * 8
    for n in (2 ** 31 - 1, 2 ** 31 - 7, 2 ** 31 - 8, 2 ** 31 - 16, 1 << 30):
        assert lib.vq_moe_route_workspace_size(c, n) == most


def _wide_block(hidden, inter, d=4, bits=9):
    K = 1 << bits
    t = [vq._CTensor(r, c, d, bits, K, 4, 4 * r, FAKE, FAKE, FAKE, None)
         for r, c in ((inter, hidden), (inter, hidden), (hidden, inter))]
    none = ctypes.POINTER(vq._CQ4)()
    return vq._CBlock(*(ctypes.pointer(x) for x in t), none, none, none, FAKE, None,
                      _route(n_experts=4, top_k=2), 1, 0, FAKE, None, None, 1e-6, 0.0, 1.0, 1.0)


@pytest.mark.parametrize("hidden,inter,n,needle", [
    (8256, 64, 1, "columns"), (64, 8256, 1, "columns"), (8256, 64, 16, "columns"),
    (16448, 64, 17, "norms"), (16448, 64, 1, "columns"),
])
def test_block_refuses_sizes_of_a_later_step_before_any(lib, hidden, inter, n, needle):
    """The routed FFN's limits and the norms' are checked ahead of the first
    step, which updates h: no launch is tried (without a GPU that would be
    VQ_ERR_HIP), and there is no workspace for such a call."""
    b = ctypes.byref(_wide_block(hidden, inter))
    assert lib.vq_moe_block_workspace_size(b, n) == 0
    _refused(lib, lib.vq_moe_block(b, n, FAKE, FAKE, None, None, None, FAKE, 1 << 34, None), 2,
             needle)


def test_block_sizes_at_the_limits(lib):
    for hidden, inter, n in ((8192, 8192, 1), (8256, 64, 17), (64, 8256, 64)):
        assert lib.vq_moe_block_workspace_size(ctypes.byref(_wide_block(hidden, inter)), n) > 0


def test_binding_refuses_tensors_that_need_a_history():
    """The results have no history: with grad enabled a backward pass would leave
    these inputs out without a word."""
    p = torch.nn.Parameter
    h, w, l = torch.zeros((2, 64)), torch.ones(64), torch.zeros((2, 8))
    with pytest.raises(ValueError, match="vq_moe_route_grad"):
        vq.vq_moe_route(p(l), 2)
    for kw in (dict(h=p(h)), dict(h=h, y=p(h)), dict(h=h, y=h, post_weight=p(w)),
               dict(h=h, pre_weight=p(w)), dict(h=h, y=h, gate=p(w))):
        with pytest.raises(ValueError, match="vq_block_norm_grad"):
            vq.vq_block_norm(**kw)
    r = torch.zeros((8, 64), dtype=torch.bfloat16)
    for a in ((p(r), h), (r, p(h))):
        with pytest.raises(ValueError, match="history"):
            vq.vq_router_logits(*a)
    q = vq.VQQ4Tensor(4, 64, 64, torch.zeros((4, 8), dtype=torch.int32),
                      torch.zeros((4, 1), dtype=torch.float16))
    with pytest.raises(ValueError, match="history"):
        vq.vq_q4_gemv(q, p(h))
    with pytest.raises(ValueError, match="history"):
        vq.vq_q4_gate_up(q, q, p(h))


def test_binding_without_grad_takes_parameters():
    """Under no_grad the same tensors go on to the checks behind (here: no GPU)."""
    h = torch.nn.Parameter(torch.zeros((2, 64)))
    with torch.no_grad():
        for call in (lambda: vq.vq_block_norm(h), lambda: vq.vq_moe_route(h, 2)):
            with pytest.raises((TypeError, RuntimeError)):
                call()


@pytest.mark.parametrize("cols", [32, 96, 160, 4128])
def test_q4_any_whole_number_of_groups(lib, cols):
    t = _q4(cols=cols, group=32)
    assert lib.vq_q4_gemv(ctypes.byref(t), 0, None, 1, None, 0, None) == 0
    assert lib.vq_q4_gate_up(ctypes.byref(t), ctypes.byref(t), 0, None, 1, None, None) == 0
    vq.VQQ4Tensor(4, cols, 32, torch.zeros((4, cols // 8), dtype=torch.int32),
                  torch.zeros((4, cols // 32), dtype=torch.float16))
    _refused(lib, lib.vq_q4_gemv(ctypes.byref(_q4(cols=cols, group=64)), 1, FAKE, 1, FAKE, 0, None),
             1, "cols")


def test_the_measured_ranges_are_accepted(lib):
    """Every case that perf/operators.py can give passes the host's checks of sizes."""
    import random

    import perf.operators as ops
    for c in ops.listed() + [ops.draw(random.Random(i)) for i in range(1000)]:
        op = c["op"]
        if op in ("q4_gemv", "q4_gate_up"):
            t = ctypes.byref(_q4(rows=c["rows"], cols=c["cols"], group=c["group"],
                                 biases=FAKE if c["affine"] else None))
            assert lib.vq_q4_gemv(t, 0, None, 1, None, 0, None) == 0, c
            assert 1 <= c["tokens"] <= 64
        elif op == "logits":
            assert lib.vq_router_logits(c["experts"], c["hidden"], FAKE, 0, None, 1, None,
                                        None) == 0, c
            assert 1 <= c["tokens"] <= 64
        elif op in ("route", "route_grad"):
            r = ctypes.byref(_route(n_experts=c["experts"], top_k=c["k"]))
            assert lib.vq_moe_route_workspace_size(r, c["tokens"]) > 0, c
        else:
            n = c["hidden"]
            a = _norm(n_tokens=c["tokens"], hidden=n, h_stride=n, y_stride=n, h_out_stride=n,
                      x_stride=n)
            assert lib.vq_block_norm_grad_workspace_size(ctypes.byref(a)) > 0, c
