"""GPU parity of the 4-bit products and the router's logits against 64-bit
definitions.  Bounds are worst-case sums of fp32 half steps along the longest
chain of additions (block_reference.q4_bound)."""
import pytest
import torch

import block_reference as ref
import vq_dequant_matmul_amd as vq
from block_reference import U, d

pytestmark = pytest.mark.gpu


def _x(n, cols, dtype, seed):
    return torch.randn((n, cols), generator=torch.Generator().manual_seed(seed)).to(dtype)


def _tensor(arrays, rows, cols, group):
    return vq.VQQ4Tensor(rows, cols, group, *(None if a is None else a.cuda() for a in arrays))


def _within(got, want, bound, what):
    err = (got.cpu().double() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = (err / bound).max().item()
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"


SHAPES = [  # rows, cols, group, tokens: one row, odd rows, one group, many groups, every tile
    (1, 64, 64, 1), (1, 128, 128, 64), (17, 64, 32, 3), (33, 192, 64, 5), (100, 320, 32, 16),
    (65, 1024, 128, 4), (257, 2048, 64, 1), (48, 4096, 64, 17), (1000, 704, 32, 33),
    (130, 5760, 64, 8), (16, 8192, 128, 64), (513, 2816, 64, 49), (31, 896, 64, 2),
]


@pytest.mark.parametrize("rows,cols,group,n", SHAPES)
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale_dtype,affine", [(torch.float16, True), (torch.bfloat16, True),
                                                (torch.bfloat16, False)])
def test_q4_gemv(rows, cols, group, n, x_dtype, scale_dtype, affine):
    arrays = ref.q4_make(rows, cols, group, scale_dtype, affine, rows + cols)
    x = _x(n, cols, x_dtype, n)
    y = vq.vq_q4_gemv(_tensor(arrays, rows, cols, group), x.cuda())
    want = d(x) @ ref.q4_weights(*arrays, group).T
    bound = ref.q4_bound(cols, group, ref.q4_magnitude(arrays[1], arrays[2], group, x))
    _within(y, want, bound, "q4_gemv")


@pytest.mark.parametrize("rows,cols,group,n", SHAPES)
@pytest.mark.parametrize("x_dtype,affine", [(torch.bfloat16, True), (torch.float32, False)])
def test_q4_gate_up(rows, cols, group, n, x_dtype, affine):
    ga = ref.q4_make(rows, cols, group, torch.float16, affine, rows)
    ua = ref.q4_make(rows, cols, group, torch.float16, affine, rows + 1)
    x = _x(n, cols, x_dtype, n + 7)
    h = vq.vq_q4_gate_up(_tensor(ga, rows, cols, group), _tensor(ua, rows, cols, group), x.cuda())
    g, u = (d(x) @ ref.q4_weights(*a, group).T for a in (ga, ua))
    dg, du = (ref.q4_bound(cols, group, ref.q4_magnitude(a[1], a[2], group, x)) for a in (ga, ua))
    s = g * torch.sigmoid(g)
    # |silu'| <= 1.1; exp's argument is off by |g| half steps, then a few roundings
    bound = 1.1 * dg * (u.abs() + du) + s.abs() * du + (8 + 4 * g.abs()) * U * (s * u).abs()
    _within(h, s * u, bound + 1e-30, "q4_gate_up")


def test_q4_gemv_accumulates_and_leaves_the_rest():
    rows, cols, n = 75, 512, 6
    arrays = ref.q4_make(rows, cols, 64, torch.float16, True, 5)
    W, x = _tensor(arrays, rows, cols, 64), _x(n, cols, torch.bfloat16, 6).cuda()
    buf = torch.full((n * rows + 64,), 7.0, device="cuda")
    out = buf[:n * rows].view(n, rows)
    base = vq.vq_q4_gemv(W, x)
    vq.vq_q4_gemv(W, x, out=out, accumulate=True)
    assert torch.equal(out, base + 7.0)
    assert (buf[n * rows:] == 7.0).all()
    vq.vq_q4_gemv(W, x, out=out)
    assert torch.equal(out, base)


def test_q4_extreme_codes_and_activations():
    """All codes 0 and 15, scales of 0, activations over fp32's range, a
    subnormal and exact zeros; a token's values stay out of its neighbours'."""
    rows, cols, group = 64, 256, 32
    codes = torch.zeros((rows, cols // 8), dtype=torch.int32)
    codes[::2] = -1
    scales = torch.full((rows, cols // group), 0.5, dtype=torch.float16)
    scales[1::4] = 0.0
    biases = torch.full_like(scales, -1.0)
    x = torch.zeros((5, cols))
    x[1] = 1e30
    x[2] = 1e-30
    x[3, 7] = 2.0 ** -140
    x[4] = _x(1, cols, torch.float32, 9)[0]
    W = _tensor((codes, scales, biases), rows, cols, group)
    y = vq.vq_q4_gemv(W, x.cuda())
    want = d(x) @ ref.q4_weights(codes, scales, biases, group).T
    # below fp32's smallest normal number a product may be flushed to zero
    bound = ref.q4_bound(cols, group, ref.q4_magnitude(scales, biases, group, x)) + 2.0 ** -126
    _within(y, want, bound, "extremes")
    assert (y[0] == 0).all()
    x[1] = float("nan")
    y2 = vq.vq_q4_gemv(W, x.cuda())
    assert y2[1].isnan().all() and torch.equal(y2[[0, 2, 3, 4]], y[[0, 2, 3, 4]])


def test_q4_repeats_bit_for_bit_on_other_streams_and_in_a_graph():
    rows, cols = 300, 1536
    W = _tensor(ref.q4_make(rows, cols, 64, torch.bfloat16, True, 1), rows, cols, 64)
    x = _x(9, cols, torch.bfloat16, 2).cuda()
    y = vq.vq_q4_gemv(W, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y1 = vq.vq_q4_gemv(W, x)
    torch.cuda.synchronize()
    assert torch.equal(y, y1)
    out = torch.empty_like(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vq.vq_q4_gemv(W, x, out=out)
    for i in range(3):
        x.copy_(_x(9, cols, torch.bfloat16, 10 + i))
        out.zero_()
        g.replay()
        assert torch.equal(out, vq.vq_q4_gemv(W, x)), i


def test_no_tokens():
    W = _tensor(ref.q4_make(8, 64, 64, torch.float16, True, 1), 8, 64, 64)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert vq.vq_q4_gemv(W, x).shape == (0, 8)
    assert vq.vq_q4_gate_up(W, W, x).shape == (0, 8)
    w = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    assert vq.vq_router_logits(w, x).shape == (0, 4)


@pytest.mark.parametrize("e,hidden,n", [(1, 64, 1), (7, 64, 64), (128, 2816, 64), (512, 4096, 1),
                                        (33, 8192, 16), (1024, 512, 17), (257, 1088, 5)])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
def test_router_logits(e, hidden, n, x_dtype):
    w, x = _x(e, hidden, torch.bfloat16, e), _x(n, hidden, x_dtype, n)
    got = vq.vq_router_logits(w.cuda(), x.cuda())
    bound = (hidden // 32 + 32 + 34) * U * (d(x).abs() @ d(w).abs().T)
    _within(got, d(x) @ d(w).T, bound, "router_logits")


def test_binding_refuses():
    arrays = ref.q4_make(8, 128, 64, torch.float16, True, 1)
    W = _tensor(arrays, 8, 128, 64)
    x = _x(2, 128, torch.bfloat16, 1).cuda()
    for bad, exc in ((x[:, :64], ValueError), (x.half(), TypeError), (x.cpu(), ValueError)):
        with pytest.raises(exc):
            vq.vq_q4_gemv(W, bad)
    with pytest.raises(vq.VQError, match="n_tokens"):
        vq.vq_q4_gemv(W, x[:1].expand(65, 128).contiguous())
    with pytest.raises(ValueError, match="out"):
        vq.vq_q4_gemv(W, x, out=torch.empty((2, 9), device="cuda"))
    with pytest.raises(ValueError, match="accumulate"):
        vq.vq_q4_gemv(W, x, accumulate=True)


@pytest.mark.parametrize("n,dtype", [(64, torch.bfloat16), (64, torch.float32), (16, torch.float32)])
def test_many_tokens_in_a_graph(n, dtype):
    """Launches that take most of a CU's shared memory."""
    rows, cols = 520, 4096
    arrays = ref.q4_make(rows, cols, 32, torch.float16, True, 3)
    W, x = _tensor(arrays, rows, cols, 32), _x(n, cols, dtype, 4).cuda()
    out = torch.empty((n, rows), device="cuda")
    h = torch.empty((n, rows), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vq.vq_q4_gemv(W, x, out=out)
        vq.vq_q4_gate_up(W, W, x, out=h)
    for i in range(3):
        x.copy_(_x(n, cols, dtype, 20 + i))
        g.replay()
        assert torch.equal(out, vq.vq_q4_gemv(W, x)) and torch.equal(h, vq.vq_q4_gate_up(W, W, x))
    bound = ref.q4_bound(cols, 32, ref.q4_magnitude(arrays[1], arrays[2], 32, x.cpu()))
    _within(out, d(x) @ ref.q4_weights(*arrays, 32).T, bound, "graph")


@pytest.mark.parametrize("rows,n", [(16500, 3), (16400, 16), (33000, 20), (70001, 1)])
def test_many_rows(rows, n):
    """Enough row tiles for the forms that split no row, or split it less."""
    cols = 320
    arrays = ref.q4_make(rows, cols, 64, torch.bfloat16, True, rows)
    x = _x(n, cols, torch.bfloat16, n)
    y = vq.vq_q4_gemv(_tensor(arrays, rows, cols, 64), x.cuda())
    bound = ref.q4_bound(cols, 64, ref.q4_magnitude(arrays[1], arrays[2], 64, x))
    _within(y, d(x) @ ref.q4_weights(*arrays, 64).T, bound, "many rows")


def test_a_bad_scale_stays_in_its_row():
    arrays = ref.q4_make(40, 192, 64, torch.float16, True, 8)
    W, x = _tensor(arrays, 40, 192, 64), _x(7, 192, torch.bfloat16, 9).cuda()
    y = vq.vq_q4_gemv(W, x)
    W.scales[11, 2] = float("nan")
    W.biases[12, 0] = float("inf")
    y2 = vq.vq_q4_gemv(W, x)
    assert not torch.isfinite(y2[:, [11, 12]]).any()
    keep = [r for r in range(40) if r not in (11, 12)]
    assert torch.equal(y2[:, keep], y[:, keep])


@pytest.mark.parametrize("rows,n,x_dtype", [(4201, 64, torch.bfloat16), (16417, 17, torch.bfloat16),
                                            (8209, 64, torch.float32), (8193, 49, torch.float32),
                                            (1033, 33, torch.float32), (257, 50, torch.bfloat16),
                                            (16500, 2, torch.float32)])
@pytest.mark.parametrize("group", [32, 128])
def test_groups_of_tokens(rows, n, x_dtype, group):
    """Row tiles by token tiles on both sides of where a wave takes two: the
    product, added to what was there, gate and up, and the memory behind."""
    cols = 384
    ga, ua = (ref.q4_make(rows, cols, group, torch.float16, True, rows + i) for i in (0, 1))
    G, UP = _tensor(ga, rows, cols, group), _tensor(ua, rows, cols, group)
    x = _x(n, cols, x_dtype, n)
    buf = torch.full(((n + 1) * rows,), 3.0, device="cuda")
    out, behind = buf[:n * rows].view(n, rows), buf[n * rows:]
    vq.vq_q4_gemv(G, x.cuda(), out=out)
    g, u = (d(x) @ ref.q4_weights(*a, group).T for a in (ga, ua))
    dg, du = (ref.q4_bound(cols, group, ref.q4_magnitude(a[1], a[2], group, x)) for a in (ga, ua))
    _within(out, g, dg, "groups of tokens")
    base = out.clone()
    vq.vq_q4_gemv(G, x.cuda(), out=out, accumulate=True)
    assert torch.equal(out, base + base)
    vq.vq_q4_gate_up(G, UP, x.cuda(), out=out)
    s = g * torch.sigmoid(g)
    bound = 1.1 * dg * (u.abs() + du) + s.abs() * du + (8 + 4 * g.abs()) * U * (s * u).abs()
    _within(out, s * u, bound + 1e-30, "groups of tokens, gate and up")
    assert (behind == 3.0).all()


@pytest.mark.parametrize("rows,n,x_dtype", [(33000, 16, torch.bfloat16), (32784, 3, torch.bfloat16),
                                            (33000, 5, torch.float32), (17000, 64, torch.bfloat16),
                                            (17000, 50, torch.float32)])
def test_a_last_round_split_over_more_waves(rows, n, x_dtype):
    """More workgroups than CUs by a few: their tiles, the last one cut short,
    are shared by several waves, alone and in a graph."""
    cols = 1344
    arrays = ref.q4_make(rows, cols, 64, torch.float16, True, rows)
    W, x = _tensor(arrays, rows, cols, 64), _x(n, cols, x_dtype, n)
    buf = torch.full(((n + 1) * rows,), 3.0, device="cuda")
    out, behind = buf[:n * rows].view(n, rows), buf[n * rows:]
    vq.vq_q4_gemv(W, x.cuda(), out=out)
    g = d(x) @ ref.q4_weights(*arrays, 64).T
    dg = ref.q4_bound(cols, 64, ref.q4_magnitude(arrays[1], arrays[2], 64, x))
    _within(out, g, dg, "last round")
    base = out.clone()
    graph, xs, h = torch.cuda.CUDAGraph(), x.cuda(), torch.empty((n, rows), device="cuda")
    with torch.cuda.graph(graph):
        vq.vq_q4_gemv(W, xs, out=out)
        vq.vq_q4_gate_up(W, W, xs, out=h)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, base)
        assert torch.equal(h, vq.vq_q4_gate_up(W, W, xs))
    s = g * torch.sigmoid(g)
    bound = 1.1 * dg * (g.abs() + dg) + s.abs() * dg + (8 + 4 * g.abs()) * U * (s * g).abs()
    _within(h, s * g, bound + 1e-30, "last round, gate and up")
    assert (behind == 3.0).all()


@pytest.mark.parametrize("e,hidden,n", [(513, 576, 64), (515, 1088, 33), (300, 4160, 25), (513, 64, 40),
                                        (1, 2048, 2), (6, 8256, 3)])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
def test_router_logits_experts_in_twos(e, hidden, n, x_dtype):
    """Many waves of two experts, the last one alone; nothing behind is touched."""
    w, x = _x(e, hidden, torch.bfloat16, e), _x(n, hidden, x_dtype, n)
    buf = torch.full(((n + 1) * e,), 5.0, device="cuda")
    got = vq.vq_router_logits(w.cuda(), x.cuda(), out=buf[:n * e].view(n, e))
    bound = (hidden // 32 + 32 + 34) * U * (d(x).abs() @ d(w).abs().T)
    _within(got, d(x) @ d(w).T, bound, "router_logits")
    assert (buf[n * e:] == 5.0).all()


@pytest.mark.parametrize("n,dtype", [(1, torch.bfloat16), (5, torch.float32), (64, torch.bfloat16)])
@pytest.mark.parametrize("group", [32, 128])
def test_the_most_columns(n, dtype, group):
    """2^20 columns: x passes through shared memory in many chunks."""
    rows, cols = 19, 1 << 20
    arrays = ref.q4_make(rows, cols, group, torch.bfloat16, True, n)
    W, x = _tensor(arrays, rows, cols, group), _x(n, cols, dtype, n)
    y = vq.vq_q4_gemv(W, x.cuda())
    bound = ref.q4_bound(cols, group, ref.q4_magnitude(arrays[1], arrays[2], group, x))
    want = d(x) @ ref.q4_weights(*arrays, group).T
    _within(y, want, bound, "most columns")
    h = vq.vq_q4_gate_up(W, W, x.cuda())
    s = want * torch.sigmoid(want)
    dg = bound
    hb = 1.1 * dg * (want.abs() + dg) + s.abs() * dg + (8 + 4 * want.abs()) * U * (s * want).abs()
    _within(h, s * want, hb + 1e-30, "most columns, gate and up")


@pytest.mark.parametrize("n", [1, 3, 17])
def test_codes_past_32_bit_offsets(n):
    """More than 2^31 words of codes (9 GB): rows on both sides of the border."""
    rows, cols, group = 140001, 1 << 17, 128
    gen = torch.Generator(device="cuda").manual_seed(n)
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, cols // 8), generator=gen, device="cuda",
                          dtype=torch.int32)
    scales = (0.5 + torch.rand((rows, cols // group), generator=gen, device="cuda")
              ).to(torch.bfloat16)
    W = vq.VQQ4Tensor(rows, cols, group, codes, scales)
    x = _x(n, cols, torch.bfloat16, n)
    y = vq.vq_q4_gemv(W, x.cuda()).cpu()
    border = 2 ** 31 // (cols // 8)
    for r in (0, border - 8, border, rows - 16):
        part = codes[r:r + 16].cpu(), scales[r:r + 16].cpu(), None
        bound = ref.q4_bound(cols, group, ref.q4_magnitude(part[1], None, group, x))
        _within(y[:, r:r + 16], d(x) @ ref.q4_weights(*part, group).T, bound, f"row {r}")


@pytest.mark.parametrize("e,hidden,n", [(1 << 20, 64, 3), (3, 1 << 20, 9), ((1 << 20) - 1, 128, 1)])
def test_router_logits_at_its_limits(e, hidden, n):
    w, x = _x(e, hidden, torch.bfloat16, 1), _x(n, hidden, torch.bfloat16, 2)
    got = vq.vq_router_logits(w.cuda(), x.cuda())
    bound = (hidden // 32 + 32 + 34) * U * (d(x).abs() @ d(w).abs().T)
    _within(got, d(x) @ d(w).T, bound, "limits")


@pytest.mark.parametrize("cols", [32, 96, 160, 608, 2080, 4128])
@pytest.mark.parametrize("rows,n", [(1, 1), (37, 4), (300, 2), (45, 17), (520, 64), (16500, 16),
                                    (33000, 20)])
@pytest.mark.parametrize("x_dtype,scale_dtype,affine", [
    (torch.bfloat16, torch.float16, True), (torch.float32, torch.bfloat16, False)])
def test_any_whole_number_of_groups(cols, rows, n, x_dtype, scale_dtype, affine):
    """Groups of 32 whose number is odd: rows of codes that end inside a unit of 128
    columns and of a load, scales that start between words; nothing behind is touched."""
    group = 32
    ga, ua = (ref.q4_make(rows, cols, group, scale_dtype, affine, rows + cols + i)
              for i in (0, 1))
    G, UP = _tensor(ga, rows, cols, group), _tensor(ua, rows, cols, group)
    x = _x(n, cols, x_dtype, n)
    buf = torch.full(((n + 1) * rows,), 3.0, device="cuda")
    out, behind = buf[:n * rows].view(n, rows), buf[n * rows:]
    vq.vq_q4_gemv(G, x.cuda(), out=out)
    g, u = (d(x) @ ref.q4_weights(*a, group).T for a in (ga, ua))
    dg, du = (ref.q4_bound(cols, group, ref.q4_magnitude(a[1], a[2], group, x)) for a in (ga, ua))
    _within(out, g, dg, "gemv")
    vq.vq_q4_gate_up(G, UP, x.cuda(), out=out)
    s = g * torch.sigmoid(g)
    bound = 1.1 * dg * (u.abs() + du) + s.abs() * du + (8 + 4 * g.abs()) * U * (s * u).abs()
    _within(out, s * u, bound + 1e-30, "gate and up")
    assert (behind == 3.0).all()


@pytest.mark.parametrize("group,cols", [(32, 512), (64, 512), (64, 1088), (128, 512), (128, 640),
                                        (128, 1536)])
@pytest.mark.parametrize("rows,n", [(4000, 1), (4000, 3), (700, 11), (3000, 34), (17000, 64)])
def test_fp32_activations_keep_their_digits(group, cols, rows, n):
    """The error as a norm over all outputs, where roundings add as independent ones.

    Codes enter as 16 + q, 24 times the scale in the mean, and weights are 4.6 scales in
    the root mean square, so a rounding of a group's sum weighs 5.2 times.  Six roundings
    (a step per 32 columns of the highest term, two where it meets the rest) of the
    products' sum and of x's, U / sqrt(3) each: 2 * 5.2 U; the sum over the groups adds
    less than 1.5 U."""
    arrays = ref.q4_make(rows, cols, group, torch.bfloat16, False, cols + n)
    x = _x(n, cols, torch.float32, n)
    y = d(vq.vq_q4_gemv(_tensor(arrays, rows, cols, group), x.cuda()))
    want = d(x) @ ref.q4_weights(*arrays, group).T
    assert (y - want).norm() <= 12 * U * want.norm()
