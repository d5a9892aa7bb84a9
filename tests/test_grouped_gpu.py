"""Grouped products and their gradients on the GPU against plain 64-bit
implementations (bounds: rows_util)."""
import numpy as np
import pytest

from rows_util import (TYPES, U, f64, grouped_ref, normal, offsets_of, random_ids, rounded,
                       wgrad_ref, within)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import persistent_stream_tiling_amd as gsk  # noqa: E402

# group sizes: no rows at all, one row, empty groups at both ends and between,
# sizes around the tiles' rows, one group with everything, many small groups
SIZES = {
    "none": [0, 0, 0],
    "one": [0, 1, 0],
    "one-group": [300],
    "around-tiles": [31, 32, 33, 0, 63, 64, 65, 127, 128, 129],
    "around-large-tiles": [255, 0, 256, 257, 1],
    "skewed": [0, 700, 1, 0, 0, 3, 0],
    "many": [(7 * i) % 5 for i in range(150)],
}
# K and N: less than any tile, odd, whole tiles, past a tile by one
DEPTHS = [(1, 1), (16, 8), (40, 72), (64, 256), (203, 101), (256, 320), (321, 257), (1000, 136)]


def tail(sizes, dropped):
    """Offsets and the number of rows, `dropped` of them past the last group."""
    off = offsets_of(sizes)
    return off, int(off[-1]) + dropped


def check_rows(sizes, dropped, K, N, dtype, half, trans, seed=1, ints=False):
    off, rows = tail(sizes, dropped)
    G = len(sizes)
    if ints:
        gen = torch.Generator().manual_seed(seed)
        a = torch.randint(-4, 5, (rows, K), generator=gen).to(TYPES[dtype])
        b = torch.randint(-4, 5, (G, K, N), generator=gen).to(TYPES[dtype])
    else:
        a, b = normal((rows, K), dtype, seed), normal((G, K, N), dtype, seed + 1)
    a[off[-1]:] = float("nan")  # rows of no group never count
    ref, size = grouped_ref(np.nan_to_num(f64(a)), f64(b), off)
    out = TYPES[dtype] if half else torch.float32
    db = b.cuda()
    if trans:
        db = db.transpose(1, 2).contiguous().transpose(1, 2)
    c = gsk.grouped_matmul(a.cuda(), db, torch.from_numpy(off).to(torch.int32).cuda(), out_dtype=out)
    assert c.dtype == out
    bound = 0.0 * size if ints else 2 * max(K, 1) * U * size
    within(c, ref, rounded(bound, ref, out), f"{sizes} K={K} N={N}")
    assert (c[off[-1]:] == 0).all()


def check_wgrad(sizes, dropped, K, N, dtype, half, seed=1):
    off, rows = tail(sizes, dropped)
    a, d = normal((rows, K), dtype, seed), normal((rows, N), dtype, seed + 1)
    ref, size = wgrad_ref(f64(a), f64(d), off)
    a[off[-1]:] = float("nan")
    d[off[-1]:] = float("inf")
    out = TYPES[dtype] if half else torch.float32
    c = gsk.grouped_matmul_wgrad(a.cuda(), d.cuda(), torch.from_numpy(off).to(torch.int32).cuda(),
                                 out_dtype=out)
    n = np.maximum(np.diff(off), 1)[:, None, None]
    within(c, ref, rounded(2 * n * U * size, ref, out), f"wgrad {sizes} K={K} N={N}")


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("trans", [False, True], ids=["b", "bT"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_product_group_sizes(sizes, trans, dtype):
    for K, N in [(72, 136), (203, 101)]:
        for half in (False, True):
            check_rows(SIZES[sizes], 37, K, N, dtype, half, trans)


@pytest.mark.parametrize("K,N", DEPTHS)
@pytest.mark.parametrize("trans", [False, True], ids=["b", "bT"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_product_depths(K, N, trans, dtype):
    check_rows([5, 0, 130, 41], 3, K, N, dtype, False, trans)
    check_rows([300, 290], 0, K, N, dtype, True, trans)


@pytest.mark.parametrize("trans", [False, True], ids=["b", "bT"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_product_is_exact_on_small_integers(trans, dtype):
    for sizes, K, N in [([9, 0, 300, 64], 520, 264), ([600, 700], 1032, 520), ([2] * 90, 136, 200)]:
        check_rows(sizes, 11, K, N, dtype, False, trans, ints=True)


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_weight_gradient_group_sizes(sizes, dtype):
    for K, N in [(72, 136), (203, 101)]:
        for half in (False, True):
            if len(SIZES[sizes]) * K * N < 3e6:
                check_wgrad(SIZES[sizes], 37, K, N, dtype, half)


@pytest.mark.parametrize("K,N", DEPTHS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_weight_gradient_depths(K, N, dtype):
    check_wgrad([5, 0, 130, 41], 3, K, N, dtype, False)
    check_wgrad([300, 290], 0, K, N, dtype, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_depth_and_empty_shapes(dtype):
    t = TYPES[dtype]
    off = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    c = gsk.grouped_matmul(torch.empty(6, 0, dtype=t, device="cuda"),
                           torch.empty(2, 0, 9, dtype=t, device="cuda"), off)
    assert c.shape == (6, 9) and (c == 0).all()
    c = gsk.grouped_matmul(torch.empty(6, 8, dtype=t, device="cuda"),
                           torch.empty(2, 8, 0, dtype=t, device="cuda"), off)
    assert c.shape == (6, 0)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    c = gsk.grouped_matmul(torch.empty(0, 8, dtype=t, device="cuda"),
                           torch.empty(2, 8, 9, dtype=t, device="cuda"), none)
    assert c.shape == (0, 9)
    c = gsk.grouped_matmul_wgrad(torch.empty(0, 8, dtype=t, device="cuda"),
                                 torch.empty(0, 9, dtype=t, device="cuda"), none)
    assert c.shape == (2, 8, 9) and (c == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_not_finite_values_stay_in_their_rows_and_groups(dtype):
    sizes, K, N = [40, 70, 33], 136, 264
    off = offsets_of(sizes)
    a, b = normal((143, K), dtype, 1), normal((3, K, N), dtype, 2)
    b[1, 5, 7] = float("inf")
    b[1, 6] = float("nan")
    a[2, 9] = float("nan")
    ref, size = grouped_ref(np.nan_to_num(f64(a)), np.nan_to_num(f64(b), posinf=0.0), off)
    c = f64(gsk.grouped_matmul(a.cuda(), b.cuda(), torch.from_numpy(off).to(torch.int32).cuda()))
    assert np.isnan(c[2]).all() and np.isnan(c[40:110]).all()
    clean = [i for i in range(143) if i != 2 and not 40 <= i < 110]
    within(c[clean], ref[clean], 2 * K * U * size[clean])
    d = normal((143, N), dtype, 3)
    d[60, 3] = float("inf")
    a = torch.nan_to_num(a)
    w = f64(gsk.grouped_matmul_wgrad(a.cuda(), d.cuda(), torch.from_numpy(off).to(torch.int32).cuda()))
    d[60, 3] = 0.0
    ref, size = wgrad_ref(f64(a), f64(d), off)
    keep = np.ones_like(ref, dtype=bool)
    keep[1, :, 3] = False
    assert not np.isfinite(w[~keep]).any()
    assert (np.abs(w - ref) <= 2 * 70 * U * size + 1e-30)[keep].all()


def test_offsets_out_of_range_or_order_touch_nothing_else():
    # the buffer may hold anything and the run still ends; offsets that
    # descend make groups overlap, whose rows are then anyone's, and offsets
    # past the rows end with them
    K, N = 72, 136
    a, b = normal((200, K), "bf16", 1), normal((4, K, N), "bf16", 2)
    for off in ([0, 50, 10 ** 9, -5, 200], [150, 20, 60, 10, 5], [-9, -1, 2 ** 31 - 1, 2 ** 31 - 1, 0],
                [-3, 50, 10 ** 9, 10 ** 9, 2 ** 31 - 1]):
        o = torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
        c = gsk.grouped_matmul(a.cuda(), b.cuda(), o)
        assert c.shape == (200, N)
        w = gsk.grouped_matmul_wgrad(a.cuda(), normal((200, N), "bf16", 3).cuda(), o)
        assert w.shape == (4, K, N)
        torch.cuda.synchronize()
    ref, size = grouped_ref(f64(a), f64(b), np.array([0, 50, 200, 200, 200]))
    within(c, ref, 2 * K * U * size)


def spread(groups, seed, most):
    """Group sizes of very different lengths, some of them zero."""
    rng = np.random.default_rng(seed)
    n = np.floor(most * rng.random(groups) ** 3).astype(int)
    n[rng.random(groups) < 0.15] = 0
    return n.tolist()


@pytest.mark.parametrize("trans", [False, True], ids=["b", "bT"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_more_tiles_than_workgroups(trans, dtype):
    # hundreds of 256x256 tiles of very different depth of work: every
    # workgroup takes several, and the queues run empty at different times
    check_rows(spread(20, 3, 3000), 700, 72, 1032, dtype, True, trans)
    check_rows([256] * 90 + [0, 1, 255, 257], 5, 40, 1096, dtype, False, trans)
    # fewer tiles than workgroups, and fewer than queues
    check_rows([300, 500], 0, 264, 300, dtype, True, trans)
    check_rows([1000], 0, 64, 100, dtype, True, trans)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_weight_gradient_of_many_groups(dtype):
    check_wgrad(spread(45, 5, 900), 30, 520, 776, dtype, False)
    check_wgrad(spread(45, 6, 900), 0, 300, 1100, dtype, True)
    # more groups than are sorted by size; and the most there can be
    check_wgrad([i % 4 for i in range(1100)], 3, 24, 40, dtype, False)
    check_wgrad([i % 2 for i in range(4096)], 0, 8, 16, dtype, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_most_groups(dtype):
    check_rows([i % 3 for i in range(4096)], 7, 24, 40, dtype, False, False)
    check_rows([0] * 4095 + [2000], 7, 24, 40, dtype, False, True)


@pytest.mark.parametrize("mean", [1, 400])
def test_rows_past_32_bit_offsets(mean):
    # A beyond 4 GiB, on the tiles of few and of many rows: the last groups
    K, N = 4096, 40
    rows = 560_000
    G = min(rows // mean, 4096)
    sizes = [mean] * (G - 1)
    off = offsets_of(sizes + [rows - sum(sizes)])
    a = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    tail = normal((300, K), "bf16", 1)
    a[-300:] = tail.cuda()
    b = normal((G, K, N), "bf16", 2) if G < 1500 else normal((1, K, N), "bf16", 2).expand(G, K, N)
    c = gsk.grouped_matmul(a, b.cuda(), torch.from_numpy(off).to(torch.int32).cuda())
    g_of = np.searchsorted(off, np.arange(rows - 300, rows), side="right") - 1
    ref, size = np.zeros((300, N)), np.zeros((300, N))
    for g in np.unique(g_of):
        m = g_of == g
        B = f64(b[g])
        ref[m], size[m] = f64(tail)[m] @ B, np.abs(f64(tail)[m]) @ np.abs(B)
    within(c[-300:], ref, 2 * K * U * size)
    assert (c[:1000] == 0).all()
    w = gsk.grouped_matmul_wgrad(a, a[:, :N].contiguous(), torch.from_numpy(off).to(torch.int32).cuda())
    m = f64(tail)[g_of == G - 1]
    ref, size = m.T @ m[:, :N], np.abs(m).T @ np.abs(m[:, :N])
    within(w[G - 1], ref, 2 * rows * U * size)


def test_strided_inputs_are_taken_as_they_are():
    off = torch.tensor([0, 70, 130], dtype=torch.int32, device="cuda")
    a, b = normal((260, 80), "f16", 1).cuda(), normal((4, 80, 96), "f16", 2).cuda()
    ref = gsk.grouped_matmul(a[::2].contiguous(), b[::2].contiguous(), off)
    assert torch.equal(gsk.grouped_matmul(a[::2], b[::2], off), ref)
    # a view that starts at an odd element
    flat = torch.empty(130 * 80 + 1, dtype=torch.float16, device="cuda")
    flat[1:] = a[::2].reshape(-1)
    assert torch.equal(gsk.grouped_matmul(flat[1:].view(130, 80), b[::2], off), ref)


def block(x, ids, weights, w, dy, groups):
    """A mixture-of-experts layer, forward and backward."""
    r = gsk.route_rows(ids, groups)
    xs = gsk.gather_rows(x, r)
    ys = gsk.grouped_matmul(xs, w, r.offsets, out_dtype=x.dtype)
    y = gsk.combine_rows(ys, weights, r)
    dys, dweights = gsk.combine_rows_backward(dy, ys, weights, r)
    dw = gsk.grouped_matmul_wgrad(xs, dys, r.offsets)
    dxs = gsk.grouped_matmul(dys, w.transpose(1, 2), r.offsets, out_dtype=x.dtype)
    return y, gsk.gather_rows_backward(dxs, r), dw, dweights


def test_layer_gradients_against_autograd_in_64_bits():
    T, k, G, K, N = 50, 3, 6, 40, 56
    ids = random_ids(T, k, G, 0.15, 8)
    x, w = normal((T, K), "f32", 1), normal((G, K, N), "f32", 2)
    p, dy = normal((T, k), "f32", 3), normal((T, N), "f32", 4)
    got = block(x.cuda(), ids.cuda(), p.cuda(), w.cuda(), dy.cuda(), G)
    X, W, P = (t.double().requires_grad_() for t in (x, w, p))
    rows = []
    for t in range(T):
        y = torch.zeros(N, dtype=torch.float64)
        for j in range(k):
            g = int(ids[t, j])
            if 0 <= g < G:
                y = y + P[t, j] * (X[t] @ W[g])
        rows.append(y)
    Y = torch.stack(rows)
    Y.backward(dy.double())
    # fp32 all the way: every stage is within its own 2 n u, so a few hundred u
    # of the largest sums involved
    for g, ref in zip(got, (Y, X.grad, W.grad, P.grad)):
        scale = float(ref.detach().abs().max()) * np.sqrt(max(T, K, N))
        within(g, f64(ref), 2 * (K + N + T) * U * scale)


def test_gradients_against_differences():
    # C is linear in a and in b: a difference of one entry is the gradient's
    # entry, up to the fp32 rounding of the two sums
    sizes, K, N = [9, 0, 20, 3], 24, 40
    off = torch.from_numpy(offsets_of(sizes)).to(torch.int32).cuda()
    a, b = normal((32, K), "f32", 1).cuda(), normal((4, K, N), "f32", 2).cuda()
    dc = normal((32, N), "f32", 3).cuda()
    da = gsk.grouped_matmul(dc, b.transpose(1, 2), off)
    db = gsk.grouped_matmul_wgrad(a, dc, off)
    loss = lambda x, y: float((gsk.grouped_matmul(x, y, off).double() * dc.double()).sum())  # noqa: E731
    here = loss(a, b)
    bound = 4 * K * U * float((a.abs().max() * b.abs().max() * dc.abs().max() * 32 * N * K))
    for r, k in [(0, 0), (8, 23), (9, 5), (31, 11)]:
        step = torch.zeros_like(a)
        step[r, k] = 1.0
        assert abs(loss(a + step, b) - here - float(da[r, k])) <= bound
    for g, k, n in [(0, 0, 0), (1, 3, 4), (2, 23, 39), (3, 7, 20)]:
        step = torch.zeros_like(b)
        step[g, k, n] = 1.0
        assert abs(loss(a, b + step) - here - float(db[g, k, n])) <= bound
    assert (db[1] == 0).all()


def test_captured_layer_replays():
    T, k, G, K, N = 96, 4, 12, 136, 72
    dev = dict(device="cuda")
    x, dy = torch.zeros(T, K, **dev).bfloat16(), torch.zeros(T, N, **dev).bfloat16()
    w, p = normal((G, K, N), "bf16", 2).cuda(), torch.zeros(T, k, **dev)
    ids = torch.zeros(T, k, dtype=torch.int32, **dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, ids, p, w, dy, G)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block(x, ids, p, w, dy, G)
    for seed in range(4):
        x.copy_(normal((T, K), "bf16", seed))
        dy.copy_(normal((T, N), "bf16", seed + 10))
        p.copy_(normal((T, k), "f32", seed + 20))
        ids.copy_(random_ids(T, k, G, 0.1 * seed, seed))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, block(x, ids, p, w, dy, G)):
            assert torch.equal(a, b), seed


def test_runs_give_the_same_bits():
    off = torch.tensor([0, 300, 300, 411, 900], dtype=torch.int32, device="cuda")
    a, b = normal((1000, 520), "bf16", 1).cuda(), normal((4, 520, 264), "bf16", 2).cuda()
    d = normal((1000, 264), "bf16", 3).cuda()
    first = [gsk.grouped_matmul(a, b, off), gsk.grouped_matmul_wgrad(a, d, off)]
    for _ in range(3):
        for x, y in zip(first, (gsk.grouped_matmul(a, b, off), gsk.grouped_matmul_wgrad(a, d, off))):
            assert torch.equal(x, y)
