"""Adapters of many requests beside a shared projection, against a plain 64-bit
implementation.

Bound: the shared product as in rows_util; H = s X A^T is an fp32 sum of K
products (2 K u of the sum of magnitudes, one more u for the scale), then held
to at least 16 bits more coarsely only where 16-bit instructions take it: split
into terms it is off by at most 2^-16 of the largest magnitude among the 16
ranks of its row that share a scale (two terms of 8 bits for bf16 with bf16
results; fp16 and three terms are finer), and H B^T is a sum of rank products.
"""
import numpy as np
import pytest

from rows_util import TYPES, U, f64, normal, rounded, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import persistent_stream_tiling_amd as gsk  # noqa: E402


def reference(x, w, a, b, ids, scales, split):
    """(Y, bound of the fp32 result); split: how far H is held, relative to its
    row's largest magnitude."""
    X, W, A, B = f64(x), f64(w), f64(a), f64(b)
    K, r = X.shape[1], A.shape[1]
    y, bound = X @ W, 2 * max(K, 1) * U * (np.abs(X) @ np.abs(W))
    for t, g in enumerate(ids.tolist()):
        if 0 <= g < A.shape[0]:
            s = float(scales[g]) if scales is not None else 1.0
            h, size = s * (A[g] @ X[t]), abs(s) * (np.abs(A[g]) @ np.abs(X[t]))
            off = 2 * (K + 1) * U * size + split * np.abs(h).max(initial=0.0)
            y[t] += B[g] @ h
            bound[t] += np.abs(B[g]) @ off + 2 * (r + 2) * U * (np.abs(B[g]) @ (np.abs(h) + off))
    return y, bound


def check(T, K, N, r, L, ids, dtype, half, trans, seed=1, scaled=True):
    x, w = normal((T, K), dtype, seed), normal((K, N), dtype, seed + 1, max(K, 1) ** -0.5)
    a, b = normal((L, r, K), dtype, seed + 2, max(K, 1) ** -0.5), normal((L, N, r), dtype, seed + 3)
    scales = torch.rand(L, generator=torch.Generator().manual_seed(seed)) * 3 if scaled else None
    dw = w.t().contiguous().cuda().t() if trans else w.cuda()
    out = TYPES[dtype] if half else torch.float32
    y = gsk.adapter_matmul(x.cuda(), dw, a.cuda(), b.cuda(), ids.cuda(),
                           None if scales is None else scales.cuda(), out_dtype=out)
    assert y.dtype == out
    split = {"f32": 0.0, "f16": 2.0 ** -21, "bf16": 2.0 ** -16 if half else 2.0 ** -23}[dtype]
    ref, bound = reference(x, w, a, b, ids, scales, split)
    within(y, ref, rounded(bound, ref, out), f"{T}x{K}x{N} r={r} L={L}")


def some_ids(T, L, seed, none=0.2):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, max(L, 1), size=T)
    gone = rng.random(T) < (none if L else 1.0)
    ids[gone] = rng.choice([-1, L, -2 ** 31, 2 ** 31 - 1, L + 3], size=int(gone.sum()))
    return torch.from_numpy(ids).to(torch.int32)


# one row, a few, each row its own adapter, tiles' ends, several row tiles
ROWS = [1, 2, 16, 17, 31, 33, 64, 65, 128, 129, 200]


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("trans", [False, True], ids=["w", "wT"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows(T, trans, dtype):
    ids = some_ids(T, 40, T)
    check(T, 520, 264, 16, 40, ids, dtype, True, trans, seed=T)
    check(T, 203, 101, 5, 40, ids, dtype, False, trans, seed=T)


@pytest.mark.parametrize("r", [1, 7, 8, 15, 16, 17, 32, 40, 64, 65, 100, 128])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_ranks(r, dtype):
    check(45, 520, 264, r, 3, some_ids(45, 3, r), dtype, False, True, seed=r)
    check(90, 264, 203, r, 30, some_ids(90, 30, r), dtype, True, False, seed=r, scaled=False)


@pytest.mark.parametrize("K,N", [(1, 1), (8, 8), (64, 128), (255, 129), (2048, 40), (4104, 257),
                                 (1000, 1000)])
@pytest.mark.parametrize("trans", [False, True], ids=["w", "wT"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_depths(K, N, trans, dtype):
    check(40, K, N, 16, 9, some_ids(40, 9, K), dtype, False, trans, seed=N)


@pytest.mark.parametrize("trans", [False, True], ids=["w", "wT"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_tiles(trans, dtype):
    # enough 256x256 tiles for the kernel of many rows; runs of rows of one
    # adapter and rows in any order
    T, K, N, L = 1300, 136, 6200, 6
    runs = torch.from_numpy(np.repeat([3, -1, 0, 5, 2, 3, 4], [300, 40, 1, 259, 300, 100, 300])).int()
    for ids in (runs, some_ids(T, L, 3)):
        check(T, K, N, 24, L, ids, dtype, True, trans)
    check(T, K, N, 16, L, runs, dtype, False, trans)


@pytest.mark.parametrize("r", [5, 16, 24, 40, 64, 100, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_rows_in_runs_and_in_any_order(r, dtype):
    # prompts: runs of rows that end inside 64-row blocks, some rows without an
    # adapter, a stretch of rows in any order (many adapters in a block); depth
    # cut into slices, the last one shorter
    T, K, N, L = 1091, 648, 3336, 40
    rng = np.random.default_rng(r)
    ids = np.repeat(rng.integers(-1, L, size=60), 30)[:T]
    ids[500:800] = rng.integers(-1, L + 1, size=300)
    check(T, K, N, r, L, torch.from_numpy(ids).int(), dtype, r % 2 == 0, True, seed=r)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_no_row_has_an_adapter(dtype):
    check(70, 136, 264, 16, 4, torch.full((70,), -1, dtype=torch.int32), dtype, True, True)
    check(5, 136, 264, 16, 0, torch.zeros(5, dtype=torch.int32), dtype, True, True)
    y = gsk.adapter_matmul(*(torch.empty(s, device="cuda", dtype=TYPES[dtype]) for s in
                             [(0, 8), (8, 4), (2, 3, 8), (2, 4, 3)]),
                           torch.empty(0, dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 4)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_no_depth(dtype):
    t = dict(device="cuda", dtype=TYPES[dtype])
    ids = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda")
    y = gsk.adapter_matmul(torch.empty(3, 0, **t), torch.empty(0, 9, **t), torch.empty(2, 4, 0, **t),
                           torch.ones(2, 9, 4, **t), ids)
    assert y.shape == (3, 9) and (y == 0).all()


@pytest.mark.parametrize("T", [40, 1300])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_an_adapter_not_finite_reaches_only_its_rows(T, dtype):
    K, N, r, L = 136, 6200 if T > 1000 else 264, 16, 5
    x, w = normal((T, K), dtype, 1), normal((K, N), dtype, 2)
    a, b = normal((L, r, K), dtype, 3), normal((L, N, r), dtype, 4)
    ids = some_ids(T, L, 5)
    clean = gsk.adapter_matmul(*(t.cuda() for t in (x, w, a, b, ids))).cpu()
    b[2, 7, 3] = float("inf")
    b[2, 8] = float("nan")
    a[4, 2, 5] = float("-inf")
    y = gsk.adapter_matmul(*(t.cuda() for t in (x, w, a, b, ids))).cpu()
    hit2, hit4 = ids == 2, ids == 4
    assert torch.equal(y[~(hit2 | hit4)], clean[~(hit2 | hit4)])
    assert torch.isnan(y[hit2][:, 8]).all() and not torch.isfinite(y[hit2][:, 7]).any()
    keep = [c for c in range(N) if c not in (7, 8)]
    assert torch.equal(y[hit2][:, keep], clean[hit2][:, keep])
    assert not torch.isfinite(y[hit4]).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_and_small_intermediates(dtype):
    # H far outside fp16's range on both sides, and ranks of very different
    # magnitude: fp32 results stay within the bound
    T, K, N, r = 40, 264, 136, 16
    x, w = normal((T, K), dtype, 1, 100.0), normal((K, N), dtype, 2)
    a, b = normal((3, r, K), dtype, 3, 100.0), normal((3, N, r), dtype, 4)
    a[1] *= 1e-4
    a[2, ::2] *= 1e-3
    b[0] *= 1e-3
    ids = torch.arange(T, dtype=torch.int32) % 3
    scales = torch.tensor([50.0, 1e-3, 7.0])
    y = gsk.adapter_matmul(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales.cuda())
    split = 2.0 ** -21 if dtype == "f16" else 2.0 ** -23
    ref, bound = reference(x, w, a, b, ids, scales, split)
    within(y, ref, bound)


def test_captured_and_on_another_stream():
    T, K, N, r, L = 32, 1032, 520, 16, 32
    x, w = normal((T, K), "bf16", 1).cuda(), normal((N, K), "bf16", 2).cuda().t()
    a, b = normal((L, r, K), "bf16", 3).cuda(), normal((L, N, r), "bf16", 4).cuda()
    ids = torch.arange(T, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = gsk.adapter_matmul(x, w, a, b, ids)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gsk.adapter_matmul(x, w, a, b, ids)
    assert torch.equal(gsk.adapter_matmul(x, w, a, b, ids), first)
    for seed in range(4):
        x.copy_(normal((T, K), "bf16", seed + 7))
        ids.copy_(some_ids(T, L, seed))
        graph.replay()
        torch.cuda.synchronize()
        for _ in range(3):  # the parts' order of arrival never shows
            assert torch.equal(gsk.adapter_matmul(x, w, a, b, ids), y)


def test_strided_and_misaligned_inputs():
    T, K, N, r, L = 20, 72, 88, 6, 4
    x, w = normal((2 * T, K), "f16", 1).cuda(), normal((K, 2 * N), "f16", 2).cuda()
    a, b = normal((L, r, K), "f16", 3).cuda(), normal((L, N, r), "f16", 4).cuda()
    ids = some_ids(2 * T, L, 1).cuda()
    ref = gsk.adapter_matmul(x[::2].contiguous(), w[:, :N].contiguous(), a, b, ids[::2].contiguous())
    assert torch.equal(gsk.adapter_matmul(x[::2], w[:, :N], a, b, ids[::2]), ref)
    flat = torch.empty(T * K + 1, dtype=torch.float16, device="cuda")
    flat[1:] = x[::2].reshape(-1)
    flat_a = torch.empty(a.numel() + 1, dtype=torch.float16, device="cuda")
    flat_a[1:] = a.reshape(-1)
    got = gsk.adapter_matmul(flat[1:].view(T, K), w[:, :N], flat_a[1:].view(L, r, K), b, ids[::2])
    assert torch.equal(got, ref)
