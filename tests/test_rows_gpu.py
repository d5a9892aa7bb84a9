"""Routing rows to groups and back on the GPU, with the gradients, against
plain 64-bit implementations (bounds: rows_util)."""
import numpy as np
import pytest

from rows_util import TYPES, U, f64, normal, random_ids, rounded, route, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import persistent_stream_tiling_amd as gsk  # noqa: E402


def routed(ids, groups):
    r = gsk.route_rows(ids.cuda(), groups)
    torch.cuda.synchronize()
    return r


# one and no tokens, one group, a wave's worth, several workgroups' worth, more
# groups than one thread each can own, groups that no counter row of sixteen
# waves holds, everything dropped
ROUTES = [(0, 2, 5, 0.0), (1, 1, 1, 0.0), (1, 8, 128, 0.0), (7, 3, 4, 0.5), (64, 1, 64, 0.1),
          (513, 8, 128, 0.0), (2048, 2, 257, 0.2), (1366, 3, 8, 0.0), (5000, 6, 60, 0.3),
          (40000, 8, 256, 0.05), (3000, 2, 1024, 0.0), (3000, 2, 5000, 0.1),
          (2500, 4, 16382, 0.0), (600, 4, 9, 1.0)]


@pytest.mark.parametrize("tokens,choices,groups,drop", ROUTES)
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_route_is_the_stable_sort(tokens, choices, groups, drop, id_type):
    ids = random_ids(tokens, choices, groups, drop, tokens + groups, id_type)
    r = routed(ids, groups)
    offsets, order, position = route(ids.numpy(), groups)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.position.cpu().numpy(), position)


def test_route_ids_beyond_32_bits_are_dropped_not_wrapped():
    ids = torch.tensor([[2 ** 32, 1], [-2 ** 32 + 1, 2 ** 40 + 2]], dtype=torch.int64)
    r = routed(ids, 4)
    assert r.offsets.cpu().tolist() == [0, 0, 1, 1, 1]
    assert r.order.cpu().tolist() == [1, -1, -1, -1]
    assert r.position.cpu().tolist() == [[-1, 0], [-1, -1]]


def test_route_one_id_per_token_and_strided_ids():
    ids = torch.tensor([3, 0, 3, 9, 1], dtype=torch.int64)
    r = routed(ids, 4)
    assert r.position.cpu().tolist() == [[2], [0], [3], [-1], [1]]
    wide = torch.randint(0, 6, (50, 8), dtype=torch.int32)
    strided = wide.cuda()[:, ::2]
    r, ref = gsk.route_rows(strided, 6), route(wide.numpy()[:, ::2], 6)
    assert np.array_equal(r.order.cpu().numpy(), ref[1])


# rows of one element, of a part of a 16-byte word, of whole words, odd, and
# longer than a workgroup covers at once
SHAPES = [(1, 1, 2, 1, 0.0), (5, 3, 4, 7, 0.3), (64, 8, 128, 256, 0.0), (33, 2, 5, 1410, 0.2),
          (130, 12, 20, 520, 0.1), (9, 17, 40, 2051, 0.4), (3, 2, 4, 9000, 0.0),
          (20, 4, 6, 64, 1.0)]


@pytest.mark.parametrize("tokens,choices,groups,cols,drop", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gather_and_its_gradient(tokens, choices, groups, cols, drop, dtype):
    ids = random_ids(tokens, choices, groups, drop, cols)
    r = routed(ids, groups)
    offsets, order, position = route(ids.numpy(), groups)
    x = normal((tokens, cols), dtype, 1)
    xs = gsk.gather_rows(x.cuda(), r).cpu()
    want = torch.zeros_like(xs)
    live = offsets[-1]
    want[:live] = x[torch.from_numpy(order[:live]) // choices]
    assert torch.equal(xs, want)

    dxs = normal((tokens * choices, cols), dtype, 2)
    dxs[live:] = float("nan")  # rows of no entry are never read
    dx = gsk.gather_rows_backward(dxs.cuda(), r)
    d = f64(dxs)
    ref, size = np.zeros((tokens, cols)), np.zeros((tokens, cols))
    for (t, j), row in np.ndenumerate(position):
        if row >= 0:
            ref[t] += d[row]
            size[t] += np.abs(d[row])
    within(dx, ref, rounded(2 * choices * U * size, ref, TYPES[dtype]), "dx")


@pytest.mark.parametrize("tokens,choices,groups,cols,drop", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_combine_and_its_gradient(tokens, choices, groups, cols, drop, dtype):
    ids = random_ids(tokens, choices, groups, drop, cols + 1)
    r = routed(ids, groups)
    offsets, order, position = route(ids.numpy(), groups)
    live = offsets[-1]
    ys = normal((tokens * choices, cols), dtype, 3)
    ys[live:] = float("nan")
    w = normal((tokens, choices), "f32", 4)
    w[position < 0] = float("nan")  # a dropped choice's weight is not used either
    dy = normal((tokens, cols), dtype, 5)
    y = gsk.combine_rows(ys.cuda(), w.cuda(), r)
    dys, dw = gsk.combine_rows_backward(dy.cuda(), ys.cuda(), w.cuda(), r)
    Y, W, D = f64(ys), f64(w), f64(dy)
    ref, size = np.zeros((tokens, cols)), np.zeros((tokens, cols))
    rdys, rdw, sdw = np.zeros(Y.shape), np.zeros(W.shape), np.zeros(W.shape)
    for (t, j), row in np.ndenumerate(position):
        if row >= 0:
            ref[t] += W[t, j] * Y[row]
            size[t] += np.abs(W[t, j] * Y[row])
            rdys[row] = W[t, j] * D[t]
            rdw[t, j] = D[t] @ Y[row]
            sdw[t, j] = np.abs(D[t]) @ np.abs(Y[row])
    within(y, ref, rounded(2 * choices * U * size, ref, TYPES[dtype]), "y")
    within(dys, rdys, rounded(U * np.abs(rdys), rdys, TYPES[dtype]), "dys")
    # (a product of two fp32 values is rounded too, or fused: within 2 (n + 1) u)
    within(dw, rdw, 2 * (cols + 1) * U * sdw + 2.0 ** -149, "dweights")
    assert (dys[live:] == 0).all()


def test_combine_gradient_against_differences():
    # y is linear in ys and in the weights: differences are exact up to rounding
    ids = random_ids(6, 3, 4, 0.2, 11)
    r = routed(ids, 4)
    ys, w = normal((18, 40), "f32", 1).cuda(), normal((6, 3), "f32", 2).cuda()
    dy = normal((6, 40), "f32", 3).cuda()
    dys, dw = gsk.combine_rows_backward(dy, ys, w, r)
    loss = lambda a, b: float((gsk.combine_rows(a, b, r).double() * dy.double()).sum())  # noqa: E731
    live = int(r.offsets[-1])
    for row, col in [(0, 0), (live - 1, 39), (live // 2, 17), (17, 3)]:
        step = torch.zeros_like(ys)
        step[row, col] = 1.0
        diff = loss(ys + step, w) - loss(ys, w)
        assert abs(diff - float(dys[row, col])) < 1e-4 if row < live else diff == 0
    for t in range(6):
        for j in range(3):
            step = torch.zeros_like(w)
            step[t, j] = 1.0
            assert abs(loss(ys, w + step) - loss(ys, w) - float(dw[t, j])) < 1e-3


def test_positions_out_of_range_touch_nothing():
    # a routing whose buffers hold nonsense: nothing outside the outputs is
    # read or written, and entries in range are still right
    tokens, choices, cols = 8, 2, 24
    position = torch.tensor([[0, 5], [10 ** 9, 1], [-5, 2], [16, 3], [2 ** 31 - 1, 4],
                             [-2 ** 31, 6], [7, 8], [9, 10]], dtype=torch.int32)
    kept = torch.tensor([0, 10 ** 9], dtype=torch.int32)
    r = gsk.Routing(kept.cuda(), torch.zeros(16, dtype=torch.int32, device="cuda"),
                    position.cuda())
    ys = normal((16, cols), "f32", 1)
    y = gsk.combine_rows(ys.cuda(), torch.ones(tokens, choices, device="cuda"), r).cpu()
    want = torch.zeros(tokens, cols)
    for t in range(tokens):
        for j in range(choices):
            p = int(position[t, j])
            if 0 <= p < 16:
                want[t] += ys[p]
    assert torch.equal(y, want)
    xs = gsk.gather_rows(ys[:8].cuda(), r).cpu()
    assert torch.equal(xs[5], ys[0]) and torch.equal(xs[8], ys[6]) and torch.equal(xs[1], ys[1])
    dys, dw = gsk.combine_rows_backward(ys[:8].cuda(), ys.cuda(), torch.ones(8, 2, device="cuda"), r)
    assert torch.equal(dys.cpu()[:11], xs[:11]) and float(dw[1, 0]) == 0.0


def test_more_tokens_than_one_launch_holds():
    # workgroups go round again past 65536 of them
    tokens, cols = 65536 * 2 + 77, 1030
    ids = torch.randint(0, 3, (tokens, 1), dtype=torch.int32, device="cuda")
    r = gsk.route_rows(ids, 3)
    x = torch.randn(tokens, cols, device="cuda").to(torch.bfloat16)
    xs = gsk.gather_rows(x, r)
    assert torch.equal(xs, x[r.order.long()])
    assert torch.equal(gsk.gather_rows_backward(xs, r), x)
    one = torch.ones(tokens, 1, device="cuda")
    dys, dw = gsk.combine_rows_backward(x, xs, one, r)
    assert torch.equal(dys, xs)
    ref = (x.double() ** 2).sum(1, keepdim=True)
    assert bool(((dw.double() - ref).abs() <= 2 * (cols + 1) * U * ref).all())


def test_rows_past_32_bit_offsets():
    # sorted rows beyond 4 GiB
    tokens, choices, cols = 290_000, 8, 1024
    ids = torch.randint(0, 16, (tokens, choices), dtype=torch.int32, device="cuda")
    r = gsk.route_rows(ids, 16)
    x = torch.randn(tokens, cols, device="cuda").to(torch.bfloat16)
    xs = gsk.gather_rows(x, r)
    last = torch.arange(tokens * choices - 5000, tokens * choices, device="cuda")
    assert torch.equal(xs[last], x[r.order[last].long() // choices])
    w = torch.ones(tokens, choices, device="cuda")
    y = gsk.combine_rows(xs, w, r)  # eight times x, exactly
    assert torch.equal(y, x * 8)
    dys, dw = gsk.combine_rows_backward(x, xs, w, r)
    assert torch.equal(dys[last], xs[last])


def test_same_bits_on_another_stream_and_again():
    ids = random_ids(700, 4, 30, 0.1, 3).cuda()
    ys, w = normal((2800, 333), "bf16", 1).cuda(), normal((700, 4), "f32", 2).cuda()
    dy = normal((700, 333), "bf16", 4).cuda()

    def all_of_it():
        r = gsk.route_rows(ids, 30)
        return [r.offsets, r.order, r.position, gsk.gather_rows(dy, r), gsk.combine_rows(ys, w, r),
                gsk.gather_rows_backward(ys, r), *gsk.combine_rows_backward(dy, ys, w, r)]

    ref = all_of_it()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = all_of_it()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(ref, again):
        # (weights of dropped entries and the like never reach an output: no NaN here)
        assert torch.equal(a, b)
