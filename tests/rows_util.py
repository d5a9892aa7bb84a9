"""Plain 64-bit implementations of the operators whose rows choose their matrix
(numpy, entry by entry), and the bounds their results are held to.

Bounds, with u = 2^-24 (half a step of fp32), h = half a step of the output
type relative to the value, and t the output type's smallest step near zero:
- a sum of n products in fp32, in any order and with each addition off by at
  most one step (matrix instructions may truncate): 2 n u * sum |products|;
- rounding a result to the output type: h * |result| + t / 2.
Products of 16-bit inputs are exact in fp32.
"""
import numpy as np
import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(bound, ref, dtype):
    """The bound of an fp32 result within `bound` of ref, once it is stored as dtype."""
    if dtype == torch.float32:
        return bound + 2.0 ** -149
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    return bound + half_step(dtype) * (np.abs(ref) + bound) + tiny / 2


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def within(got, ref, bound, what=""):
    g = f64(got) if isinstance(got, torch.Tensor) else got
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert not np.isnan(g).any(), f"{what}: NaN"
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} out of bound, first at "
                           f"{np.argwhere(bad)[0]}: {g[bad][0]} against {ref[bad][0]}")


def route(ids, groups):
    """offsets, order, position of ids (numpy, tokens x choices)."""
    flat = ids.reshape(-1)
    buckets = [[] for _ in range(groups)]
    for i, g in enumerate(flat):
        if 0 <= g < groups:
            buckets[g].append(i)
    kept = [i for b in buckets for i in b]
    offsets = np.cumsum([0] + [len(b) for b in buckets])
    order = np.full(flat.size, -1)
    order[:len(kept)] = kept
    position = np.full(flat.size, -1)
    position[kept] = np.arange(len(kept))
    return offsets, order, position.reshape(ids.shape)


def random_ids(tokens, choices, groups, drop, seed, dtype=torch.int32):
    """Ids with a share `drop` out of range on both sides."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, groups, size=(tokens, choices))
    gone = rng.random((tokens, choices)) < drop
    ids[gone] = rng.choice([-1, -7, groups, groups + 5], size=int(gone.sum()))
    return torch.from_numpy(ids).to(dtype)


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TYPES[dtype])


def grouped_ref(a, b, offsets):
    """(C, sum |a||b|) in 64 bits; a rows x K, b groups x K x N (numpy)."""
    c = np.zeros((a.shape[0], b.shape[2]))
    s = np.zeros_like(c)
    for g in range(b.shape[0]):
        lo, hi = offsets[g], offsets[g + 1]
        c[lo:hi] = a[lo:hi] @ b[g]
        s[lo:hi] = np.abs(a[lo:hi]) @ np.abs(b[g])
    return c, s


def wgrad_ref(a, d, offsets):
    parts = [(a[lo:hi].T @ d[lo:hi], np.abs(a[lo:hi]).T @ np.abs(d[lo:hi]))
             for lo, hi in zip(offsets, offsets[1:])]
    return np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])


def offsets_of(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
