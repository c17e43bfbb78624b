"""The calls around a layer's projections in plain numpy: the residual norms in the fp32 steps of their definition (the
sums in 64 bits, rounded once), the adapters in 64 bits with the error that the kernels' sums allow.

Adapters.  low_i = sum_j A_ij x_j and out_o = base_o + s sum_i B_oi low_i.  Products are exact or fused; a term of low meets
at most c roundings of partial sums (half a step, 2^-24, each; the tensor cores' sums drop bits instead of rounding them:
a step), c = 96 + in / 128: at most 32 terms of a thread or 32 steps of a run of matrix products, 5 + 3 levels of a tree or
8 or 16 parts, in / 256 runs, the scale.  x and low enter the tensor cores to 24 bits: 2^-24 each.  A term of out meets at
most r + 4 roundings, r the rank.
"""
import numpy as np

U = 2.0 ** -24


def inverse_rms(x, eps):
    total = (x.astype(np.float64) ** 2).sum(-1, keepdims=True).astype(np.float32)
    mean = (total / np.float32(x.shape[-1])).astype(np.float32)
    return np.float32(1.0) / np.sqrt(mean + np.float32(eps), dtype=np.float32)


def residual_norm(h, y, gamma_next, eps, gamma_post=None, post=False, gate=None, scale=1.0, store=lambda v: v):
    """fp32 arrays; store rounds h' to the stream's type and back.  -> n, h' (fp32)."""
    u = y
    if post:
        u = u * inverse_rms(y, eps)
        if gamma_post is not None:
            u = u * gamma_post
    if gate is not None:
        u = gate * u
    h = store(np.float32(scale) * h + u)
    n = h * inverse_rms(h, eps)
    if gamma_next is not None:
        n = n * gamma_next
    return n, h


def lora(x, a, b, ids, ranks, scales, base):
    """float64 arrays.  -> out, bound on |error|."""
    n, n_in = x.shape
    out = np.zeros((n, b.shape[1])) if base is None else base.astype(np.float64).copy()
    err = np.zeros_like(out)
    c = 96 + n_in / 128
    for k in np.unique(ids[(ids >= 0) & (ids < a.shape[0])]):
        t = np.flatnonzero(ids == k)
        r, s = int(np.clip(ranks[k], 0, a.shape[1])), float(scales[k])
        ak, bk = a[k, :r], b[k, :, :r]
        low, low_abs = x[t] @ ak.T, np.abs(x[t]) @ np.abs(ak).T
        out[t] += s * (low @ bk.T)
        err[t] += abs(s) * (((c + 2) * U * low_abs + (r + 4) * U * np.abs(low)) @ np.abs(bk).T)
    return out, err + U * np.abs(out) + 1e-37
