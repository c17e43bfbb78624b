"""Attention in 64 bits from its definition, with the error that the kernels' roundings allow.

For weights w_j = softmax(z)_j and A = sum_j w_j |v_j| the kernels' output differs from the exact one by at most
  u_p A                          weights rounded to 16 bit (half a step: 2^-8 bf16, 2^-11 fp16; Q8_0 caches fp16)
  + 2 dz A                       scores: dz = (D + 8) 2^-23 scale sum_i |q_i k_i| + 4 |z| 2^-23, products' sums and
                                 the conversion to log2 units in fp32; it enters numerator and denominator
  + (2^-21 + (n/8 + 16) 2^-23) A the exponential (2^-22), n products and weights summed in fp32, n/8 steps
  + 2^-24 max|v| n               fp16 weights below 2^-14: absolute steps of 2^-24 against a largest weight of 1
  + u_out |out|                  the output's own rounding
"""
import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def attend(q, k, v, see, scale, sink, weight_type, out_type):
    """One head: q [rows, D], k and v [keys, D] float64, see [rows, keys] bool, sink or None.
    -> out, lse, bound on out, bound on lse.  k and v are read only where some row sees them."""
    rows, d = q.shape
    n = k.shape[0]
    out, bound = np.zeros((rows, d)), np.full((rows, d), 1e-30)
    lse, lse_bound = np.full(rows, -np.inf), np.zeros(rows)
    for r in range(rows):
        j = np.flatnonzero(see[r])
        z = k[j] @ q[r] * scale
        m = max([*z, *([sink] if sink is not None else [])], default=-np.inf)
        if m == -np.inf:
            continue
        total = np.exp(z - m).sum() + (np.exp(sink - m) if sink is not None else 0.0)
        lse[r] = m + np.log(total)
        dz = 0.0
        if len(j):
            dz = ((d + 8) * 2.0 ** -23 * scale * (np.abs(k[j]) @ np.abs(q[r]))).max() + 4 * np.abs(z).max() * 2.0 ** -23
        sums = 2.0 ** -21 + (len(j) / 8 + 16) * 2.0 ** -23
        lse_bound[r] = 2 * dz + sums + 8 * abs(lse[r]) * 2.0 ** -24
        if not len(j):
            continue
        w = np.exp(z - m) / total
        out[r] = w @ v[j]
        a = w @ np.abs(v[j])
        bound[r] = a * (HALF_STEP[weight_type] + 2 * dz + sums) + HALF_STEP[out_type] * np.abs(out[r]) + 1e-30
        if weight_type == "f16":
            bound[r] += 2.0 ** -24 * np.abs(v[j]).max() * len(j)
    return out, lse, bound, lse_bound
