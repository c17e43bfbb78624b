"""What q8_residual_norm promises of its sums of squares, shown in numpy steps of fp32 (no GPU): two words, each square with its
rounding error, each addition with its own (Knuth), joined over threads.

Bound: of a sum of L additions in a row (L <= 16 of a thread's pairs + 16 warps + 6 of a tree), the low word is at most L halves of a step,
L 2^-24 S, and is itself rounded L times: L^2 2^-48 S < 2^-37 S.  That holds as long as the squares' errors are numbers of fp32, which is so
for |x| >= 2^-51 (the last bit of x^2 is then at least 2^-149)."""
import numpy as np
import pytest

F = np.float32


def add(ah, al, bh, bl):
    h = ah + bh
    b = h - ah
    e = (ah - (h - b)) + (bh - b)
    return h, (al + bl) + e


def squares(x):
    p = x * x
    e = (x.astype(np.float64) ** 2 - p.astype(np.float64)).astype(F)     # fma(x, x, -p): exact in 64 bits, rounded once
    return p, e


def two_words(x, per_thread, one_warp):
    """x [dim] fp32: threads take chunks of 8, `per_thread` of them; even and odd values apart."""
    chunks = x.size // 8
    threads = -(-(-(-chunks // per_thread)) // 32) * 32
    pad = np.zeros((per_thread * threads, 8), F)
    pad[:chunks] = x.reshape(-1, 8)
    v = pad.reshape(per_thread, threads, 4, 2).transpose(1, 0, 2, 3).reshape(threads, -1, 2)
    h, l = squares(v[:, 0])
    for i in range(1, v.shape[1]):
        p, e = squares(v[:, i])
        s = h + p
        b = s - h
        r = (h - (s - b)) + (p - b)
        h, l = s, l + (r + e)
    h, l = add(h[:, 0], l[:, 0], h[:, 1], l[:, 1])
    h, l = h.reshape(-1, 32), l.reshape(-1, 32)

    def lanes(h, l):
        for o in (16, 8, 4, 2, 1):
            h, l = add(h, l, h[..., np.arange(32) ^ o], l[..., np.arange(32) ^ o])
        return h[..., 0], l[..., 0]
    if one_warp:
        H, L = h[0], l[0]
        for w in range(1, h.shape[0]):
            H, L = add(H, L, h[w], l[w])
        return lanes(H, L)
    h, l = lanes(h, l)
    H, L = np.zeros(32, F), np.zeros(32, F)
    H[:h.size], L[:h.size] = h, l
    return lanes(H, L)


@pytest.mark.parametrize("dim,per_thread,one_warp", [(32, 1, False), (2080, 1, True), (4096, 1, True), (4096, 1, False), (8192, 1, False), (8192, 4, False),
                                                     (32768, 4, False)])
# 1e15: S, up to 32768 (1e15)^2 e^4.5 = 3e36 in the mean, stays a number of fp32 (with 1e18 it would be 3e42, infinite)
@pytest.mark.parametrize("size", [1.0, 1e15, 1e-13])
def test_the_sum_of_squares_in_two_words(dim, per_thread, one_warp, size):
    rng = np.random.default_rng(dim)
    errors = []
    for kind in range(30):
        x = (size * (rng.standard_normal(dim) if kind % 2 else rng.lognormal(0, 1.5, dim))).astype(F)
        x[np.abs(x) < 2.0 ** -51] = 0
        want = np.sum(x.astype(np.longdouble) ** 2)
        h, l = two_words(x, per_thread, one_warp)
        errors.append(abs(float((np.longdouble(h) + np.longdouble(l) - want) / want)))
    assert max(errors) < 2.0 ** -37
    assert np.median(errors) < 2.0 ** -45      # what is usual: the words' roundings fall to either side


def test_smaller_values_lose_their_squares_errors():
    """Below 2^-51 the bound does not hold: by how much is why an eps above 1e-25 leaves nothing of it in the norm."""
    x = np.full(4096, 1.2345e-20, F)
    want = np.sum(x.astype(np.float64) ** 2)
    h, l = two_words(x, 1, True)
    assert 2.0 ** -37 < abs(float(h) + float(l) - want) / want < 2.0 ** -8
    assert want / 4096 / 1e-25 < 2.0 ** -24
