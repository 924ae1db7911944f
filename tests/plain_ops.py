"""Plain 64-bit forms of the operators around the cache (numpy, one row at a time),
for the parity tests.  They share no code with the library."""
import numpy as np

from synth.workloads import bf16_bits_to_f32

U = 2.0 ** -24          # a rounding to fp32, relative
HALF_STEP = 2.0 ** -8   # a rounding to bf16, relative


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def norm_rope(x, weight, eps, cos, sin, interleaved):
    """(y, bound) of head rows x [T, H, d] in float64; cos, sin [T, R/2].

    bound: how far the fp32 computation and its rounding to bf16 may be from y.  The norm's
    factor comes from at most 19 additions of squares (half of their error after the square
    root), a division, an addition and a reciprocal square root of 2 units, then two products;
    the rotation adds a product and an fma: under 32 U of |a| + |b| in all."""
    d = x.shape[-1]
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    out, size = y.copy(), np.abs(y)
    if half:
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., a] * sin + y[..., b] * cos
        both = np.abs(y[..., a]) + np.abs(y[..., b])
        size[..., a] = both
        size[..., b] = both
    assert d % 2 == 0
    return out, HALF_STEP * np.abs(out) + 32 * U * size


def slots_of(page_table_row, page_size, n):
    j = np.arange(n)
    return page_table_row[j // page_size].astype(np.int64) * page_size + j % page_size


def decode_weights(q, k_pool, v_pool, page_table, seq_lens, scale):
    """Per sequence: (out [Hq, d], weights [Hkv, L], bound of out, bound of weights).

    The scores are fp32 sums of d products (q * scale * log2 e rounded, then at most 22 steps a
    product passes through), so a weight's exponent is off by at most 23 U of the sum of |q k|;
    the exponential by 2^-22; the sum over the keys passes through at most L / 8 + 64 steps.
    Numerator and denominator both.  The exponential flushes results under 2^-126 to zero, and
    the sum that it is divided by is at least 1 (the reference that is subtracted is a score that
    occurs): at most 2^-126 of a query head's weight is lost that way, which no relative bound
    covers."""
    Hq, d = q.shape[1:]
    ps, Hkv = k_pool.shape[1:3]
    G = Hq // Hkv
    k_rows, v_rows = k_pool.reshape(-1, Hkv, d), v_pool.reshape(-1, Hkv, d)
    results = []
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        out, w = np.zeros((Hq, d)), np.zeros((Hkv, L))
        tol_out, tol_w = np.zeros((Hq, d)), np.zeros((Hkv, L))
        if L:
            slots = slots_of(page_table[b], ps, L)
            K, V = f64(k_rows[slots]), f64(v_rows[slots])
            Q = f64(q[b])
            for h in range(Hq):
                g = h // G
                s = K[:, g] @ Q[h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                size = (np.abs(K[:, g]) @ np.abs(Q[h])).max() * abs(scale)
                delta = 2 * (23 * U * size + 2.0 ** -22 + (L / 8 + 64) * U)
                out[h] = p @ V[:, g]
                w[g] += p
                tol_w[g] += delta * p + 2.0 ** -126
                tol_out[h] = HALF_STEP * np.abs(out[h]) + delta * (p @ np.abs(V[:, g]))
        results.append((out, w, tol_out, tol_w))
    return results


def evict_kept(sums, n, num_first, num_recent):
    """The kept positions (rising) of a row of sums [L]."""
    L = len(sums)
    n = min(n, L)
    first = min(num_first, n)
    recent = min(num_recent, n - first)
    middle = range(first, L - recent)

    def rank(j):
        x = float(sums[j])
        return (1, 0.0, j) if x != x else (0, -x + 0.0, j)

    heavy = sorted(middle, key=rank)[:n - first - recent]
    return np.array(list(range(first)) + sorted(heavy) + list(range(L - recent, L)), dtype=np.int32)
