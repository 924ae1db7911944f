"""With how many bits softmax weights enter the product with V: at least 16 wherever the interface
says so, in blocks of up to 16 query rows."""
import numpy as np
import pytest

from tests.common_keys_util import Cross, Shared, attention, status_of
from tests.gpu_util import as_f64
from synth.workloads import bf16_bits_to_f32, f32_to_bf16_bits
from tests.plain_ops import f64, slots_of

pytestmark = pytest.mark.gpu


def cancel(x, q, row, n):
    """One query for all the rows that read the n keys of a page-table row, and values, as many of either
    sign, each the reciprocal of its key's weight, so that the output is a small rest: its own rounding
    hides nothing.  Returns (out, bound) and the output with weights of 8 bits, by KV head."""
    G = x.Hq // x.Hkv
    q[:] = np.repeat(q[:1, ::G], G, axis=1)
    slots = slots_of(row, x.ps, n)
    k, v = (p.reshape(-1, x.Hkv, x.d) for p in (x.pool.k, x.pool.v))
    one = f64(q[:1, ::G])
    rounded = np.zeros((x.Hkv, x.d))
    for g in range(x.Hkv):
        s = f64(k[slots, g]) @ one[0, g] * x.scale
        p = np.exp(s - s.max())
        sign = x.pool.rng.permuted(np.where(np.arange(n) % 2, 1.0, -1.0)[:, None].repeat(x.d, 1), axis=0)
        v[slots, g] = f32_to_bf16_bits((sign * p.sum() / (n * p[:, None])).astype(np.float32))
        eight = bf16_bits_to_f32(f32_to_bf16_bits(p.astype(np.float32))).astype(np.float64)
        rounded[g] = eight / p.sum() @ f64(v[slots, g])
    out, bound = attention(one, f64(k[slots]), f64(v[slots]), x.scale, np.full(n, False))
    return out[0], bound[0], rounded


def check(x, got, seen):
    for rows, (out, bound, rounded) in seen:
        G = x.Hq // x.Hkv
        assert (np.abs(got[rows] - np.repeat(out, G, axis=0)) <= np.repeat(bound, G, axis=0)).all(), rows
        # weights of 8 bits would have been seen
        assert (np.abs(rounded - out) > 1.5 * bound).any(), rows
    assert status_of(x) == 0


@pytest.mark.parametrize("Hq,Hkv,d,tokens,requests", [
    (8, 8, 64, 9, 60), (8, 8, 64, 16, 60), (16, 2, 64, 2, 90), (4, 2, 64, 5, 90),  # heads of 64: always
    (16, 8, 128, 4, 100), (32, 4, 128, 1, 100),                                   # up to 8 rows: always
    (16, 8, 128, 5, 4), (16, 2, 128, 2, 9), (8, 8, 128, 16, 3)])                  # few segments
def test_cross_attention(Hq, Hkv, d, tokens, requests):
    x = Cross(tokens, [tokens] * requests, [8] * requests, Hq, Hkv, d, page_size=8)
    seen = [(slice(x.cu[r], x.cu[r + 1]), cancel(x, x.q[x.cu[r]:x.cu[r + 1]], x.table[r], 8)) for r in range(requests)]
    x.device()
    check(x, as_f64(x.call()), seen)


@pytest.mark.parametrize("Hq,Hkv,d,members,groups", [
    (8, 8, 64, 9, 60), (8, 8, 64, 16, 60), (16, 2, 64, 2, 90), (16, 8, 128, 4, 100), (32, 4, 128, 1, 100),
    (16, 8, 128, 5, 4), (16, 2, 128, 2, 9), (8, 8, 128, 16, 3)])
def test_decode_with_groups(Hq, Hkv, d, members, groups):
    """Shared keys alone."""
    x = Shared(members, [([0] * members, 1)] * groups, Hq, Hkv, d, page_size=8)
    seen = []
    for g in range(groups):
        rows = slice(x.start[g], x.start[g + 1])
        seen.append((rows, cancel(x, x.q[rows], x.table[x.start[g]], 8)))
    x.device()
    check(x, as_f64(x.call()), seen)
