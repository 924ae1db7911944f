"""paged_decode_attn_weights where its output is a small difference of large terms, so that bf16
shows errors far below the rounding of a usual output: the softmax weights have to be carried in 32
bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from tests.gpu_util import as_f64, dev
from tests.plain_ops import U

pytestmark = pytest.mark.gpu


def call(k, v, q, table, lens, scale):
    """k, v [pages, page size, Hkv, d], q [B, Hq, d]: the output in float64."""
    B, longest = len(lens), max(lens)
    acc = torch.zeros(B, k.shape[2], longest, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = pkv.paged_decode_attn_weights(q.bfloat16(), k.bfloat16(), v.bfloat16(), table,
                                        torch.tensor(lens, dtype=torch.int32, device=dev()), scale, acc, longest,
                                        dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return as_f64(out), acc.cpu().numpy()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [1, 8])
@pytest.mark.parametrize("c,n", [(2, 3), (4, 7), (6, 7), (5, 6), (9, 11), (5, 9)])
def test_every_bit_of_a_weight_counts(c, n, heads, d):
    """One key of score s with value -c, n keys of score 0 with value 1, exp(-s) = x = c / n nearly:
    the output is (n x - c) / (n x + 1), nearly 0.  x has no short binary form: the next 16 bits
    after a rounding to bf16's 8 would leave 1.8e-6 to 3.3e-6 of an output here.

    How far fp32 may be off, in U = 2^-24: the scores' products are exact, the exponent (at most
    0.85) takes 4 roundings: 2.4 of x; the exponential 2^-22 = 4 of x; the sums of at most 12
    products 2 in the last place of c = n x: 4, and one more where their parts meet; together
    11.4 n x / (n x + 1) < 12.  What multiplies the output afterwards is nothing next to that."""
    scale = float(np.float32(math.log(n / c)))
    k, v = torch.zeros(1, 16, 1, d, device=dev()), torch.ones(1, 16, 1, d, device=dev())
    k[0, 0, 0, 0], v[0, 0] = 1, -c
    q = torch.zeros(1, heads, d, device=dev())
    q[..., 0] = 1
    out, acc = call(k, v, q, torch.zeros(1, 1, dtype=torch.int32, device=dev()), [n + 1], scale)
    x = math.exp(-scale)
    want = (n * x - c) / (n * x + 1)
    assert abs(want) < 1e-8
    assert (np.abs(out - want) <= 12 * U).all()
    weights = heads * np.array([1.0] + [x] * n) / (n * x + 1)
    assert (np.abs(acc[0, 0] - weights) <= (12 + heads) * U * weights).all()
