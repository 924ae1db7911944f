"""paged_decode_attn_weights where its output is a small difference of large terms, so that bf16
shows errors far below the rounding of a usual output: the softmax weights and the sums over the
keys have to be carried in 32 bits."""
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


@pytest.mark.parametrize("d,heads", [(64, 1), (128, 1), (128, 8)])
def test_a_long_sum_does_not_drift(d, heads):
    """65536 keys with values from 1 to 1.25, and the same keys again with the negatives of their
    values: the output is 0.  Sequences enough that no block has more than one of them, all on the
    same pages.

    A running sum that loses half a unit in its last place, U / 2 of itself at least, with each of N
    tiles, and is half of its largest on average, ends N U / 4 of that largest sum from 0, N U / 8
    of the divisor: 256 U with the 2048 tiles of 64 keys, 512 U with 4096 of 32 keys.  Added up in
    128 parts of 32 sums, each of them off by at most 2 units in the last place (4 U) of the part's
    sum so far, 17 / 32 of the part on average: 68 U of the divisor for all parts, and where the
    parts meet at most U of the largest sum each, 64 U of the divisor.  With 13 U for the weights
    (see above) 145 U at the worst for values of 1, so 182 U here."""
    L, blocks = 131072, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    k, v = torch.zeros(L // 256, 256, 1, d, device=dev()), torch.empty(L // 256, 256, 1, d, device=dev())
    gen = torch.Generator(device=dev()).manual_seed(d + heads)
    scores = torch.rand(L // 2, generator=gen, device=dev()).div_(2).bfloat16().float().repeat(2)
    k.view(-1, d)[:, 0] = scores
    values = 1 + torch.rand(L // 2, d, generator=gen, device=dev()).mul_(32).floor_().div_(128)
    v.view(-1, d)[:L // 2], v.view(-1, d)[L // 2:] = values, -values
    q = torch.zeros(blocks, heads, d, device=dev())
    q[..., 0] = 1
    table = torch.arange(L // 256, dtype=torch.int32, device=dev()).repeat(blocks, 1)
    out, acc = call(k, v, q, table, [L] * blocks, 1.0)
    assert (np.abs(out) <= 182 * U).all(), np.abs(out).max() / U
    weights = heads * torch.softmax(scores.double(), 0).cpu().numpy()
    # a lane's share of the divisor is one addition per tile, each rounded; the rest as above
    assert (np.abs(acc[::50, 0] - weights) <= (L * d / 4096 + 64) * U * weights).all()
