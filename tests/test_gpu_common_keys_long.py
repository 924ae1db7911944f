"""Attention over common keys of very long sequences: a few pages that a row lists over and over, so
that the 64-bit form is a softmax over them with the number of times each key comes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from tests.common_keys_util import bits
from tests.gpu_util import as_f64, dev, to_dev
from tests.plain_ops import HALF_STEP, f64

pytestmark = pytest.mark.gpu


class Repeated:
    """`pages` pages of a pool of one more, listed in turn by every row of a page table."""

    def __init__(self, seed, rows, width, pages, page_size, Hkv, d, bias=0.0):
        rng = np.random.default_rng(seed)
        self.ps, self.pages, self.Hkv, self.d, self.rng = page_size, pages, Hkv, d, rng
        shape = (pages + 1, page_size, Hkv, d)
        self.k, self.v = bits(rng, *shape), bits(rng, *shape)
        self.dk, self.dv = to_dev(self.k), to_dev(self.v)
        if bias:
            self.dv += bias
            self.v = self.dv.view(torch.int16).cpu().numpy().view(np.uint16)
        self.table = torch.empty(rows, width, dtype=torch.int32, device=dev())
        for r in range(rows):
            torch.remainder(torch.arange(width, dtype=torch.int32, device=dev()), pages, out=self.table[r])

    def want(self, q, n, scale):
        """q [m, Hq, d] over the first n keys: (out, the mean size of what is summed)."""
        period = self.pages * self.ps
        times = np.full(period, n // period, np.float64)
        times[:n % period] += 1
        k, v = (f64(x[:self.pages]).reshape(period, self.Hkv, self.d) for x in (self.k, self.v))
        q, out, size = f64(q), np.zeros(q.shape), np.zeros(q.shape)
        for h in range(q.shape[1]):
            g = h // (q.shape[1] // self.Hkv)
            s = q[:, h] @ k[:, g].T * scale
            p = np.exp(s - s.max(1, keepdims=True)) * times
            p /= p.sum(1, keepdims=True)
            out[:, h], size[:, h] = p @ v[:, g], p @ np.abs(v[:, g])
        return out, size


def rounding(out, size, steps):
    """The output's rounding, the weights' (one bf16 term), and `steps` sums on one accumulator that
    grows evenly, each cut off below an fp32 step of it: half of steps x 2^-23 (both of the numerator
    and of the denominator)."""
    return HALF_STEP * (np.abs(out) + size) + steps * 2.0 ** -23 * size


# Rows as long as 31 bits number keys.  A piece is at most a 608th of the keys for few rows, whose four
# warps add 16 keys in two instructions, and a 152nd for many, 16 keys an instruction.
FEW_STEPS, MANY_STEPS = 2 ** 31 / 608 / 4 / 16 * 2, 2 ** 31 / 152 / 16


@pytest.mark.parametrize("tokens,d", [(1, 64), (1, 128), (20, 64), (20, 128)])
@pytest.mark.parametrize("page_size", [4, 64, 256])
def test_cross_attention_over_two_billion_states(tokens, d, page_size):
    width = (2 ** 31 - 1) // page_size
    x = Repeated(1, 1, width, 5, page_size, 1, d)
    q = bits(x.rng, tokens, 1, d)
    n = width * page_size - 1
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = pkv.paged_cross_attn(to_dev(q), to_dev(np.array([0, tokens], np.int32)), x.dk, x.dv, x.table,
                               to_dev(np.array([n], np.int32)), d ** -0.5, dev_status=status)
    o, size = x.want(q, n, d ** -0.5)
    assert status.item() == 0
    assert (np.abs(as_f64(out) - o) <= rounding(o, size, FEW_STEPS if tokens == 1 else MANY_STEPS)).all()


@pytest.mark.parametrize("d", [64, 128])
def test_decode_with_two_billion_shared_keys(d):
    """Three sequences whose own keys lie behind them."""
    width = (2 ** 31 - 1) // 256
    x = Repeated(2, 3, width, 5, 256, 1, d)
    q = bits(x.rng, 3, 8, d)
    lens = np.array([width * 256, width * 256 - 2560, width * 256 - 1000], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = pkv.paged_decode_attn_shared(
        to_dev(q), x.dk, x.dv, x.table, to_dev(lens), d ** -0.5, to_dev(np.array([0, 3], np.int32)),
        to_dev(np.array([(width - 10) * 256], np.int32)), dev_status=status)
    assert status.item() == 0
    for b in range(3):
        o, size = x.want(q[b:b + 1], int(lens[b]), d ** -0.5)
        assert (np.abs(as_f64(out)[b:b + 1] - o) <= rounding(o, size, MANY_STEPS)).all(), b


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [1, 20])
def test_sums_of_long_pieces_do_not_drift(tokens, d):
    """A million keys in one piece, whose first half's values come again with the other sign and the
    same keys in the second: the output is the error of its sums and nothing else, since equal scores
    have equal weights.

    1216 segments, so that ranges of both kernels hold whole ones.  An instruction cuts off below an
    fp32 step of its accumulator, which grows to half of `size` and falls again: on average a quarter
    of it is what 2^-23 is taken of."""
    n, pages, R, Hkv = 1 << 20, 4, 76, 16
    x = Repeated(3, 1, n // 256, pages, 256, Hkv, d)
    x.dv.abs_()
    k, v = torch.cat([x.dk[:pages], x.dk[:pages]]), torch.cat([x.dv[:pages], -x.dv[:pages]])
    table = x.table.clone()
    table[:, n // 512:] += pages
    q = torch.randn(R * tokens, Hkv, d, dtype=torch.bfloat16, device=dev(),
                    generator=torch.Generator(device=dev()).manual_seed(4))
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = pkv.paged_cross_attn(q, torch.arange(0, R * tokens + 1, tokens, dtype=torch.int32, device=dev()), k, v,
                               table.expand(R, -1).contiguous(), torch.full((R,), n, dtype=torch.int32, device=dev()),
                               d ** -0.5, dev_status=status)
    assert status.item() == 0
    # the mean of |v| is 0.8; few rows: a warp's 16 keys in two instructions, 4 warps
    steps = n / 4 / 16 * 2 if tokens == 1 else n / 16
    assert out.float().abs().max().item() <= 0.25 * steps * 2.0 ** -23 * 0.8


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,requests", [(1, 76), (20, 38), (200, 38)])
@pytest.mark.parametrize("n", [1 << 14, (1 << 14) + 16, 1 << 20])
def test_outputs_of_long_pieces_are_not_biased(n, tokens, requests, d):
    """Values of one sign, in pieces of few rows, of one query tile and of two: what the sums lose adds up.

    At most 1024 instructions (16384 keys) go to one accumulator.  Each aligns 17 terms to the largest and
    may cut each off below its fp32 step, 17 x 2^-23 of an accumulator that grows evenly, half of it on
    average.  The outputs' own roundings, at most 2^-8 each and as often up as down, leave four of their
    mean's deviations, 2^-8 / sqrt(3 N)."""
    Hkv, page_size = 16, 16
    x = Repeated(5, 1, n // page_size, 64, page_size, Hkv, d)
    x.dv.abs_()
    x.v = x.dv.view(torch.int16).cpu().numpy().view(np.uint16)
    q = bits(x.rng, tokens, Hkv, d)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = pkv.paged_cross_attn(
        to_dev(q).repeat(requests, 1, 1), torch.arange(0, requests * tokens + 1, tokens, dtype=torch.int32, device=dev()),
        x.dk, x.dv, x.table.expand(requests, -1).contiguous(),
        torch.full((requests,), n, dtype=torch.int32, device=dev()), d ** -0.5, dev_status=status)
    assert status.item() == 0
    o, size = x.want(q, n, d ** -0.5)
    off = as_f64(out).reshape(requests, *o.shape) / o - 1
    assert np.abs(off).max() <= 2 * HALF_STEP
    assert np.abs(off.mean((1, 2, 3))).max() <= 512 * 17 * 2.0 ** -23 + 4 * HALF_STEP / (3 * o.size) ** 0.5


@pytest.mark.parametrize("d", [64, 128])
def test_decode_with_long_shared_keys_is_not_biased(d):
    """Groups of few rows, of up to 128 and of up to 256; own keys behind them, some long as well."""
    Hkv, page_size, members = 16, 256, [1, 20, 200] * 8
    B, n = sum(members), 1 << 18
    x = Repeated(6, 1, 2 * n // page_size, 8, page_size, Hkv, d)
    x.dv.abs_()
    x.v = x.dv.view(torch.int16).cpu().numpy().view(np.uint16)
    q = bits(x.rng, 1, Hkv, d)
    lens = np.full(B, n + 300, np.int32)
    lens[np.cumsum(members)[:-1]] = 2 * n
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    out = as_f64(pkv.paged_decode_attn_shared(
        to_dev(q).repeat(B, 1, 1), x.dk, x.dv, x.table.expand(B, -1).contiguous(), to_dev(lens), d ** -0.5,
        to_dev(np.concatenate([[0], np.cumsum(members)]).astype(np.int32)),
        torch.full((len(members),), n, dtype=torch.int32, device=dev()), dev_status=status))
    assert status.item() == 0
    for length in (n + 300, 2 * n):
        o, size = x.want(q, length, d ** -0.5)
        off = out[lens == length] / o - 1
        assert np.abs(off).max() <= 2 * HALF_STEP
        assert np.abs(off.mean((1, 2))).max() <= 512 * 17 * 2.0 ** -23 + 4 * HALF_STEP / (3 * o.size) ** 0.5
