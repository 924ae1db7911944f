"""kv_evict in the form of two launches: long rows of few heads, which move in large rounds by large
clusters, at both head sizes, and offsets past 32 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from tests import plain_ops
from tests.gpu_util import dev
from tests.test_gpu_evict import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,Hkv", [(2049, 1), (5000, 4), (17000, 2), (49152, 1), (49153, 1), (70001, 4)])
@pytest.mark.parametrize("copy", [False, True])
def test_one_sequence_of_few_heads(L, Hkv, d, copy):
    for part in (3, 20):   # a third, and nearly all
        Case(L + d, [L], [L - L // part if part == 20 else L // part], Hkv=Hkv, d=d, ps=16, first=4, recent=64,
             copy=copy).call(not copy).check()


@pytest.mark.parametrize("sums", ["equal", "few", "odd"])
@pytest.mark.parametrize("L", [8193, 50011])
def test_sums_of_every_kind_at_head_size_128(L, sums):
    Case(L, [L, 30, 0, 3000], [L // 2, 20, 0, 2999], Hkv=1, d=128, ps=64, sums=sums, first=3, recent=40).call().check()


@pytest.mark.parametrize("ps", [1, 256])
@pytest.mark.parametrize("kept", [511, 512, 513, 4095, 4096, 4097, 8191])
def test_kept_rows_around_a_round(ps, kept):
    """A cluster of 16 blocks moves 4096 rows in a round, one of 2 blocks 512."""
    Case(kept, [8192], [kept], Hkv=1, d=128, ps=ps, first=1, recent=1).call().check()


@pytest.mark.parametrize("Hkv,d,rows", [(1, 128, 1), (8, 128, 1), (8, 64, 40)])
def test_past_32_bit_offsets(Hkv, d, rows):
    """Rows of sums behind 2^31 elements and pages behind 2^32; rows 1: large rounds on one head."""
    ps, stride, L, n = 256, 2100, 2050, 900
    pages = (1 << 32) // (ps * Hkv * d) + 10
    k = torch.empty(pages, ps, Hkv, d, dtype=torch.bfloat16, device=dev())
    v = torch.empty(pages, ps, Hkv, d, dtype=torch.bfloat16, device=dev())
    gen = torch.Generator(device=dev()).manual_seed(Hkv)
    ids = [pages - 1, 2, pages - 3, 0, pages - 5, 7, pages - 8, 9, pages - 10]
    table = torch.full((rows, len(ids)), -1, dtype=torch.int32, device=dev())
    table[0] = torch.tensor(ids, dtype=torch.int32)
    for p in ids:
        k[p] = torch.randn(ps, Hkv, d, generator=gen, device=dev()).bfloat16()
        v[p] = torch.randn(ps, Hkv, d, generator=gen, device=dev()).bfloat16()
    R = (1 << 31) // (Hkv * stride) + 2
    acc = torch.empty(R, Hkv, stride, device=dev())
    acc[R - 1] = torch.rand(Hkv, stride, generator=gen, device=dev())
    old_k, old_v = (torch.cat([c[p] for p in ids]) for c in (k, v))
    sums = acc[R - 1].cpu().numpy()
    lens, keep, acc_rows = (torch.zeros(rows, dtype=torch.int32, device=dev()) for _ in range(3))
    lens[0], keep[0], acc_rows[0] = L, n, R - 1      # the other sequences are empty
    kept, new = pkv.kv_evict(k, v, table, lens, keep, acc, 4, 32, max_keep=n, acc_rows=acc_rows)
    assert new.tolist() == [n] + [0] * (rows - 1)
    now_k, now_v = (torch.cat([c[p] for p in ids]) for c in (k, v))
    for g in range(Hkv):
        stay = plain_ops.evict_kept(sums[g, :L], n, 4, 32)
        assert np.array_equal(kept[0, g].cpu().numpy(), stay)
        at = torch.from_numpy(stay.astype(np.int64)).to(dev())
        assert torch.equal(now_k[:n, g], old_k[at, g]) and torch.equal(now_v[:n, g], old_v[at, g])
        assert torch.equal(now_k[n:, g], old_k[n:, g]) and torch.equal(now_v[n:, g], old_v[n:, g])
        assert np.array_equal(acc[R - 1, g, :n].cpu().numpy(), sums[g, stay])
