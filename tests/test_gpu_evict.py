"""kv_evict against the plain form: the kept positions, the moved rows and sums, and everything
that must not change, all bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from tests import plain_ops
from tests.gpu_util import dev, to_dev, to_host_bits

pytestmark = pytest.mark.gpu

FREE = -7  # what kept holds where nothing is to be written


class Case:
    """Sequences of `lens` keys on shuffled pages; row bits are random, so that every row is known."""

    def __init__(self, seed, lens, keep, Hkv=2, d=64, ps=16, first=2, recent=5, stride=None, copy=False,
                 sums="random", extra_pages=3):
        rng = np.random.default_rng(seed)
        self.Hkv, self.d, self.ps, self.first, self.recent = Hkv, d, ps, first, recent
        self.lens, self.keep = np.asarray(lens, np.int32), np.asarray(keep, np.int32)
        B = len(self.lens)
        n = np.maximum(0, np.minimum(self.lens, self.keep))
        per, per_out = -(-np.maximum(self.lens, 0) // ps), -(-n // ps)
        pages = int(per.sum() + (per_out.sum() if copy else 0)) + extra_pages
        ids = rng.permutation(pages)
        self.table = np.full((B, max(1, int(per.max()) + 1)), -1, np.int32)
        self.table_out = np.full((B, max(1, int(per_out.max()))), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :per[b]] = ids[at:at + per[b]]
            at += per[b]
        for b in range(B):
            if copy:
                self.table_out[b, :per_out[b]] = ids[at:at + per_out[b]]
                at += per_out[b]
        if not copy:
            self.table_out = self.table
        self.k = rng.integers(0, 1 << 16, (pages, ps, Hkv, d), dtype=np.uint16)
        self.v = rng.integers(0, 1 << 16, (pages, ps, Hkv, d), dtype=np.uint16)
        S = stride or int(max(1, self.lens.max()))
        R = B + 2
        self.rows = rng.permutation(R)[:B].astype(np.int32)
        if sums == "random":
            self.acc = rng.random((R, Hkv, S), dtype=np.float32) ** 4
        elif sums == "equal":
            self.acc = np.full((R, Hkv, S), 0.5, np.float32)
        elif sums == "few":                                     # many ties, both zeros, both signs
            self.acc = rng.choice(np.array([0.0, -0.0, 1.0, 2.0, -1.0], np.float32), (R, Hkv, S))
        elif sums == "close":                                   # neighbours in the last bits
            self.acc = (np.float32(1.0) + rng.integers(0, 1100, (R, Hkv, S)).astype(np.float32) * np.float32(2.0 ** -23))
        else:                                                   # what a broken row may hold
            self.acc = rng.standard_normal((R, Hkv, S)).astype(np.float32)
            odd = rng.random((R, Hkv, S))
            self.acc[odd < 0.2] = np.nan
            self.acc.view(np.uint32)[(odd > 0.2) & (odd < 0.25)] = 0xFFC00001   # a NaN with its sign set
            self.acc[(odd > 0.25) & (odd < 0.3)] = np.inf
            self.acc[(odd > 0.3) & (odd < 0.4)] = -np.inf
            self.acc[(odd > 0.4) & (odd < 0.5)] = 1e-41
        self.max_keep = max(1, int(n.max()))
        self.status = torch.zeros(1, dtype=torch.int32, device=dev())

    def call(self, in_place_sums=True, **kw):
        self.dk, self.dv, self.dacc = to_dev(self.k), to_dev(self.v), to_dev(self.acc)
        self.dout = self.dacc if in_place_sums else torch.full_like(self.dacc, 3.5)
        self.acc_out0 = self.acc if in_place_sums else np.full_like(self.acc, 3.5)
        self.kept = torch.full((len(self.lens), self.Hkv, self.max_keep), FREE, dtype=torch.int32, device=dev())
        table = to_dev(self.table)
        args = dict(acc_rows=to_dev(self.rows), acc_out=self.dout, kept=self.kept, dev_status=self.status,
                    page_table_out=table if self.table_out is self.table else to_dev(self.table_out))
        args.update(kw)
        _, self.new = pkv.kv_evict(self.dk, self.dv, table, to_dev(self.lens), to_dev(self.keep), self.dacc,
                                   self.first, self.recent, **args)
        return self

    def check(self, nothing=()):
        k, v = self.k.reshape(-1, self.Hkv, self.d).copy(), self.v.reshape(-1, self.Hkv, self.d).copy()
        k0, v0 = k.copy(), v.copy()
        kept = np.full((len(self.lens), self.Hkv, self.max_keep), FREE, np.int32)
        acc, new = self.acc_out0.copy(), self.lens.copy()
        for b, (L, keep, row) in enumerate(zip(self.lens, self.keep, self.rows)):
            if b in nothing:
                continue
            n = new[b] = min(int(L), int(keep))
            if n == 0:
                continue
            source = plain_ops.slots_of(self.table[b], self.ps, int(L))
            target = plain_ops.slots_of(self.table_out[b], self.ps, n)
            for g in range(self.Hkv):
                stay = plain_ops.evict_kept(self.acc[row, g, :L], n, self.first, self.recent)
                kept[b, g, :n] = stay
                acc.view(np.uint32)[row, g, :n] = self.acc.view(np.uint32)[row, g, stay]
                k[target, g], v[target, g] = k0[source[stay], g], v0[source[stay], g]
        assert np.array_equal(self.kept.cpu().numpy(), kept)
        assert np.array_equal(self.new.cpu().numpy(), new)
        assert np.array_equal(self.dout.cpu().numpy().view(np.uint32), acc.view(np.uint32))
        assert np.array_equal(to_host_bits(self.dk).reshape(k.shape), k)
        assert np.array_equal(to_host_bits(self.dv).reshape(v.shape), v)


LENS = [1, 2, 7, 8, 40, 300, 513, 1000, 64]
KEEP = [1, 1, 7, 3, 20, 150, 512, 90, 64]


@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("Hkv,d", [(1, 128), (8, 128), (3, 64), (8, 64)])
@pytest.mark.parametrize("ps", [1, 4, 16, 256])
def test_matches_the_plain_form(ps, Hkv, d, copy):
    Case(ps + Hkv, LENS, KEEP, Hkv, d, ps, copy=copy).call().check()


@pytest.mark.parametrize("in_place_sums", [False, True])
@pytest.mark.parametrize("sums", ["random", "equal", "few", "close", "odd"])
def test_sums_of_every_kind(sums, in_place_sums):
    Case(1, [700, 90, 5000, 33], [350, 60, 700, 30], sums=sums, first=1, recent=3, stride=5003).call(
        in_place_sums).check()


@pytest.mark.parametrize("first,recent", [(0, 0), (0, 50), (50, 0), (3, 1000), (1000, 3), (40, 40), (25, 25)])
def test_the_protected_ends(first, recent):
    Case(2, [100, 50, 49, 200, 51], [50, 50, 50, 50, 50], first=first, recent=recent).call().check()


def test_keep_nothing_everything_and_more_than_everything():
    c = Case(3, [60, 0, 33, 17, 0], [0, 5, 33, 100, 0]).call()
    assert int(c.status.item()) == 0
    c.check()


@pytest.mark.parametrize("L", [17000, 49152, 49153, 70001])
def test_rows_longer_than_what_a_block_holds(L):
    for in_place in (False, True):
        Case(L, [L, 30], [L // 3, 20], Hkv=1, ps=256, sums="few" if L == 49153 else "random",
             first=4, recent=64).call(in_place).check()


@pytest.mark.parametrize("in_place_sums", [False, True])
@pytest.mark.parametrize("sums", ["random", "equal", "few", "close", "odd"])
@pytest.mark.parametrize("L", [8193, 20011])
def test_long_rows_of_few_sequences(L, sums, in_place_sums):
    """Sums of every kind in long rows, short rows and an empty one among them."""
    Case(L, [L, 30, 0, 5000, 33], [L // 2, 20, 0, 4999, 1], Hkv=1, ps=64, sums=sums, first=3, recent=40).call(
        in_place_sums).check()


def test_short_sequences_in_long_rows():
    Case(4, [100, 2000, 9], [50, 1999, 8], stride=60000).call().check()


def test_new_pages_for_some_of_the_keys():
    """The first pages of sequence 0 are shared with sequence 1: both get new ones there and keep
    the rest of their own."""
    c = Case(5, [200, 150], [120, 100], ps=16, extra_pages=10)
    used = np.unique(c.table[c.table >= 0])
    free = np.setdiff1d(np.arange(c.k.shape[0]), used)
    c.table[1, :3] = c.table[0, :3]
    c.table_out = c.table.copy()
    c.table_out[0, :3] = free[:3]
    c.table_out[1, :3] = free[3:6]
    shared = c.table[0, :3].copy()
    c.call().check()
    assert np.array_equal(to_host_bits(c.dk)[shared], c.k[shared])


def test_sequences_without_a_row_and_bad_arguments_stay_as_they_are():
    c = Case(6, [60, 60, 60, 60, 60, -3, 60, 60], [30] * 8, stride=60)
    c.max_keep = 30
    c.rows[1] = -1
    c.rows[2] = len(c.acc)
    c.keep[3] = -1
    c.keep[4] = 31                        # more than max_keep
    c.lens[6] = 61                        # longer than a row of sums
    c.call()
    assert int(c.status.item()) == pkv.DEV_BAD_SEQLEN | pkv.DEV_BAD_ROW
    c.check(nothing=(1, 2, 3, 4, 5, 6))


def test_keys_that_do_not_fit_the_tables():
    c = Case(7, [200, 60], [150, 30], copy=True, ps=16)
    c.table_out = c.table_out[:, :5].copy()          # 80 keys
    c.call()
    assert int(c.status.item()) == pkv.DEV_BAD_SEQLEN
    c.check(nothing=(0,))
    c = Case(8, [200, 60], [150, 30], ps=16)
    c.table = c.table_out = c.table[:, :6].copy()    # 96 keys
    c.call()
    assert int(c.status.item()) == pkv.DEV_BAD_SEQLEN
    c.check(nothing=(0,))


@pytest.mark.parametrize("page", [-1, 1 << 20, -(1 << 31)])
def test_rows_on_bad_pages_are_not_copied(page):
    for out in (False, True):
        c = Case(9, [64, 64], [48, 48], copy=out, ps=16, first=48, recent=0)   # kept = 0 .. 47
        c.keep[:] = 48
        pages_in, pages_out = c.table.copy(), c.table_out.copy()
        if out:
            c.table_out[0, 1] = page
        else:
            c.table = c.table.copy()
            c.table[0, 1] = page
            c.table_out = pages_in
        c.call()
        assert int(c.status.item()) == pkv.DEV_BAD_PAGE
        assert c.new.tolist() == [48, 48]
        want_k = c.k.copy()
        for b in range(2):
            for i in range(3):
                if (b, i) != (0, 1):
                    want_k[pages_out[b, i]] = c.k[pages_in[b, i]]
        assert np.array_equal(to_host_bits(c.dk), want_k)


@pytest.mark.parametrize("L", [700, 50000])
def test_two_sequences_with_one_row_of_sums_touch_nothing_else(L):
    """A caller error: their own results are open, but rows of other sequences, what lies past a
    sequence's kept positions and every other page stay."""
    c = Case(30, [L, L - 5, 90], [L // 2, L // 3, 40], Hkv=2, ps=16)
    c.rows[1] = c.rows[0]
    c.call()
    other = c.kept.cpu().numpy()
    for g in range(2):
        stay = plain_ops.evict_kept(c.acc[c.rows[2], g, :90], 40, c.first, c.recent)
        assert np.array_equal(other[2, g, :40], stay)
    assert (other[2, :, 40:] == FREE).all() and (other[1, :, L // 3:] == FREE).all()
    assert c.new.tolist() == [L // 2, L // 3, 40]
    own = np.zeros(c.k.shape[0], bool)
    for b, n in ((0, L // 2), (1, L // 3), (2, 40)):
        own[c.table[b, :-(-n // 16)]] = True
    assert np.array_equal(to_host_bits(c.dk)[~own], c.k[~own])
    sums = np.ones(len(c.acc), bool)
    sums[c.rows] = False
    assert np.array_equal(c.dout.cpu().numpy().view(np.uint32)[sums], c.acc.view(np.uint32)[sums])


def test_no_sequences():
    c = Case(10, [5], [2])
    none = torch.empty(0, dtype=torch.int32, device=dev())
    kept, new = pkv.kv_evict(to_dev(c.k), to_dev(c.v), torch.empty(0, 4, dtype=torch.int32, device=dev()), none,
                             none, torch.zeros(1, 2, 8, device=dev()), 1, 1, max_keep=4)
    assert kept.shape == (0, 2, 4) and new.shape == (0,)


def test_defaults_allocate_and_work_in_place():
    c = Case(11, [90, 40], [30, 30])
    c.rows = np.array([0, 1], np.int32)
    c.dk, c.dv, c.dacc = to_dev(c.k), to_dev(c.v), to_dev(c.acc)
    kept, c.new = pkv.kv_evict(c.dk, c.dv, to_dev(c.table), to_dev(c.lens), to_dev(c.keep), c.dacc, c.first,
                               c.recent)
    assert kept.shape == (2, 2, 90)
    c.kept = torch.full((2, 2, 30), FREE, dtype=torch.int32, device=dev())
    c.kept.copy_(kept[:, :, :30])
    c.dout, c.acc_out0 = c.dacc, c.acc
    c.check()


def test_on_another_stream_and_equal_calls_give_equal_bits():
    c = Case(12, [3000, 700, 50], [1000, 699, 2], Hkv=8, d=128, sums="few")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        c.call(stream=s)
        s.synchronize()
        c.check()


def test_captured_and_replayed_with_other_inputs():
    cases = [Case(20, [300, 50, 700], [100, 50, 33], stride=800, extra_pages=9),
             Case(21, [700, 0, 301], [699, 4, 1], stride=800, extra_pages=9)]
    a = cases[0]
    width, pages = max(c.table.shape[1] for c in cases), max(len(c.k) for c in cases)
    for c in cases:
        c.table = c.table_out = np.pad(c.table, ((0, 0), (0, width - c.table.shape[1])), constant_values=-1)
        grow = ((0, pages - len(c.k)), (0, 0), (0, 0), (0, 0))
        c.k, c.v, c.max_keep = np.pad(c.k, grow), np.pad(c.v, grow), 700
    buf = dict(k=to_dev(a.k), v=to_dev(a.v), pt=to_dev(a.table), sl=to_dev(a.lens), keep=to_dev(a.keep),
               acc=to_dev(a.acc), rows=to_dev(a.rows), kept=torch.zeros(3, 2, 700, dtype=torch.int32, device=dev()),
               new=torch.zeros(3, dtype=torch.int32, device=dev()))

    def call(**kw):
        pkv.kv_evict(buf["k"], buf["v"], buf["pt"], buf["sl"], buf["keep"], buf["acc"], 2, 5, acc_rows=buf["rows"],
                     kept=buf["kept"], new_seq_lens=buf["new"], **kw)

    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(stream=s)
    for c in (cases[1], cases[0], cases[1]):
        for name, x in (("k", c.k), ("v", c.v), ("pt", c.table), ("sl", c.lens), ("keep", c.keep), ("acc", c.acc),
                        ("rows", c.rows)):
            buf[name].copy_(to_dev(x))
        buf["kept"].fill_(FREE)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.dk, c.dv, c.dout, c.acc_out0 = buf["k"], buf["v"], buf["acc"], c.acc
        c.kept, c.new = buf["kept"], buf["new"]
        c.check()


def test_sums_and_pool_rows_past_32_bit_offsets():
    pages, ps, Hkv, d = (1 << 32) // (256 * 8 * 128) + 4, 256, 8, 128
    k = torch.empty(pages, ps, Hkv, d, dtype=torch.bfloat16, device=dev())
    v = torch.empty(pages, ps, Hkv, d, dtype=torch.bfloat16, device=dev())
    gen = torch.Generator(device=dev()).manual_seed(1)
    table = torch.tensor([[pages - 1, 2, pages - 3]], dtype=torch.int32, device=dev())
    for p in table[0].tolist():
        k[p] = torch.randn(ps, Hkv, d, generator=gen, device=dev()).bfloat16()
        v[p] = torch.randn(ps, Hkv, d, generator=gen, device=dev()).bfloat16()
    R = (1 << 31) // (8 * 1000) + 2
    acc = torch.empty(R, Hkv, 1000, device=dev())
    acc[R - 1] = torch.rand(Hkv, 1000, generator=gen, device=dev())
    old_k, old_v = (torch.cat([c[p] for p in table[0].tolist()]) for c in (k, v))
    sums = acc[R - 1].cpu().numpy()
    kept, new = pkv.kv_evict(k, v, table, torch.tensor([700], dtype=torch.int32, device=dev()),
                             torch.tensor([300], dtype=torch.int32, device=dev()), acc, 4, 32, max_keep=300,
                             acc_rows=torch.tensor([R - 1], dtype=torch.int32, device=dev()))
    assert new.tolist() == [300]
    now_k, now_v = (torch.cat([c[p] for p in table[0].tolist()]) for c in (k, v))
    for g in range(Hkv):
        stay = plain_ops.evict_kept(sums[g, :700], 300, 4, 32)
        assert np.array_equal(kept[0, g].cpu().numpy(), stay)
        at = torch.from_numpy(stay.astype(np.int64)).to(dev())
        assert torch.equal(now_k[:300, g], old_k[at, g]) and torch.equal(now_v[:300, g], old_v[at, g])
        assert np.array_equal(acc[R - 1, g, :300].cpu().numpy(), sums[g, stay])


def test_refused_tensors():
    c = Case(13, [60, 60], [30, 30])
    bad_calls = (dict(acc_rows=to_dev(c.rows).long()), dict(acc_out=torch.zeros(4, 2, 59, device=dev())),
                 dict(kept=torch.zeros(2, 3, 30, dtype=torch.int32, device=dev())),
                 dict(new_seq_lens=torch.zeros(3, dtype=torch.int32, device=dev())),
                 dict(page_table_out=torch.zeros(1, 8, dtype=torch.int32, device=dev())),
                 dict(dev_status=torch.zeros(1, device=dev())))
    for bad in bad_calls:
        with pytest.raises(ValueError):
            c.call(**bad)
        assert np.array_equal(to_host_bits(c.dk), c.k)
    lens = to_dev(c.lens)
    with pytest.raises(pkv.PkvError):                # would be read while it is written
        pkv.kv_evict(to_dev(c.k), to_dev(c.v), to_dev(c.table), lens, to_dev(c.keep), to_dev(c.acc), 1, 1,
                     acc_rows=to_dev(c.rows), new_seq_lens=lens)
