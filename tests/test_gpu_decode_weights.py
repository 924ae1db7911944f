"""paged_decode_attn_weights against the 64-bit form: its output, and the sums of weights."""
import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from synth import make_inputs
from tests import plain_ops
from tests.gpu_util import Run, as_f64, dev, to_dev, to_host_bits

pytestmark = pytest.mark.gpu


def inputs(seed, lens, Hq=16, Hkv=8, d=128, page_size=16, **kw):
    lens = np.asarray(lens)
    new = np.minimum(lens, 1)
    x = make_inputs(seed=seed, Hq=Hq, Hkv=Hkv, d=d, page_size=page_size, new_lens=new, prefix_lens=lens - new, **kw)
    # a query row for every sequence, those without keys too
    x.q = make_inputs(seed=seed + 1, Hq=Hq, Hkv=Hkv, d=d, page_size=16, new_lens=[len(lens)], prefix_lens=[0]).q
    return x


class State(Run):
    """An input's device copies and the running sums: rows of the batch in shuffled order among
    more rows, NaN wherever nothing may be read."""

    def __init__(self, x, stride=None, extra_rows=2):
        super().__init__(x)
        self.store()
        rng = np.random.default_rng(7)
        longest = int(max(1, x.seq_lens.max()))
        stride = stride or longest
        R = x.B + extra_rows
        self.rows = rng.permutation(R)[:x.B].astype(np.int32)
        self.acc0 = np.full((R, x.Hkv, stride), np.nan, np.float32)
        for b, L in enumerate(x.seq_lens):
            if L > 0:
                self.acc0[self.rows[b], :, :L - 1] = rng.random((x.Hkv, L - 1), dtype=np.float32)
        self.acc = to_dev(self.acc0)
        self.max_len = longest
        self.drows = to_dev(self.rows)

    def weights(self, **kw):
        args = dict(acc_rows=self.drows, dev_status=self.status)
        args.update(kw)
        return pkv.paged_decode_attn_weights(self.q, self.k, self.v, self.page_table, self.seq_lens, self.x.scale,
                                             args.pop("acc", self.acc), args.pop("max_seq_len", self.max_len), **args)

    def pools(self):
        return to_host_bits(self.k), to_host_bits(self.v)

    def check(self, out, calls=1, skip=()):
        x = self.x
        want = plain_ops.decode_weights(x.q, *self.pools(), x.page_table, x.seq_lens, x.scale)
        got_out, got = as_f64(out), self.acc.cpu().numpy()
        touched = np.zeros(got.shape, bool)
        for b, (o, w, tol_o, tol_w) in enumerate(want):
            L = int(x.seq_lens[b])
            assert (np.abs(got_out[b] - o) <= tol_o).all(), b
            if b in skip or self.rows[b] < 0 or L == 0:
                continue
            total = w.copy()
            total[:, :L - 1] += self.acc0[self.rows[b], :, :L - 1].astype(np.float64)
            row = got[self.rows[b], :, :L].astype(np.float64)
            assert (np.abs(row - total) <= tol_w + plain_ops.U * np.abs(total)).all(), b
            touched[self.rows[b], :, :L] = True
        assert np.array_equal(got.view(np.uint32)[~touched], self.acc0.view(np.uint32)[~touched])


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 8, 128), (16, 8, 128), (8, 2, 128), (8, 1, 128),
                                      (4, 4, 64), (4, 2, 64), (32, 8, 64), (16, 2, 64)])
@pytest.mark.parametrize("page_size", [1, 4, 16, 256])
def test_matches_the_plain_form(Hq, Hkv, d, page_size):
    r = State(inputs(Hq + page_size, [1, 2, 31, 32, 33, 0, 63, 64, 65, 700, 255, 1500], Hq, Hkv, d, page_size),
              stride=1601)
    out = r.weights(max_seq_len=1500)
    assert r.dev_status() == 0
    r.check(out)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [5], [4097], [1] * 40, [3000, 1, 1, 1]])
def test_small_and_lopsided_batches(lens):
    r = State(inputs(len(lens), lens))
    out = r.weights()
    assert r.dev_status() == 0
    r.check(out)


def test_a_long_sequence_cut_over_all_blocks():
    r = State(inputs(3, [40000, 17], Hq=4, Hkv=1, d=64, page_size=64))
    out = r.weights()
    r.check(out)


def test_many_sequences():
    rng = np.random.default_rng(4)
    r = State(inputs(4, rng.integers(0, 120, 900), Hq=4, Hkv=2, d=64, page_size=8))
    r.check(r.weights())


@pytest.mark.parametrize("page_size", [1, 16])
def test_the_largest_batch(page_size):
    """4096 sequences, most of them of a few keys, some empty."""
    rng = np.random.default_rng(page_size)
    lens = rng.integers(0, 12, 4096)
    lens[::500] = 150
    r = State(inputs(40, lens, Hq=2, Hkv=1, d=64, page_size=page_size))
    r.check(r.weights())
    assert r.dev_status() == 0


def test_one_sequence_and_one_head_cut_over_every_block():
    """Eight query heads on one KV head: every block of the grid has a piece of the one segment."""
    for d in (64, 128):
        r = State(inputs(41, [33001], Hq=8, Hkv=1, d=d, page_size=16))
        r.check(r.weights())
        assert r.dev_status() == 0


def test_steps_add_up_and_the_newest_key_starts_afresh():
    """Two calls at one length, then one a key later: sums of the weights of all three; the new
    key's slot in the sums holds NaN before."""
    x = inputs(5, [70, 300])
    r = State(x, stride=400)
    r.weights()
    r.weights()
    w1 = plain_ops.decode_weights(x.q, *r.pools(), x.page_table, x.seq_lens, x.scale)
    short = torch.from_numpy(x.seq_lens - 1).int().to(dev())
    pkv.paged_decode_attn_weights(r.q, r.k, r.v, r.page_table, short, x.scale, r.acc, 400, acc_rows=r.drows)
    w2 = plain_ops.decode_weights(x.q, *r.pools(), x.page_table, x.seq_lens - 1, x.scale)
    got = r.acc.cpu().numpy().astype(np.float64)
    for b, L in enumerate(x.seq_lens):
        row = got[r.rows[b]]
        old = r.acc0[r.rows[b]].astype(np.float64)
        tol = 3 * (w1[b][3][:, :L - 2].max() + w2[b][3][:, :L - 2].max()) + 8 * plain_ops.U
        assert (np.abs(row[:, :L - 2] - (old[:, :L - 2] + 2 * w1[b][1][:, :L - 2] + w2[b][1][:, :L - 2])) <= tol).all()
        assert (np.abs(row[:, L - 2] - w2[b][1][:, L - 2]) <= tol).all()       # newest of the last call
        assert (np.abs(row[:, L - 1] - w1[b][1][:, L - 1]) <= tol).all()       # twice its own first weight
        assert np.isnan(row[:, L:]).all()


def test_rows_default_to_the_batch_and_negative_rows_are_left_out():
    x = inputs(6, [100, 50, 7])
    r = State(x, extra_rows=0)
    r.rows[:] = [0, 1, 2]
    r.acc0[:] = 0.25
    r.acc = to_dev(r.acc0)
    r.check(r.weights(acc_rows=None))
    r.acc = to_dev(r.acc0)
    r.rows[:] = [2, -1, 0]
    r.check(r.weights(acc_rows=to_dev(r.rows)))
    assert r.dev_status() == 0


def test_bad_rows_lengths_and_pages():
    x = inputs(7, [100, 50, 7, 300, 33], Hkv=2, Hq=4)
    r = State(x, stride=300)
    r.rows[1] = len(r.acc0)
    out = r.weights(acc_rows=to_dev(r.rows))
    assert r.dev_status() == pkv.DEV_BAD_ROW
    r.check(out, skip=(1,))

    r = State(x, stride=300)
    out = r.weights(max_seq_len=299)                # sequence 3 is longer than the caller said
    assert r.dev_status() == pkv.DEV_BAD_SEQLEN
    assert torch.isnan(out[3]).all()
    got = r.acc.cpu().numpy()
    assert np.array_equal(got[r.rows[3]].view(np.uint32), r.acc0[r.rows[3]].view(np.uint32))
    x.seq_lens[3] = 0
    out[3] = 0
    r.check(out)
    x.seq_lens[3] = -5
    r = State(x, stride=300)
    out = r.weights(max_seq_len=300)
    assert r.dev_status() == pkv.DEV_BAD_SEQLEN
    assert torch.isnan(out[3]).all()
    out[3] = 0
    x.seq_lens[3] = 0
    r.check(out)


@pytest.mark.parametrize("page_size", [1, 2, 8, 16, 64])
@pytest.mark.parametrize("key", [0, 37, 99, 280, 299])
def test_keys_on_bad_pages(page_size, key):
    x = inputs(7, [100, 50, 7, 300, 33], Hkv=2, Hq=4, page_size=page_size)
    r = State(x, stride=300)
    pt = x.page_table.copy()
    pt[3, key // page_size] = x.num_pages
    pt[0, min(key, 99) // page_size] = -1
    r.page_table = to_dev(pt)
    out = r.weights()
    assert r.dev_status() == pkv.DEV_BAD_PAGE
    assert torch.isnan(out[[0, 3]]).all()
    got = r.acc.cpu().numpy()
    for b in (0, 3):
        assert np.array_equal(got[r.rows[b]].view(np.uint32), r.acc0[r.rows[b]].view(np.uint32))
    keep = r.acc0.copy()
    out[[0, 3]] = 0
    x.seq_lens[[0, 3]] = 0
    r.acc0 = keep
    r.check(out)


def test_nan_and_infinite_keys_stay_in_their_head():
    x = inputs(8, [64, 200], Hq=4, Hkv=2, d=64)
    r = State(x)
    slots = plain_ops.slots_of(x.page_table[1], 16, 200)
    r.k.view(-1, 2, 64)[int(slots[20]), 1, 5] = float("nan")
    out = as_f64(r.weights())
    assert np.isnan(out[1, 2:]).all() and np.isfinite(out[1, :2]).all() and np.isfinite(out[0]).all()
    got = r.acc.cpu().numpy()[r.rows[1]][:, :200]
    assert np.isnan(got[1]).all() and np.isfinite(got[0]).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 6.0])
def test_flat_negative_and_peaked_softmax(scale):
    x = inputs(9, [90, 400], Hq=8, Hkv=4, d=64)
    x.scale = scale
    r = State(x)
    r.check(r.weights())


def test_workspace_contents_do_not_matter_and_equal_calls_give_equal_bits():
    x = inputs(10, [500, 3, 0, 2000, 90])
    r = State(x)
    ws = pkv.decode_weights_workspace(x.B, x.Hq, x.Hkv, x.d, r.max_len)
    seen = []
    for fill in (0, 255, 127):
        ws.fill_(fill)
        r.acc = to_dev(r.acc0)
        out = r.weights(workspace=ws)
        r.check(out)
        seen.append((to_host_bits(out), r.acc.cpu().numpy().view(np.uint32)))
    for o, a in seen[1:]:
        assert np.array_equal(o, seen[0][0]) and np.array_equal(a, seen[0][1])


def test_a_workspace_on_a_16_byte_boundary_is_left_alone_outside():
    x = inputs(42, [500, 3, 2000])
    r = State(x)
    n = pkv.decode_weights_workspace_size(x.B, x.Hq, x.Hkv, x.d, r.max_len)
    big = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=dev())
    r.check(r.weights(workspace=big[1040:1040 + n]))
    assert (big[:1040] == 0xA5).all() and (big[1040 + n:] == 0xA5).all()


def test_graph_replays_with_other_lengths_and_a_padded_batch():
    a = inputs(11, [100, 700, 33, 1000], pool_pages=400, pt_stride=64)
    b = inputs(12, [5, 0, 1024, 64], pool_pages=400, pt_stride=64)
    ra, rb = State(a, stride=1024), State(b, stride=1024)
    rb.rows = ra.rows.copy()
    rb.rows[1] = -1
    out = torch.empty_like(ra.q)
    ws = pkv.decode_weights_workspace(4, 16, 8, 128, 1024)
    ra.weights(max_seq_len=1024, workspace=ws)      # sets kernel attributes
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ra.weights(max_seq_len=1024, workspace=ws, out=out, stream=s)
    own_pools = {ra: ra.pools(), rb: rb.pools()}     # ra's are the captured buffers
    for r in (ra, rb, ra):
        x = r.x
        r.pools = lambda bits=own_pools[r]: bits
        fresh = np.full(ra.acc0.shape, 0.5, np.float32)
        ra.k.copy_(to_dev(own_pools[r][0])), ra.v.copy_(to_dev(own_pools[r][1]))
        ra.q.copy_(to_dev(x.q)), ra.page_table.copy_(to_dev(x.page_table))
        ra.seq_lens.copy_(to_dev(x.seq_lens)), ra.drows.copy_(to_dev(r.rows))
        ra.acc.copy_(to_dev(fresh))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        r.acc0 = fresh
        keep, r.acc = r.acc, ra.acc
        r.check(out)
        r.acc = keep
    assert ra.dev_status() == 0


def test_two_streams_with_workspaces_of_their_own():
    xs = [inputs(13 + i, [900, 40, 2000, 600]) for i in range(2)]
    rs = [State(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in rs]
    torch.cuda.synchronize()
    outs = []
    for r, s in zip(rs, streams):
        outs.append(r.weights(stream=s))             # workspace and out allocated inside, on s
    torch.cuda.synchronize()
    for r, o in zip(rs, outs):
        r.check(o)


def test_sums_and_pool_rows_past_32_bit_offsets():
    """A row of sums behind 2^31 elements, keys in a pool behind 2^32 elements."""
    x = inputs(15, [300, 50], Hq=16, Hkv=8, d=128, page_size=256)
    r = State(x)
    pages = (1 << 32) // (256 * 8 * 128) + 4
    k = torch.empty(pages, 256, 8, 128, dtype=torch.bfloat16, device=dev())
    v = torch.empty(pages, 256, 8, 128, dtype=torch.bfloat16, device=dev())
    ids = np.array([[pages - 1, 3], [pages - 2, -1]], np.int32)
    for b, n in enumerate((2, 1)):
        for i in range(n):
            k[int(ids[b, i])] = r.k[int(x.page_table[b, i])]
            v[int(ids[b, i])] = r.v[int(x.page_table[b, i])]
    R = (1 << 31) // (8 * 1000) + 2
    acc = torch.empty(R, 8, 1000, device=dev())
    rows = np.array([R - 1, R - 2], np.int32)
    acc[[R - 1, R - 2]] = 0.25
    out = pkv.paged_decode_attn_weights(r.q, k, v, to_dev(ids), r.seq_lens, x.scale, acc, 300,
                                        acc_rows=to_dev(rows), dev_status=r.status)
    assert r.dev_status() == 0
    want = plain_ops.decode_weights(x.q, *r.pools(), x.page_table, x.seq_lens, x.scale)
    for b, (o, w, tol_o, tol_w) in enumerate(want):
        L = int(x.seq_lens[b])
        assert (np.abs(as_f64(out)[b] - o) <= tol_o).all()
        total = w + 0.25
        total[:, L - 1] -= 0.25
        assert (np.abs(as_f64(acc[int(rows[b])])[:, :L] - total) <= tol_w + plain_ops.U * total).all()
        assert (acc[int(rows[b]), :, L:] == 0.25).all()


def test_refused_tensors():
    x = inputs(16, [20, 30])
    r = State(x)
    with pytest.raises(pkv.PkvError):
        r.weights(workspace=torch.empty(1024, dtype=torch.uint8, device=dev()))
    with pytest.raises(pkv.PkvError):
        r.weights(max_seq_len=31)                    # longer than a row of acc
    for bad in (dict(acc=r.acc.double()), dict(acc=r.acc[:, :4]), dict(acc_rows=r.drows[:1]),
                dict(acc_rows=r.drows.long()), dict(out=r.q[:1]), dict(acc=r.acc.cpu())):
        with pytest.raises(ValueError):
            r.weights(**bad)
    wide = torch.zeros(2, 8, dtype=torch.int32, device=dev())
    with pytest.raises(ValueError):                  # the last row would be read past the tensor
        pkv.paged_decode_attn_weights(r.q, r.k, r.v, wide[:, 6:], r.seq_lens, 1.0, r.acc, 30, acc_rows=r.drows)
    assert np.array_equal(r.acc.cpu().numpy().view(np.uint32), r.acc0.view(np.uint32))
