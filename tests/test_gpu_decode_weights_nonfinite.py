"""paged_decode_attn_weights with infinities and NaN in the cache: they reach the outputs and sums
that they belong to and no others, in segments of one piece and in ones cut over many blocks."""
import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from tests import plain_ops
from tests.gpu_util import as_f64, dev, to_host_bits
from tests.test_gpu_decode_weights import State, inputs

pytestmark = pytest.mark.gpu

INF = float("inf")
# lengths, and the one the odd values go to: whole segments, and one that every block has a piece of
SHAPES = [([64, 200, 33], 1), ([33001], 0)]


def rows_of(r, b, page_size):
    return plain_ops.slots_of(r.x.page_table[b], page_size, int(r.x.seq_lens[b]))


@pytest.mark.parametrize("lens,b", SHAPES)
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 2), (128, 8, 1)])
def test_values_that_are_not_finite_stay_in_their_column(d, Hq, Hkv, lens, b):
    r = State(inputs(50, lens, Hq=Hq, Hkv=Hkv, d=d))
    L, G, g = lens[b], Hq // Hkv, Hkv - 1
    slots = rows_of(r, b, 16)
    v = r.v.view(-1, Hkv, d)
    odd = {3: INF, 9: -INF, 17: float("nan"), d - 1: INF}
    for at, (c, x) in zip((0, L // 2, L - 1, L - 2), odd.items()):
        v[int(slots[at]), g, c] = x
    v[int(slots[5]), g, d - 1] = -INF     # both infinities in one column
    out = as_f64(r.weights())
    heads = slice(g * G, (g + 1) * G)
    assert (out[b, heads, 3] == INF).all() and (out[b, heads, 9] == -INF).all()
    assert np.isnan(out[b, heads, 17]).all() and np.isnan(out[b, heads, d - 1]).all()
    # everything else as if those columns held zeros
    for c in odd:
        v[torch.from_numpy(slots).to(dev()), g, c] = 0
        out[b, heads, c] = 0
    r.check(torch.from_numpy(out))


@pytest.mark.parametrize("lens,b", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 20, -1])
def test_a_key_of_score_minus_infinity_has_no_weight(d, lens, b, at):
    r = State(inputs(51, lens, Hq=2, Hkv=2, d=d, page_size=1))
    L = lens[b]
    at %= L
    q = as_f64(r.q)
    slot = int(rows_of(r, b, 1)[at])
    keys = r.k.view(-1, 2, d)
    keys[slot, 1, 7] = -INF if q[b, 1, 7] > 0 else INF
    out, got = as_f64(r.weights()), r.acc.cpu().numpy()[r.rows[b]].astype(np.float64)
    assert r.dev_status() == 0
    # head 1 attends to the other keys; head 0 to all
    short = r.x.page_table[b:b + 1, :L].copy()
    short = np.delete(short, at, axis=1)
    k, v = r.pools()
    (o, w, tol_o, tol_w), = plain_ops.decode_weights(r.x.q[b:b + 1], k, v, short, [L - 1], r.x.scale)
    assert (np.abs(out[b, 1] - o[1]) <= tol_o[1]).all()
    old = r.acc0[r.rows[b], 1, :L].astype(np.float64)
    old[L - 1] = 0
    weights, tol = np.insert(w[1], at, 0), np.insert(tol_w[1], at, 0)
    total = old + weights
    assert (np.abs(got[1, :L] - total) <= tol + plain_ops.U * np.abs(total)).all()
    k.reshape(-1, 2, d)[slot, 1, 7] = 0
    (o, w, tol_o, tol_w), = plain_ops.decode_weights(r.x.q[b:b + 1], k, v, r.x.page_table[b:b + 1], [L], r.x.scale)
    assert (np.abs(out[b, 0] - o[0]) <= tol_o[0]).all()


@pytest.mark.parametrize("lens,b", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 20, -1])
def test_a_key_of_infinite_score_leaves_no_number_in_its_head(d, lens, b, at):
    """(infinity less infinity, as in the definition)"""
    r = State(inputs(52, lens, Hq=2, Hkv=2, d=d))
    L = lens[b]
    q = as_f64(r.q)
    slot = int(rows_of(r, b, 16)[at])
    r.k.view(-1, 2, d)[slot, 1, 7] = INF if q[b, 1, 7] > 0 else -INF
    out, got = as_f64(r.weights()), r.acc.cpu().numpy()
    assert r.dev_status() == 0
    assert np.isnan(out[b, 1]).all() and np.isnan(got[r.rows[b], 1, :L]).all()
    r.k.view(-1, 2, d)[slot, 1, 7] = 0
    want = plain_ops.decode_weights(r.x.q, *r.pools(), r.x.page_table, r.x.seq_lens, r.x.scale)
    for i, (o, w, tol_o, tol_w) in enumerate(want):
        for h in range(2):
            if (i, h) != (b, 1):
                assert (np.abs(out[i, h] - o[h]) <= tol_o[h]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_in_a_long_piece(d):
    """More tiles in one block than an accumulator sums up, the infinities in the first and the last."""
    L, blocks = 6000, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pages = -(-L // 16)
    gen = torch.Generator(device=dev()).manual_seed(d)
    draw = lambda *s: torch.randn(*s, generator=gen, device=dev()).bfloat16()  # noqa: E731
    k, v, q = draw(pages, 16, 1, d), draw(pages, 16, 1, d), draw(blocks, 2, d)
    rows = v.view(-1, d)
    rows[2, 1], rows[L - 1, 2], rows[3, 3], rows[L - 2, 3] = INF, -INF, INF, -INF
    table = torch.arange(pages, dtype=torch.int32, device=dev()).repeat(blocks, 1)
    lens = torch.full((blocks,), L, dtype=torch.int32, device=dev())
    acc = torch.zeros(blocks, 1, L, device=dev())
    out = as_f64(pkv.paged_decode_attn_weights(q, k, v, table, lens, d ** -0.5, acc, L))
    assert (out[..., 1] == INF).all() and (out[..., 2] == -INF).all() and np.isnan(out[..., 3]).all()
    rows[:, 1:4] = 0
    out[..., 1:4] = 0
    some = [0, 1, blocks // 2, blocks - 1]
    want = plain_ops.decode_weights(to_host_bits(q)[some], to_host_bits(k), to_host_bits(v), table[some].cpu().numpy(),
                                    [L] * len(some), d ** -0.5)
    for b, (o, w, tol_o, tol_w) in zip(some, want):
        assert (np.abs(out[b] - o) <= tol_o).all()
        assert (np.abs(as_f64(acc[b]) - w) <= tol_w + plain_ops.U * w).all()
