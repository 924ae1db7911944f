"""qk_norm_rope_store against the 64-bit form: queries and stored keys within rounding,
stored values and everything that must not change bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from synth.workloads import f32_to_bf16_bits
from tests import plain_ops
from tests.gpu_util import as_f64, dev, to_dev, to_host_bits

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, seed, T, Hq, Hkv, d, rot, norm=True, interleaved=False, ps=16, context=5000, pad=0,
                 spread=0, weight_scale=1.0):
        rng = np.random.default_rng(seed)
        draw = lambda *s: f32_to_bf16_bits(rng.standard_normal(s, dtype=np.float32) * weight_scale)  # noqa: E731
        self.T, self.Hq, self.Hkv, self.d, self.rot, self.inter = T, Hq, Hkv, d, rot, interleaved
        self.q, self.k, self.v = draw(T, Hq, d), draw(T, Hkv, d), draw(T, Hkv, d)
        self.qw = f32_to_bf16_bits((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)) if norm else None
        self.kw = f32_to_bf16_bits((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)) if norm else None
        self.eps = 1e-6
        self.pos = rng.integers(0, context, T).astype(np.int32)
        angle = np.arange(context)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
        self.table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
        pages = -(-(T + 7) // ps) + 2
        self.loc = rng.permutation(pages * ps)[:T].astype(np.int32)
        if pad:
            self.loc[-pad:] = -1
        self.kc, self.vc = draw(pages, ps, Hkv, d), draw(pages, ps, Hkv, d)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev())
        self.dkc, self.dvc = to_dev(self.kc), to_dev(self.vc)

    def weights(self):
        return dict(q_weight=None if self.qw is None else to_dev(self.qw),
                    k_weight=None if self.kw is None else to_dev(self.kw))

    def call(self, q=None, k=None, v=None, **kw):
        q, k, v = (to_dev(x) if t is None else t for x, t in ((self.q, q), (self.k, k), (self.v, v)))
        args = dict(eps=self.eps, interleaved=self.inter, dev_status=self.status, **self.weights())
        args.update(kw)
        return pkv.qk_norm_rope_store(q, k, v, to_dev(self.pos) if self.rot else None,
                                      to_dev(self.table) if self.rot else None, to_dev(self.loc), self.dkc,
                                      self.dvc, **args)

    def want(self):
        half = self.rot // 2
        row = self.table[self.pos].astype(np.float64)
        cos, sin = row[:, :half], row[:, half:]
        w = lambda x: None if x is None else plain_ops.f64(x)  # noqa: E731
        q = plain_ops.norm_rope(plain_ops.f64(self.q), w(self.qw), self.eps, cos, sin, self.inter)
        k = plain_ops.norm_rope(plain_ops.f64(self.k), w(self.kw), self.eps, cos, sin, self.inter)
        return q, k

    def check(self, out, skip_k=(), skip_q=()):
        (q, q_tol), (k, k_tol) = self.want()
        rows = [t for t in range(self.T) if t not in skip_q]
        assert (np.abs(as_f64(out) - q)[rows] <= q_tol[rows]).all()
        stored = [t for t in range(self.T) if self.loc[t] >= 0 and t not in skip_k]
        at = self.loc[stored]
        got_k = as_f64(self.dkc).reshape(-1, self.Hkv, self.d)
        assert (np.abs(got_k[at] - k[stored]) <= k_tol[stored]).all()
        rest = np.ones(len(got_k), bool)
        rest[at] = False
        bits_k = to_host_bits(self.dkc).reshape(-1, self.Hkv, self.d)
        bits_v = to_host_bits(self.dvc).reshape(-1, self.Hkv, self.d)
        assert np.array_equal(bits_k[rest], self.kc.reshape(bits_k.shape)[rest])
        assert np.array_equal(bits_v[rest], self.vc.reshape(bits_v.shape)[rest])
        assert np.array_equal(bits_v[at], self.v[stored])


HEADS = [(16, 8, 128), (32, 8, 64), (8, 1, 128), (1, 1, 64), (5, 3, 128), (7, 2, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("T", [1, 2, 33, 700])
def test_matches_the_plain_form(T, Hq, Hkv, d, interleaved):
    c = Case(T + Hq, T, Hq, Hkv, d, d, interleaved=interleaved, ps=4, pad=min(2, T - 1))
    c.check(c.call())
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("d,rot", [(128, 0), (128, 16), (128, 64), (128, 112), (64, 0), (64, 16), (64, 32), (64, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_partial_rotation(d, rot, interleaved, norm):
    c = Case(rot, 45, 6, 2, d, rot, norm=norm, interleaved=interleaved)
    c.check(c.call())


@pytest.mark.parametrize("Hq,Hkv,d,rot,norm,interleaved", [
    (16, 8, 128, 128, True, False), (32, 8, 64, 64, False, False), (8, 1, 128, 64, True, True),
    (1, 1, 64, 16, True, False), (5, 3, 128, 112, True, False), (7, 2, 64, 0, True, False),
    (7, 2, 64, 64, False, True), (4, 4, 128, 0, False, False), (32, 32, 128, 128, True, False)])
@pytest.mark.parametrize("T", [690, 1367, 5003])
def test_many_tokens(T, Hq, Hkv, d, rot, norm, interleaved):
    c = Case(T, T, Hq, Hkv, d, rot, norm=norm, interleaved=interleaved, ps=16, pad=5)
    bad = [7, T // 2, T - 6]
    if rot:
        c.pos[bad[0]], c.pos[bad[1]] = -3, len(c.table)
    c.loc[bad[2]] = c.kc.shape[0] * 16
    out = c.call()
    assert int(c.status.item()) == pkv.DEV_BAD_SLOT | (pkv.DEV_BAD_POS if rot else 0)
    if rot:
        assert torch.isnan(out[bad[:2]]).all()
        c.pos[bad[:2]] = 0                  # for the plain form; these rows are not looked at
        c.loc[bad[:2]] = -1
    c.loc[bad[2]] = -1
    c.check(out, skip_q=bad[:2] if rot else ())


def test_many_tokens_in_place_from_one_buffer():
    """Queries in place; keys and values as column ranges."""
    c = Case(19, 4000, 16, 8, 128, 128, pad=3)
    joined = torch.zeros(4000, 16 * 128 + 8, dtype=torch.bfloat16, device=dev())
    k, v = joined[:, :1024].view(4000, 8, 128), joined[:, 1024:2048].view(4000, 8, 128)
    k.copy_(to_dev(c.k)), v.copy_(to_dev(c.v))
    before, q = joined.clone(), to_dev(c.q)
    c.call(q=q, k=k, v=v, out=q)
    c.check(q)
    assert torch.equal(joined, before) and int(c.status.item()) == 0


def test_without_norm_and_rotation_everything_is_copied():
    c = Case(5, 61, 16, 8, 128, 0, norm=False)
    assert np.array_equal(to_host_bits(c.call()), c.q)
    assert np.array_equal(to_host_bits(c.dkc).reshape(-1, 8, 128)[c.loc], c.k)


def test_norm_of_the_queries_only():
    c = Case(6, 20, 4, 4, 64, 64)
    c.kw = None
    c.check(c.call())


@pytest.mark.parametrize("scale", [1e-18, 1e-4, 1e4, 3e17])
def test_small_and_large_rows(scale):
    """eps stands beside squares down to 1e-36 and up to 1e35."""
    c = Case(7, 24, 4, 2, 128, 128, weight_scale=scale)
    c.check(c.call())


def test_zero_rows_stay_zero():
    c = Case(8, 9, 4, 2, 128, 128)
    c.q[3] = 0
    c.k[5] = 0
    out = c.call()
    c.check(out)
    assert not to_host_bits(out)[3].astype(np.int16).__and__(0x7fff).any()


def test_column_ranges_of_one_buffer_and_far_strides():
    c = Case(9, 50, 16, 8, 128, 128, pad=3)
    joined = torch.zeros(50, 32 * 128 + 64, dtype=torch.bfloat16, device=dev())
    views, col = [], 0
    for x, H in ((c.q, 16), (c.k, 8), (c.v, 8)):
        views.append(joined[:, col:col + H * 128].view(50, H, 128))
        views[-1].copy_(to_dev(x))
        col += H * 128
    before = joined.clone()
    c.check(c.call(*views))
    assert torch.equal(joined, before)


def test_in_place_queries():
    c = Case(10, 77, 16, 8, 128, 128)
    q = to_dev(c.q)
    assert c.call(q=q, out=q).data_ptr() == q.data_ptr()
    c.check(q)


def test_bad_positions_and_slots():
    c = Case(11, 40, 4, 2, 64, 64)
    c.pos[3], c.pos[8] = -1, len(c.table)
    c.loc[5] = c.kc.shape[0] * 16
    out = c.call()
    assert int(c.status.item()) == pkv.DEV_BAD_POS | pkv.DEV_BAD_SLOT
    assert torch.isnan(out[[3, 8]]).all()
    loc = c.loc.copy()
    c.pos[[3, 8]] = 0                       # for the plain form; these rows are not looked at
    c.loc = np.where(np.isin(np.arange(40), [3, 5, 8]), -1, loc).astype(np.int32)
    c.check(out, skip_q=(3, 8))


def test_nan_stays_in_its_row():
    c = Case(12, 30, 4, 2, 128, 128)
    c.q[4, 1, 7] = 0x7FC0
    c.k[9, 0, 3] = 0x7FC0
    out = as_f64(c.call())
    assert np.isnan(out[4, 1]).all()
    out[4, 1] = 0
    assert np.isfinite(out).all()
    got = as_f64(c.dkc).reshape(-1, 2, 128)
    assert np.isnan(got[c.loc[9], 0]).all()
    got[c.loc[9], 0] = 0
    assert np.isfinite(got).all()


def test_no_tokens():
    c = Case(13, 1, 4, 2, 128, 128)
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=dev())
    kv = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=dev())
    none = torch.empty(0, dtype=torch.int32, device=dev())
    out = pkv.qk_norm_rope_store(e, kv, kv, none, to_dev(c.table), none, c.dkc, c.dvc)
    assert out.shape == (0, 4, 128)
    assert np.array_equal(to_host_bits(c.dkc), c.kc)


def test_captured_and_replayed_on_another_stream():
    c = Case(14, 12, 16, 8, 128, 128)
    q, k, v = to_dev(c.q), to_dev(c.k), to_dev(c.v)
    pos, table, loc, w = to_dev(c.pos), to_dev(c.table), to_dev(c.loc), c.weights()
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pkv.qk_norm_rope_store(q, k, v, pos, table, loc, c.dkc, c.dvc, eps=c.eps, dev_status=c.status, out=out,
                               stream=s, **w)
    other = Case(15, 12, 16, 8, 128, 128)
    other.qw, other.kw, other.table = c.qw, c.kw, c.table
    other.dkc, other.dvc = c.dkc, c.dvc
    for x in (c, other):
        c.dkc.copy_(to_dev(x.kc)), c.dvc.copy_(to_dev(x.vc))
        q.copy_(to_dev(x.q)), k.copy_(to_dev(x.k)), v.copy_(to_dev(x.v))
        pos.copy_(to_dev(x.pos)), loc.copy_(to_dev(x.loc))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        x.check(out)


def test_slots_past_two_to_the_31_elements():
    """A pool of 2^32 + elements each for K and V: the last slots are reached."""
    ps, Hkv, d = 256, 8, 128
    pages = (1 << 32) // (ps * Hkv * d) + 2
    c = Case(16, 5, 16, Hkv, d, d, ps=ps)
    k = torch.empty(pages, ps, Hkv, d, dtype=torch.bfloat16, device=dev())
    v = torch.empty(pages, ps, Hkv, d, dtype=torch.bfloat16, device=dev())
    last = pages * ps
    loc = np.array([last - 1, last - 2, last - 300, 0, 77], np.int32)
    out = pkv.qk_norm_rope_store(to_dev(c.q), to_dev(c.k), to_dev(c.v), to_dev(c.pos), to_dev(c.table),
                                 to_dev(loc), k, v, dev_status=c.status, **c.weights())
    (q, q_tol), (kk, k_tol) = c.want()
    assert (np.abs(as_f64(out) - q) <= q_tol).all()
    at = torch.from_numpy(loc.astype(np.int64)).to(dev())
    assert (np.abs(as_f64(k.view(-1, Hkv, d)[at]) - kk) <= k_tol).all()
    assert np.array_equal(to_host_bits(v.view(-1, Hkv, d)[at]), c.v)
    assert int(c.status.item()) == 0


def test_refused_tensors():
    c = Case(17, 6, 4, 2, 64, 64)
    wide = torch.zeros(6, 8, 64, dtype=torch.bfloat16, device=dev())
    for bad in (dict(q=wide[:, ::2]), dict(k=to_dev(c.k).float()), dict(v=to_dev(c.v)[:5]),
                dict(q=to_dev(c.q).cpu()), dict(out=wide), dict(q_weight=wide[0, 0, :32])):
        with pytest.raises(ValueError):
            c.call(**bad)
    assert np.array_equal(to_host_bits(c.dkc), c.kc)
