"""The plain forms that the operators' parity tests go by, checked against closed forms,
torch and differences of their own, on the CPU."""
import math

import numpy as np
import pytest
import torch

from synth import make_inputs
from tests import plain_ops


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_turns_each_pair_and_keeps_its_length(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64))
    angle = rng.uniform(-50, 50, (3, 16))
    y, _ = plain_ops.norm_rope(x, None, 0.0, np.cos(angle), np.sin(angle), interleaved)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    a, b = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    turned = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle)[:, None]
    assert np.allclose(y[..., a], turned.real) and np.allclose(y[..., b], turned.imag)


def test_scores_of_rotated_rows_depend_on_the_distance_only():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    freq = 10000.0 ** (-np.arange(32) / 32)

    def score(i, j):
        a, _ = plain_ops.norm_rope(q, None, 0.0, np.cos(i * freq)[None], np.sin(i * freq)[None], False)
        b, _ = plain_ops.norm_rope(k, None, 0.0, np.cos(j * freq)[None], np.sin(j * freq)[None], False)
        return float((a * b).sum())

    assert math.isclose(score(7, 3), score(1007, 1003), rel_tol=1e-9)


def test_norm_matches_torch():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((5, 3, 128)), rng.standard_normal(128)
    y, _ = plain_ops.norm_rope(x, w, 1e-6, np.ones((5, 0)), np.ones((5, 0)), False)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (128,), torch.from_numpy(w), 1e-6)
    assert np.allclose(y, want.numpy(), rtol=1e-12)


def test_decode_weights_sum_to_the_query_heads_and_match_sdpa():
    x = make_inputs(seed=3, Hq=8, Hkv=2, d=64, page_size=4, new_lens=[1, 1, 1], prefix_lens=[0, 6, 20])
    k, v = x.k_cache.copy(), x.v_cache.copy()
    k.reshape(-1, 2, 64)[x.out_loc], v.reshape(-1, 2, 64)[x.out_loc] = x.k_new, x.v_new
    for b, (out, w, _, _) in enumerate(plain_ops.decode_weights(x.q, k, v, x.page_table, x.seq_lens, x.scale)):
        assert np.allclose(w.sum(1), 4)
        slots = plain_ops.slots_of(x.page_table[b], 4, x.seq_lens[b])
        K, V = (torch.from_numpy(plain_ops.f64(p.reshape(-1, 2, 64)[slots])).transpose(0, 1) for p in (k, v))
        Q = torch.from_numpy(plain_ops.f64(x.q[b]))[:, None]
        want = torch.nn.functional.scaled_dot_product_attention(
            Q, K.repeat_interleave(4, 0), V.repeat_interleave(4, 0), scale=x.scale)[:, 0]
        assert np.allclose(out, want.numpy())


def test_kept_positions():
    s = [9.0, 0.1, 0.5, 0.3, 0.5, 0.2, 0.0]
    assert plain_ops.evict_kept(s, 4, 1, 1).tolist() == [0, 2, 4, 6]
    assert plain_ops.evict_kept(s, 3, 1, 1).tolist() == [0, 2, 6]          # equal sums: the lower position
    assert plain_ops.evict_kept(s, 3, 0, 0).tolist() == [0, 2, 4]
    assert plain_ops.evict_kept(s, 2, 5, 5).tolist() == [0, 1]             # the first come before the last
    assert plain_ops.evict_kept(s, 99, 1, 1).tolist() == list(range(7))
    assert plain_ops.evict_kept(s, 0, 1, 1).tolist() == []
    nan = float("nan")
    assert plain_ops.evict_kept([nan, -math.inf, nan, 1.0], 3, 0, 0).tolist() == [0, 1, 3]
    assert plain_ops.evict_kept([-0.0, 0.0, 0.0], 1, 0, 0).tolist() == [0]
