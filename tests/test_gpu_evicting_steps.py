"""The three operators as an engine runs them: decode steps that norm, rotate and store the new
token, attend and add up the weights, and an eviction whenever the sequences reach their limit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from synth.workloads import f32_to_bf16_bits
from tests import plain_ops
from tests.gpu_util import as_f64, dev, to_dev, to_host_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,d,ps", [(16, 8, 128, 16), (8, 2, 64, 1)])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_steps_with_evictions(Hq, Hkv, d, ps, graph):
    B, limit, budget, first, recent, steps = 3, 48, 32, 2, 6, 40
    rng = np.random.default_rng(Hq + ps)
    lens = np.array([40, 12, 47], np.int32)
    context = 200
    angle = np.arange(context)[:, None] * 10000.0 ** (-np.arange(d // 2) / (d // 2))
    table = to_dev(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    cos, sin = np.split(table.cpu().numpy().astype(np.float64), 2, axis=1)
    w = f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(d)).astype(np.float32))
    per = limit // ps
    pt = rng.permutation(B * per + 2)[:B * per].reshape(B, per).astype(np.int32)
    draw = lambda *s: f32_to_bf16_bits(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    pages = B * per + 2
    k, v = to_dev(draw(pages, ps, Hkv, d)), to_dev(draw(pages, ps, Hkv, d))
    acc = to_dev(np.where(np.arange(limit) < lens[:, None, None], rng.random((B, Hkv, limit)), np.nan).astype(np.float32))
    # the device's state of the step
    q_in, k_in, v_in = (torch.empty(B, H, d, dtype=torch.bfloat16, device=dev()) for H in (Hq, Hkv, Hkv))
    positions, loc, sl, keep = (torch.zeros(B, dtype=torch.int32, device=dev()) for _ in range(4))
    new = torch.zeros_like(sl)
    kept = torch.zeros(B, Hkv, limit, dtype=torch.int32, device=dev())
    out, status, dw, dpt = torch.empty_like(q_in), torch.zeros(1, dtype=torch.int32, device=dev()), to_dev(w), to_dev(pt)
    ws = pkv.decode_weights_workspace(B, Hq, Hkv, d, limit)

    def step(**kw):
        q = pkv.qk_norm_rope_store(q_in, k_in, v_in, positions, table, loc, k, v, q_weight=dw, k_weight=dw,
                                   dev_status=status, **kw)
        pkv.paged_decode_attn_weights(q, k, v, dpt, sl, d ** -0.5, acc, limit, workspace=ws, dev_status=status,
                                      out=out, **kw)
        # sequences that are not full keep everything
        pkv.kv_evict(k, v, dpt, sl, keep, acc, first, recent, kept=kept, new_seq_lens=new, dev_status=status, **kw)

    run = step
    if graph:
        sl.fill_(0), loc.fill_(-1)
        step()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(stream=s)
        run = g.replay
        torch.cuda.synchronize()

    position = lens.astype(np.int64) + 5           # a sequence that was shortened before
    evictions = 0
    for _ in range(steps):
        lens = lens + 1
        x = [draw(B, H, d) for H in (Hq, Hkv, Hkv)]
        for t, h in zip((q_in, k_in, v_in), x):
            t.copy_(to_dev(h))
        slot = np.array([plain_ops.slots_of(pt[b], ps, int(lens[b]))[-1] for b in range(B)], np.int32)
        n = np.where(lens >= limit, budget, limit).astype(np.int32)
        for t, h in ((positions, position.astype(np.int32)), (loc, slot), (sl, lens), (keep, n)):
            t.copy_(to_dev(h))
        k0, v0, acc0 = to_host_bits(k), to_host_bits(v), acc.cpu().numpy()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        # the plain step, from the state before it; the rounded rows that it stores and attends
        # with are taken from the kernel once they are found within rounding
        k1, v1 = to_host_bits(k).reshape(-1, Hkv, d), to_host_bits(v).reshape(-1, Hkv, d)
        k_ref, v_ref = k0.reshape(-1, Hkv, d).copy(), v0.reshape(-1, Hkv, d).copy()
        args = (plain_ops.f64(w), 1e-6, cos[position], sin[position], False)
        k_new, k_tol = plain_ops.norm_rope(plain_ops.f64(x[1]), *args)
        q_new, _ = plain_ops.norm_rope(plain_ops.f64(x[0]), *args)
        stays = kept.cpu().numpy()
        for b in range(B):
            m = min(int(n[b]), int(lens[b]))
            for h in range(Hkv):
                # the newest key is among the recent ones: it is the last that stays
                at = plain_ops.slots_of(pt[b], ps, m)[-1]
                assert stays[b, h, m - 1] == lens[b] - 1
                assert (np.abs(plain_ops.f64(k1[at, h]) - k_new[b, h]) <= k_tol[b, h]).all()
                k_ref[slot[b], h] = k1[at, h]
                v_ref[slot[b], h] = x[2][b, h]
        q_bits = f32_to_bf16_bits(q_new.astype(np.float32))
        want = plain_ops.decode_weights(q_bits, k_ref.reshape(k0.shape), v_ref.reshape(v0.shape), pt, lens, d ** -0.5)
        got_out, got_acc = as_f64(out), acc.cpu().numpy()
        for b, (o, wt, tol_o, tol_w) in enumerate(want):
            # q_bits may differ from the kernel's queries by one rounding here and there, so a
            # score by HALF_STEP of the sum of |q k| at most
            L = int(lens[b])
            slots = plain_ops.slots_of(pt[b], ps, L)
            size = np.abs(plain_ops.f64(k_ref[slots])).sum(-1).max() * np.abs(plain_ops.f64(q_bits[b])).max() * d ** -0.5
            loose = 2 * (np.exp(2 * plain_ops.HALF_STEP * size) - 1)
            vmax = np.abs(plain_ops.f64(v_ref[slots])).max()
            assert (np.abs(got_out[b] - o) <= tol_o + loose * vmax).all()
            m = min(int(n[b]), L)
            for h in range(Hkv):
                total = np.where(np.arange(L) < L - 1, acc0[b, h, :L], 0).astype(np.float64) + wt[h]
                stay = stays[b, h, :m]
                assert (np.diff(stay) > 0).all() and stay[0] >= 0 and stay[-1] < L
                assert np.isin(np.arange(min(first, m)), stay).all()
                assert np.isin(np.arange(L - min(recent, m), L), stay).all()
                tol = tol_w[h] + loose * wt[h] + 2 * plain_ops.U * np.abs(total)
                assert (np.abs(got_acc[b, h, :m] - total[stay]) <= tol[stay]).all()
                gone = np.setdiff1d(np.arange(L), stay)
                free = [j for j in stay if first <= j < L - recent]
                if len(gone) and free:
                    # nothing that went was heavier than what stayed, up to the sums' tolerance
                    assert (total[gone] - tol[gone]).max() <= (total[free] + tol[free]).min()
                to, frm = plain_ops.slots_of(pt[b], ps, m), slots[stay]
                assert np.array_equal(k1[to, h], k_ref[frm, h]) and np.array_equal(v1[to, h], v_ref[frm, h])
            evictions += m < L
            lens[b] = m
        assert np.array_equal(new.cpu().numpy(), lens)
        position = position + 1
    assert evictions >= 4
