"""Every attention call with tensors that begin on a 16-byte boundary and on no wider one, which is
all that the library asks for."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_out_gb300 as pkv
from synth import make_inputs
from tests.common_keys_util import Cross, Shared, status_of
from tests.gpu_util import TOL, Run, as_f64, dev, max_err

pytestmark = pytest.mark.gpu


def placed(t):
    """A copy of t that begins 16 bytes past a 32-byte boundary, and the buffer around it."""
    room = torch.full((t.numel() + 16,), 3.0, dtype=torch.bfloat16, device=dev())
    at = room[8:8 + t.numel()].view(t.shape)
    at.copy_(t)
    assert at.data_ptr() % 32 == 16 and at.is_contiguous()
    return at, room


def output_like(q):
    return placed(torch.full_like(q, 3.0))


def untouched(room):
    return bool((room[:8] == 3.0).all() and (room[-8:] == 3.0).all())


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 8, 128), (8, 1, 128), (4, 4, 64), (32, 8, 64)])
@pytest.mark.parametrize("page_size", [1, 16])
def test_cross_attention(Hq, Hkv, d, page_size):
    """Whole blocks of few rows, of up to 128 and of up to 256, and cut ones."""
    tokens = [1, 3, 0, 20, 100, 33, 64, 200, 256, 300, 2, 40] * 4
    states = [100, 0, 7, 128, 90, 1, 300, 60, 128, 40, 2000, 1500] * 4
    x = Cross(Hq, tokens, states, Hq, Hkv, d, page_size, extra_rows=3)
    x.dq, x.dk, x.dv = placed(x.dq)[0], placed(x.dk)[0], placed(x.dv)[0]
    out, room = output_like(x.dq)
    x.call(out=out)
    assert status_of(x) == 0
    x.check(out)
    assert untouched(room) and (out[x.cu[-1]:] == 3.0).all()


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 8, 128), (8, 1, 128), (4, 4, 64)])
@pytest.mark.parametrize("page_size", [1, 16])
def test_decode_with_groups(Hq, Hkv, d, page_size):
    groups = [([17, 1, None, 129], 20), ([5], 0), ([2] * 35 + [0] * 3, 9), ([30] * 130, 8)]
    x = Shared(Hq, groups, Hq, Hkv, d, page_size)
    x.dq, x.dk, x.dv = placed(x.dq)[0], placed(x.dk)[0], placed(x.dv)[0]
    out, room = output_like(x.dq)
    x.call(out=out)
    assert status_of(x) == 0
    x.check(out)
    assert untouched(room)


def moved(x):
    r = Run(x).store()
    r.q, r.k, r.v = placed(r.q)[0], placed(r.k)[0], placed(r.v)[0]
    return r


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("ps", [1, 16])
def test_prefill(d, G, ps):
    x = make_inputs(seed=60 + G, Hq=2 * G, Hkv=2, d=d, page_size=ps, new_lens=[1, 17, 128, 129, 300],
                    prefix_lens=[0, 100, 5, 256, 77])
    r = moved(x)
    out, room = output_like(r.q)
    r.prefill(out=out)
    assert r.dev_status() == 0
    assert max_err(as_f64(out), oracle.run_inputs(x, threads=8)) <= TOL and untouched(room)


@pytest.mark.parametrize("ps", [1, 16])
def test_prefill_with_groups(ps):
    x = make_inputs(seed=62, Hq=16, Hkv=8, d=128, page_size=ps, new_lens=[130, 5, 40, 70], prefix_lens=[256] * 4)
    r = moved(x)
    r.page_table[1:3, :256 // ps] = r.page_table[0, :256 // ps]
    out, room = output_like(r.q)
    want = r.prefill()
    r.prefill_shared(group_start=[0, 3, 4], prefix_len=[256, 0], out=out)
    assert r.dev_status() == 0
    # two results of the same rows, each within the bound of one
    assert max_err(as_f64(out), as_f64(want)) <= 2 * TOL and untouched(room)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [1, 16])
def test_decode(d, ps):
    lens = np.array([77, 300, 1024, 5000])
    x = make_inputs(seed=61, Hq=16, Hkv=8, d=d, page_size=ps, new_lens=np.ones(4, np.int64), prefix_lens=lens - 1)
    r = moved(x)
    out, room = output_like(r.q)
    r.decode(out=out)
    ref = oracle.run_inputs(x, threads=8)
    assert r.dev_status() == 0
    assert max_err(as_f64(out), ref) <= TOL and untouched(room)
    out, room = output_like(r.q)
    acc = torch.zeros(4, 8, x.page_table.shape[1] * ps, dtype=torch.float32, device=dev())
    pkv.paged_decode_attn_weights(r.q, r.k, r.v, r.page_table, r.seq_lens, x.scale, acc, 5000, out=out,
                                  dev_status=r.status)
    assert r.dev_status() == 0
    assert max_err(as_f64(out), ref) <= TOL and untouched(room)
