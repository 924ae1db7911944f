"""Decode attention over page tables that name pages outside the pool, at page sizes whose rows are
gathered by several warps: wherever the bad page lies in a tile, it is reported, its sequence's
output is NaN, and no other sequence notices."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_out_gb300 as pkv
from synth import make_inputs
from tests.gpu_util import TOL, Run, as_f64, max_err

pytestmark = pytest.mark.gpu


def decode_case(seed, lens, Hq, Hkv, d, ps):
    lens = np.asarray(lens)
    return make_inputs(seed=seed, Hq=Hq, Hkv=Hkv, d=d, page_size=ps, new_lens=np.ones(len(lens), np.int64),
                       prefix_lens=lens - 1)


def check_bad(x, r, out, bad):
    assert r.dev_status() == pkv.DEV_BAD_PAGE
    got, ref = as_f64(out), oracle.run_inputs(x)
    good = [b for b in range(x.B) if b not in bad]
    assert np.isnan(got[bad]).all()
    assert max_err(got[good], ref[good]) <= TOL


# a tile holds 32 keys of head size 128, 64 of 64; its halves are gathered by two warps each
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 16, 8), (64, 32, 8), (128, 8, 1)])
@pytest.mark.parametrize("ps", [1, 2, 4, 16])
@pytest.mark.parametrize("key", [0, 15, 16, 31, 32, 37, 63, 99, 280, 299])
def test_a_bad_page_anywhere_in_a_tile(ps, key, d, Hq, Hkv):
    x = decode_case(60, [100, 50, 7, 300, 33], Hq, Hkv, d, ps)
    r = Run(x).store()
    r.page_table[3, key // ps] = x.num_pages
    r.page_table[0, min(key, 99) // ps] = -1
    check_bad(x, r, r.decode(), [0, 3])


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 16, 8), (64, 32, 8)])
@pytest.mark.parametrize("ps", [1, 2, 4])
@pytest.mark.parametrize("length", [1, 5, 16, 17, 33, 48])
@pytest.mark.parametrize("page", [1 << 30, -(1 << 31)])
def test_a_bad_first_page_of_a_tile_that_ends_early(ps, length, page, d, Hq, Hkv):
    """Keys past the end are read from no page that was not looked at."""
    x = decode_case(61, [40, length, 90], Hq, Hkv, d, ps)
    r = Run(x).store()
    r.page_table[1, (length - 1) // (4096 // d) * (4096 // d) // ps] = page
    check_bad(x, r, r.decode(), [1])


@pytest.mark.parametrize("ps", [1, 2, 4])
@pytest.mark.parametrize("key", [0, 20, 40])
def test_a_bad_page_under_the_fused_store(ps, key):
    x = decode_case(62, [100, 50, 70], 16, 8, 128, ps)
    r = Run(x)
    r.page_table[1, key // ps] = x.num_pages + 3
    out = pkv.paged_decode_attn_store(r.q, r.k_new, r.v_new, r.out_loc, r.k, r.v, r.page_table, r.seq_lens, x.scale,
                                      dev_status=r.status)
    check_bad(x, r, out, [1])


@pytest.mark.parametrize("ps", [1, 4])
def test_a_call_with_good_pages_follows(ps):
    """What a bad tile leaves in a ring stage or its flags does not reach the next sequences."""
    x = decode_case(63, [900] * 6, 16, 8, 128, ps)
    r = Run(x).store()
    table = r.page_table.clone()
    r.page_table[[0, 2, 4], 777 // ps] = -1
    check_bad(x, r, r.decode(), [0, 2, 4])
    r.page_table.copy_(table)
    r.status.zero_()
    out = r.decode()
    assert r.dev_status() == 0
    assert max_err(as_f64(out), oracle.run_inputs(x)) <= TOL
    assert torch.isfinite(out).all()
