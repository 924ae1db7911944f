"""Decode attention over page tables that name pages outside the pool, at page sizes whose rows are
gathered by several warps: wherever the bad page lies in a tile, it is reported, its sequence's
output is NaN, and no other sequence notices."""
import numpy as np
import pytest

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
