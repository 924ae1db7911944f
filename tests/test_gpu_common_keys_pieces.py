"""Orders of pieces within a block of the kernels of attention over common keys."""
import numpy as np
import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from tests.common_keys_util import Cross, Shared, status_of
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_pairs_and_single_tiles_in_turn(d, seed):
    """Blocks of up to 256 rows and of up to 128, most of them over one tile of keys, several to a
    thread block."""
    rng = np.random.default_rng(seed)
    tokens = rng.choice([32, 16, 20, 9, 3, 41, 60], 900).tolist()
    states = rng.choice([1, 60, 128, 128, 129, 300, 0, 700], 900).tolist()
    x = Cross(seed, tokens, states, Hq=16, Hkv=2, d=d)
    first = x.call()
    x.check(first)
    for _ in range(20):
        assert (x.call() == first).all()
    assert status_of(x) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_groups_of_many_forms(d):
    rng = np.random.default_rng(d)
    groups = [(rng.integers(0, 40, int(rng.choice([33, 20, 2, 9]))).tolist(), int(rng.choice([4, 8, 8, 9, 20])))
              for _ in range(180)]
    x = Shared(4, groups, Hq=16, Hkv=2, d=d)
    first = x.call()
    x.check(first)
    for _ in range(20):
        assert (x.call() == first).all()
    assert status_of(x) == 0


@pytest.mark.parametrize("make", [
    lambda: Cross(7, [1, 40, 3, 150, 2, 1, 1, 16], [900, 700, 0, 130, 40, 333, 64, 512], extra_rows=4),
    lambda: Shared(8, [([17, 200, 5], 40), ([9], 0), ([1] * 40, 16), ([None, 3], 1)])])
def test_calls_in_a_row_on_the_same_buffers_see_the_last_contents(make):
    """Queries, lengths and stored values change in place between calls, with nothing waited for and one
    workspace: both kernels work in every call, and the one that starts beside the other reads what the
    kernels before wrote."""
    x = make()
    gen = torch.Generator(device=dev()).manual_seed(9)
    n, live = 30, (x.dl > 8).int()
    sets = [(torch.randn(x.dq.shape, dtype=torch.bfloat16, device=dev(), generator=gen), x.dl - live * (i % 4),
             torch.randn(x.dv.shape, dtype=torch.bfloat16, device=dev(), generator=gen)) for i in range(n)]
    ws = (pkv.cross_workspace(len(x.lens), x.Hq, x.Hkv, x.d) if isinstance(x, Cross)
          else pkv.decode_shared_workspace(len(x.lens), x.Hq, x.Hkv, x.d))

    def run(wait):
        outs = [torch.zeros_like(x.dq) for _ in range(n)]
        torch.cuda.synchronize()
        for (q, lens, v), out in zip(sets, outs):
            x.dq.copy_(q), x.dl.copy_(lens), x.dv.copy_(v)
            if wait:
                torch.cuda.synchronize()
                ws.fill_(255)
            x.call(workspace=ws, out=out)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(run(False), want))
    # (the 40 sequences with one key of their own fall below their group's shared ones: NaN)
    assert status_of(x) == (0 if isinstance(x, Cross) else 64)
