"""Orders of pieces within a block of the kernels of attention over common keys."""
import numpy as np
import pytest

from tests.common_keys_util import Cross, Shared, status_of

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
