"""Arguments that the operators around the cache refuse before they touch the device."""
import ctypes

import pytest
import torch

import paged_kv_cache_out_gb300 as pkv
from paged_kv_cache_out_gb300 import build as cuda_build

E, U = pkv.binding.EINVAL, pkv.binding.EUNSUPPORTED
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10002)


def at(n):
    return ctypes.c_void_p(n)


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return pkv.load_library()


def _store(lib, **kw):
    a = dict(q=FAKE, qs=2048, k=FAKE, ks=1024, v=FAKE, vs=1024, qw=None, kw=None, eps=1e-6, pos=FAKE, cs=FAKE,
             rows=64, rot=128, inter=0, loc=FAKE, T=4, Hq=16, Hkv=8, d=128, kc=FAKE, vc=FAKE, P=8, ps=16,
             out=at(0x90000), status=None, stream=None)
    a.update(kw)
    return lib.pkv_qk_norm_rope_store(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E), (dict(k=None), E), (dict(v=None), E), (dict(out=None), E), (dict(loc=None), E),
    (dict(kc=None), E), (dict(pos=None), E), (dict(cs=None), E), (dict(T=-1), E), (dict(Hq=0), E),
    (dict(Hkv=0), E), (dict(P=-1), E), (dict(ps=0), E), (dict(rows=-1), E), (dict(rot=-16), E),
    (dict(rot=144), E), (dict(eps=-1.0), E), (dict(eps=float("nan")), E), (dict(eps=float("inf")), E),
    (dict(qs=2040), E), (dict(ks=1016), E), (dict(vs=1000), E), (dict(qs=2052), E), (dict(ks=1028), E),
    (dict(q=ODD), E), (dict(kw=ODD), E), (dict(cs=ODD), E), (dict(out=ODD), E), (dict(vc=ODD), E),
    (dict(out=FAKE, qs=4096), E),                        # in place needs dense queries
    (dict(d=96, rot=96), U), (dict(rot=8), U), (dict(P=1 << 40), U),
    (dict(T=0, q=None, out=None), 0),
])
def test_store_refusals(lib, kw, want):
    assert _store(lib, **kw) == want


def _weights(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, pt=FAKE, stride=4, sl=FAKE, B=2, Hq=16, Hkv=8, d=128, ps=16, P=64,
             scale=0.088, acc=FAKE, rows=None, nrows=2, astride=64, maxlen=64, ws=FAKE, ws_bytes=1 << 40,
             status=None, out=FAKE, stream=None)
    a.update(kw)
    return lib.pkv_paged_decode_attn_weights(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), E), (dict(acc=None), E), (dict(acc=ODD), E), (dict(maxlen=-1), E), (dict(astride=63), E),
    (dict(nrows=1), E), (dict(nrows=-1), E), (dict(Hq=12), E), (dict(B=-1), E), (dict(ws=None), E),
    (dict(scale=float("nan")), E), (dict(out=ODD), E), (dict(d=96), U), (dict(Hq=24), U), (dict(ps=24), U),
    (dict(ps=512), U), (dict(B=5000, nrows=5000), U), (dict(B=0, acc=None), 0),
])
def test_decode_weights_refusals(lib, kw, want):
    assert _weights(lib, **kw) == want


def test_decode_weights_workspace_of_bad_sizes_is_zero(lib):
    size = lib.pkv_decode_weights_workspace_size
    assert size(4, 12, 8, 128, 100) == 0 and size(4, 16, 8, 96, 100) == 0 and size(4, 16, 8, 128, -1) == 0


def _evict(lib, **kw):
    a = dict(k=FAKE, v=FAKE, pt=FAKE, stride=4, pto=FAKE, strideo=4, sl=at(0x20000), keep=at(0x30000), B=2,
             Hkv=8, d=128, ps=16, P=64, first=4, recent=16, acc=at(0x100000), acco=at(0x100000), rows=None,
             nrows=2, astride=64, kept=at(0x40000), maxkeep=32, new=at(0x50000), status=None, stream=None)
    a.update(kw)
    return lib.pkv_kv_evict(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), E), (dict(v=None), E), (dict(pt=None), E), (dict(pto=None), E), (dict(sl=None), E),
    (dict(keep=None), E), (dict(acc=None), E), (dict(acco=None), E), (dict(kept=None), E), (dict(new=None), E),
    (dict(B=-1), E), (dict(Hkv=0), E), (dict(P=0), E), (dict(first=-1), E), (dict(recent=-1), E),
    (dict(nrows=1), E), (dict(astride=-1), E), (dict(maxkeep=-1), E), (dict(k=ODD), E), (dict(acc=ODD), E),
    (dict(new=at(0x20000)), E), (dict(new=at(0x20004)), E),      # would be read while it is written
    (dict(new=at(0x30004)), E), (dict(rows=at(0x50000)), E),
    (dict(acco=at(0x100100)), E),                                # overlaps acc, but is not acc
    (dict(d=96), U), (dict(ps=24), U), (dict(ps=512), U), (dict(B=5000, nrows=5000), U),
    (dict(Hkv=70000), U), (dict(P=1 << 40), U), (dict(B=0, k=None), 0),
])
def test_evict_refusals(lib, kw, want):
    assert _evict(lib, **kw) == want


def test_tensors_off_the_gpu_are_refused(lib):
    b, i, f = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, 8)
    cache, table = torch.zeros(4, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    calls = [lambda: pkv.qk_norm_rope_store(b, b, b, None, None, i, cache, cache),
             lambda: pkv.paged_decode_attn_weights(b, cache, cache, table, i, 1.0, f, 8,
                                                   workspace=torch.zeros(16, dtype=torch.uint8)),
             lambda: pkv.kv_evict(cache, cache, table, i, i, f, 1, 1)]
    for call in calls:
        with pytest.raises(ValueError, match="on the current CUDA device"):
            call()
