"""Loading the compiled binding from several threads at once."""
import threading
import time

import pytest

from paged_kv_cache_out_gb300 import binding


@pytest.fixture
def loads(tmp_path, monkeypatch):
    """Loads of a binding that takes a while to come up."""
    made = []

    class Loader:
        def __init__(self, name, path):
            assert path == str(tmp_path / "ext.so")

        def create_module(self, spec):
            return None

        def exec_module(self, module):
            made.append(module)
            time.sleep(0.2)
            module.kv_evict = lambda *args: 0

    (tmp_path / "ext.so").write_text("")
    monkeypatch.setattr(binding, "EXT_PATH", str(tmp_path / "ext.so"))
    monkeypatch.setattr(binding, "_ext", None)
    monkeypatch.setattr(binding, "load_library", lambda: None)
    monkeypatch.setattr(binding.importlib.machinery, "ExtensionFileLoader", Loader)
    return made


def test_threads_load_it_once_and_none_sees_it_half_made(loads):
    results, start = [], threading.Barrier(4)

    def first_call(delay):
        start.wait()
        time.sleep(delay)
        try:
            results.append((binding._ext or binding.load_extension()).kv_evict())
        except Exception as e:
            results.append(e)

    threads = [threading.Thread(target=first_call, args=(d,)) for d in (0, 0, 0.05, 0.1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert results == [0, 0, 0, 0] and len(loads) == 1


def test_a_missing_binding_is_an_error_each_time(loads, tmp_path, monkeypatch):
    monkeypatch.setattr(binding, "EXT_PATH", str(tmp_path / "none.so"))
    for _ in range(2):
        with pytest.raises(RuntimeError, match="is not built"):
            binding.load_extension()
