"""Where a cache's arrays may be, checked by the binding before anything is launched (no GPU needed)."""
from types import SimpleNamespace

import pytest


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_nvfp4_b200 import build
    build.build()
    import fp4_kv_cache_nvfp4_b200 as m
    return m


def _cache(**where):
    """A handle whose arrays only know their GPU (-1: host memory)."""
    at = dict(page_table=0, codes=0, scales=0)
    at.update(where)
    return SimpleNamespace(**{k: SimpleNamespace(get_device=lambda n=n: n, device=f"cuda:{n}" if n >= 0 else "cpu")
                              for k, n in at.items()})


def test_dense_attention_reads_one_gpus_arrays(csa2):
    ok = csa2._binding._cache_on
    ok(_cache(), 0)
    ok(_cache(codes=-1, scales=-1), 0)  # the library has the answer to these
    for bad in (dict(page_table=1), dict(page_table=-1), dict(codes=1), dict(scales=1)):
        with pytest.raises(ValueError):
            ok(_cache(**bad), 0)
    with pytest.raises(ValueError):
        ok(_cache(), 1)
