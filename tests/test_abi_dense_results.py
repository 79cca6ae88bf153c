"""Dense attention refuses results that lie over its queries or over one another (no GPU needed)."""
import pytest
from test_abi_dense import _call


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_nvfp4_b200 import build
    build.build()
    import fp4_kv_cache_nvfp4_b200 as m
    return m


@pytest.mark.parametrize("prefill", [False, True])
def test_lse_over_queries_or_results_is_refused(csa2, prefill):
    rows, q, out = (5 if prefill else 2) * 16, 0x100000, 0x200000
    for dt, size in ((csa2.F32, 4), (csa2.BF16, 2)):
        for at, n in ((q, rows * 256), (out, rows * 128 * size)):
            for lse in (at, at + 4, at + n - 4, at - rows * 4 + 4):  # the last two share four bytes
                assert _call(csa2, prefill, q=q, out=out, lse=lse, dt=dt, ws=0x1000000) == 1
