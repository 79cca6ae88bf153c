"""Page operations: what the host refuses, before the GPU is touched (no GPU needed)."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def csa2():
    from fp4_kv_cache_nvfp4_b200 import build
    build.build()
    import fp4_kv_cache_nvfp4_b200 as m
    return m


def _caches(csa2, n=2, **over):
    C = (csa2._binding._Cache * max(n, 1))()
    for i in range(max(n, 1)):
        C[i] = csa2._binding._Cache(0x10000 * (i + 1), 0x2000, 0x3000, 0x4000, 0x5000, 64, 16, 40)
    for k, v in over.items():
        setattr(C[n - 1], k, v)
    return C


def _call(csa2, what, C, n_caches=2, **over):
    a = dict(src=0x1000, dst=0x1000, table=0x1000, n_seqs=4, refs=0x1000, lens=0x1000, n=3, map=0x1000, live=0x1000,
             ws=0x100000, size=1 << 40, err=0x1000)
    a.update(over)
    p = {k: P(v) if k not in ("n_seqs", "n", "size") else v for k, v in a.items()}
    L = csa2.lib()
    if what == "copy":
        return L.csa2_kv_pages_copy(n_caches, C, p["src"], p["dst"], p["n"], p["err"], None)
    if what == "fork":
        return L.csa2_kv_pages_fork(n_caches, C, p["table"], p["n_seqs"], p["refs"], p["lens"], p["src"], p["dst"],
                                    p["n"], p["ws"], p["size"], p["err"], None)
    if what == "free":
        return L.csa2_kv_pages_free(C, p["table"], p["n_seqs"], p["refs"], p["lens"], p["src"], p["n"], p["err"], None)
    return L.csa2_kv_pages_compact(n_caches, C, p["table"], p["n_seqs"], p["refs"], p["map"], p["live"], p["ws"],
                                   p["size"], p["err"], None)


def test_refusals(csa2):
    ok = _caches(csa2)
    bad = {"copy": [dict(src=None), dict(dst=0x1001), dict(n=-1), dict(err=0x1001)],
           "fork": [dict(src=None), dict(dst=None), dict(table=0x1002), dict(refs=0x1004), dict(lens=None), dict(n=-1),
                    dict(n_seqs=0), dict(err=0x1001)],
           "free": [dict(src=None), dict(table=None), dict(refs=0x1002), dict(lens=None), dict(n=-1), dict(n_seqs=0)],
           "compact": [dict(table=None), dict(refs=0x1008), dict(map=None), dict(live=0x1001), dict(n_seqs=-1)]}
    for what, cases in bad.items():
        for o in cases:
            assert _call(csa2, what, ok, **o) == 1, (what, o)
    for what in ("copy", "fork", "compact"):
        assert _call(csa2, what, ok, n_caches=0) == 1
        assert _call(csa2, what, _caches(csa2, 17), n_caches=17) == 2
        for o in (dict(page_size=32), dict(n_phys_pages=41), dict(max_pages_per_seq=15), dict(codes=0x10000),
                  dict(codes=None), dict(scales=0x2001), dict(idx_k=0x3002), dict(idx_k_pooled=0x4008)):
            assert _call(csa2, what, _caches(csa2, 2, **o)) == 1, (what, o)
        assert _call(csa2, what, _caches(csa2, 1, n_phys_pages=(1 << 22) + 1), n_caches=1) == 2
    for what in ("fork", "compact"):
        for o in (dict(ws=None), dict(ws=0x100080), dict(size=8)):
            assert _call(csa2, what, ok, **o) == 4, (what, o)
    assert _call(csa2, "fork", ok, n=1025) == 2
    for what in ("copy", "fork", "free"):
        assert _call(csa2, what, ok, n=0, src=None, dst=None, table=None, refs=None, lens=None, ws=None) == 0


def test_workspace(csa2):
    assert csa2.kv_pages_workspace_bytes(1000, 64) % 256 == 0
    assert csa2.kv_pages_workspace_bytes(1 << 22, 1024) >= 3 * 4 << 22
    for bad in ((0, 1), ((1 << 22) + 1, 1), (10, -1), (10, 1025)):
        with pytest.raises(ValueError):
            csa2.kv_pages_workspace_bytes(*bad)


def test_binding_checks_tensors(csa2):
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    mk = lambda pt: csa2.KVCache.from_tensors(z(64, 128, dt=torch.uint8), z(64, 16, dt=torch.uint8), pt, 8)  # noqa: E731
    a, b = mk(z(2, 4)), mk(z(2, 4))
    ws = z(4096, dt=torch.uint8)
    for bad in (lambda: csa2.kv_pages_fork([a, b], z(8), z(2), z(1), z(1), ws),  # two tables
                lambda: csa2.kv_pages_fork([], z(8), z(2), z(1), z(1), ws),
                lambda: csa2.kv_pages_free(a, z(8), z(2), z(1)),                  # on the CPU
                lambda: csa2.kv_pages_copy([a], z(1), z(1))):
        with pytest.raises(ValueError):
            bad()


def test_pooled_alone_is_refused(csa2):
    """Pooled indexer keys without the keys they pool: they would not be copied."""
    for what in ("copy", "fork", "compact"):
        assert _call(csa2, what, _caches(csa2, 2, idx_k=None)) == 1
        assert _call(csa2, what, _caches(csa2, 2, idx_k=None, idx_k_pooled=None), n=0, table=None) == \
            (0 if what != "compact" else 1)
