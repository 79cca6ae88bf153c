"""Dense attention: what the host refuses, before the GPU is touched (no GPU needed)."""
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


def _call(csa2, prefill=False, desc=None, cache=None, **over):
    """Status of a call whose pointers are never followed: everything here is rejected or empty."""
    a = dict(q=0x1000, cu=0x1000, st=0x1000, lens=0x1000, out=0x1000, dt=0, lse=0x1000, B=2, T=5, max_len=1024,
             ws=0x100000, size=1 << 40, err=0x1000)
    a.update(over)
    d = csa2.default_desc(csa2.FULL, 1) if desc is None else desc
    c = csa2._binding._Cache(0x1000, 0x2000, None, None, 0x5000, 64, 16, 4) if cache is None else cache
    L = csa2.lib()
    if prefill:
        return L.csa2_dense_attn_prefill(ctypes.byref(d), ctypes.byref(c), P(a["q"]), P(a["cu"]), P(a["st"]),
                                         P(a["lens"]), P(a["out"]), a["dt"], P(a["lse"]), a["B"], a["T"], a["max_len"],
                                         P(a["ws"]), a["size"], P(a["err"]), None)
    return L.csa2_dense_attn_decode(ctypes.byref(d), ctypes.byref(c), P(a["q"]), P(a["lens"]), P(a["out"]), a["dt"],
                                    P(a["lse"]), a["B"], a["max_len"], P(a["ws"]), a["size"], P(a["err"]), None)


@pytest.mark.parametrize("prefill", [False, True])
def test_refusals(csa2, prefill):
    call = lambda **o: _call(csa2, prefill, **o)  # noqa: E731
    cache = lambda **o: csa2._binding._Cache(*[o.get(n, v) for n, v in (  # noqa: E731
        ("codes", 0x1000), ("scales", 0x2000), ("idx_k", None), ("idx_k_pooled", None), ("page_table", 0x5000),
        ("page_size", 64), ("max_pages", 16), ("n_phys", 4))])
    invalid = [dict(q=None), dict(q=0x1008), dict(lens=None), dict(lens=0x1002), dict(out=None), dict(out=0x1004),
               dict(dt=2), dict(dt=-1), dict(lse=None), dict(lse=0x1001), dict(B=-1), dict(max_len=0),
               dict(max_len=1025), dict(err=0x1002), dict(cache=cache(codes=None)), dict(cache=cache(scales=0x2008)),
               dict(cache=cache(page_table=None)), dict(cache=cache(page_size=48)), dict(cache=cache(page_size=4)),
               dict(cache=cache(n_phys=0)), dict(desc=csa2.default_desc(csa2.FULL, 3))]
    if prefill:
        invalid += [dict(cu=None), dict(cu=0x1001), dict(st=0x1002), dict(T=-1)]
    for o in invalid:
        assert call(**o) == 1, o
    for o in (dict(desc=csa2.default_desc(csa2.FULL, 1, n_heads=32)), dict(B=65537), dict(cache=cache(n_phys=1 << 25))):
        assert call(**o) == 2, o
    for o in (dict(ws=None), dict(ws=0x100010), dict(size=16)):
        assert call(**o) == 4, o
    assert call(B=0, q=None, lens=None, out=None, lse=None, ws=None, cu=None) == 0
    if prefill:
        assert call(T=0, q=None, lens=None, out=None, lse=None, ws=None, cu=None) == 0
        assert call(T=(1 << 26) + 1) == 2


@pytest.mark.parametrize("prefill", [False, True])
def test_results_over_queries_are_refused(csa2, prefill):
    q, n = 0x100000, (5 if prefill else 2) * 16 * 128
    for dt, size in ((csa2.F32, 4), (csa2.BF16, 2)):
        for out in (q, q + 16, q + n * 2 - 16, q - n * size + 16):  # the last two share 16 bytes
            assert _call(csa2, prefill, q=q, out=out, dt=dt, ws=0x1000000) == 1


def test_workspace(csa2):
    d = csa2.default_desc(csa2.FULL, 1)
    for prefill in (False, True):
        n = csa2.dense_attn_workspace_bytes(d, 8, prefill)
        assert n > 0 and n % 256 == 0
    assert csa2.lib().csa2_dense_attn_workspace_bytes(None, 8, 0) == 0
    assert csa2.dense_attn_workspace_bytes(d, -1) == 0


def test_binding_checks_tensors(csa2):
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)  # noqa: E731
    K = csa2.KVCache.from_tensors
    pt = z(2, 4, dt=torch.int32)
    c = K(z(64, 128), z(64, 16), pt, 8, idx_k=z(64, 64, dt=torch.int16), pooled=z(8, 64, dt=torch.bfloat16))
    assert c.n_phys_pages == 8 and c.struct().max_pages_per_seq == 4
    for bad in (lambda: K(z(60, 128), z(60, 16), pt, 8), lambda: K(z(64, 128), z(64, 8), pt, 8),
                lambda: K(z(64, 256)[:, ::2], z(64, 16), pt, 8), lambda: K(z(64, 128), z(64, 16), pt[0], 8),
                lambda: K(z(64, 128), z(64, 16), pt, 8, pooled=z(64, 64, dt=torch.int16)), lambda: K(z(64, 128), z(64, 16), pt, 0)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        K(z(64, 128, dt=torch.int8), z(64, 16), pt, 8)
    d = csa2.default_desc(csa2.FULL, 1)
    with pytest.raises(ValueError):  # on the CPU
        csa2.dense_attn_decode(d, c, z(2, 16, 128, dt=torch.bfloat16), z(2, dt=torch.int32), z(2, 16, 128, dt=torch.float32),
                               z(2, 16, dt=torch.float32), 32, z(1024))
