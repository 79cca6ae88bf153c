"""Where a cache's arrays may be, checked by the binding before anything is launched (no GPU needed)."""
from types import SimpleNamespace

import pytest
import torch


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


def test_calls_refuse_arrays_that_kernels_cannot_read(csa2):
    """A handle made on ordinary host memory reaches no kernel."""
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    u8, i16, f32 = torch.uint8, torch.int16, torch.float32
    c = csa2.KVCache.from_tensors(z(64, 128, dt=u8), z(64, 16, dt=u8), z(2, 4), 8, idx_k=z(64, 64, dt=i16),
                                  pooled=z(8, 64, dt=i16))
    d = csa2.default_desc(csa2.FULL, 1)
    q, w, lens, ids, ws = z(2, 4, 64, dt=i16), z(2, 4, dt=f32), z(2), z(2, 512), z(1 << 20, dt=u8)
    qh, swa, out, lse = z(2, 16, 128, dt=i16), z(2, 128, 256, dt=i16), z(2, 16, 128, dt=f32), z(2, 16, dt=f32)
    for call in (lambda: csa2.kv_quant_append(c, z(2, 256, dt=f32), None, z(2, dt=torch.int64)),
                 lambda: csa2.indexer_topk(d, c, csa2.TOKEN, q, w, lens, ids, 2, 32, ws),
                 lambda: csa2.indexer_topk_noalloc(d, c, csa2.TOKEN, q, w, lens, ids, 2, 32),
                 lambda: csa2.indexer_score_ids(d, c, csa2.TOKEN, q, w, lens, ids, 0, z(2, 512, dt=f32), ids, 2, 32),
                 lambda: csa2.sparse_attn_decode(d, c, qh, ids, swa, lens, out, lse, 2),
                 lambda: csa2.sparse_attn_prefill(d, c, qh, ids, lens, swa, 0, 2, out, lse, 2),
                 lambda: csa2.decode_layers([d], c, [q], [w], [qh], [swa], lens, ids, ids, [out], [lse], 2, 32, ws)):
        with pytest.raises(ValueError, match="page_table on cpu"):
            call()
