"""ctypes marshalling for include/csa2.h.  No arithmetic of the method lives here."""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libcsa2.so")

FULL, REINDEX, REUSE = 0, 1, 2
BLOCK, TOKEN = 0, 1
F32, BF16 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported dimension or size", 3: "CUDA error",
          4: "workspace missing or too small"}


class CSA2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: csa2 status {status} ({STATUS.get(status, '?')})")
        self.status = status


class LayerDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("mode", "ratio", "topk", "block", "keep_blocks", "window", "n_heads",
                                                "head_dim", "idx_heads", "idx_dim")]


class _Cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("idx_k", ctypes.c_void_p),
                ("idx_k_pooled", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("n_phys_pages", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None
_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """The loaded libcsa2.so.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(lib_path):
                raise ImportError(f"libcsa2.so not built ({lib_path}); run python -m fp4_kv_cache_nvfp4_b200.build")
            L = ctypes.CDLL(lib_path)
            L.csa2_layer_desc_default.argtypes = [ctypes.POINTER(LayerDesc), _I32, _I32]
            L.csa2_layer_desc_default.restype = None
            L.csa2_schedule.argtypes = [_I32, _P]
            L.csa2_schedule.restype = _I32
            L.csa2_kv_quant_append.argtypes = [ctypes.POINTER(_Cache), _P, _I32, _P, _I64, _I32, _P, _P, _P]
            L.csa2_indexer_workspace_bytes.argtypes = [ctypes.POINTER(LayerDesc), _I32, _I32, _I64, _I32]
            L.csa2_indexer_workspace_bytes.restype = _SZ
            L.csa2_indexer_topk.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(_Cache), _I32, _P, _P, _P, _P,
                                            _P, _P, _P, _I32, _I64, _P, _SZ, _P, _P]
            L.csa2_sparse_attn_decode.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(_Cache), _P, _P, _P, _P,
                                                  _P, _P, _P, _I32, _P, _P]
            L.csa2_sparse_attn_prefill.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(_Cache), _P, _P, _P, _P,
                                                   _I32, _I32, _P, _P, _I32, _P, _P]
            L.csa2_decode_layers.argtypes = [_I32, ctypes.POINTER(LayerDesc), ctypes.POINTER(_Cache), _P, _P, _P, _P,
                                             _P, _P, _P, _P, _P, _P, _I32, _I64, _P, _SZ, _P, _P]
            for n in ("csa2_kv_quant_append", "csa2_indexer_topk", "csa2_sparse_attn_decode",
                      "csa2_sparse_attn_prefill", "csa2_decode_layers"):
                getattr(L, n).restype = _I32
            L.csa2_indexer_topk_noalloc.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(_Cache), _I32, _P, _P,
                                                    _P, _P, _P, _I32, _I64, _P, _P]
            L.csa2_indexer_topk_noalloc.restype = _I32
            L.csa2_status_string.argtypes = [_I32]
            L.csa2_status_string.restype = ctypes.c_char_p
            L.csa2_abi_version.restype = _I32
            L.csa2_device_accessible.argtypes = [_P]
            L.csa2_device_accessible.restype = _I32
            L.csa2_indexer_score_ids.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(_Cache), _I32, _P, _P,
                                                 _P, _P, _I32, _I32, _P, _P, _I32, _I64, _P, _P]
            L.csa2_topk_merge.argtypes = [_P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _I32, _P]
            L.csa2_attn_lse_merge.argtypes = [_I32, _P, _P, _P, _P, _I32, _P]
            for n in ("csa2_indexer_score_ids", "csa2_topk_merge", "csa2_attn_lse_merge"):
                getattr(L, n).restype = _I32
            L.csa2_dense_attn_workspace_bytes.argtypes = [ctypes.POINTER(LayerDesc), _I32, _I32]
            L.csa2_dense_attn_workspace_bytes.restype = _SZ
            L.csa2_dense_attn_decode.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(_Cache), _P, _P, _P, _I32,
                                                 _P, _I32, _I64, _P, _SZ, _P, _P]
            L.csa2_dense_attn_prefill.argtypes = [ctypes.POINTER(LayerDesc), ctypes.POINTER(_Cache), _P, _P, _P, _P,
                                                  _P, _I32, _P, _I32, _I32, _I64, _P, _SZ, _P, _P]
            for n in ("csa2_dense_attn_decode", "csa2_dense_attn_prefill"):
                getattr(L, n).restype = _I32
            caches, i32p = ctypes.POINTER(_Cache), _P
            L.csa2_kv_pages_workspace_bytes.argtypes = [_I64, _I32]
            L.csa2_kv_pages_workspace_bytes.restype = _SZ
            L.csa2_kv_pages_copy.argtypes = [_I32, caches, i32p, i32p, _I32, i32p, _P]
            L.csa2_kv_pages_fork.argtypes = [_I32, caches, i32p, _I32, i32p, i32p, i32p, i32p, _I32, _P, _SZ, i32p, _P]
            L.csa2_kv_pages_free.argtypes = [caches, i32p, _I32, i32p, i32p, i32p, _I32, i32p, _P]
            L.csa2_kv_pages_compact.argtypes = [_I32, caches, i32p, _I32, i32p, i32p, i32p, _P, _SZ, i32p, _P]
            for n in ("csa2_kv_pages_copy", "csa2_kv_pages_fork", "csa2_kv_pages_free", "csa2_kv_pages_compact"):
                getattr(L, n).restype = _I32
            L.csa2_swa_replay.argtypes = [_P, _P, _P, _P, _I32, _I32, _I32, _P, _P]
            L.csa2_swa_replay.restype = _I32
            L.csa2_test_empty_chain.argtypes = [_I32, _I32, _I32, _P, _P]
            L.csa2_test_empty_chain.restype = _I32
            L.csa2_test_set_wait_limit.argtypes = [ctypes.c_uint32]
            L.csa2_test_set_wait_limit.restype = ctypes.c_uint32
            _lib = L
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    """The raw handle of a stream; of the current device's current stream for None."""
    if stream is None:
        if not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(status: int, what: str) -> None:
    if status != 0:
        raise CSA2Error(status, what)


_BITS16 = (torch.bfloat16, torch.int16, torch.uint16)


def _tensor(name: str, t, dtypes, shape, optional: bool = False) -> None:
    """Raise unless t is a contiguous tensor of one of the dtypes and of that
    shape (None: any size).  What is on a GPU has to be on the current one."""
    if t is None and optional:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if len(t.shape) != len(shape) or any(w is not None and w != g for g, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous (strides {t.stride()})")
    if t.is_cuda and t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _on_gpu(name: str, t, dtypes, shape, dev: int, optional: bool = False) -> None:
    """_tensor, and on GPU `dev`: one quick look where all is well (a decode call
    makes half a dozen of these)."""
    if t is None and optional:
        return
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.get_device() == dev and t.is_contiguous() and \
            (t.shape == shape or (shape[-1] is None and t.dim() == len(shape))):
        return
    _tensor(name, t, dtypes, shape)
    raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")


def _readable(cache: KVCache):
    """The cache's struct, for a call whose kernels read its arrays: none of them may
    be in host memory that is not pinned (a handle made by from_tensors can be)."""
    if not cache._seen_readable:
        for name in ("page_table", "codes", "scales", "idx_k", "pooled"):
            t = getattr(cache, name)
            if t is not None and not t.is_cuda and not t.is_pinned():
                raise ValueError(f"cache: {name} on {t.device}, which kernels cannot read")
        cache._seen_readable = True
    return ctypes.byref(cache._s)


def abi_version() -> int:
    return int(lib().csa2_abi_version())


def device_accessible(t) -> int:
    """1 if kernels can read the tensor (or raw address) in place, 0 if not, -1 on a CUDA error."""
    return int(lib().csa2_device_accessible(_ptr(t)))


def indexer_score_ids(desc: LayerDesc, cache: KVCache, level: int, q_idx, w, seq_lens, ids, id_offset: int,
                      scores, ids_out, n: int, max_len: int, err=None, stream=None) -> None:
    """Scores of the given ids (exact chains) and the ids plus id_offset."""
    _check(lib().csa2_indexer_score_ids(ctypes.byref(desc), _readable(cache), level, _ptr(q_idx),
                                        _ptr(w), _ptr(seq_lens), _ptr(ids), ids.shape[-1], id_offset, _ptr(scores),
                                        _ptr(ids_out), n, max_len, _ptr(err), _stream(stream)), "indexer_score_ids")


def topk_merge(scores, ids, k: int, out, out_local=None, lo: int = 0, hi: int = 0, stream=None) -> None:
    """Top-k of gathered (score, id) pairs [parts, n, part_len]; ids ascending in pair order."""
    parts, n, plen = scores.shape
    _check(lib().csa2_topk_merge(_ptr(scores), _ptr(ids), parts, plen, k, lo, hi, _ptr(out), _ptr(out_local), n,
                                 _stream(stream)), "topk_merge")


def attn_lse_merge(out_parts, lse_parts, out, lse, stream=None) -> None:
    """Log-sum-exp merge of partial attention outputs [G, rows, 16, 128] / [G, rows, 16]."""
    _check(lib().csa2_attn_lse_merge(out_parts.shape[0], _ptr(out_parts), _ptr(lse_parts), _ptr(out), _ptr(lse),
                                     out_parts.shape[1], _stream(stream)), "attn_lse_merge")


def swa_replay(h, w_kv, seq_lens, swa_kv, B: int, window: int = 128, err=None, stream=None) -> None:
    """Recompute the window K|V rows of B sequences from their hidden states
    h [B, window, d_model] and the projection w_kv [256, d_model] (bf16 bits)."""
    _check(lib().csa2_swa_replay(_ptr(h), _ptr(w_kv), _ptr(seq_lens), _ptr(swa_kv), B, h.shape[-1], window,
                                 _ptr(err), _stream(stream)), "swa_replay")


def test_set_wait_limit(polls: int) -> int:
    """Test hook: poll limit of the waits of the block-level indexer's cp.async
    copy ring and of dense attention (returns the previous limit)."""
    return int(lib().csa2_test_set_wait_limit(polls))


def test_empty_chain(n_kernels: int, ctas: int, threads: int = 128, sink=None, stream=None) -> None:
    """Measurement helper: n_kernels empty dependent kernels (programmatic
    dependent launch) on the stream."""
    _check(lib().csa2_test_empty_chain(n_kernels, ctas, threads, _ptr(sink), _stream(stream)), "test_empty_chain")


def default_desc(mode: int = FULL, ratio: int = 1, **over) -> LayerDesc:
    d = LayerDesc()
    lib().csa2_layer_desc_default(ctypes.byref(d), mode, ratio)
    for k, v in over.items():
        setattr(d, k, v)
    return d


def schedule(decoder: bool = True) -> list[int]:
    buf = (ctypes.c_int32 * 20)()
    n = lib().csa2_schedule(1 if decoder else 0, ctypes.cast(buf, _P))
    return list(buf[:n])


class KVCache:
    """Paged FP4 main-KV cache + indexer K (+ pooled indexer K) in device memory.

    page_table: int32 [n_seqs, max_pages] (host or device tensor) mapping the
    entry pages of each sequence to physical pages (-1 = none).
    main_kv_on_host: keep codes and scales (the main KV) in pinned host memory
    that the device reads in place; the indexer K stays in device memory."""

    _seen_readable = False  # _readable found every array in place

    def __init__(self, n_phys_pages: int, page_size: int, page_table: torch.Tensor, device="cuda",
                 pooled: bool = True, main_kv_on_host: bool = False):
        n = n_phys_pages * page_size
        self.page_size, self.n_phys_pages = page_size, n_phys_pages
        if main_kv_on_host:
            self.codes = torch.zeros((n, 128), dtype=torch.uint8, pin_memory=True)
            self.scales = torch.zeros((n, 16), dtype=torch.uint8, pin_memory=True)
            for t in (self.codes, self.scales):
                if device_accessible(t) != 1:
                    raise RuntimeError("pinned host memory is not mapped into the device address space")
        else:
            self.codes = torch.zeros((n, 128), dtype=torch.uint8, device=device)
            self.scales = torch.zeros((n, 16), dtype=torch.uint8, device=device)
        self.idx_k = torch.zeros((n, 64), dtype=torch.int16, device=device)
        self.pooled = torch.zeros((n // 8, 64), dtype=torch.int16, device=device) if pooled else None
        self.page_table = page_table.to(device=device, dtype=torch.int32).contiguous()
        self._s = _Cache(self.codes.data_ptr(), self.scales.data_ptr(), self.idx_k.data_ptr(),
                         self.pooled.data_ptr() if pooled else None, self.page_table.data_ptr(), page_size,
                         self.page_table.shape[1], n_phys_pages)

    @classmethod
    def from_tensors(cls, codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor, page_size: int,
                     idx_k: torch.Tensor | None = None, pooled: torch.Tensor | None = None) -> "KVCache":
        """A handle on arrays the caller keeps (nothing is copied; the page table
        may be rewritten in place): codes [n_slots, 128] and scales [n_slots, 16]
        uint8, page_table int32 [n_seqs, max_pages], idx_k [n_slots, 64] and
        pooled [n_slots / 8, 64] 16-bit.  Without idx_k and pooled the handle
        serves the attention and page calls and appends without an indexer K.
        Arrays in host memory that is not pinned are refused by every call."""
        n = codes.shape[0]
        if page_size < 1 or n % page_size:
            raise ValueError(f"{n} slots are not whole pages of {page_size}")
        _tensor("codes", codes, (torch.uint8,), (n, 128))
        _tensor("scales", scales, (torch.uint8,), (n, 16))
        _tensor("page_table", page_table, (torch.int32,), (None, None))
        _tensor("idx_k", idx_k, _BITS16, (n, 64), optional=True)
        _tensor("pooled", pooled, _BITS16, (n // 8, 64), optional=True)
        v = cls.__new__(cls)
        v.page_size, v.n_phys_pages = page_size, n // page_size
        v.codes, v.scales, v.idx_k, v.pooled, v.page_table = codes, scales, idx_k, pooled, page_table
        v._s = _Cache(codes.data_ptr(), scales.data_ptr(), _ptr(idx_k), _ptr(pooled), page_table.data_ptr(),
                      page_size, page_table.shape[1], v.n_phys_pages)
        return v

    def struct(self) -> _Cache:
        return self._s

    def shard(self, page_lo: int, n_pages: int) -> "KVCache":
        """A view of pages [page_lo, page_lo + n_pages) of every sequence: the
        same cache arrays with that slice of the page table, so entry e of the
        view is entry page_lo * page_size + e of the sequence (a context-parallel
        shard)."""
        v = KVCache.__new__(KVCache)
        v.page_size, v.n_phys_pages = self.page_size, self.n_phys_pages
        v.codes, v.scales, v.idx_k, v.pooled = self.codes, self.scales, self.idx_k, self.pooled
        v.page_table = self.page_table[:, page_lo:page_lo + n_pages].contiguous()
        v._s = _Cache(self._s.codes, self._s.scales, self._s.idx_k, self._s.idx_k_pooled, v.page_table.data_ptr(),
                      self.page_size, v.page_table.shape[1], self.n_phys_pages)
        return v


def kv_quant_append(cache: KVCache, kv_src: torch.Tensor, idx_k_src, slot_mapping: torch.Tensor, ratio: int = 1,
                    err=None, stream=None) -> None:
    dt = BF16 if kv_src.dtype == torch.bfloat16 else F32
    n = slot_mapping.numel()
    _check(lib().csa2_kv_quant_append(_readable(cache), _ptr(kv_src), dt, _ptr(idx_k_src), n, ratio,
                                      _ptr(slot_mapping), _ptr(err), _stream(stream)), "kv_quant_append")


def workspace_bytes(desc: LayerDesc, level: int, n: int, max_len: int, prefill: bool = False) -> int:
    return int(lib().csa2_indexer_workspace_bytes(ctypes.byref(desc), level, n, max_len, 1 if prefill else 0))


def indexer_topk(desc: LayerDesc, cache: KVCache, level: int, q_idx, w, seq_lens, out, n: int, max_len: int,
                 workspace: torch.Tensor, q_pos=None, cand_blocks=None, err=None, stream=None) -> None:
    _check(lib().csa2_indexer_topk(ctypes.byref(desc), _readable(cache), level, _ptr(q_idx), _ptr(w),
                                   _ptr(seq_lens), _ptr(q_pos), _ptr(cand_blocks), _ptr(out), None, n, max_len,
                                   _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err),
                                   _stream(stream)), "indexer_topk")


def sparse_attn_decode(desc: LayerDesc, cache: KVCache, q, topk_idx, swa_kv, seq_lens, out, lse, B: int,
                       swa_lens=None, err=None, stream=None) -> None:
    _check(lib().csa2_sparse_attn_decode(ctypes.byref(desc), _readable(cache), _ptr(q), _ptr(topk_idx),
                                         _ptr(swa_kv), _ptr(seq_lens), _ptr(swa_lens), _ptr(out), _ptr(lse), B,
                                         _ptr(err), _stream(stream)), "sparse_attn_decode")


def sparse_attn_prefill(desc: LayerDesc, cache: KVCache, q, topk_idx, q_pos, swa_kv, swa_start: int, seq_len: int,
                        out, lse, T: int, err=None, stream=None) -> None:
    _check(lib().csa2_sparse_attn_prefill(ctypes.byref(desc), _readable(cache), _ptr(q), _ptr(topk_idx),
                                          _ptr(q_pos), _ptr(swa_kv), swa_start, seq_len, _ptr(out), _ptr(lse), T,
                                          _ptr(err), _stream(stream)), "sparse_attn_prefill")


_OUT = {torch.float32: F32, torch.bfloat16: BF16}


def dense_attn_workspace_bytes(desc: LayerDesc, B: int, prefill: bool = False) -> int:
    return int(lib().csa2_dense_attn_workspace_bytes(ctypes.byref(desc), B, 1 if prefill else 0))


_I32T, _U8T, _F32T, _OUTT = (torch.int32,), (torch.uint8,), (torch.float32,), (torch.float32, torch.bfloat16)


def _device(t) -> int:
    """The current GPU, where the call's tensors have to be (t decides nothing: it
    only keeps a CPU tensor from initialising CUDA)."""
    if isinstance(t, torch.Tensor) and not t.is_cuda:
        raise ValueError(f"a tensor on {t.device}, expected the GPU")
    return torch.cuda.current_device()


def _cache_on(cache: KVCache, dev: int) -> None:
    """The page table is on GPU `dev` and the main KV on no other GPU (the library
    refuses one in host memory)."""
    for name, t in (("page_table", cache.page_table), ("codes", cache.codes), ("scales", cache.scales)):
        at = t.get_device()
        if at != dev and (at >= 0 or t is cache.page_table):
            raise ValueError(f"cache: {name} on {t.device}, expected cuda:{dev}")


def _dense_checks(cache: KVCache, q, seq_lens, out, lse, workspace, err, B: int) -> tuple[int, int]:
    dev, T = _device(q), q.shape[0]
    _on_gpu("q", q, _BITS16, (T, 16, 128), dev)
    _on_gpu("seq_lens", seq_lens, _I32T, (B,), dev)
    _on_gpu("out", out, _OUTT, (T, 16, 128), dev)
    _on_gpu("lse", lse, _F32T, (T, 16), dev)
    _on_gpu("workspace", workspace, _U8T, (None,), dev)
    _on_gpu("err", err, _I32T, (1,), dev, optional=True)
    if cache.page_table.shape[0] < B:
        raise ValueError(f"seq_lens: {B} sequences, the page table has {cache.page_table.shape[0]}")
    _cache_on(cache, dev)
    return _OUT[out.dtype], dev


def dense_attn_decode(desc: LayerDesc, cache: KVCache, q, seq_lens, out, lse, max_len: int, workspace: torch.Tensor,
                      err=None, stream=None) -> None:
    """One token per sequence (q [B, 16, 128] bf16) over every entry of its
    sequence; out fp32 or bf16, lse fp32 [B, 16]."""
    B = seq_lens.numel()
    dt, _ = _dense_checks(cache, q, seq_lens, out, lse, workspace, err, B)
    if q.shape[0] != B:
        raise ValueError(f"q: {q.shape[0]} rows for {B} sequences")
    _check(lib().csa2_dense_attn_decode(ctypes.byref(desc), ctypes.byref(cache._s), q.data_ptr(), seq_lens.data_ptr(),
                                        out.data_ptr(), dt, lse.data_ptr(), B, max_len, workspace.data_ptr(),
                                        workspace.numel(), _ptr(err), _stream(stream)), "dense_attn_decode")


def dense_attn_prefill(desc: LayerDesc, cache: KVCache, q, cu_q, seq_lens, out, lse, max_len: int,
                       workspace: torch.Tensor, q_start=None, err=None, stream=None) -> None:
    """Chunks of tokens (sequence b: rows cu_q[b] .. cu_q[b+1]-1 of q [T, 16, 128])
    over their sequence's entries: causal from position q_start[b] on (desc.ratio
    tokens per entry), or over every entry without q_start."""
    B = seq_lens.numel()
    dt, dev = _dense_checks(cache, q, seq_lens, out, lse, workspace, err, B)
    _on_gpu("cu_q", cu_q, _I32T, (B + 1,), dev)
    _on_gpu("q_start", q_start, _I32T, (B,), dev, optional=True)
    _check(lib().csa2_dense_attn_prefill(ctypes.byref(desc), ctypes.byref(cache._s), q.data_ptr(), cu_q.data_ptr(),
                                         _ptr(q_start), seq_lens.data_ptr(), out.data_ptr(), dt, lse.data_ptr(), B,
                                         q.shape[0], max_len, workspace.data_ptr(), workspace.numel(), _ptr(err),
                                         _stream(stream)), "dense_attn_prefill")


def kv_pages_workspace_bytes(n_phys_pages: int, n: int = 0) -> int:
    """Workspace of n forks (or, with n = 0, of a compaction) over that many pages."""
    size = int(lib().csa2_kv_pages_workspace_bytes(n_phys_pages, n))
    if size == 0:
        raise ValueError(f"{n_phys_pages} pages and {n} forks: out of range")
    return size


def _mapped(caches, dev: int) -> None:
    """Every array of the caches is where kernels of GPU `dev` can write it."""
    for c in caches:
        for t in (c.codes, c.scales, c.idx_k, c.pooled):
            if t is not None and t.get_device() != dev and (t.is_cuda or not t.is_pinned()):
                raise ValueError(f"a cache's array is on {t.device}: neither on cuda:{dev} nor pinned")


def _page_args(caches, refs, seq_lens, err):
    """The caches as a C array, their common table and the device."""
    if not caches:
        raise ValueError("caches: empty")
    c0 = caches[0]
    table = c0.page_table
    dev = _device(table)
    _mapped(caches, dev)
    for c in caches[1:]:
        if c.page_table.data_ptr() != table.data_ptr() or c.page_table.shape != table.shape:
            raise ValueError("caches: they do not share one page table")
    _on_gpu("page_table", table, _I32T, tuple(table.shape), dev)
    _on_gpu("refs", refs, _I32T, (c0.n_phys_pages,), dev)
    _on_gpu("seq_lens", seq_lens, _I32T, (table.shape[0],), dev, optional=True)
    _on_gpu("err", err, _I32T, (1,), dev, optional=True)
    return ctypes.byref(c0._s) if len(caches) == 1 else (_Cache * len(caches))(*[c._s for c in caches]), table, dev


def kv_pages_copy(caches: list[KVCache], src, dst, err=None, stream=None) -> None:
    """Physical pages src[i] -> dst[i] in every cache (int32; a -1 skips the pair)."""
    if not caches:
        raise ValueError("caches: empty")
    dev = _device(src)
    _mapped(caches, dev)
    _on_gpu("src", src, _I32T, (None,), dev)
    _on_gpu("dst", dst, _I32T, (src.numel(),), dev)
    _on_gpu("err", err, _I32T, (1,), dev, optional=True)
    C = (_Cache * len(caches))(*[c._s for c in caches])
    _check(lib().csa2_kv_pages_copy(len(caches), C, _ptr(src), _ptr(dst), src.numel(), _ptr(err), _stream(stream)),
           "kv_pages_copy")


def kv_pages_fork(caches: list[KVCache], refs, seq_lens, parents, children, workspace: torch.Tensor, err=None,
                  stream=None) -> None:
    """Rows children[i] of the caches' page table share what rows parents[i] hold.
    Caches of one call share the table itself (build them on one CUDA tensor)."""
    C, table, dev = _page_args(caches, refs, seq_lens, err)
    _on_gpu("parents", parents, _I32T, (None,), dev)
    _on_gpu("children", children, _I32T, (parents.numel(),), dev)
    _on_gpu("workspace", workspace, _U8T, (None,), dev)
    _check(lib().csa2_kv_pages_fork(len(caches), C, _ptr(table), table.shape[0], _ptr(refs), _ptr(seq_lens),
                                    _ptr(parents), _ptr(children), parents.numel(), _ptr(workspace),
                                    workspace.numel(), _ptr(err), _stream(stream)), "kv_pages_fork")


def kv_pages_free(cache: KVCache, refs, seq_lens, seqs, err=None, stream=None) -> None:
    """Rows seqs[i] of the page table become free; their pages lose one holder each."""
    C, table, dev = _page_args([cache], refs, seq_lens, err)
    _on_gpu("seqs", seqs, _I32T, (None,), dev)
    _check(lib().csa2_kv_pages_free(C, _ptr(table), table.shape[0], _ptr(refs), _ptr(seq_lens), _ptr(seqs),
                                    seqs.numel(), _ptr(err), _stream(stream)), "kv_pages_free")


def kv_pages_compact(caches: list[KVCache], refs, page_map, n_live, workspace: torch.Tensor, err=None,
                     stream=None) -> None:
    """Live pages move into the free numbers below their count; the page table and
    refs follow, page_map [n_phys_pages] tells each page's new number (-1: free)
    and n_live [1] their count."""
    C, table, dev = _page_args(caches, refs, None, err)
    _on_gpu("page_map", page_map, _I32T, (caches[0].n_phys_pages,), dev)
    _on_gpu("n_live", n_live, _I32T, (1,), dev)
    _on_gpu("workspace", workspace, _U8T, (None,), dev)
    _check(lib().csa2_kv_pages_compact(len(caches), C, _ptr(table), table.shape[0], _ptr(refs), _ptr(page_map),
                                       _ptr(n_live), _ptr(workspace), workspace.numel(), _ptr(err), _stream(stream)),
           "kv_pages_compact")


def decode_layers(descs: list[LayerDesc], cache: KVCache, q_idx: list, w: list, q: list, swa_kv: list, seq_lens,
                  cand_blocks, idx_sets, out: list, lse: list, B: int, max_len: int, workspace: torch.Tensor,
                  swa_lens=None, err=None, stream=None) -> None:
    n = len(descs)
    D = (LayerDesc * n)(*descs)
    arr = lambda xs: (ctypes.c_void_p * n)(*[_ptr(x) for x in xs])  # noqa: E731
    keep = [arr(q_idx), arr(w), arr(q), arr(swa_kv), arr(out), arr(lse)]
    _check(lib().csa2_decode_layers(n, D, _readable(cache), ctypes.cast(keep[0], _P),
                                    ctypes.cast(keep[1], _P), ctypes.cast(keep[2], _P), ctypes.cast(keep[3], _P),
                                    _ptr(seq_lens), _ptr(swa_lens), _ptr(cand_blocks), _ptr(idx_sets),
                                    ctypes.cast(keep[4], _P), ctypes.cast(keep[5], _P), B, max_len,
                                    _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err),
                                    _stream(stream)), "decode_layers")


def indexer_topk_noalloc(desc: LayerDesc, cache: KVCache, level: int, q_idx, w, seq_lens, out, n: int, max_len: int,
                         cand_blocks=None, err=None, stream=None) -> None:
    """Decode indexer without a caller workspace (static 16 MiB library scratch);
    for callers that cannot allocate device memory at this point."""
    _check(lib().csa2_indexer_topk_noalloc(ctypes.byref(desc), _readable(cache), level, _ptr(q_idx),
                                           _ptr(w), _ptr(seq_lens), _ptr(cand_blocks), _ptr(out), n, max_len,
                                           _ptr(err), _stream(stream)), "indexer_topk_noalloc")
