// Dense attention over the whole FP4 main KV: the C ABI of decode
// (dense_decode.cu) and prefill (dense_prefill.cu).
#include "checks.h"
#include "common.cuh"
#include "kernels.h"

using namespace csa2;

namespace {

constexpr int kMaxDenseSeqs = 65536;
constexpr int kMaxDenseRows = 1 << 26;

// The host's checks of both calls; fills what they share.
csa2_status dense_args(const csa2_layer_desc* desc, const csa2_kv_cache* cache, const uint16_t* q,
                       const int32_t* seq_lens, void* out, int32_t out_dtype, float* lse, int32_t B, int32_t rows,
                       int64_t max_len, void* ws, size_t ws_bytes, int32_t prefill, int32_t* err, DenseArgs& a) {
    csa2_status s = check_desc(desc);
    if (s != CSA2_OK) return s;
    s = check_cache(cache, false, false);
    if (s != CSA2_OK) return s;
    if (out_dtype != CSA2_SRC_F32 && out_dtype != CSA2_SRC_BF16) return CSA2_ERR_INVALID_ARG;
    if (B < 0 || rows < 0) return CSA2_ERR_INVALID_ARG;
    if (B == 0 || rows == 0) return CSA2_OK;
    if (!q || !seq_lens || !out || !lse || max_len < 1) return CSA2_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) || !aligned(lse, 4) || (err && !aligned(err, 4)))
        return CSA2_ERR_INVALID_ARG;
    if (max_len > (int64_t)cache->max_pages_per_seq * cache->page_size) return CSA2_ERR_INVALID_ARG;
    if (B > kMaxDenseSeqs || rows > kMaxDenseRows || max_len > INT32_MAX - 65536 ||
        cache->n_phys_pages * cache->page_size > INT32_MAX || B * ((max_len + 63) / 64 + 16) > INT32_MAX)
        return CSA2_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256) || ws_bytes < csa2_dense_attn_workspace_bytes(desc, B, prefill))
        return CSA2_ERR_WORKSPACE;
    {
        // a CTA stores rows while another may still read its queries or store its own
        const uintptr_t at[3] = {(uintptr_t)q, (uintptr_t)out, (uintptr_t)lse};
        const uint64_t n = (uint64_t)rows * kH, size[3] = {n * kD * 2, n * kD * (out_dtype == CSA2_SRC_F32 ? 4 : 2), n * 4};
        for (int i = 0; i < 3; ++i)
            for (int j = 0; j < i; ++j)
                if (at[i] < at[j] + size[j] && at[j] < at[i] + size[i]) return CSA2_ERR_INVALID_ARG;
    }
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return from_cuda(e);
    for (const void* p : {(const void*)cache->codes, (const void*)cache->scales}) {
        cudaPointerAttributes at{};
        if (cudaPointerGetAttributes(&at, p) != cudaSuccess) return from_cuda(cudaErrorInvalidValue);
        if (at.type == cudaMemoryTypeHost || at.type == cudaMemoryTypeUnregistered) return CSA2_ERR_UNSUPPORTED;
        if (at.type == cudaMemoryTypeDevice && at.device != dev) return CSA2_ERR_INVALID_ARG;
    }
    a.cache = *cache;
    a.q = q;
    a.seq_lens = seq_lens;
    a.out = out;
    a.lse = lse;
    a.err = err;
    a.B = B;
    a.T = rows;
    a.max_len = (int32_t)max_len;
    a.ratio = desc->ratio;
    a.page_shift = page_shift_of(*cache);
    a.out_bf16 = out_dtype == CSA2_SRC_BF16;
    a.wait_limit = test_wait_limit();
    return CSA2_OK;
}

}  // namespace

extern "C" {

size_t csa2_dense_attn_workspace_bytes(const csa2_layer_desc* desc, int32_t B, int32_t prefill) {
    if (!desc || B < 0) return 0;
    return ((prefill ? dense_prefill_ws_bytes() : dense_decode_ws_bytes()) + 255) & ~size_t(255);
}

csa2_status csa2_dense_attn_decode(const csa2_layer_desc* desc, const csa2_kv_cache* cache, const uint16_t* q,
                                   const int32_t* seq_lens, void* out, int32_t out_dtype, float* lse, int32_t B,
                                   int64_t max_len, void* workspace, size_t ws_bytes, int32_t* err_word,
                                   void* stream) {
    DenseArgs a{};
    csa2_status s = dense_args(desc, cache, q, seq_lens, out, out_dtype, lse, B, B, max_len, workspace, ws_bytes, 0,
                               err_word, a);
    if (s != CSA2_OK || B == 0) return s;
    return from_cuda(launch_dense_decode(a, static_cast<char*>(workspace), (cudaStream_t)stream));
}

csa2_status csa2_dense_attn_prefill(const csa2_layer_desc* desc, const csa2_kv_cache* cache, const uint16_t* q,
                                    const int32_t* cu_q, const int32_t* q_start, const int32_t* seq_lens, void* out,
                                    int32_t out_dtype, float* lse, int32_t B, int32_t T, int64_t max_len,
                                    void* workspace, size_t ws_bytes, int32_t* err_word, void* stream) {
    DenseArgs a{};
    if (B > 0 && T > 0 && (!cu_q || !aligned(cu_q, 4) || (q_start && !aligned(q_start, 4))))
        return CSA2_ERR_INVALID_ARG;
    csa2_status s = dense_args(desc, cache, q, seq_lens, out, out_dtype, lse, B, T, max_len, workspace, ws_bytes, 1,
                               err_word, a);
    if (s != CSA2_OK || B == 0 || T == 0) return s;
    a.cu_q = cu_q;
    a.q_start = q_start;
    if (((int64_t)T / 16 + B) * ((max_len + 127) / 128 + 8) > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
    return from_cuda(launch_dense_prefill(a, static_cast<char*>(workspace), (cudaStream_t)stream));
}

}  // extern "C"
