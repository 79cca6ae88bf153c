// Dense attention over the whole FP4 main KV: decode (one token per sequence)
// and prefill (ragged chunks, causal or over every entry).
#include "checks.h"
#include "common.cuh"
#include "kernels.h"

namespace csa2 {

constexpr int DS_KEYS = 32;          // entries per tile
constexpr int DS_THREADS = kH * 32;  // one warp per head
constexpr int DS_ROW = kCh + 1;      // floats per staged entry (odd: lanes read distinct banks)

// One CTA per query token, one warp per head.  A tile of 32 entries is
// dequantised to fp32 in shared memory; lane j scores entry j, the warp keeps
// the running maximum and sum, and each lane accumulates four output dims.
__global__ void __launch_bounds__(DS_THREADS) dense_attn_kernel(DenseArgs a) {
    __shared__ float kv[DS_KEYS * DS_ROW];
    __shared__ float qs[kH][kD];
    __shared__ int ok[DS_KEYS];
    __shared__ int nan_row[DS_KEYS];
    __shared__ int s_seq;
    const int tid = threadIdx.x, h = tid >> 5, lane = tid & 31, row = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    if (tid == 0) s_seq = a.cu_q ? -1 : row;
    __syncthreads();
    if (a.cu_q)
        for (int b = tid; b < a.B; b += DS_THREADS) {
            const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
            if (lo < 0 || hi < lo || hi > a.T) {
                if (row == 0) dev_error(a.err, CSA2_DEV_LEN);
            } else if (row >= lo && row < hi) {
                s_seq = b;
            }
        }
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    int64_t n = a.seq_lens[b];
    if (n < 0 || n > a.max_len) {
        if (tid == 0) dev_error(a.err, CSA2_DEV_LEN);
        n = 0;
    }
    if (a.q_start) {
        const int64_t p0 = a.q_start[b];
        if (p0 < 0) {
            if (tid == 0) dev_error(a.err, CSA2_DEV_LEN);
            n = 0;
        }
        n = min(n, (p0 + row - a.cu_q[b] + 1) / a.ratio);
    }
    for (int i = tid; i < kH * kD; i += DS_THREADS)
        qs[i / kD][i % kD] = bf16_bits_to_f32(a.q[(int64_t)row * kH * kD + i]);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t j0 = 0; j0 < n; j0 += DS_KEYS) {
        __syncthreads();
        if (tid < DS_KEYS) {
            const int64_t slot = j0 + tid < n ? entry_slot(a.cache, a.page_shift, b, (int)(j0 + tid), a.err) : -1;
            ok[tid] = slot >= 0;
            int bad = 0;
            if (slot >= 0)
                for (int i = 0; i < kScales; ++i) bad |= (a.cache.scales[slot * kScales + i] & 0x7f) == 0x7f;
            nan_row[tid] = bad;
        }
        __syncthreads();
        for (int i = tid; i < DS_KEYS * kCodeBytes / 4; i += DS_THREADS) {
            const int k = i / (kCodeBytes / 4), c = i % (kCodeBytes / 4);  // word c: channels 8c .. 8c + 7
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (ok[k]) {
                const int64_t slot = entry_slot(a.cache, a.page_shift, b, (int)(j0 + k), nullptr);
                const float s = e4m3_to_f32(a.cache.scales[slot * kScales + c / 2]);
                uint32_t h[4];
                e2m1x8_to_h2x4(reinterpret_cast<const uint32_t*>(a.cache.codes + slot * kCodeBytes)[c], h[0], h[1], h[2],
                               h[3]);
                for (int e = 0; e < 8; ++e) {
                    __half_raw r;
                    r.x = (unsigned short)(h[e >> 1] >> (16 * (e & 1)));
                    x[e] = __half2float(__half(r)) * s;
                }
            }
            for (int e = 0; e < 8; ++e) kv[k * DS_ROW + 8 * c + e] = x[e];
        }
        __syncthreads();
        float s = 0.f;
        for (int d = 0; d < kD; ++d) s += qs[h][d] * kv[lane * DS_ROW + d];
        s = ok[lane] ? (nan_row[lane] ? NAN : s * 0.08838834764831845f) : -INFINITY;
        float tm = s;
        for (int w = 16; w > 0; w >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, w));
        const float mn = fmaxf(m, tm), base = mn == -INFINITY ? 0.f : mn;
        const float f = m == -INFINITY ? 0.f : expf(m - base);
        const float p = expf(s - base);
        float ps = p;
        for (int w = 16; w > 0; w >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, w);
        l = l * f + ps;
        for (int i = 0; i < 4; ++i) o[i] *= f;
        for (int k = 0; k < DS_KEYS; ++k) {
            const float pk = __shfl_sync(0xffffffffu, p, k);
            for (int i = 0; i < 4; ++i) o[i] += pk * kv[k * DS_ROW + kD + lane + 32 * i];
        }
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = ((int64_t)row * kH + h) * kD;
    for (int i = 0; i < 4; ++i) {
        if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at + lane + 32 * i] = __float2bfloat16_rn(o[i] * inv);
        else static_cast<float*>(a.out)[at + lane + 32 * i] = o[i] * inv;
    }
    if (lane == 0) a.lse[(int64_t)row * kH + h] = l == 0.f ? -INFINITY : m + logf(l);
}

cudaError_t launch_dense_attn(const DenseArgs& a, char*, cudaStream_t stream) {
    LaunchCfg c(dim3((unsigned)(a.cu_q ? a.T : a.B)), dim3(DS_THREADS), 0, stream);
    return cudaLaunchKernelEx(&c.cfg, dense_attn_kernel, a);
}

}  // namespace csa2

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
        cache->n_phys_pages * cache->page_size > INT32_MAX || B * ((max_len + 63) / 64) > INT32_MAX)
        return CSA2_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256) || ws_bytes < csa2_dense_attn_workspace_bytes(desc, B, prefill))
        return CSA2_ERR_WORKSPACE;
    for (const void* p : {(const void*)cache->codes, (const void*)cache->scales}) {
        cudaPointerAttributes at{};
        if (cudaPointerGetAttributes(&at, p) != cudaSuccess) return from_cuda(cudaErrorInvalidValue);
        if (at.type == cudaMemoryTypeHost || at.type == cudaMemoryTypeUnregistered) return CSA2_ERR_UNSUPPORTED;
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
    return CSA2_OK;
}

}  // namespace

extern "C" {

size_t csa2_dense_attn_workspace_bytes(const csa2_layer_desc* desc, int32_t B, int32_t prefill) {
    if (!desc || B < 0) return 0;
    return prefill ? 256 : (dense_decode_ws_bytes() + 255) & ~size_t(255);
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
    return from_cuda(launch_dense_attn(a, static_cast<char*>(workspace), (cudaStream_t)stream));
}

}  // extern "C"
