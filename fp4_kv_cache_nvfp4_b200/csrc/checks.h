// Host-side argument checks shared by the C-ABI entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/csa2.h"
#include "common.cuh"

namespace csa2 {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline csa2_status check_desc(const csa2_layer_desc* d) {
    if (!d) return CSA2_ERR_INVALID_ARG;
    if (d->n_heads != 16 || d->head_dim != 128 || d->idx_heads != 4 || d->idx_dim != 64 || d->block != 8)
        return CSA2_ERR_UNSUPPORTED;
    if (d->ratio != 1 && d->ratio != 2) return CSA2_ERR_INVALID_ARG;
    if (d->topk < 1 || d->topk > kMaxTopk) return CSA2_ERR_INVALID_ARG;
    if (d->keep_blocks < 0 || d->keep_blocks > kMaxKeep) return CSA2_ERR_INVALID_ARG;  // 0: flat indexer
    if (d->window < 1 || d->window > kMaxWindow) return CSA2_ERR_INVALID_ARG;
    if (d->mode < CSA2_MODE_FULL || d->mode > CSA2_MODE_REUSE) return CSA2_ERR_INVALID_ARG;
    return CSA2_OK;
}

inline csa2_status check_cache(const csa2_kv_cache* c, bool need_idx, bool need_pooled) {
    if (!c || !c->codes || !c->scales || !c->page_table) return CSA2_ERR_INVALID_ARG;
    if (!aligned(c->codes, 16) || !aligned(c->scales, 16) || !aligned(c->page_table, 4)) return CSA2_ERR_INVALID_ARG;
    if (c->page_size < 8 || (c->page_size & (c->page_size - 1)) != 0 || c->page_size > (1 << 20) ||
        c->max_pages_per_seq < 1 || c->n_phys_pages < 1)
        return CSA2_ERR_INVALID_ARG;
    if ((int64_t)c->max_pages_per_seq * c->page_size > (int64_t(1) << 31)) return CSA2_ERR_INVALID_ARG;
    if (c->n_phys_pages > (int64_t(1) << 40) / c->page_size) return CSA2_ERR_INVALID_ARG;
    if (need_idx && (!c->idx_k || !aligned(c->idx_k, 16))) return CSA2_ERR_INVALID_ARG;
    if (need_pooled && (!c->idx_k_pooled || !aligned(c->idx_k_pooled, 16))) return CSA2_ERR_INVALID_ARG;
    if (c->idx_k_pooled && !aligned(c->idx_k_pooled, 16)) return CSA2_ERR_INVALID_ARG;
    return CSA2_OK;
}

inline csa2_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return CSA2_OK;
    (void)cudaGetLastError();
    return CSA2_ERR_CUDA;
}

}  // namespace csa2
