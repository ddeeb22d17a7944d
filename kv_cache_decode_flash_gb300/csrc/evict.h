// evict.h - eviction of the rows of least accumulated attention weight (k_evict.cu).  Not part of the ABI.
#pragma once

#include "kvc_internal.h"

namespace kvc {

struct EvictArgs {
    int32_t n;            // rows of the sequence
    int32_t n_cand;       // candidates: rows first .. first + n_cand - 1, or rows[0 .. n_cand)
    int32_t first;
    const int32_t *rows;  // ascending; null: the contiguous range
    int32_t n_remove;     // 1 .. n_cand
    float *w;             // [Hk][w_stride]
    int64_t w_stride;
    uint32_t *keys;       // work: [n_cand]
    int32_t *gone;        // out: the removed rows, ascending [n_remove]
    int4 *pairs;          // work: hole's and mover's pool rows of KV head 0, layer 0, the hole; [n_remove], -1 where none
    // the pools
    const int32_t *pt;    // the sequence's page table
    int32_t pt_len, n_pages, off, P, Hk, L;
    uint8_t *base[4];     // K codes, V codes, K scales, V scales (null: absent)
    int32_t rowb[4];
    int64_t pool_rows;
    uint32_t *err;        // set: nothing is changed
};
cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st);

} // namespace kvc
