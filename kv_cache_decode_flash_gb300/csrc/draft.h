// draft.h - kernels around the attention over a drafted block: the append of
// rows as a model's projections leave them (kvc_append_rope) and the rows that
// stay of a block (kvc_seq_keep).  Not part of the ABI.
#pragma once

#include "kvc_internal.h"

namespace kvc {

// Consecutive tokens of one sequence of an append: token t of the piece becomes
// the sequence's row row0 + t.
struct RopePiece {
    int32_t id;    // row of the page table
    int32_t off;   // offset of logical row 0 in the first page
    int32_t row0;  // logical row of the first token
    int32_t first; // first token of the piece in the launch
    int32_t tok0;  // and in q, k, v and q_out
    int32_t pos;   // position of the first token, the others' follow it (listed < 0)
    int32_t listed; // place of the tokens' positions in RopeArgs.pos, or -1
};
constexpr int ROPE_PIECES = 64, ROPE_LISTED = 320; // of one launch

struct RopeArgs {
    const void *q, *k, *v; // q may be null, and q_out with it
    int64_t q_stride, k_stride, v_stride; // elements from token to token
    const float *q_norm, *k_norm; // [D] or null
    void *q_out;
    float eps;
    int32_t H, Hk, P, type_k, type_v;
    int32_t neox;
    int32_t n_pieces, n_tok, passes, warps; // passes over a token's head-rows, and warps that share them
    int32_t max_pages, n_pages;
    const int32_t *pt;
    LayerView lv;
    uint32_t *err;
    uint64_t turn[64]; // base^(-2i/D) / (2 pi), the fraction of a turn, in units of 2^-64
    RopePiece piece[ROPE_PIECES];
    int32_t pos[ROPE_LISTED];
};
static_assert(sizeof(RopeArgs) <= 4000, "launch parameters stay within 4 KB");

cudaError_t launch_rope_append(int D, int act, const RopeArgs &a, cudaStream_t st);
// Head-rows that a warp takes at a time.
constexpr int rope_rows(int D) { return 256 / D; }

// RopeArgs.turn of a rotary base.
void rope_turns(float base, int D, uint64_t *turn);

// Rows that move: (from, to), layer-0 pool rows of KV head 0 in the order in which a sequence's are to be moved.
constexpr int KEEP_ENTRIES = 64, KEEP_MOVES = 384;
struct KeepArgs {
    uint8_t *base[4];  // K codes, V codes, K scales, V scales (null: absent)
    int32_t rowb[4];   // bytes per row of each
    int64_t pool_rows; // rows of one layer pool
    int32_t L, Hk, P;
    int32_t n_entries;
    int32_t first[KEEP_ENTRIES + 1]; // an entry's (sequence's) moves
    int2 move[KEEP_MOVES];
};
static_assert(sizeof(KeepArgs) <= 4000, "launch parameters stay within 4 KB");
cudaError_t launch_keep(const KeepArgs &a, cudaStream_t st);

} // namespace kvc
