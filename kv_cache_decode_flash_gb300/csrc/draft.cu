// draft.cu - host side of the calls around the attention over a drafted block:
// kvc_append_rope (rows as a model's projections leave them, normalised and
// turned on the way into the cache) and kvc_seq_keep (the block's rows that stay).
#include "draft.h"
#include "ctx.h"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

namespace kvc {

#define KVC_CU(c, call)                                                                                            \
    do {                                                                                                           \
        cudaError_t e_ = (call);                                                                                   \
        if (e_ != cudaSuccess) return cuda_fail((c), e_, #call);                                                   \
    } while (0)

// theta_i = base^(-2i/D), as kvc_seq_add has it: the double nearest to it, an integer of 53 bits times a power of two.
// That integer times 1 / 2 pi in 128 bits is an integer product: the same on every machine, good to 2^-64 of a turn
// whatever the position.
void rope_turns(float base, int D, uint64_t *turn) {
    const uint64_t inv_hi = 0x28BE60DB9391054Aull, inv_lo = 0x7F09D5F47D4D3770ull; // 2^128 / 2 pi
    for (int i = 0; i < D / 2; ++i) {
        int k;
        const double f = std::frexp(std::pow((double)base, -2.0 * i / (double)D), &k);
        const uint64_t m = (uint64_t)std::ldexp(f, 53);
        const unsigned __int128 q = (unsigned __int128)m * inv_hi + (((unsigned __int128)m * inv_lo) >> 64);
        const int down = 53 - k; // theta <= 1: k <= 1
        turn[i] = down >= 128 ? 0 : (uint64_t)((q + ((unsigned __int128)1 << (down - 1))) >> down);
    }
}

static bool overlaps(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

// Distinct ids in range: the first fault's message, or null.
static const char *check_ids(const Ctx *c, int n_seq, const int32_t *ids) {
    std::vector<char> seen(c->seqs.size(), 0);
    for (int i = 0; i < n_seq; ++i) {
        if (ids[i] < 0 || ids[i] >= (int)c->seqs.size()) return "sequence id out of range";
        if (seen[(size_t)ids[i]]) return "duplicate sequence id";
        seen[(size_t)ids[i]] = 1;
    }
    return nullptr;
}

// What the launches of an append read, as the call has it.
struct RopeCall {
    int n_seq;
    const int32_t *ids, *n_tok, *pos;
    int act;
};

static void make_room(std::vector<int32_t> &v, size_t n) {
    if (v.capacity() < n) v.reserve(std::max(n, 2 * v.capacity()));
}

static bool run_of(const int32_t *pos, int n) {
    for (int i = 1; i < n; ++i)
        if (pos[i] != (int64_t)pos[0] + i) return false;
    return true;
}

static int append_rope(Ctx *c, int layer, const RopeCall &call, RopeArgs &a, cudaStream_t st) {
    const int n_seq = call.n_seq, el = call.act == KVC_ACT_F32 ? 4 : 2;
    const int32_t *ids = call.ids, *n_tok = call.n_tok, *pos = call.pos;
    if (c->host) return c->fail(KVC_EINVAL, "this append needs a device-resident context");
    if (layer < 0 || layer >= c->L) return c->fail(KVC_EINVAL, "layer out of range");
    if (n_seq < 1 || !ids || !n_tok) return c->fail(KVC_EINVAL, "n_seq >= 1, seq_ids and n_tok required");
    if (call.act != KVC_ACT_F32 && call.act != KVC_ACT_F16 && call.act != KVC_ACT_BF16)
        return c->fail(KVC_EINVAL, "act must be KVC_ACT_F32, KVC_ACT_F16 or KVC_ACT_BF16");
    if (const char *why = check_ids(c, n_seq, ids)) return c->fail(KVC_EINVAL, why);
    int64_t total = 0;
    for (int i = 0; i < n_seq; ++i) {
        if (n_tok[i] < 0) return c->fail(KVC_EINVAL, "n_tok must not be negative");
        total += n_tok[i];
    }
    if (total > INT32_MAX / 64 / (c->H + 2 * c->Hk)) return c->fail(KVC_EINVAL, "too many tokens in one block");
    if (total == 0) return KVC_OK;
    if (!pos || !a.k || !a.v) return c->fail(KVC_EINVAL, "pos, k and v must be non-null");
    if (!a.q != !a.q_out) return c->fail(KVC_EINVAL, "q and q_out come together");
    if (((uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q_out | (uintptr_t)a.q_norm | (uintptr_t)a.k_norm) & 15)
        return c->fail(KVC_EINVAL, "device pointers must be 16-byte aligned");
    const int64_t least[3] = {(int64_t)c->H * c->D, (int64_t)c->Hk * c->D, (int64_t)c->Hk * c->D};
    const int64_t stride[3] = {a.q ? a.q_stride : least[0], a.k_stride, a.v_stride};
    for (int i = 0; i < 3; ++i) {
        if (stride[i] < least[i] || stride[i] > INT32_MAX) return c->fail(KVC_EINVAL, "a stride is below a token's head-rows");
        if (stride[i] * el % 16) return c->fail(KVC_EINVAL, "strides must be multiples of 16 bytes");
    }
    if ((a.q_norm || a.k_norm) && !(std::isfinite(a.eps) && a.eps >= 0.f))
        return c->fail(KVC_EINVAL, "eps must be finite and not negative");
    if (a.q_out) {
        const int64_t out_bytes = total * least[0] * el;
        auto span = [&](int i) { return ((total - 1) * stride[i] + least[i]) * el; };
        // (in place: a warp has read its head-rows before it writes them)
        if (!(a.q_out == a.q && stride[0] == least[0]) && overlaps(a.q_out, out_bytes, a.q, span(0)))
            return c->fail(KVC_EINVAL, "q_out may overlap q only where both are the same rows");
        if (overlaps(a.q_out, out_bytes, a.k, span(1)) || overlaps(a.q_out, out_bytes, a.v, span(2)))
            return c->fail(KVC_EINVAL, "q_out may not overlap k or v");
    }
    // Positions, rows and pages: everything is checked before anything changes.
    std::vector<char> creates((size_t)n_seq, 0);
    int64_t new_pages = 0, t0 = 0;
    for (int i = 0; i < n_seq; t0 += n_tok[i++]) {
        const Seq &q = c->seqs[(size_t)ids[i]];
        for (int t = 0; t < n_tok[i]; ++t)
            if (pos[t0 + t] < 0) return c->fail(KVC_ERANGE, "positions out of range");
        if (n_tok[i] == 0) continue;
        const int32_t fill = q.lfill[(size_t)layer];
        creates[(size_t)i] = fill == q.n;
        if (!creates[(size_t)i]) {
            if ((int64_t)fill + n_tok[i] > q.n) return c->fail(KVC_EINVAL, "append runs past the rows other layers created");
            if (!std::equal(pos + t0, pos + t0 + n_tok[i], q.pos.begin() + fill))
                return c->fail(KVC_EINVAL, "append positions differ from the rows other layers created");
            continue;
        }
        if ((int64_t)q.n + n_tok[i] > INT32_MAX / 2) return c->fail(KVC_ENOSPC, "sequence would exceed the page table");
        const int32_t need = pages_for(c, q.off, (int64_t)q.n + n_tok[i]);
        if (need > c->max_pages) return c->fail(KVC_ENOSPC, "sequence would exceed the page table");
        new_pages += std::max<int64_t>(0, need - (int64_t)q.pages.size());
    }
    if (new_pages > (int64_t)c->free_pages.size()) return c->fail(KVC_ENOSPC, "no free pages");
    KVC_CU(c, cudaSetDevice(c->dev));
    // (host memory for all of it before the first change)
    std::vector<int32_t> written;
    written.reserve((size_t)n_seq);
    for (int i = 0; i < n_seq; ++i) {
        if (n_tok[i] > 0) written.push_back(ids[i]);
        if (!creates[(size_t)i]) continue;
        Seq &q = c->seqs[(size_t)ids[i]];
        const size_t pages = std::max(q.pages.size(), (size_t)pages_for(c, q.off, (int64_t)q.n + n_tok[i]));
        make_room(q.pos, (size_t)q.n + (size_t)n_tok[i]);
        make_room(q.pages, pages);
        make_room(q.dev_table, pages);
    }
    for (int i = 0; i < n_seq; ++i) {
        if (!creates[(size_t)i]) continue;
        size_t first_new;
        int rc = grow_pages(c, c->seqs[(size_t)ids[i]], n_tok[i], &first_new);
        if (rc) return rc; // (cannot happen: checked above)
    }
    if (int rc = send_pages(c, written.data(), (int)written.size(), st)) return rc;
    // The launches: pieces of consecutive positions need no list, the others' positions travel with them.
    if (!c->has_turns) rope_turns(c->prm.rope_base, c->D, c->rope_turn);
    c->has_turns = true;
    std::copy(c->rope_turn, c->rope_turn + c->D / 2, a.turn);
    const int rows = rope_rows(c->D);
    a.H = c->H;
    a.Hk = c->Hk;
    a.P = c->P;
    a.type_k = c->tk;
    a.type_v = c->tv;
    a.neox = c->prm.rope_mode == KVC_ROPE_NEOX;
    a.max_pages = c->max_pages;
    a.n_pages = c->n_pages;
    a.pt = c->pt_dev;
    a.err = c->err_dev;
    const int64_t lo = (int64_t)layer * c->pool_rows;
    a.lv.k.data = c->kdata + lo * c->krow;
    a.lv.k.scales = c->ksb ? reinterpret_cast<uint16_t *>(c->kscales + lo * c->ksb) : nullptr;
    a.lv.v.data = c->vdata + lo * c->vrow;
    a.lv.v.scales = c->vsb ? reinterpret_cast<uint16_t *>(c->vscales + lo * c->vsb) : nullptr;
    a.passes = (a.q ? (c->H + rows - 1) / rows : 0) + 2 * ((c->Hk + rows - 1) / rows);
    a.n_pieces = a.n_tok = 0;
    int listed = 0;
    auto flush = [&]() -> int {
        if (a.n_tok == 0) return KVC_OK;
        // Few tokens: a warp a pass, as latency is all there is.  Many: four warps a token, so that its angles serve
        // several passes and the warps still fill the machine.
        a.warps = (int)std::min<int64_t>(a.passes, std::max<int64_t>(4, (int64_t)c->sms * 48 / a.n_tok));
        cudaError_t e = launch_rope_append(c->D, call.act, a, st);
        a.n_pieces = a.n_tok = listed = 0;
        if (e == cudaSuccess) return KVC_OK;
        for (int32_t id : written) release_tail_pages(c, c->seqs[(size_t)id]);
        return cuda_fail(c, e, "append kernel");
    };
    t0 = 0;
    for (int i = 0; i < n_seq; t0 += n_tok[i++]) {
        const Seq &q = c->seqs[(size_t)ids[i]];
        const bool run = run_of(pos + t0, n_tok[i]);
        for (int t = 0; t < n_tok[i];) {
            if (a.n_pieces == ROPE_PIECES || (!run && listed == ROPE_LISTED))
                if (int rc = flush()) return rc;
            const int n = run ? n_tok[i] - t : std::min(n_tok[i] - t, ROPE_LISTED - listed);
            RopePiece &pc = a.piece[a.n_pieces++];
            pc.id = ids[i];
            pc.off = q.off;
            pc.row0 = q.lfill[(size_t)layer] + t;
            pc.first = a.n_tok;
            pc.tok0 = (int32_t)(t0 + t);
            pc.pos = pos[t0 + t];
            pc.listed = run ? -1 : listed;
            if (!run) {
                std::copy(pos + t0 + t, pos + t0 + t + n, a.pos + listed);
                listed += n;
            }
            a.n_tok += n;
            t += n;
        }
    }
    if (int rc = flush()) return rc;
    t0 = 0;
    for (int i = 0; i < n_seq; t0 += n_tok[i++]) {
        if (n_tok[i] == 0) continue;
        Seq &q = c->seqs[(size_t)ids[i]];
        if (creates[(size_t)i]) {
            q.linear = (q.pos.empty() || (q.linear && (int64_t)q.pos.back() + 1 == pos[t0])) && run_of(pos + t0, n_tok[i]);
            q.pos.insert(q.pos.end(), pos + t0, pos + t0 + n_tok[i]);
            q.n += n_tok[i];
        }
        q.lfill[(size_t)layer] += n_tok[i];
        c->appended(ids[i], layer, n_tok[i]);
    }
    return KVC_OK;
}

static int seq_keep(Ctx *c, int n_seq, const int32_t *ids, const int32_t *n_last, const int32_t *n_keep, const int32_t *keep,
                    cudaStream_t st) {
    if (c->host) return c->fail(KVC_EINVAL, "sequence operations need a device-resident context");
    if (n_seq < 1 || !ids || !n_last || !n_keep) return c->fail(KVC_EINVAL, "n_seq >= 1, seq_ids, n_last and n_keep required");
    if (const char *why = check_ids(c, n_seq, ids)) return c->fail(KVC_EINVAL, why);
    int64_t k0 = 0;
    for (int i = 0; i < n_seq; k0 += n_keep[i++]) {
        const Seq &q = c->seqs[(size_t)ids[i]];
        if (!q.synced()) return c->fail(KVC_EINVAL, "layers are not in sync (a step's appends are incomplete)");
        if (n_last[i] < 0 || n_last[i] > q.n) return c->fail(KVC_EINVAL, "n_last must be at most the sequence's rows");
        if (n_keep[i] < 0 || n_keep[i] > n_last[i]) return c->fail(KVC_EINVAL, "n_keep must be at most n_last");
        if (n_keep[i] > 0 && !keep) return c->fail(KVC_EINVAL, "keep must be non-null");
        for (int k = 0; k < n_keep[i]; ++k)
            if (keep[k0 + k] < (k ? keep[k0 + k - 1] + 1 : 0) || keep[k0 + k] >= n_last[i])
                return c->fail(KVC_EINVAL, "keep must be ascending places among the last rows");
    }
    KVC_CU(c, cudaSetDevice(c->dev));
    KeepArgs a;
    std::memset(&a, 0, sizeof(a));
    a.base[0] = c->kdata;
    a.base[1] = c->vdata;
    a.base[2] = c->ksb ? c->kscales : nullptr;
    a.base[3] = c->vsb ? c->vscales : nullptr;
    a.rowb[0] = c->krow;
    a.rowb[1] = c->vrow;
    a.rowb[2] = c->ksb;
    a.rowb[3] = c->vsb;
    a.pool_rows = c->pool_rows;
    a.L = c->L;
    a.Hk = c->Hk;
    a.P = c->P;
    int moves = 0;
    auto flush = [&]() -> int {
        if (a.n_entries == 0) return KVC_OK;
        cudaError_t e = launch_keep(a, st);
        a.n_entries = moves = 0;
        return e == cudaSuccess ? KVC_OK : cuda_fail(c, e, "keep kernel");
    };
    k0 = 0;
    for (int i = 0; i < n_seq; k0 += n_keep[i++]) {
        const Seq &q = c->seqs[(size_t)ids[i]];
        const int64_t base = (int64_t)q.n - n_last[i];
        int k = 0;
        while (k < n_keep[i] && keep[k0 + k] == k) ++k; // these stay where they are
        while (k < n_keep[i]) {
            // (a sequence's moves that do not fit go on in the next launch, behind this one)
            if (a.n_entries == KEEP_ENTRIES || moves == KEEP_MOVES)
                if (int rc = flush()) return rc;
            for (; k < n_keep[i] && moves < KEEP_MOVES; ++k) {
                int32_t page, cell;
                phys(c, q, base + keep[k0 + k], page, cell);
                a.move[moves].x = (int32_t)prow(c, page, 0, cell);
                phys(c, q, base + k, page, cell);
                a.move[moves++].y = (int32_t)prow(c, page, 0, cell);
            }
            a.first[++a.n_entries] = moves;
        }
    }
    if (int rc = flush()) return rc;
    k0 = 0;
    for (int i = 0; i < n_seq; k0 += n_keep[i++]) {
        Seq &q = c->seqs[(size_t)ids[i]];
        if (n_keep[i] == n_last[i]) continue;
        const size_t base = (size_t)(q.n - n_last[i]);
        for (int k = 0; k < n_keep[i]; ++k) q.pos[base + (size_t)k] = q.pos[base + (size_t)keep[k0 + k]];
        q.n = (int32_t)base + n_keep[i];
        q.pos.resize((size_t)q.n);
        if (!q.linear) q.linear = consecutive(q.pos.data(), q.n);
        else if (n_keep[i]) q.linear = consecutive(q.pos.data() + base, n_keep[i]) && (base == 0 || q.pos[base] == (int64_t)q.pos[base - 1] + 1);
        release_tail_pages(c, q);
        for (auto &f : q.lfill) f = q.n;
        // rows that moved were written by a kernel that the next one may overlap; those that left need no wait
        for (auto &r : c->recent[(size_t)ids[i]]) r = std::max(r - (n_last[i] - n_keep[i]), n_keep[i]);
    }
    return KVC_OK;
}

} // namespace kvc

using namespace kvc;

extern "C" int kvc_append_rope(kvc_ctx *cc, int layer, int n_seq, const int32_t *seq_ids, const int32_t *n_tok,
                               const int32_t *pos, int act, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                               const void *v, int64_t v_stride, const float *q_norm, const float *k_norm, float eps,
                               void *q_out, void *stream) {
    if (!cc) return KVC_EINVAL;
    Ctx *c = reinterpret_cast<Ctx *>(cc);
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.q_out = q_out;
    try { // (lists, made before anything changes)
        return append_rope(c, layer, RopeCall{n_seq, seq_ids, n_tok, pos, act}, a, reinterpret_cast<cudaStream_t>(stream));
    } catch (const std::bad_alloc &) {
        c->err.assign("no host memory"); // (fits a string's own room: no allocation)
        return KVC_ENOMEM;
    }
}

extern "C" int kvc_seq_keep(kvc_ctx *cc, int n_seq, const int32_t *seq_ids, const int32_t *n_last, const int32_t *n_keep,
                            const int32_t *keep, void *stream) {
    if (!cc) return KVC_EINVAL;
    Ctx *c = reinterpret_cast<Ctx *>(cc);
    try {
        return seq_keep(c, n_seq, seq_ids, n_last, n_keep, keep, reinterpret_cast<cudaStream_t>(stream));
    } catch (const std::bad_alloc &) {
        c->err.assign("no host memory");
        return KVC_ENOMEM;
    }
}

extern "C" int kvc_debug_rope_turns(float rope_base, int head_dim, uint64_t *turns) {
    if (!(rope_base > 1.0f) || !std::isfinite(rope_base) || (head_dim != 64 && head_dim != 128) || !turns) return KVC_EINVAL;
    rope_turns(rope_base, head_dim, turns);
    return KVC_OK;
}

