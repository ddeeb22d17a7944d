// k_cross_tc.cu - the block attention for 16-bit queries on the fifth
// generation's tensor cores (tcgen05): same items, masks and results as
// k_cross.cu, whose comment has the definition.
//
// One CTA per SM: two groups of four softmax warps (one thread owns a query row),
// four warps that bring the rows' K (eight for codes) and four that bring their V,
// and a group of four of which one thread issues the products.  Steps are 128 cached rows:
//   S = Q K^T    128 x 128 x D, both operands fp16 in shared memory, S in TMEM;
//   O += P V     P (fp16) written over S in TMEM, V from shared memory, O stays in TMEM.
// Two jobs are always in flight, so that one's softmax runs under the other's
// products.  A query tile of more than 128 rows is two halves that share every
// step (job 2s + h: step s, half h); a smaller one is one half whose even and odd
// steps run apart, with sums of their own that are joined at the end.
//
// What comes from the cache is turned into fp16 on the way to shared memory:
// halves as they are (cp.async), codes times their block's scale.  Of V those
// products are rounded once to 11 bits (a choice that fits results of 8 or 11
// bits; P is rounded to as many).  K they leave whole, as two fp16 parts that hold
// the 18 bits: scores make the log-sum-exp, a result of 32 bits, whose error from
// 11 bits of K was 2e-4 for tokens of few rows and 3e-3 for peaked softmaxes, and
// every row weight formed from it was off by as much.  Both parts are multiplied
// with Q into the same scores.  Scales may lie anywhere in fp16's range, their
// products need not: a step's K is scaled by a power of two that brings its largest
// scale to [2^7, 2^8), undone in the score's factor; V's exponent is that of the
// largest scale met so far, and O is rescaled when it grows.
// The softmax rescales O only when a row's maximum has grown by more than 2^8
// since the last time (the final quotient is the same), so O is hardly ever read
// back before the end.  P stands 2^7 above its value for that maximum: it is 2^15
// at most, inside fp16, and keeps its 11 bits down to weights of 2^-21 of the
// largest; below, it is off by 2^-32 of the largest at most, where a long row's
// many small weights beside a great one would otherwise vanish.  The sum is
// formed under the same factor, which lse and the parts' maxima take back.
// What bounds it: with many query rows the chain of a half's job, softmax and its
// products, against the other half's, whose products the one issuing thread takes
// in turn (2048 tokens of 40 heads over 16384 rows, causal: halves 606 us, 1.07
// PFLOP/s of seen pairs, 57 % of a plain matrix product's rate; codes, with three
// products a job, 789 us, 0.82 PFLOP/s).  With few, halves run at the memory's rate
// (131072 rows, 5 tokens: 90 us, 6.0 TB/s of 6.8), codes at that of their
// conversion (136 us, 2.1 TB/s), short ones at start, first tiles and join (16384
// rows, 5 tokens: 31 us, of which the seven steps are half).
#include "tc_tile.cuh"

namespace kvc {
namespace {

constexpr int TM = 128;      // query rows of a half
constexpr int TN = 128;      // cached rows of a step
// Roles by groups of four warps: softmax of half 0, of half 1, K, V, then the issuing thread's.  K's codes have two groups:
// one takes about 2200 cycles to form a tile, and there are two a step (5 tokens over 131072 rows: 199 us by one, 139 by two).
template <bool CODES> constexpr int K_GROUPS = CODES ? 2 : 1;
template <bool CODES> constexpr int THREADS = (4 + K_GROUPS<CODES>) * GROUP;
// Registers: a launch gives every thread LAUNCH.  The loading groups and the issuing thread's hand some back (those that turn
// codes into values need more), the softmax groups take them, so that a thread holds all or half of its row's 128 scores.  (No function of
// theirs may stay a call: its registers would have to fit the smallest role's.)  Few are to spare: shared memory leaves
// spilled ones next to no cache (V's codes by two groups as well, with 72 a thread at launch: 139 to 199 us).
template <bool CODES> struct Regs {
    static constexpr int LAUNCH = CODES ? 80 : 96;
    static constexpr int SOFT = CODES ? 136 : 184, K = CODES ? 56 : 40, V = CODES ? 72 : 40, MMA = 24;
    static constexpr int HOLD = CODES ? 2 : 4; // blocks of 32 scores that a softmax thread keeps
    static_assert(2 * SOFT + K_GROUPS<CODES> * K + V + MMA <= THREADS<CODES> / GROUP * LAUNCH, "the roles' registers come from the launch's");
};
// Steps whose places, V exponents and reports are kept.  The V loaders write those of step s + 1 once P V of step s - 2 is
// done, before which the softmax groups are through with step s - 3.
constexpr int SLOTS = 4;
// Steps whose score factors are kept.  The K loaders write that of step s + 1 once Q K of step s - 2 is done; in a tile of
// one half that product comes after P V of step s - 4, and step s - 3's softmax may not even have begun: five are
// needed, and eight make the place a mask.
constexpr int KFACS = 8;
constexpr float GROW = 8.f; // log2 growth of a maximum that is let pass before O is rescaled
constexpr float LIFT = 7.f; // log2 of P at the reference maximum: P <= 2^(GROW + LIFT), inside fp16

enum Bar { KF0, KF1, KF2, KF3, KE0, KE1, KE2, KE3, VF0, VF1, VE0, VE1, SF0, SF1, PF0, PF1, OD0, OD1, XF0, XF1, XF2, XF3, DRAIN, N_BARS };

// A step's K is one tile, or with codes two, its values' first and second parts, which take the K tiles' places in turn.
template <int D, bool CODES> struct Lay {
    static constexpr int REG = TN * 128;          // a region: 128 rows of 64 fp16, 128-byte swizzled
    static constexpr int TILE = D / 64 * REG;     // bytes of a 128-row tile of fp16
    static constexpr int PARTS = CODES ? 2 : 1;
    static constexpr int K_TILES = CODES && D == 64 ? 4 : 2; // (D 128 has room for no more)
    static constexpr int Q = 0, K = 2 * TILE, V = K + K_TILES * TILE, AUX = V + 2 * TILE;
    // a query tile of one half leaves the other half's place free: one more for K
    static constexpr int MORE = CODES && D == 128 ? 1 : 0;
    __device__ static __forceinline__ int k_tiles(bool wide) { return K_TILES + (wide ? 0 : MORE); }
    __device__ static __forceinline__ int k(bool wide) { return K - (wide ? 0 : MORE) * TILE; }
};

// A tree's masks (TREE): which of the block's rows the tile's tokens see; a word of zeros behind them.
template <bool TREE> struct TreeMasks {};
template <> struct TreeMasks<true> {
    static constexpr int WORDS = TREE_MAX / 32 + 1;
    int32_t parent[TREE_MAX];
    uint32_t sees[2 * TM][WORDS]; // by the token's place from the tile's first
};

struct Aux {
    uint64_t bar[N_BARS];
    int32_t row[2][SLOTS][TN];   // K's and V's loaders: pool rows of a step, -1 past the end
    float qscale[2 * TM];
    int32_t vis[2 * TM];
    float kfac[KFACS];           // score factor of the step's K exponent
    int32_t vexp[SLOTS];         // V's exponent as of the step, twice, and whether rows of it are reported in badrow
    alignas(16) uint32_t badrow[SLOTS][TN / 32]; // rows of the step whose V values that are not finite were left out
    alignas(16) uint32_t red[2][2][GROUP / 32];
    float2 ml[TM];
    uint16_t scale[2][2][TN * 4]; // K's and V's block scales of a step, [row][block]
    uint32_t tmem;
    int32_t vis_max, vis_min, any_bad;
    volatile int32_t abort;
};

__device__ __forceinline__ bool any_bad(const uint32_t (&rows)[TN / 32]) {
    const uint4 b = *reinterpret_cast<const uint4 *>(rows);
    return (b.x | b.y | b.z | b.w) != 0;
}

template <int D, bool CODES, bool TREE> constexpr int smem_bytes() {
    // TMEM is allocated whole: one CTA per SM, whatever D
    const int need = Lay<D, CODES>::AUX + (int)sizeof(Aux) + 2 * TM * (D / 16) * 4 + 1024 + (TREE ? (int)sizeof(TreeMasks<TREE>) : 0);
    return need > 120 * 1024 ? need : 120 * 1024;
}

// ------------------------------------------------------------- loading ----
// A loading group's work: tensor T's rows of every step (IS_V: V, else K) into its n_tiles stages (two, but for K's codes).
template <int D, int T, bool IS_V>
__device__ __forceinline__ void load_rows(const BlockParams &p, const BlockSeq &q, int g, uint8_t *tiles, int n_tiles, Aux &x, int r0,
                                          int r_end, int t) {
    constexpr bool TWO = !IS_V && T != KVC_F16; // a step is two tiles
    constexpr int TILE = Lay<D, TWO>::TILE;
    const uint8_t *data = IS_V ? p.vdata : p.kdata;
    uint64_t *full = &x.bar[IS_V ? VF0 : KF0], *empty = &x.bar[IS_V ? VE0 : KE0];
    int32_t(*row)[TN] = x.row[IS_V];
    int steps = 1 << 24, vis_min = 0, r1 = 0; // known with the query rows; r1: the end of the rows that some token sees
    constexpr int SYNC = IS_V ? 4 : 3, NT = IS_V ? GROUP : K_GROUPS<TWO> * GROUP; // threads
    const bool has_row = NT == TN || t < TN;   // whose place and scales it sees to
    Lookup next; // of the step whose rows the group gets next
    auto look_up = [&](int s) { next.ask(p, q, r0 + s * TN + t, has_row && s < steps); };
    auto find = [&](int s) { // for all threads after the next barrier
        if (has_row) row[s % SLOTS][t] = next.row(p, g);
        look_up(s + 1);
    };
    auto clear = [&](int s) { // a step's reports; the slot's last step, four before, is done with (its V was used up)
        if (IS_V && t < TN / 32) x.badrow[s % SLOTS][t] = 0;
    };
    auto begin = [&] { // the query rows are there: how far the tokens see
        __syncthreads();
        tc_after();
        r1 = min(r_end, x.vis_max);
        steps = r1 > r0 ? (r1 - r0 + TN - 1) / TN : 0;
        vis_min = x.vis_min;
    };
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (has_row) row[k][t] = pool_row(p, q, g, r0 + k * TN + t);
    look_up(3);
    clear(0);
    named_sync<SYNC, NT>();
    if constexpr (T == KVC_F16) {
        // A step's copies are under way while those of the step before are waited for, if their stage is free by then;
        // a step that has landed is not held back for a stage.
        copy_halves<D>(tiles, data, row[0], t);
        begin();
        if (steps == 0) { // no token sees a row: the results are put together where step 0 lands, so they wait for it
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            bar_arrive(&full[0]);
        }
        for (int s = 0; s <= steps && steps > 0; ++s) {
            bool ahead = false;
            if (s < steps) {
                ahead = s < 2 || bar_try(&empty[s & 1], ((s >> 1) - 1) & 1);
                if (ahead && s > 0) copy_halves<D>(tiles + (s & 1) * TILE, data, row[s % SLOTS], t);
                if (!IS_V && t == 0) x.kfac[s % KFACS] = 1.f;
            }
            if (s > 0) {
                if (ahead)
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                else
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                if (IS_V && r0 + s * TN > vis_min)
                    drop_halves<D>(tiles + ((s - 1) & 1) * TILE, x.badrow[(s - 1) % SLOTS], t);
                fence_async();
                bar_arrive(&full[(s - 1) & 1]);
            }
            if (s < steps && !ahead) {
                bar_wait(&empty[s & 1], ((s >> 1) - 1) & 1, p.err, &x.abort);
                copy_halves<D>(tiles + (s & 1) * TILE, data, row[s % SLOTS], t);
            }
            find(s + 3);
            clear(s + 1);
            named_sync<SYNC, NT>();
        }
    } else {
        // A thread's piece of the next step is requested as soon as this step's is stored.  It looks after one row's
        // scales too, a step earlier: the largest scale, which gives a step its exponent, is known before the step's turn.
        using C = Codes<D, T, NT>;
        const int c = t % C::PIECES, j0 = t / C::PIECES;
        const uint8_t *codes = data + c * 16;
        const uint16_t *scales = IS_V ? p.vs : p.ks;
        uint32_t a[4];
        constexpr bool f = false; // (avoiding the stores' bank conflicts costs more instructions here than it saves)
        C::places(j0, c, a, f);
        uint4 u[C::MINE];
        uint32_t sc[D / 64];
        auto at_row = [&](int s, int j) { return max(row[s % SLOTS][j], 0); };
        int E = E_MIN;
        auto exponent = [&](int s) { // of step s, whose scales are sc
            uint32_t m = 0;
            const bool in = r0 + s * TN + t < r1; // a row past the end, or that nobody sees: scales 0
#pragma unroll
            for (int k = 0; has_row && k < D / QK; ++k) {
                uint32_t h = sc[k >> 1] >> (16 * (k & 1)) & 0xffffu;
                if (!in) h = 0;
                if ((h & 0x7fffu) < 0x7c00u) {
                    m = max(m, h & 0x7fffu);
                } else if (IS_V) { // not finite: reported and left out
                    h = 0;
                    atomicOr(&x.badrow[s % SLOTS][t >> 5], 1u << (t & 31));
                }
                x.scale[IS_V][s & 1][t * (D / QK) + k] = (uint16_t)h;
            }
            m = __reduce_max_sync(0xffffffffu, m);
            if (has_row && (t & 31) == 0) x.red[IS_V][s & 1][t >> 5] = m;
            find(s + 3);
            clear(s + 1);
            named_sync<SYNC, NT>();
            const uint4 r = *reinterpret_cast<const uint4 *>(x.red[IS_V][s & 1]);
            const uint32_t top = max(max(r.x, r.y), max(r.z, r.w));
            const int e = top ? ilogbf(__half2float(__ushort_as_half((uint16_t)top))) : E_MIN;
            E = IS_V ? max(E, e) : e;
            if (t == 0) {
                if (IS_V) {
                    x.vexp[s % SLOTS] = 2 * E + any_bad(x.badrow[s % SLOTS]);
                    bar_arrive(&x.bar[XF0 + s % SLOTS]);
                } else {
                    x.kfac[s % KFACS] = ldexpf(1.f, E - 7);
                }
            }
        };
        if (has_row) C::load(sc, scales, at_row(0, t));
#pragma unroll
        for (int i = 0; i < C::MINE; ++i) C::load(u[i], codes, at_row(0, j0 + i * C::ROWS));
        begin();
        if (steps == 0) return;
        exponent(0);
        if (has_row) C::load(sc, scales, at_row(1, t));
        int place = 0, use = 0; // TWO: of the next tile, and how often the places have been used
        for (int s = 0; s < steps; ++s) {
            const float up = ldexpf(1.f, 7 - E);
            const uint16_t *d = &x.scale[IS_V][s & 1][j0 * (D / QK) + (T == KVC_Q4_0 ? c : c / 2)];
            if constexpr (TWO) {
                // (scales and rows first: a shared load would wait for the stores before it)
                __half2 ds[C::MINE];
                int32_t next_row[C::MINE];
#pragma unroll
                for (int i = 0; i < C::MINE; ++i) {
                    ds[i] = scaled(d[i * C::ROWS * (D / QK)], up);
                    next_row[i] = at_row(s + 1, j0 + i * C::ROWS);
                }
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (use > 0) bar_wait(&empty[place], (use - 1) & 1, p.err, &x.abort);
                    uint8_t *tile = tiles + place * TILE;
#pragma unroll
                    for (int i = 0; i < C::MINE; ++i) {
                        if (part == 0) {
                            C::store(tile + i * C::ROWS * 128, a, u[i], ds[i], f);
                        } else {
                            // (opaque: the first part's values are formed again, there are no registers to keep them)
                            asm volatile("" : "+r"(u[i].x), "+r"(u[i].y), "+r"(u[i].z), "+r"(u[i].w));
                            C::store_rest(tile + i * C::ROWS * 128, a, u[i], ds[i], f);
                            C::load(u[i], codes, next_row[i]); // (behind the last step: a row that is there)
                        }
                    }
                    fence_async();
                    bar_arrive(&full[place]);
                    if (++place == n_tiles) {
                        place = 0;
                        ++use;
                    }
                }
            } else {
                if (s >= 2) bar_wait(&empty[s & 1], ((s >> 1) - 1) & 1, p.err, &x.abort);
                uint8_t *tile = tiles + (s & 1) * TILE;
#pragma unroll
                for (int i = 0; i < C::MINE; ++i) {
                    C::store(tile + i * C::ROWS * 128, a, u[i], scaled(d[i * C::ROWS * (D / QK)], up), f);
                    C::load(u[i], codes, at_row(s + 1, j0 + i * C::ROWS)); // (behind the last step: a row that is there)
                }
                fence_async();
                bar_arrive(&full[s & 1]);
            }
            if (s + 1 < steps) {
                exponent(s + 1);
                if (has_row) C::load(sc, scales, at_row(s + 2, t));
            }
        }
    }
}

// ------------------------------------------------------------ softmax ----
// Which of a step's 128 rows a thread's token sees: the first n, or (a tree) the rows whose bits are set.
struct Leading {
    int n;
    __device__ __forceinline__ bool operator()(int c, int e) const { return c * 32 + e < n; }
    __device__ __forceinline__ uint32_t block(int c) const { // of 32 rows
        const int k = n - c * 32;
        return k >= 32 ? 0xffffffffu : (k > 0 ? (1u << k) - 1u : 0u);
    }
};
struct Picked {
    uint32_t w[4];
    __device__ __forceinline__ bool operator()(int c, int e) const { return w[c] >> e & 1; }
    __device__ __forceinline__ uint32_t block(int c) const { return w[c]; }
};

// A thread's 128 scores, of which it sees some (MASK): 32 of them from registers, unseen ones -inf; the largest.
template <bool MASK, class Seen> __device__ __forceinline__ void score_block(uint32_t (&r)[32], int c, const Seen &n, float (&m)[4]) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float v0 = __uint_as_float(r[e]), v1 = __uint_as_float(r[e + 1]);
        if (MASK) {
            v0 = n(c, e) ? v0 : -INFINITY;
            v1 = n(c, e + 1) ? v1 : -INFINITY;
            r[e] = __float_as_uint(v0);
            r[e + 1] = __float_as_uint(v1);
        }
        m[e / 2 % 4] = max3(m[e / 2 % 4], v0, v1);
    }
}
// HOLD: blocks of 32 scores that stay in registers between the maximum and the weights; the others are read again (P's
// 64 columns go over the first two blocks, so those stay).
template <bool MASK, int HOLD, class Seen>
__device__ __forceinline__ float row_scores(uint32_t S, const Seen &n, uint32_t (&r)[HOLD][32]) {
    static_assert(HOLD == 2 || HOLD == 4, "all, or what P overwrites");
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if constexpr (HOLD == 4) {
#pragma unroll
        for (int c = 0; c < 4; ++c) tm_ld(r[c], S + c * 32);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            tm_wait(r[c]);
            score_block<MASK>(r[c], c, n, m);
        }
    } else {
        uint32_t t[32];
        tm_ld(r[0], S);
        tm_ld(r[1], S + 32);
        tm_ld(t, S + 64);
        tm_wait(r[0]);
        score_block<MASK>(r[0], 0, n, m);
        tm_wait(r[1]);
        score_block<MASK>(r[1], 1, n, m);
        tm_wait(t);
        score_block<MASK>(t, 2, n, m);
        tm_ld(t, S + 96);
        tm_wait(t);
        score_block<MASK>(t, 3, n, m);
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// exp2 of the scores (times f, less use; f >= 0, an unseen one is -inf) as fp16 pairs over them; returns their sum.
// mark(c, rows): a look at column block c's 32 rows (MASK); with all scores held, rows are those that are seen, of whatever
// weight.  (Gathered on the way, where the registers are there: 6 tokens over 16384 rows, halves 23.0 us so and 24.2 with the
// bits made when they are needed; codes 31.9 and 30.3, and their trees 386 and 370 us of 32 sequences of 20 to 80 tokens.)
template <bool MASK, int HOLD, class Seen, class Mark>
__device__ __forceinline__ float row_exp(uint32_t S, const Seen &n, uint32_t (&r)[HOLD][32], float f, float use, Mark mark) {
    const uint64_t ff = pair(f, f), mm = pair(-use, -use);
    uint64_t a0 = 0, a1 = 0;
    auto block = [&](int c, const uint32_t(&x)[32]) {
        uint32_t w[16], own = 0;
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float2 y = unpair(fma2(pair(x[e], x[e + 1]), ff, mm));
            if (MASK) {
                y.x = n(c, e) ? y.x : -INFINITY;
                y.y = n(c, e + 1) ? y.y : -INFINITY;
            }
            if (MASK && HOLD == 4) own |= (n(c, e) ? 1u << e : 0u) | (n(c, e + 1) ? 2u << e : 0u);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            w[e / 2] = h2(y.x, y.y);
            if (e & 2)
                a1 = add2(a1, pair(y.x, y.y));
            else
                a0 = add2(a0, pair(y.x, y.y));
        }
        if (MASK) mark(c, own);
        tm_st16(S + c * 16, w);
    };
    if constexpr (HOLD == 4) {
#pragma unroll
        for (int c = 0; c < 4; ++c) block(c, r[c]);
    } else {
        uint32_t t[32];
        tm_ld(t, S + 64);
        block(0, r[0]);
        tm_ld(r[0], S + 96);
        block(1, r[1]);
        tm_wait(t);
        block(2, t);
        tm_wait(r[0]);
        block(3, r[0]);
    }
    const float2 s = unpair(add2(a0, a1));
    return s.x + s.y;
}

// TREE: the block's tokens are the sequence's last rows, and each sees the rows before them, its ancestors' and its own
// (kvc_attn_tree); else a token sees its n_vis leading rows.  K's codes have two parts there too, although no log-sum-exp
// comes with a tree: with one of 11 bits (26 tokens over 16384 rows 36 us, 40 with both; 64 over 32768 95 and 99) scores of
// 300 were off by 0.07 and results by as much, ten roundings of bf16.
template <int D, int KT, int VT, bool TREE>
__global__ void __launch_bounds__(THREADS<KT != KVC_F16>, 1) cross_tc_kernel(const __grid_constant__ BlockParams p) {
    constexpr bool CODES = KT != KVC_F16;
    using L = Lay<D, CODES>;
    using R = Regs<CODES>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u); // swizzled tiles need 1024-byte alignment
    Aux &x = *reinterpret_cast<Aux *>(smem + L::AUX);
    uint32_t(*poison)[D / 16] = reinterpret_cast<uint32_t(*)[D / 16]>(smem + L::AUX + sizeof(Aux));
    TreeMasks<TREE> &tree = *reinterpret_cast<TreeMasks<TREE> *>(smem + L::AUX + sizeof(Aux) + 2 * TM * (D / 16) * 4);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const BlockSeq q = p.seq[item_seq(p, (int)blockIdx.x)];
    const int local = (int)blockIdx.x - q.item0;
    int unit, part, parts;
    item_unit(q, local, unit, part, parts);
    const int g = unit / q.tiles, tile = q.tile0 + q.tiles - 1 - unit % q.tiles; // later tokens see more: they begin first
    const int m_all = q.n_tok * p.r, m0 = tile * 2 * TM, mrows = min(2 * TM, m_all - m0);
    const bool wide = mrows > TM;
    constexpr int WK = 8, WV = WK + 4 * K_GROUPS<CODES>, WI = WV + 4; // first warps of K's, V's and the issuing role

    if (tid == 0) {
        for (int i = 0; i < N_BARS; ++i) {
            const bool load = (i >= KF0 && i <= KF3) || i == VF0 || i == VF1;
            bar_init(&x.bar[i], load || i == PF0 || i == PF1 ? (i <= KF3 ? K_GROUPS<CODES> : 1) * GROUP : 1);
        }
        x.vis_max = 0;
        x.vis_min = 0x7fffffff;
        x.any_bad = 0;
        x.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&x.tmem)), "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    __syncthreads();
    if (TREE) wait_for_previous();
    const int r0 = part * q.split_rows, r_end = parts == 1 ? q.n_rows : min(r0 + q.split_rows, q.n_rows);
    if (warp >= WK && warp < WV) {
        regs_dec<R::K>();
        load_rows<D, KT, false>(p, q, g, smem + L::k(wide), L::k_tiles(wide), x, r0, r_end, tid - WK * 32);
        return;
    } else if (warp >= WV && warp < WI) {
        regs_dec<R::V>();
        load_rows<D, VT, true>(p, q, g, smem + L::V, 2, x, r0, r_end, tid - WV * 32);
        return;
    }
    // The other warps see to the query rows: a warp each, QR of its rows under way together, normalised by a power of two
    // that takes the scale's sign too; rows that are not there are zero.
    constexpr int QR = 6, QW = 12; // (the loading warps are at their first rows already)
    const int qw = warp < 8 ? warp : warp - WI + 8;
    for (int mb = qw; mb < mrows; mb += QW * QR) {
        Query<D> y[QR];
#pragma unroll
        for (int k = 0; k < QR; ++k)
            if (mb + k * QW < mrows) y[k].ask(p, q, g, m0 + mb + k * QW, m_all, lane);
#pragma unroll
        for (int k = 0; k < QR; ++k) {
            const int m = mb + k * QW;
            if (m >= mrows) break;
            float v[D / 32];
            uint32_t h[D / 64], l[D / 64];
            int vis = y[k].get(p, q, v);
            if (TREE) vis = q.n_rows - q.n_tok; // the rows that all of the block see
            float scale = query_pack<D, false>(p, v, h, l);
            if (scale < 0.f) {
                scale = -scale;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) h[i] ^= 0x80008000u;
            }
            uint8_t *dst = smem + L::Q + (m >> 7) * L::TILE + at(m & 127, lane * (D / 32));
            if constexpr (D == 128)
                *reinterpret_cast<uint2 *>(dst) = make_uint2(h[0], h[1]);
            else
                *reinterpret_cast<uint32_t *>(dst) = h[0];
            if (lane == 0) {
                x.qscale[m] = scale;
                x.vis[m] = vis;
                atomicMax(&x.vis_max, TREE ? q.n_rows : vis);
                atomicMin(&x.vis_min, vis);
            }
        }
    }
    {
        const int ft = qw * 32 + lane, all = wide ? 2 * TM : TM;
        for (int i = ft; i < (all - mrows) * (D / 8); i += QW * 32) {
            const int m = mrows + i / (D / 8), c = i % (D / 8); // 16 bytes of the row, whichever the swizzle makes of them
            *reinterpret_cast<uint4 *>(smem + L::Q + (m >> 7) * L::TILE + (c >> 3) * L::REG + (m & 127) * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
            if (c == 0) x.qscale[m] = 0.f;
        }
        for (int i = ft; i < all * (D / 16); i += QW * 32) poison[i / (D / 16)][i % (D / 16)] = 0;
    }
    if constexpr (TREE) {
        // The tokens' masks, where the part holds rows of the block: by walks from each token to its root (a parent is
        // below its child).
        if (r_end > q.n_rows - q.n_tok) {
            const int ft = qw * 32 + lane, first = token_of(p, m0), count = token_of(p, m0 + mrows - 1) - first + 1;
            if (p.parent)
                for (int i = ft; i < q.n_tok; i += QW * 32) {
                    const int up = p.parent[(int64_t)q.tok0 + i];
                    tree.parent[i] = up >= 0 && up < i ? up : -1;
                }
            named_sync<5, QW * 32>();
            for (int i = ft; i < count; i += QW * 32) {
                const int t = first + i;
                for (int k = 0; k < tree.WORDS; ++k) {
                    const int n = t + 1 - k * 32; // without a tree: a chain
                    tree.sees[i][k] = p.parent ? 0u : (n >= 32 ? 0xffffffffu : (n > 0 ? (1u << n) - 1u : 0u));
                }
                if (p.parent)
                    for (int u = t; u >= 0; u = tree.parent[u]) tree.sees[i][u >> 5] |= 1u << (u & 31);
            }
        }
    }
    fence_async();
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tm = x.tmem;
    const uint32_t tS = tm, tO = tm + 256; // S0, S1: 128 columns each (P over them); O0, O1: D columns each
    const int r1 = min(r_end, x.vis_max);
    const int steps = r1 > r0 ? (r1 - r0 + TN - 1) / TN : 0;
    const int jobs = wide ? 2 * steps : steps;
    const int vis_min = x.vis_min;

    if (warp < 8) {
        // -------------------------------------------------- softmax of half h
        regs_inc<R::SOFT>();
        const int h = warp >> 2, mr = wide ? tid : (tid & 127);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21; // TMEM lane 32 * (warp % 4)
        const uint32_t S = tS + h * 128 + lanes, O = tO + h * D + lanes;
        const bool live = __any_sync(0xffffffffu, mr < mrows);
        const float cq = x.qscale[mr];
        const int vis = mr < mrows ? x.vis[mr] : 0x7fffffff;
        const int slot_t = TREE ? token_of(p, min(m0 + mr, m_all - 1)) - token_of(p, m0) : 0; // its token's mask
        const int wvis = __reduce_min_sync(0xffffffffu, vis);
        float mx = -INFINITY, sum = 0.f; // the row's reference maximum and sum
        int E = E_MIN;
        int done = 0; // jobs of this half
        for (int i = h; i < jobs; i += 2, ++done) {
            const int s = wide ? i >> 1 : i, base = r0 + s * TN, slot = s % SLOTS;
            bar_wait_warp(&x.bar[SF0 + h], done & 1, p.err, &x.abort);
            tc_after();
            if (live) {
                const bool masked = base + TN > wvis;
                auto seen = [&] {
                    if constexpr (TREE) {
                        Picked w;
#pragma unroll
                        for (int c = 0; c < 4; ++c) { // rows base + 32 c on: the tree's place t on, and all before it
                            const int t = base + c * 32 - (q.n_rows - q.n_tok);
                            const uint32_t *m = tree.sees[slot_t];
                            if (t <= -32)
                                w.w[c] = 0xffffffffu;
                            else if (t < 0)
                                w.w[c] = m[0] << -t | ((1u << -t) - 1u);
                            else
                                w.w[c] = t < TREE_MAX ? __funnelshift_r(m[t >> 5], m[(t >> 5) + 1], t & 31) : 0u;
                        }
                        return w;
                    } else {
                        return Leading{vis - base};
                    }
                };
                const float f = cq * x.kfac[s % KFACS];
                constexpr int HOLD = R::HOLD;
                uint32_t sc[HOLD][32];
                const float raw = masked ? row_scores<true>(S, seen(), sc) : row_scores<false>(S, Leading{0}, sc);
                const float top = raw == -INFINITY ? raw : raw * f;
                float al = 1.f;
                if (top > mx + GROW || (mx == -INFINITY && top > mx)) {
                    al = ex2(mx - top); // 0 for a first maximum
                    mx = top;
                }
                sum *= al;
                // V's exponent, and whether values were left out: a row that sees those takes them from the reports, whatever
                // the tile's other rows see
                bool reported = false;
                if (VT != KVC_F16) {
                    bar_wait_warp(&x.bar[XF0 + slot], (s / SLOTS) & 1, p.err, &x.abort);
                    const int e2 = x.vexp[slot], e = e2 >> 1;
                    reported = e2 & 1;
                    if (e != E) al *= ldexpf(1.f, max(E - e, -126));
                    E = e;
                } else if (base + TN > vis_min) {
                    bar_wait_warp(&x.bar[VF0 + (s & 1)], (s >> 1) & 1, p.err, &x.abort);
                    reported = any_bad(x.badrow[slot]);
                }
                if (done > 0 && __any_sync(0xffffffffu, al != 1.f)) {
                    bar_wait_warp(&x.bar[OD0 + h], (done - 1) & 1, p.err, &x.abort);
                    tc_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float v[32];
                        tm_ld32(v, O + c * 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] *= al;
                        tm_st32(O + c * 32, v);
                    }
                }
                const float use = mx == -INFINITY ? 0.f : mx - LIFT;
                if (!masked && !reported) {
                    sum += row_exp<false>(S, Leading{0}, sc, f, use, [](int, uint32_t) {});
                } else {
                    sum += row_exp<true>(S, seen(), sc, f, use, [&](int c, uint32_t own) {
                        const uint32_t rows = x.badrow[slot][c];
                        if (rows == 0) return;
                        if (HOLD != 4) own = seen().block(c);
#pragma unroll 1
                        for (int e = 0; e < 32; ++e) {
                            if (!(rows >> e & 1)) continue;
                            const int32_t R = pool_row(p, q, g, base + c * 32 + e);
                            if (mr < mrows && (own >> e & 1) && R >= 0) {
                                mark_poison<D, VT>(poison[mr], p.vdata, p.vs, R);
                                x.any_bad = 1;
                            }
                        }
                        __syncwarp();
                    });
                }
                tm_wait_st();
            }
            tc_before();
            bar_arrive(&x.bar[PF0 + h]);
        }
        if (done > 0) bar_wait_warp(&x.bar[OD0 + h], (done - 1) & 1, p.err, &x.abort);
        if (KT == KVC_F16 && steps == 0) { // halves were requested before it was known that nobody sees them
            bar_wait_warp(&x.bar[KF0], 0, p.err, &x.abort);
            bar_wait_warp(&x.bar[VF0], 0, p.err, &x.abort);
        }
        tc_after();
        // -------------------------------------------------- results
        named_sync<2, 2 * GROUP>(); // both halves' products are done: the K and V tiles are free
        float *join = reinterpret_cast<float *>(smem + L::K); // [TM][D + 4]: the odd steps' sums
        constexpr int JP = D + 4;
        const float back = VT == KVC_F16 ? 1.f : ldexpf(1.f, E - 7);
        if (!wide && h == 1 && live) {
            x.ml[mr] = make_float2(mx, sum);
            if (done > 0) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    __syncwarp();
                    tm_ld32(v, O + c * 32);
                    if (mr < mrows) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(&join[mr * JP + c * 32 + e]) =
                                make_float4(v[e] * back, v[e + 1] * back, v[e + 2] * back, v[e + 3] * back);
                    }
                }
            }
        }
        named_sync<2, 2 * GROUP>();
        const bool whole = parts == 1;
        const int prow = q.part_row0 + (local - q.whole) * p.part_rows;
        if (live && (wide || h == 0)) {
            float f0 = 1.f, f1 = 0.f;
            bool two = false;
            if (!wide && jobs > 1) { // the even and the odd steps' sums
                const float2 o = x.ml[mr];
                const float M = fmaxf(mx, o.x), use = M == -INFINITY ? 0.f : M;
                f0 = ex2(mx - use);
                f1 = ex2(o.x - use);
                sum = sum * f0 + o.y * f1;
                mx = M;
                two = true;
            }
            mx -= LIFT; // what the sum's terms are relative to
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            auto head_of = [&](int row) {
                const int m = m0 + row, t = token_of(p, m), j = m - t * p.r;
                return ((int64_t)q.tok0 + t) * p.H + (int64_t)g * p.r + j;
            };
            constexpr int SP = 36; // floats of a staging row: 16 bytes off a multiple of 128
            float *stage = join + (wide ? 0 : TM * JP) + (warp & (wide ? 7 : 3)) * (32 * SP);
            static_assert((TM * JP + 4 * 32 * SP) * 4 <= L::AUX - L::K && 8 * 32 * SP * 4 <= L::AUX - L::K, "within the K and V tiles");
            const bool bad = x.any_bad != 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float v[32];
                __syncwarp();
                if (done > 0) {
                    tm_ld32(v, O + c * 32);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                if (mr < mrows) {
                    const float s0 = back * f0;
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = sum == 0.f ? 0.f : v[e] * s0;
                    if (two && sum != 0.f) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 y = *reinterpret_cast<const float4 *>(&join[mr * JP + c * 32 + e]);
                            v[e] = fmaf(y.x, f1, v[e]);
                            v[e + 1] = fmaf(y.y, f1, v[e + 1]);
                            v[e + 2] = fmaf(y.z, f1, v[e + 2]);
                            v[e + 3] = fmaf(y.w, f1, v[e + 3]);
                        }
                    }
                    if (bad) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = poisoned(v[e], poison[mr][(c * 32 + e) / 16] >> (2 * (e % 16)) & 3u);
                    }
                }
                // through the warp's staging rows, so that memory is written a row's 32 columns at a time
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(&stage[lane * SP + e]) =
                        make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
                __syncwarp();
                const int mw = mr - lane; // the warp's first row
                if (whole) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = k * 8 + (lane >> 2), e = (lane & 3) * 8;
                        const float4 a = *reinterpret_cast<const float4 *>(&stage[row * SP + e]);
                        const float4 b = *reinterpret_cast<const float4 *>(&stage[row * SP + e + 4]);
                        if (mw + row < mrows)
                            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.out) + head_of(mw + row) * D + c * 32 + e) =
                                make_uint4(pack16(p.act, a.x, a.y), pack16(p.act, a.z, a.w), pack16(p.act, b.x, b.y),
                                           pack16(p.act, b.z, b.w));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int row = k * 4 + (lane >> 3), e = (lane & 7) * 4;
                        const float4 a = *reinterpret_cast<const float4 *>(&stage[row * SP + e]);
                        if (mw + row < mrows)
                            *reinterpret_cast<float4 *>(p.part + (int64_t)(prow + mw + row) * D + c * 32 + e) = a;
                    }
                }
            }
            if (mr < mrows) {
                if (whole) {
                    if (p.lse) p.lse[head_of(mr)] = sum == 0.f ? -INFINITY : mx * 0.6931471805599453f + logf(sum);
                } else {
                    *reinterpret_cast<float2 *>(p.part + p.part_cap * D + 2 * (int64_t)(prow + mr)) = make_float2(mx, sum);
                }
            }
        }
        tc_before();
        named_sync<2, 2 * GROUP>();
        if (warp == 0) {
            tc_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(TMEM_COLS));
        }
    } else {
        regs_dec<R::MMA>();
        if (warp > WI || lane > 0) return;
        // -------------------------------------------------- products
        const int n_tiles = L::k_tiles(wide);
        const uint64_t dq = desc(smem_u32(smem + L::Q), 16), dk = desc(smem_u32(smem + L::k(wide)), 16);
        const uint32_t sv = smem_u32(smem + L::V);
        int place = 0, odd = 0; // of the step's first K tile, and its barriers' phase
        auto qk = [&](int i) {  // job i's scores
            const int h = i & 1;
            int at = place, phase = odd;
#pragma unroll
            for (int part = 0; part < L::PARTS; ++part) { // (the larger part first)
                bar_wait(&x.bar[KF0 + at], phase, p.err, &x.abort);
                tc_after();
                const uint64_t a = dq + (uint32_t)(wide ? h * (L::TILE >> 4) : 0), b = dk + (uint32_t)(at * (L::TILE >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t o = ((k >> 2) * L::REG + (k & 3) * 32) >> 4;
                    mma_ss(tS + h * 128, a + o, b + o, inst(TN, false), part > 0 || k > 0);
                }
                if (part == L::PARTS - 1) tc_commit(&x.bar[SF0 + h]);
                if (!wide || h) tc_commit(&x.bar[KE0 + at]);
                if (++at == n_tiles) {
                    at = 0;
                    phase ^= 1;
                }
            }
            if (!wide || h) {
                place = at;
                odd = phase;
            }
        };
        if (jobs > 0) qk(0);
        if (jobs > 1) qk(1);
        for (int i = 0; i < jobs; ++i) {
            const int s = wide ? i >> 1 : i, h = i & 1, k0 = i >> 1; // k0: the half's job
            bar_wait(&x.bar[VF0 + (s & 1)], (s >> 1) & 1, p.err, &x.abort);
            bar_wait(&x.bar[PF0 + h], k0 & 1, p.err, &x.abort);
            tc_after();
#pragma unroll
            for (int k = 0; k < TN / 16; ++k)
                mma_ts(tO + h * D, tS + h * 128 + k * 8, desc(sv + (s & 1) * L::TILE + k * 2048, L::REG), inst(D, true),
                       k0 > 0 || k > 0);
            tc_commit(&x.bar[OD0 + h]);
            if (!wide || h) tc_commit(&x.bar[VE0 + (s & 1)]);
            if (i + 2 < jobs) qk(i + 2);
        }
        // nothing may be in flight when the CTA gives its memory back
        tc_commit(&x.bar[DRAIN]);
        const uint64_t t0 = now_ns();
        while (!bar_try(&x.bar[DRAIN], 0) && now_ns() - t0 < WAIT_NS) {
        }
    }
}

template <bool TREE, int D, int KT, int VT> cudaError_t go(const BlockParams &p, cudaStream_t st) {
    constexpr bool CODES = KT != KVC_F16;
    auto k = cross_tc_kernel<D, KT, VT, TREE>;
    constexpr int bytes = smem_bytes<D, CODES, TREE>();
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    static SharedMemory set;
    cudaError_t e = set.allow((const void *)k, bytes, Regs<CODES>::LAUNCH);
    if (e != cudaSuccess) return e;
    if (TREE) {
        e = launch_behind(k, (unsigned)p.n_items, THREADS<CODES>, bytes, st, p);
    } else {
        k<<<(unsigned)p.n_items, THREADS<CODES>, bytes, st>>>(p);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? launch_join(p, st) : e;
}
template <bool TREE> cudaError_t pick(int type_k, int type_v, const BlockParams &p, cudaStream_t st) {
    if (p.n_items <= 0) return cudaSuccess;
    if (p.D == 64)
        return type_k == KVC_F16 ? go<TREE, 64, KVC_F16, KVC_F16>(p, st) : go<TREE, 64, KVC_Q8_0, KVC_Q8_0>(p, st);
    if (type_k == KVC_F16) return go<TREE, 128, KVC_F16, KVC_F16>(p, st);
    if (type_v == KVC_Q4_0) return go<TREE, 128, KVC_Q8_0, KVC_Q4_0>(p, st);
    return go<TREE, 128, KVC_Q8_0, KVC_Q8_0>(p, st);
}

} // namespace

cudaError_t launch_cross_tc(int type_k, int type_v, const BlockParams &p, cudaStream_t st) {
    return pick<false>(type_k, type_v, p, st);
}
cudaError_t launch_tree_tc(int type_k, int type_v, const BlockParams &p, cudaStream_t st) {
    return pick<true>(type_k, type_v, p, st);
}

} // namespace kvc
