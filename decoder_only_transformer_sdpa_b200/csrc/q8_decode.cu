// q8_decode.cu -- attention of the newest tokens over the 8-bit block cache.
//
// Sequence b holds L = lens[b] tokens, its Tq newest ones included; query r is
// the token at position L - Tq + r and sees the positions up to its own (a
// position below zero sees none: o = 0, lse = -inf).  H = G * Hkv query heads
// share Hkv key/value heads, so a key/value head serves R = G * Tq rows:
//
//   s_ij = scale * kscale_J * <q_i, code_j - 128>,  J = j / 64
//   o_i  = sum_j p_ij vscale_J (vcode_j - 128) / sum_j p_ij,  p_ij = exp(s_ij - max)
//
// Both products run on the tensor cores with the tokens (for S^T = K q^T) and
// the channels (for O^T = V^T P^T) as the 16 rows of an m16n8k16 fragment and
// eight query rows as its columns, so that one query row wastes seven eighths
// of a tile and not fifteen sixteenths; tcgen05 tiles start at 64 rows.  Codes
// turn into f16 exactly (|code - 128| <= 127); queries are scaled by a power of
// two that brings the row's largest value to [2^14, 2^15), which keeps all
// eight bits of anything down to 2^-31 of it (where that power is at most
// 2^114: a row whose largest value is below 2^-100 keeps eight bits down to
// 2^-131, with errors of 2^-139 at most).  P is rounded to f16 (half a step:
// 2^-11, an eighth of the bf16 output's 2^-8) as 2^13 exp(s - m) with a reference
// m that is at most 2^2 below the running maximum.  Weights below 2^-27 of the
// reference, some 19 below the largest score, would lose bits there, and they are
// all of the output where the heavier tokens' values are zero: such a block's take
// products of their own, 2^29 times as large for each 2^29 that they are smaller
// (light_weights), down to where exp underflows in float32.  Sums of P, the scores
// and both accumulators are float32.
//
// What bounds it is the stream of codes, 128 D bytes a block: every warp has a
// ring of its own in shared memory, filled by bulk copies that its first lane
// issues (a block a slot, or its keys and its values each at D = 128), so a warp
// never waits for another and some 100 KB are in flight on an SM.
//
// How the work is shared out goes by its size alone (shares_for):
//   * little work: the CTAs of a cluster share a row tile, each block going to
//     the next of their warps, and they join their results through distributed
//     shared memory: one launch;
//   * much of it: as many CTAs as the GPU holds, or twice as many, take equal runs
//     of all blocks of all row tiles, whatever the sequences' lengths (which only
//     the kernel knows); a second kernel joins what the runs left of each row tile.
//
// The open block comes first, in bf16 from the ring of recent positions, 16
// tokens a warp, with exact products and P as the sum of two bf16 numbers.
#include "q8_cache.cuh"

#include <cooperative_groups.h>

namespace attn {
namespace {

using namespace sm100;
using namespace q8;
namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
// P is held as 2^13 exp2(s - m), and a score may pass m by 2 before m moves: the two share f16's 2^15.  The more slack,
// the less often m moves and the more often weights are too light (below kLeastF16 = 2^-14, from where on f16 has its
// eleven bits): 8, 3, 2 and 1 take 37.0, 33.9, 33.6 and 33.9 us over 16411 tokens of 4 x 8 heads of 128 with 16 rows,
// whose scores spread by 1.8; without the light weights' check and products it were 31.8.
constexpr float kPShift = 13.f, kSlack = 2.f, kLeastF16 = 0x1p-14f;
constexpr float kUnit = 0x1p-13f;  // brings sums of P to those of exp2(s - m), whose logarithms are smaller and round less
// Outputs are summed as 2^7 exp2(s - m) times the values (what P gives times kOutputs), so that values of 10^30 do not
// overflow over 10^5 tokens of one weight; smaller sums would cost bits where a block's value scale is next to underflow
// (10^-35 keeps 16 of them).
constexpr float kOutputs = 0x1p-6f;
constexpr float kLeastFactor = 0x1p-126f;  // of a block's sums, for scores
constexpr int kMaxCluster = 8;   // portable cluster size

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {  // off by 2^-22 at most
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Warps of a CTA, slots of a warp's ring (a block, or half of one at D = 128),
// and CTAs that an SM holds: three of 168 registers a thread, or two of 255 where
// the sums take more.  In between (32 rows of 32 channels, 16 of 64, 8 of 128),
// where three CTAs spill 30 to 80 bytes a thread, three only where two would
// leave row tiles waiting.  Us with three / two: 16 rows of 64, 432 row tiles of
// 2000 tokens 27.5 / 42.5, 273 of 300 tokens 8.3 / 8.2, 6 of 17000 13.6 / 12.7; 32
// rows of 32, 400 row tiles of 1000 tokens 18.9 / 28.2; one row of 128, 400 row
// tiles of 100 tokens 7.7 / 11.6 and of 2000 tokens 38.3 / 42.0, 128 of up to 16384
// tokens 61.3 / 60.8.
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int ctas_on_sm(int D, int nt, bool crowded) {
    const int sums = D * nt;  // (of a thread, D / 4 each)
    return sums <= 64 ? 3 : sums <= 128 && crowded ? 3 : 2;
}
template <int D, int NT, int Ctas>
struct Cfg {
    static constexpr int kCtas = Ctas;
    static constexpr int kHalves = D == 128 ? 2 : 1;  // slots of a block
    static constexpr int kSlots = D == 32 ? 4 : (kCtas == 3 ? 2 : 3);
    static constexpr bool kQueriesInSmem = NT > 1;  // a warp prepares a row tile; else each the only one, in registers
    static_assert(NT <= kWarps, "a warp a row tile");
    // tiles of 16 tokens (keys) or 16 channels (values) whose sums a warp forms side by side
    static constexpr int kAtOnce = NT == 4 ? 1 : D == 32 ? 2 : 4 / NT;
};

// Layout of the workspace: what each run left of a row tile (its unnormalised
// output, and its maximum in log2 units and sum per row), at place `run + tile`,
// which no other pair of the two has, as runs and row tiles follow one another;
// and each block's log2-sum per row, when the blocks' weights are kept.
struct Parts {
    float *o;    // [run + tile][rows][D]
    float2 *ml;  // [run + tile][rows]
    float *total;  // [tile][rows] log2 of each row's sum, for the kernel that writes the weights, or NULL
    float *lb;     // [B * Hkv][blocks][R]
};

template <int D, int NT, int Ctas>
struct Smem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kSlots = Cfg<D, NT, Ctas>::kSlots;
    static constexpr int kSlot = 2 * kBlock * D / Cfg<D, NT, Ctas>::kHalves;
    static constexpr int kPitch = D + 4;  // rows of partial outputs: four rows apart are on other banks
    // the rings; once they are empty, the warps' outputs and then the CTA's
    union {
        alignas(128) uint8_t ring[kWarps][kSlots][kSlot];
        struct {
            float part[kWarps][kRows][kPitch];
            float o[kRows][D];
        };
    };
    uint2 q[Cfg<D, NT, Ctas>::kQueriesInSmem ? NT : 1][Cfg<D, NT, Ctas>::kQueriesInSmem ? D / 16 : 1][32];  // fragments
    float down[kRows];  // their rows' factors
    int seen[kRows];    // and the last position each sees
    uint64_t full[kWarps][kSlots];
    float m[kWarps][kRows], l[kWarps][kRows];
    float mc[kRows], lc[kRows];  // the CTA's maximum and sum
    float by[kRows];             // what the CTA's outputs are multiplied by
    float total[kRows];          // log2 of each row's sum (for the blocks' weights)
    long long to[kRows];         // where each row's output goes, in elements of o
    int abort;
};

struct DecodeArgs {
    Q8Cache c;
    const __nv_bfloat16 *q;
    TStrides sq;
    __nv_bfloat16 *o;
    TStrides so;
    float *lse;
    const int32_t *lens;
    const int32_t *list;  // NULL: every block
    int list_n;
    int H, G, Tq;   // query heads, heads of a group, new tokens
    unsigned per_tq;  // 2^16 / Tq rounded up: (r * per_tq) >> 16 is r / Tq for r * Tq < 2^16, and r < 64 * 16
    int rows;       // rows of a group: G * Tq, or G with lists (a group is then one token)
    int tiles;      // row tiles of a group
    int tile_rows;  // rows of a tile
    int cluster;    // CTAs of a cluster, which share a row tile; 0: no clusters, but
    int runs;       // this many runs
    bool weigh;     // the decode kernel writes the blocks' weights
    float qscale;   // scale * log2(e)
    int weight;     // 0: not kept, 1: set, 2: add
    Parts part;
    int *err;
};

// Which sequence, key head, token (with lists) and row tile a CTA works for.
struct Where {
    int b, h, r0, tile;
    long long bh;
};
__device__ __forceinline__ Where where(const DecodeArgs &a, unsigned index) {
    Where w;
    w.tile = (int)(index % a.tiles);
    unsigned grp = index / a.tiles;
    w.r0 = 0;
    if (a.list) {
        w.r0 = (int)(grp % a.Tq);
        grp /= a.Tq;
    }
    w.bh = grp;
    w.b = (int)(grp / a.c.H);
    w.h = (int)(grp % a.c.H);
    return w;
}
// ---- runs.  All row tiles' work is laid end to end in units of a block's time:
// kPad units that stand for what a CTA's warps spend on a row tile beside its
// blocks, the places of the list or the closed blocks, and kOpen units for an
// open block.  Run r takes the units from r * units_of_run on, at least kLeastRun
// of them.  A row tile without a token is nobody's.
constexpr int kPad = 12, kOpen = 2, kLeastRun = 8;
__device__ __forceinline__ unsigned units_of(const DecodeArgs &a, int b) {
    int L = a.lens[b];
    if (L < 0 || L / kBlock > a.c.blocks) L = 0;
    const int places = a.list ? a.list_n : L / kBlock;
    return L == 0 ? 0u : (unsigned)(kPad + places + (L % kBlock != 0 ? kOpen : 0));
}
__device__ __forceinline__ unsigned tiles_of_sequence(const DecodeArgs &a) {
    return (unsigned)(a.c.H * (a.list ? a.Tq : 1) * a.tiles);
}
// Inclusive sum over the lanes.
__device__ __forceinline__ unsigned sum_up_to(unsigned x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    return x;
}
// Units of a run (all units are below 2^31, which the host sees to); `mine`:
// units_of sequence `lane`.  The whole warp calls it.
__device__ __forceinline__ unsigned units_of_run(const DecodeArgs &a, unsigned mine) {
    unsigned all = mine;
    for (int i = 32 + (threadIdx.x & 31); i < a.c.B; i += 32) all += units_of(a, i);
    all = __reduce_add_sync(0xffffffffu, all) * tiles_of_sequence(a);
    return max((unsigned)kLeastRun, (all + a.runs - 1) / (unsigned)a.runs);
}
// The row tile with unit u, and u's place in it and the tile's units; false: u
// lies behind all of them.  The whole warp calls it.
__device__ __forceinline__ bool tile_at(const DecodeArgs &a, unsigned mine, unsigned u, unsigned &group, unsigned &at,
                                        unsigned &units) {
    const int lane = threadIdx.x & 31;
    const unsigned per = tiles_of_sequence(a);
    unsigned before = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += 32) {
        const unsigned n = b0 == 0 ? mine : (b0 + lane < a.c.B ? units_of(a, b0 + lane) : 0u);
        const unsigned upto = before + sum_up_to(n);
        const unsigned in = __ballot_sync(0xffffffffu, u < upto * per);
        if (in) {
            const int src = __ffs(in) - 1;
            units = __shfl_sync(0xffffffffu, n, src);
            u -= (__shfl_sync(0xffffffffu, upto, src) - units) * per;
            const unsigned tile = u / units;
            group = (unsigned)(b0 + src) * per + tile;
            at = u - tile * units;
            return true;
        }
        before = __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}
// The runs with units of row tile `group` that it leaves something of: first ..
// last, none where last < first.  The whole warp calls it.
__device__ __forceinline__ void runs_of_tile(const DecodeArgs &a, unsigned group, int &first, int &last) {
    const int lane = threadIdx.x & 31;
    const unsigned per = tiles_of_sequence(a);
    const int b = (int)(group / per);
    const unsigned each = units_of_run(a, lane < a.c.B ? units_of(a, lane) : 0u);
    unsigned before = 0;
    for (int i = lane; i < b; i += 32) before += units_of(a, i);
    before = __reduce_add_sync(0xffffffffu, before) * per;
    const unsigned n = units_of(a, b);
    first = 0;
    last = -1;
    if (n == 0) return;
    const unsigned u0 = before + (group - b * per) * n;
    first = (int)((u0 + kPad) / each);
    last = (int)((u0 + n - 1) / each);
}

// Head in the group and token of row `row` of a group.
__device__ __forceinline__ int row_head(const DecodeArgs &a, int row) {
    return a.list ? row : (int)((unsigned)row * a.per_tq >> 16);
}
__device__ __forceinline__ int row_token(const DecodeArgs &a, const Where &w, int row) {
    return a.list ? w.r0 : row - row_head(a, row) * a.Tq;
}
__device__ __forceinline__ const __nv_bfloat16 *query_row(const DecodeArgs &a, const Where &w, int row) {
    return a.q + (long long)w.b * a.sq.b + (long long)(w.h * a.G + row_head(a, row)) * a.sq.h +
           (long long)row_token(a, w, row) * a.sq.t;
}

// Running softmax state of a warp: this lane's rows 2t and 2t + 1 of each row
// tile (t = lane % 4), and O^T with channels 16 i + g, + 8 (g = lane / 4).
template <int D, int NT>
struct State {
    float m[NT][2], l[NT][2];
    float o[D / 16][NT][4];
};

// Folds the scores f * s[i][nt] (log2 units, f >= 0; s = -inf where masked) of
// 16 * Tiles tokens into the running softmax and replaces them by
// 2^13 exp2(f s - m); the sums of this lane's weights go to `sum`.  The
// reference m moves (to the maximum so far) only when a score passes it by more
// than kSlack, which after the first blocks is rare: one vote a block
// instead of two butterflies.
template <int D, int NT, int Tiles>
__device__ __forceinline__ void softmax_step(State<D, NT> &st, float (&s)[Tiles][NT][4], const float (&f)[NT][2],
                                             float (&sum)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float mx[2];
        bool past = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            mx[x] = fmaxf(s[0][nt][x], s[0][nt][x + 2]);
#pragma unroll
            for (int i = 1; i < Tiles; ++i) mx[x] = fmaxf(mx[x], fmaxf(s[i][nt][x], s[i][nt][x + 2]));
            mx[x] *= f[nt][x];
            past = past || mx[x] > st.m[nt][x] + kSlack;
        }
        if (__any_sync(0xffffffffu, past)) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], off));
                const float m_new = fmaxf(st.m[nt][x], mx[x]);
                const float alpha = m_new == -INFINITY ? 1.f : ex2(st.m[nt][x] - m_new);
                st.m[nt][x] = m_new;
                st.l[nt][x] *= alpha;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    st.o[i][nt][x] *= alpha;
                    st.o[i][nt][x + 2] *= alpha;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float base = (st.m[nt][x] == -INFINITY ? 0.f : st.m[nt][x]) - kPShift;  // (nothing seen yet)
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < Tiles; ++i) {
                s[i][nt][x] = ex2(fmaf(s[i][nt][x], f[nt][x], -base));
                s[i][nt][x + 2] = ex2(fmaf(s[i][nt][x + 2], f[nt][x], -base));
                t += s[i][nt][x] + s[i][nt][x + 2];
            }
            sum[nt][x] = t;
            st.l[nt][x] += t;
        }
    }
}

// Adds the weights of row tile nt that f16 does not hold with all of its bits,
// below kLeastF16, times the block's values to the outputs, and takes them out of
// s.  Each pass has those within 2^29 of one another, times a power of two; `v`:
// the lane's 16 tokens of channel g.  The whole warp calls it.
template <int D, int NT>
__device__ __forceinline__ void light_weights(State<D, NT> &st, float (&s)[4][NT][4], int nt, float scale,
                                              const uint8_t *v) {
    constexpr float kUp = 0x1p29f, kDown = 0x1p-29f, kMost = kLeastF16 * kUp;
    bool some = false;  // lighter ones than those of the passes so far
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x) some = some || (s[u][nt][x] > 0.f && s[u][nt][x] < kLeastF16);
    float up = kUp, down = kDown;
#pragma unroll 1
    for (; __any_sync(0xffffffffu, some); up *= kUp, down *= kDown) {  // (four times at most: weights are normal numbers)
        uint32_t p[4][2];
        some = false;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float w[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float x = s[u][nt][2 * y + z] * up;
                    some = some || (x > 0.f && x < kLeastF16);
                    w[z] = x >= kLeastF16 && x < kMost ? x : 0.f;
                }
                p[u][y] = transpose8(pack_f16x2(w[0], w[1]));
            }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const uint4 a = *reinterpret_cast<const uint4 *>(v + 16 * c * kBlock);
            const uint4 b = *reinterpret_cast<const uint4 *>(v + (16 * c + 8) * kBlock);
            const uint32_t r0[4] = {a.x, a.y, a.z, a.w}, r1[4] = {b.x, b.y, b.z, b.w};
            float acc[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t va[4] = {codes_f16x2<0>(r0[u]), codes_f16x2<0>(r1[u]), codes_f16x2<1>(r0[u]),
                                        codes_f16x2<1>(r1[u])};
                if (u == 0)
                    mma_f16_first(acc, va, p[u][0], p[u][1]);
                else
                    mma_f16(acc, va, p[u][0], p[u][1]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) st.o[c][nt][x] = fmaf(scale, acc[x] * down, st.o[c][nt][x]);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (s[u][nt][x] < kLeastF16) s[u][nt][x] = 0.f;
}

// A load that stays where it is written, ahead of what it overlaps with.
__device__ __forceinline__ uint4 load_now(const void *p) {
    uint4 w;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
    return w;
}

// One bf16 row chunk of the lane: channels slab * S + (S / 4) t + 0 .. S / 4 - 1.
template <int D, bool Now = false>
__device__ __forceinline__ void load_row(uint32_t (&w)[D / 8], const __nv_bfloat16 *row, int t) {
    constexpr int S = slab(D);
#pragma unroll
    for (int i = 0; i < D / 8; i += 4) {  // four words = eight channels
        const int sl = i / (S / 8), in = i % (S / 8);
        const __nv_bfloat16 *from = row + sl * S + (S / 4) * t + 2 * in;
        const uint4 x = Now ? load_now(from) : *reinterpret_cast<const uint4 *>(from);
        w[i] = x.x;
        w[i + 1] = x.y;
        w[i + 2] = x.z;
        w[i + 3] = x.w;
    }
}

__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], const void *row) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(row))
                 : "memory");
}
// A pair of bf16 numbers with what lies behind the end, infinities and NaN
// replaced by 0; the latter are noted in `odd`.
__device__ __forceinline__ uint32_t clean_pair(uint32_t w, bool first, bool second, bool &odd) {
    w &= (first ? 0xffffu : 0u) | (second ? 0xffff0000u : 0u);
    if ((w & 0x7f80u) == 0x7f80u) {
        odd = true;
        w &= 0xffff0000u;
    }
    if ((w & 0x7f800000u) == 0x7f800000u) {
        odd = true;
        w &= 0xffffu;
    }
    return w;
}

// 16 tokens of the open block, positions p0 .. p0 + 15 of a sequence of length
// L: keys k and values v [16][D] in shared memory.
template <int D, int NT, typename Queries, typename Sees>
__device__ __forceinline__ void open_tokens(State<D, NT> &st, float qscale, Queries queries, Sees sees,
                                            const __nv_bfloat16 *k, const __nv_bfloat16 *v, int p0, int L, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float s[1][NT][4], f[NT][2], sum[NT][2];
    {
        uint32_t k0[D / 8], k1[D / 8];  // tokens p0 + g and p0 + g + 8
        load_row<D>(k0, k + g * D, t);
        load_row<D>(k1, k + (g + 8) * D, t);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t q[D / 8];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) q[i] = 0;
            const __nv_bfloat16 *row = queries(nt);
            if (row) load_row<D>(q, row, t);
            s[0][nt][0] = s[0][nt][1] = s[0][nt][2] = s[0][nt][3] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint32_t ka[4] = {k0[2 * i], k1[2 * i], k0[2 * i + 1], k1[2 * i + 1]};
                mma_bf16(s[0][nt], ka, q[2 * i], q[2 * i + 1]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (p0 + g + (x & 2) * 4 > sees(nt, x & 1)) s[0][nt][x] = -INFINITY;
            f[nt][0] = f[nt][1] = qscale;
        }
    }
    softmax_step<D, NT, 1>(st, s, f, sum);
    // P as a bf16 number and what that leaves, another one
    uint32_t b[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            s[0][nt][2 * y] *= kOutputs;
            s[0][nt][2 * y + 1] *= kOutputs;
            const uint32_t h = pack_bf16x2(s[0][nt][2 * y], s[0][nt][2 * y + 1]);
            const float2 r = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&h));
            b[nt][y] = transpose8(h);
            b[nt][2 + y] = transpose8(pack_bf16x2(s[0][nt][2 * y] - r.x, s[0][nt][2 * y + 1] - r.y));
        }
    bool odd = false;
    const int n0 = L - p0 - 2 * t;  // tokens from this lane's first pair on
    const __nv_bfloat16 *row = v + ((lane & 7) + (lane & 16 ? 8 : 0)) * D + (lane & 8);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t va[4];  // channels 16 i + g, + 8 of tokens 2 t, 2 t + 1; the same of tokens 8 further
        load_transposed(va, row + 16 * i);
#pragma unroll
        for (int x = 0; x < 4; ++x) va[x] = clean_pair(va[x], n0 > (x & 2) * 4, n0 > (x & 2) * 4 + 1, odd);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mma_bf16(st.o[i][nt], va, b[nt][0], b[nt][1]);
            mma_bf16(st.o[i][nt], va, b[nt][2], b[nt][3]);
        }
    }
    if (__any_sync(0xffffffffu, odd)) {
        // Infinities and NaN reach only the rows that see their token: added one by one, never as 0 * inf.
        for (int y = 0; y < 16 && p0 + y < L; ++y)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int src = 4 * (y & 7) + t;
                const float pa = __shfl_sync(0xffffffffu, y < 8 ? s[0][nt][0] : s[0][nt][2], src);
                const float pb = __shfl_sync(0xffffffffu, y < 8 ? s[0][nt][1] : s[0][nt][3], src);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float e = __bfloat162float(v[y * D + 16 * i + g + (x & 2) * 4]);
                        if (!isfinite(e) && p0 + y <= sees(nt, x & 1))
                            st.o[i][nt][x] = fmaf((x & 1) ? pb : pa, e, st.o[i][nt][x]);
                    }
            }
    }
}

// f times one output into a joint one.
__device__ __forceinline__ void add(float4 &o, float f, const float4 &o1) {
    o.x = fmaf(f, o1.x, o.x);
    o.y = fmaf(f, o1.y, o.y);
    o.z = fmaf(f, o1.z, o.z);
    o.w = fmaf(f, o1.w, o.w);
}

// log2 of a row's sum, in the units of the blocks' sums; a row that sees nothing gives nothing.
__device__ __forceinline__ float row_total(float m, float l) { return l == 0.f ? INFINITY : m + lg2(l * kUnit); }

// Row `r` of a group: where its output goes, and its lse.
__device__ __forceinline__ long long row_place(const DecodeArgs &a, const Where &w, int r) {
    return (long long)w.b * a.so.b + (long long)(w.h * a.G + row_head(a, r)) * a.so.h +
           (long long)row_token(a, w, r) * a.so.t;
}
__device__ __forceinline__ void write_lse(const DecodeArgs &a, const Where &w, int r, float m, float l) {
    a.lse[((long long)w.b * a.H + w.h * a.G + row_head(a, r)) * a.Tq + row_token(a, w, r)] =
        l == 0.f ? -INFINITY : (m + log2f(l * kUnit)) * kLn2;
    if (a.part.total) a.part.total[w.bh * (a.tiles * a.tile_rows) + r] = row_total(m, l);
}
// What a row's sums are multiplied by; nothing seen: zeros.
__device__ __forceinline__ float row_factor(float l) { return l == 0.f ? 0.f : 1.f / (kOutputs * l); }
__device__ __forceinline__ void write_four(__nv_bfloat16 *to, const float4 &o, float by) {
    *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16x2(o.x * by, o.y * by), pack_bf16x2(o.z * by, o.w * by));
}

// weight[j] (+)= sum over the rows of exp(block j's log-sum - the row's log-sum),
// by eight consecutive lanes a block (all lanes of a warp call it; j < 0: none).
constexpr int kWeightLanes = 8;
__device__ __forceinline__ void write_weight(const DecodeArgs &a, long long bh, int j, const float *total) {
    const int part = threadIdx.x % kWeightLanes;
    float sum = 0.f;
    if (j >= 0) {
        const float *lb = a.part.lb + (bh * a.c.blocks + j) * a.rows;
#pragma unroll 4
        for (int row = part; row < a.rows; row += kWeightLanes) sum += ex2(lb[row] - total[row]);
    }
#pragma unroll
    for (int off = 1; off < kWeightLanes; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (j >= 0 && part == 0) {
        float *out = a.c.weight + bh * a.c.blocks + j;
        *out = a.weight == 2 ? *out + sum : sum;
    }
}

// The first block that counts at place i or a whole number of steps behind it in
// a list out of order, and its place; -1: none.  Those count that are closed and
// above all closed ones before them, up to the first negative entry.  The whole
// warp calls it.
__device__ __noinline__ int2 block_out_of_order(const int32_t *list, int i, int count, int step, int closed) {
    for (; i < count; i += step) {
        const int id = list[i];
        int most = -1;
        bool ended = id < 0;
        for (int y = threadIdx.x & 31; y < i; y += 32) {
            const int other = list[y];
            ended = ended || other < 0;
            if (other < closed) most = max(most, other);
        }
        if (__any_sync(0xffffffffu, ended)) break;
        if (id < closed && id > __reduce_max_sync(0xffffffffu, most)) return make_int2(id, i);
    }
    return make_int2(-1, i);
}

template <int D, int NT, int Ctas>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT, Ctas>::kCtas) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using Sm = Smem<D, NT, Ctas>;
    constexpr int SL = Sm::kSlots, kRows = Sm::kRows, S = slab(D), kHalves = Cfg<D, NT, Ctas>::kHalves,
                  kAtOnce = Cfg<D, NT, Ctas>::kAtOnce;
    constexpr bool kShared = Cfg<D, NT, Ctas>::kQueriesInSmem;
    constexpr int kSide = kBlock * D;  // bytes of a block's keys, and of its values
    static_assert(sizeof(float) * kWarps * kRows * Sm::kPitch + sizeof(float) * kRows * D <= sizeof(Sm::ring),
                  "the outputs take no more than the rings");
    extern __shared__ uint8_t smem_raw[];
    Sm &sm = *reinterpret_cast<Sm *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    volatile int *abort = &sm.abort;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    if (lane < SL) mbar_init(&sm.full[warp][lane], 1);
    fence_mbar_init();
    if (tid == 0) sm.abort = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();

    // ---- this CTA's work: with clusters every a.cluster-th kWarps blocks of a row tile, else a run
    unsigned group, left = 1, skip = 0;  // units still to do, and those of the row tile that are not this CTA's
    int rank = 0;
    if (a.cluster) {
        group = blockIdx.x / a.cluster;
        rank = (int)(blockIdx.x - group * a.cluster);
    } else {
        const unsigned mine = lane < a.c.B ? units_of(a, lane) : 0u;
        left = units_of_run(a, mine);
        unsigned units;
        if (!tile_at(a, mine, blockIdx.x * left, group, skip, units)) return;
    }
    int slot = 0, put_slot = 0, ahead = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (true) {
        const Where w = where(a, group);
        // ---- queries: this lane's row g of the warp's row tile (on their way while the lengths are)
        uint32_t qx[D / 8];
        const int my_tile = kShared ? warp : 0, my_row = w.tile * kRows + my_tile * 8 + g;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) qx[i] = 0;
        const __nv_bfloat16 *my_q = my_tile < NT && my_row < a.rows ? query_row(a, w, my_row) : nullptr;
        if (my_q) load_row<D, true>(qx, my_q, t);
        auto queries = [&](int nt) -> const __nv_bfloat16 * {  // this lane's row of row tile nt
            if constexpr (!kShared) return my_q;
            const int row = w.tile * kRows + 8 * nt + g;
            return row < a.rows ? query_row(a, w, row) : nullptr;
        };
        int L = checked_length(a.lens[w.b], a.c.blocks, a.err);
        if (L < 0) L = 0;
        // ---- this warp's blocks: places first, first + step, ... below `count` (of all closed blocks, or of the list),
        // and its tokens of the open block: open_at, + 16 step, ... below `open`
        const int closed = L / kBlock;
        int count = a.list ? a.list_n : closed;
        int step = kWarps, first = warp, open = L - closed * kBlock, open_at = 16 * (kWarps - 1 - warp);
        if (a.cluster) {
            step = a.cluster * kWarps;
            first = rank * kWarps + warp;
            open_at = 16 * (step - 1 - first);  // the last warp of the last CTA first
            left = 0;
        } else {
            const unsigned units = (unsigned)(kPad + count + (open ? kOpen : 0)), end = min(units, skip + left);
            left -= end - skip;
            if (skip > kPad) first += (int)skip - kPad;
            // the open block goes with the first of its units
            if (skip > (unsigned)(kPad + count) || end <= (unsigned)(kPad + count)) open = 0;
            count = min(count, max(0, (int)end - kPad));
            skip = 0;
        }
        const int32_t *list = a.list ? a.list + (w.bh * a.Tq + w.r0) * a.list_n : nullptr;
        const uint8_t *kc = a.c.k_codes + w.bh * a.c.blocks * (long long)(kBlock * D);
        const uint8_t *vc = a.c.v_codes + w.bh * a.c.blocks * (long long)(kBlock * D);
        const float2 *scales = reinterpret_cast<const float2 *>(a.c.scales) + w.bh * a.c.blocks;
        // Whether the list, as far as this CTA's places go, is one of ascending closed blocks ended by negative entries
        bool in_order = true;
        if (list) {
#pragma unroll 4
            for (int i = tid; i < count; i += kThreads) {
                const int id = list[i], before = i > 0 ? list[i - 1] : -1;
                if (id >= 0 && (id >= closed || id <= before || (i > 0 && before < 0))) in_order = false;
            }
            if (!in_order) atomicExch(a.err, kErrLength);
            in_order = __syncthreads_and(in_order);
        }
        // The first block at place i or a whole number of steps behind it, or -1.
        auto block_from = [&](int &i) -> int {
            if (!list) return i < count ? i : -1;
            if (in_order) return i < count ? max(list[i], -1) : -1;
            const int2 found = block_out_of_order(list, i, count, step, closed);
            i = found.y;
            return found.x;
        };

        // ---- bulk copies run SL slots ahead of what is read: first 16 tokens of the open block, then the blocks
        int put_at = first, put_id = block_from(put_at), put_half = 0;
        auto put = [&]() {
            if (put_id < 0) return;
            if (lane == 0) {
                ATTN_DCHECK(put_id < a.c.blocks && put_slot < SL, a.err);
                uint8_t *to = sm.ring[warp][put_slot];
                uint64_t *bar = &sm.full[warp][put_slot];
                mbar_arrive_expect_tx(bar, Sm::kSlot);
                const long long from = (long long)put_id * kSide;
                if (kHalves == 1) {
                    bulk_load(to, kc + from, kSide, bar);
                    bulk_load(to + kSide, vc + from, kSide, bar);
                } else {
                    bulk_load(to, (put_half ? vc : kc) + from, kSide, bar);
                }
            }
            ++ahead;
            put_slot = put_slot + 1 == SL ? 0 : put_slot + 1;
            if (kHalves == 2) put_half ^= 1;
            if (put_half == 0) {
                put_at += step;
                put_id = block_from(put_at);
            }
        };
        auto wait = [&]() { return mbar_wait_warp(&sm.full[warp][slot], phase, a.err, abort); };
        auto next = [&]() {  // the slot is read: what is SL slots on comes in
            --ahead;
            __syncwarp();
            put();
            slot = slot + 1 == SL ? 0 : slot + 1;
            phase ^= slot == 0;
        };
        const bool tokens = open_at < open;  // (step is 4 or more: 16 tokens are all of a warp's)
        if (tokens) {
            constexpr int kBytes = 16 * D * 2;  // of 16 tokens' keys
            static_assert(2 * kBytes <= Sm::kSlot, "a slot holds 16 tokens in bf16");
            if (lane == 0) {
                const int row = (closed * kBlock + open_at) % kRing;
                ATTN_DCHECK(row <= kRing - 16, a.err);
                uint64_t *bar = &sm.full[warp][put_slot];
                mbar_arrive_expect_tx(bar, 2 * kBytes);
                bulk_load(sm.ring[warp][put_slot], a.c.recent_k + (w.bh * kRing + row) * D, kBytes, bar);
                bulk_load(sm.ring[warp][put_slot] + kBytes, a.c.recent_v + (w.bh * kRing + row) * D, kBytes, bar);
            }
            ++ahead;
            put_slot = put_slot + 1 == SL ? 0 : put_slot + 1;
        }
#pragma unroll 1
        for (int s = tokens; s < SL; ++s) put();
        int at = first, id = block_from(at);
        float2 sc = id >= 0 ? scales[id] : make_float2(0.f, 0.f);

        // ---- the queries as f16 fragments, and the factors of rows 2t, 2t + 1
        float rowf[2];
        if (my_tile < NT) {
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) mx = __vmaxu2(mx, qx[i] & 0x7fff7fffu);
            mx = max(mx & 0xffffu, mx >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // 2^e with the largest value in [2^14, 2^15); e within what a float32 power of two and its inverse hold
            int e = 14 - ((int)(mx >> 7) - 127);
            e = e > 114 ? 114 : e;
            const float up = __uint_as_float((uint32_t)(e + 127) << 23);
            const float down = __uint_as_float((uint32_t)(127 - e) << 23) * a.qscale;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qx[i]));
                qx[i] = pack_f16x2(f.x * up, f.y * up);
            }
            if constexpr (kShared) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) sm.q[my_tile][i][lane] = make_uint2(qx[2 * i], qx[2 * i + 1]);
                if (t == 0) sm.down[8 * my_tile + g] = down;
            } else {
#pragma unroll
                for (int y = 0; y < 2; ++y) rowf[y] = __shfl_sync(0xffffffffu, down, 4 * (2 * t + y));
            }
        }
        // the last position that row r of the tile sees
        auto last_seen = [&](int r) { return r < a.rows - w.tile * kRows ? L - a.Tq + row_token(a, w, w.tile * kRows + r) : -1; };
        int seen[2];
        if constexpr (kShared) {
            if (tid < kRows) sm.seen[tid] = last_seen(tid);
            __syncthreads();
        } else {
            seen[0] = last_seen(2 * t);
            seen[1] = last_seen(2 * t + 1);
        }
        // of rows 2t, 2t + 1 of a row tile: that, and their factors
        auto sees = [&](int nt, int y) {
            if constexpr (kShared)
                return sm.seen[8 * nt + 2 * t + y];
            else
                return seen[y];
        };
        auto factor = [&](int nt, int y) {
            if constexpr (kShared)
                return sm.down[8 * nt + 2 * t + y];
            else
                return rowf[y];
        };
        auto query = [&](int nt, int i) -> uint2 {
            if constexpr (kShared)
                return sm.q[nt][i][lane];
            else
                return make_uint2(qx[2 * i], qx[2 * i + 1]);
        };

        State<D, NT> st;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            st.m[nt][0] = st.m[nt][1] = -INFINITY;
            st.l[nt][0] = st.l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) st.o[i][nt][0] = st.o[i][nt][1] = st.o[i][nt][2] = st.o[i][nt][3] = 0.f;
        }

        // ---- the open block
        if (tokens && (ok = wait())) {
            const __nv_bfloat16 *k = reinterpret_cast<const __nv_bfloat16 *>(sm.ring[warp][slot]);
            open_tokens<D, NT>(st, a.qscale, queries, sees, k, k + 16 * D, closed * kBlock + open_at, L, lane);
            next();
        }

        // ---- the closed blocks
        const int all_see = L - a.Tq;  // positions up to here are seen by every query
#pragma unroll 1
        while (id >= 0 && ok) {
            int at_next = at + step;
            const int id_next = block_from(at_next);
            const float2 sc_next = id_next >= 0 ? scales[id_next] : make_float2(0.f, 0.f);
            if (!(ok = wait())) break;
            // S^T: four tiles of 16 tokens; row y of tile u is token 16 (y >> 1) + 4 u + (y & 1), row y + 8 the token two
            // further, which is the order in which a lane's 16 value bytes pair up below
            float sv[4][NT][4];
#pragma unroll
            for (int sl = 0; sl < D / S; ++sl) {
                const uint8_t *kb = sm.ring[warp][slot] + sl * (kBlock * S) + (16 * (g >> 1) + (g & 1)) * S + t * (S / 4);
#pragma unroll
                for (int u0 = 0; u0 < 4; u0 += kAtOnce) {
                    uint32_t r0[kAtOnce][S / 16], r1[kAtOnce][S / 16];
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        const uint8_t *from = kb + 4 * (u0 + u) * S;
                        if constexpr (S == 64) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(from);
                            const uint4 y = *reinterpret_cast<const uint4 *>(from + 2 * S);
                            r0[u][0] = x.x, r0[u][1] = x.y, r0[u][2] = x.z, r0[u][3] = x.w;
                            r1[u][0] = y.x, r1[u][1] = y.y, r1[u][2] = y.z, r1[u][3] = y.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2 *>(from);
                            const uint2 y = *reinterpret_cast<const uint2 *>(from + 2 * S);
                            r0[u][0] = x.x, r0[u][1] = x.y;
                            r1[u][0] = y.x, r1[u][1] = y.y;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < S / 16; ++k) {
                        uint32_t ka[kAtOnce][4];
#pragma unroll
                        for (int u = 0; u < kAtOnce; ++u) {
                            ka[u][0] = codes_f16x2<0>(r0[u][k]);
                            ka[u][1] = codes_f16x2<0>(r1[u][k]);
                            ka[u][2] = codes_f16x2<1>(r0[u][k]);
                            ka[u][3] = codes_f16x2<1>(r1[u][k]);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 q = query(nt, sl * (S / 16) + k);
#pragma unroll
                            for (int u = 0; u < kAtOnce; ++u) {
                                if (sl == 0 && k == 0)
                                    mma_f16_first(sv[u0 + u][nt], ka[u], q.x, q.y);
                                else
                                    mma_f16(sv[u0 + u][nt], ka[u], q.x, q.y);
                            }
                        }
                    }
                }
            }
            if (kHalves == 2) next();
            const int p0 = id * kBlock;
            if (p0 + kBlock - 1 > all_see) {  // only the newest positions are masked
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (p0 + 16 * (g >> 1) + 4 * u + (g & 1) + (x & 2) > sees(nt, x & 1))
                                sv[u][nt][x] = -INFINITY;
            }
            float f[NT][2], sum[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    f[nt][x] = sc.x * factor(nt, x);
                    // A factor of 0 would turn -inf into NaN.  It stands for a block of zeros, or for scores below
                    // 2^-120 (sums are below 2^29, and the factor was below 2^-149): with the smallest normal number
                    // those stay next to nothing, -inf what it is and a NaN one.
                    if (f[nt][x] == 0.f) f[nt][x] = kLeastFactor;
                }
            softmax_step<D, NT, 4>(st, sv, f, sum);
            if (a.weight) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float v = sum[nt][x];
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
                        const int row = w.tile * kRows + nt * 8 + 2 * t + x;
                        if (g == 0 && row < a.rows)
                            a.part.lb[(w.bh * a.c.blocks + id) * a.rows + row] =
                                v == 0.f ? -INFINITY : st.m[nt][x] + lg2(v * kUnit);
                    }
            }
            const float vscale = sc.y * kOutputs;
            const uint8_t *vb = sm.ring[warp][slot] + (kHalves == 2 ? 0 : kSide) + g * kBlock + 16 * t;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float least = sv[0][nt][0];
#pragma unroll
                for (int x = 1; x < 16; ++x) least = fminf(least, sv[x / 4][nt][x % 4]);
                // (a wait that runs out here does so again below)
                if (__any_sync(0xffffffffu, least < kLeastF16) && (kHalves == 1 || wait()))
                    light_weights<D, NT>(st, sv, nt, vscale, vb);
            }
            uint32_t p[4][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    p[u][nt][0] = transpose8(pack_f16x2(sv[u][nt][0], sv[u][nt][1]));
                    p[u][nt][1] = transpose8(pack_f16x2(sv[u][nt][2], sv[u][nt][3]));
                }
            // O^T: channels 16 c + g and + 8, the lane's 16 tokens 16 t ..; a block's sum is scaled as it joins the rest
            if (kHalves == 2 && !(ok = wait())) break;
#pragma unroll
            for (int c0 = 0; c0 < D / 16; c0 += kAtOnce) {
                uint32_t r0[kAtOnce][4], r1[kAtOnce][4];
                float acc[kAtOnce][NT][4];
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(vb + 16 * (c0 + c) * kBlock);
                    const uint4 y = *reinterpret_cast<const uint4 *>(vb + (16 * (c0 + c) + 8) * kBlock);
                    r0[c][0] = x.x, r0[c][1] = x.y, r0[c][2] = x.z, r0[c][3] = x.w;
                    r1[c][0] = y.x, r1[c][1] = y.y, r1[c][2] = y.z, r1[c][3] = y.w;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int c = 0; c < kAtOnce; ++c) {
                        const uint32_t va[4] = {codes_f16x2<0>(r0[c][u]), codes_f16x2<0>(r1[c][u]),
                                                codes_f16x2<1>(r0[c][u]), codes_f16x2<1>(r1[c][u])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (u == 0)
                                mma_f16_first(acc[c][nt], va, p[u][nt][0], p[u][nt][1]);
                            else
                                mma_f16(acc[c][nt], va, p[u][nt][0], p[u][nt][1]);
                        }
                    }
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            st.o[c0 + c][nt][x] = fmaf(vscale, acc[c][nt][x], st.o[c0 + c][nt][x]);
            }
            next();
            at = at_next;
            id = id_next;
            sc = sc_next;
        }
        if (!ok) {
            // A wait ran out: this warp's copies in flight land before its shared memory is used again.
            for (; ahead > 0; --ahead) {
                if (lane == 0) mbar_wait_drain(&sm.full[warp][slot], phase);
                slot = slot + 1 == SL ? 0 : slot + 1;
                phase ^= slot == 0;
            }
            __syncwarp();
        }

        // ---- the warps' results into one
        __syncthreads();  // every ring is empty
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float l = st.l[nt][x];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
                if (g == 0) {
                    sm.m[warp][nt * 8 + 2 * t + x] = st.m[nt][x];
                    sm.l[warp][nt * 8 + 2 * t + x] = l;
                }
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    sm.part[warp][nt * 8 + 2 * t + (x & 1)][16 * c + g + (x & 2) * 4] = st.o[c][nt][x];
        }
        __syncthreads();
        const int here = min(kRows, a.rows - w.tile * kRows);
        if (tid < here) {
            // a thread a row: its maximum and sum, the warps' factors (in their maxima's place), where it goes
            float m = -INFINITY, l = 0.f, f[kWarps];
#pragma unroll
            for (int y = 0; y < kWarps; ++y) m = fmaxf(m, sm.m[y][tid]);
            const float safe = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int y = 0; y < kWarps; ++y) {
                f[y] = ex2(sm.m[y][tid] - safe);
                l = fmaf(f[y], sm.l[y][tid], l);
            }
            const float by = a.cluster == 1 ? row_factor(l) : 1.f;
#pragma unroll
            for (int y = 0; y < kWarps; ++y) sm.m[y][tid] = f[y];
            sm.by[tid] = by;
            const int r = w.tile * kRows + tid;
            if (a.cluster) {
                sm.mc[tid] = m;
                sm.lc[tid] = l;
                sm.to[tid] = row_place(a, w, r);
                if (a.cluster == 1) write_lse(a, w, r, m, l);
            } else {
                a.part.ml[((long long)blockIdx.x + group) * kRows + tid] = make_float2(m, l);
            }
        }
        __syncthreads();
#pragma unroll 2
        for (int e = tid; e < here * (D / 4); e += kThreads) {
            const int row = e / (D / 4), ch = 4 * (e % (D / 4));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int y = 0; y < kWarps; ++y) add(o, sm.m[y][row], *reinterpret_cast<const float4 *>(&sm.part[y][row][ch]));
            if (a.cluster == 1)
                write_four(a.o + sm.to[row] + ch, o, sm.by[row]);
            else if (a.cluster)
                *reinterpret_cast<float4 *>(&sm.o[row][ch]) = o;
            else
                *reinterpret_cast<float4 *>(a.part.o + (((long long)blockIdx.x + group) * kRows + row) * D + ch) = o;
        }
        if (!a.cluster) {
            // ---- the next row tile with units
            if (left == 0) return;
            do {
                if (++group >= (unsigned)a.c.B * tiles_of_sequence(a)) return;
            } while (units_of(a, where(a, group).b) == 0);
            fence_proxy_async_smem();
            __syncthreads();  // the rings take blocks again
            continue;
        }
        // ---- the cluster's results into one, every CTA a part of them
        if (a.cluster > 1)
            cluster.sync();
        else
            __syncthreads();
        if (a.cluster > 1) {
            for (int e = rank * kThreads + tid; e < here * (D / 4); e += a.cluster * kThreads) {
                const int row = e / (D / 4), ch = 4 * (e % (D / 4));
                float ms[kMaxCluster];
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int y = 0; y < kMaxCluster; ++y) {
                    ms[y] = y < a.cluster ? *cluster.map_shared_rank(&sm.mc[row], y) : -INFINITY;
                    m = fmaxf(m, ms[y]);
                }
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                const float safe = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int y = 0; y < kMaxCluster; ++y)
                    if (y < a.cluster) {
                        const float f = ex2(ms[y] - safe);
                        l = fmaf(f, *cluster.map_shared_rank(&sm.lc[row], y), l);
                        add(o, f, *reinterpret_cast<const float4 *>(cluster.map_shared_rank(&sm.o[row][ch], y)));
                    }
                write_four(a.o + sm.to[row] + ch, o, row_factor(l));
                if (ch == 0) write_lse(a, w, w.tile * kRows + row, m, l);
            }
        }
        if (a.weigh) {
            // ---- the weights of this CTA's blocks
            if (tid < here) {
                float ms[kMaxCluster], ls[kMaxCluster];
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int y = 0; y < kMaxCluster; ++y) {
                    ms[y] = y < a.cluster ? *cluster.map_shared_rank(&sm.mc[tid], y) : -INFINITY;
                    ls[y] = y < a.cluster ? *cluster.map_shared_rank(&sm.lc[tid], y) : 0.f;
                    m = fmaxf(m, ms[y]);
                }
                const float safe = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int y = 0; y < kMaxCluster; ++y) l = fmaf(ex2(ms[y] - safe), ls[y], l);
                sm.total[tid] = row_total(m, l);
            }
            __syncthreads();
            // places rank * kWarps + (0 .. kWarps - 1) + a multiple of step are this CTA's
            constexpr int kOnce = kThreads / kWeightLanes;
            for (int e0 = 0; (e0 / kWarps) * step + rank * kWarps < closed; e0 += kOnce) {
                const int e = e0 + tid / kWeightLanes, j = (e / kWarps) * step + rank * kWarps + e % kWarps;
                write_weight(a, w.bh, j < closed ? j : -1, sm.total);
            }
        }
        if (a.cluster > 1) cluster.sync();  // the CTAs keep their shared memory until it has been read
        return;
    }
}

// Joins what the runs left of a row: blockIdx.x is its row tile, blockIdx.y its
// place there.  A row of D / 4 threads takes every kParts-th run.
constexpr int kJoinThreads = 256;
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int kRows = 8 * NT, kLanes = D / 4, kParts = kJoinThreads / kLanes;
    __shared__ float4 so[kParts][kLanes];
    __shared__ float sl[kParts], sm[kJoinThreads / 32];
    const int tid = threadIdx.x;
    const unsigned group = blockIdx.x;
    const int row = (int)blockIdx.y;
    const Where w = where(a, group);
    if (w.tile * kRows + row >= a.rows) return;
    // The lengths are there: the attention, which does not write them, waited for what came before it.
    checked_length(a.lens[w.b], a.c.blocks, a.err);  // (a sequence without units is in no run)
    int first, last;
    runs_of_tile(a, group, first, last);
    grid_dep_wait();
    grid_dep_launch();
    const float2 *ml = a.part.ml + (long long)group * kRows + row;
    const float *po = a.part.o + ((long long)group * kRows + row) * D + 4 * (tid % kLanes);
    float m = -INFINITY;
    for (int y = first + tid; y <= last; y += kJoinThreads) m = fmaxf(m, ml[(long long)y * kRows].x);
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (tid % 32 == 0) sm[tid / 32] = m;
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kJoinThreads / 32; ++y) m = fmaxf(m, sm[y]);
    const float safe = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int y = first + tid / kLanes; y <= last; y += kParts) {
        const float2 x = ml[(long long)y * kRows];
        const float f = ex2(x.x - safe);
        l = fmaf(f, x.y, l);
        add(o, f, *reinterpret_cast<const float4 *>(po + (long long)y * kRows * D));
    }
    so[tid / kLanes][tid % kLanes] = o;
    if (tid % kLanes == 0) sl[tid / kLanes] = l;
    __syncthreads();
    if (tid < kLanes) {
#pragma unroll
        for (int y = 1; y < kParts; ++y) {
            l += sl[y];
            add(o, 1.f, so[y][tid]);
        }
        const int r = w.tile * kRows + row;
        write_four(a.o + row_place(a, w, r) + 4 * tid, o, row_factor(l));
        if (tid == 0) write_lse(a, w, r, m, l);
    }
}

// The blocks' weights where a key head's rows are joined from runs, or lie in
// several row tiles.
// blockIdx.x: key head; blockIdx.y: kWeightBlocks blocks at a time.
constexpr int kWeightBlocks = 2 * kJoinThreads / kWeightLanes;
__global__ void __launch_bounds__(kJoinThreads) weight_kernel(const __grid_constant__ DecodeArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const long long bh = blockIdx.x;
    int L = a.lens[bh / a.c.H];
    if (L < 0 || L / kBlock > a.c.blocks) L = 0;  // recorded by the attention
    const int closed = L / kBlock, j0 = (int)blockIdx.y * kWeightBlocks;
    for (int j = j0 + threadIdx.x / kWeightLanes; j < j0 + kWeightBlocks; j += kWeightBlocks / 2)
        // (a key head's row tiles follow one another, so its rows do too)
        write_weight(a, bh, j < closed ? j : -1, a.part.total + bh * (a.tiles * a.tile_rows));
}

// CTAs that the GPU holds at once in clusters of 1 .. 8, with up to 1, 2 and 3
// CTAs an SM (cudaOccupancyMaxActiveClusters on B200: a cluster lies within a
// part of the GPU, and the parts' sizes leave SMs over).
constexpr int kRoom[3][kMaxCluster] = {{148, 148, 135, 132, 130, 132, 105, 120},
                                       {296, 296, 279, 284, 280, 270, 259, 264},
                                       {444, 444, 426, 416, 410, 426, 392, 384}};

// Clusters (the CTAs of one, 0: none) or runs, by what each costs in the time a
// warp takes for a block, as if every sequence filled its cache.  Clusters of n
// CTAs a row tile: the rounds that the GPU needs for all of them times the blocks
// a warp reads and kPerCta beside them.  Runs: each warp's even share of all units
// and kPerRuns for finding them and joining what they leave.  Measured (us,
// clusters / runs; row tiles x blocks): 144 x 16 8.1 / 11.8, 200 x up to 64 with
// weights 22.1 / 23.1, 32 x 257 (head size 128, 16 rows) 33.9 / 36.1, 432 x 24 (16
// rows) 22.7 / 51.5, 6 x 265 (16 rows) 17.8 / 12.7, 1 x 2048 69.3 / 12.0, 192 x up
// to 512 99.8 / 84.5.  Runs where the
// two come out alike: unequal lengths, which they even out, cost clusters more.
constexpr int kPerCta = 3, kPerRuns = 5;
// Where a run is long, two for each CTA that the GPU holds let an SM that is
// quicker than others take more of them (84.4 us against 85.6 at 230 units a run;
// 60.8 against 59.4 at 120).
constexpr int kLongRun = 100;
struct Shares {
    int cluster, runs;
};
Shares shares_for(long long tiles, int on_sm, int blocks) {
    const int(&held)[kMaxCluster] = kRoom[on_sm - 1];
    int best = 1;
    long long least = 0;
    for (int n = 1; n <= kMaxCluster; ++n) {
        if (n > 1 && (long long)(n - 1) * kWarps > blocks) break;  // warps without a block
        const long long rounds = (tiles * n + held[n - 1] - 1) / held[n - 1];
        const long long cost = rounds * ((blocks + (long long)n * kWarps - 1) / ((long long)n * kWarps) + kPerCta);
        if (n == 1 || cost < least) {
            least = cost;
            best = n;
        }
    }
    const long long units = tiles * (blocks + kPad + kOpen), each = units / held[0];
    if (units < (1ll << 31) && each / kWarps + 1 + kPerRuns <= least) return Shares{0, held[0] * (each >= kLongRun ? 2 : 1)};
    return Shares{best, 0};
}

struct Plan {
    int rows, nt, tiles, ctas;
    Shares shares;
    bool weigh;
    long long groups;  // row groups x row tiles
    size_t o, ml, total, lb, bytes;  // places in the workspace, and its size
};
Plan make_plan(const Q8Cache &c, int H, int Tq, int list_n, bool weight) {
    const bool lists = list_n > 0;
    Plan p;
    const int G = H / c.H;
    p.rows = lists ? G : G * Tq;
    p.nt = p.rows > 16 && c.D < 128 ? 4 : p.rows > 8 ? 2 : 1;
    p.tiles = (p.rows + 8 * p.nt - 1) / (8 * p.nt);
    p.groups = (long long)c.B * c.H * (lists ? Tq : 1) * p.tiles;
    p.ctas = ctas_on_sm(c.D, p.nt, p.groups > kRoom[1][0]);
    p.shares = shares_for(p.groups, p.ctas, lists ? list_n : c.blocks);  // (the kernel counts a list's places too)
    p.weigh = weight && p.shares.cluster && p.tiles == 1;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = p.shares.cluster ? 0 : (size_t)(p.groups + p.shares.runs) * 8 * p.nt;
    p.o = 0;
    p.ml = up(rows * c.D * sizeof(float));
    p.total = p.ml + up(rows * sizeof(float2));
    p.lb = p.total + (weight && !p.weigh ? up((size_t)p.groups * 8 * p.nt * sizeof(float)) : 0);
    p.bytes = p.lb + (weight ? up((size_t)c.B * c.H * p.rows * c.blocks * sizeof(float)) : 0);
    return p;
}

template <int D, int NT, int Ctas>
cudaError_t launch(const DecodeArgs &a, const Plan &p, cudaStream_t st, LaunchInfo &li) {
    int dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    // CTAs fill one SM after another, so a grid that leaves room asks for as much shared memory as keeps it spread out
    // (144 row tiles of 16 blocks in 288 CTAs: 8.4 us on 127 SMs, 7.9 us with two CTAs on each).
    const size_t smem_most = 227 * 1024;
    static std::atomic<unsigned long long> smem_set{0};
    if ((e = set_max_smem_once(reinterpret_cast<const void *>(decode_kernel<D, NT, Ctas>), smem_most, dev, smem_set)) !=
        cudaSuccess)
        return e;
    const long long grid = a.cluster ? p.groups * a.cluster : a.runs;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    size_t smem = sizeof(Smem<D, NT, Ctas>) + 128;
    for (int per = 1; per < Ctas; ++per)
        if (grid <= kRoom[per - 1][a.cluster ? a.cluster - 1 : 0]) {
            smem = smem_most / per / 1024 * 1024 - 1024;
            break;
        }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    if ((e = mark_main_start(li, st)) != cudaSuccess) return e;
    if ((e = cudaLaunchKernelEx(&cfg, decode_kernel<D, NT, Ctas>, a)) != cudaSuccess) return e;
    li.kernels += 1;
    if ((e = mark_main_end(li, st)) != cudaSuccess) return e;
    if (!a.cluster) {
        if ((e = launch_pdl(join_kernel<D, NT>, dim3((unsigned)p.groups, (unsigned)(a.rows < 8 * NT ? a.rows : 8 * NT)),
                            dim3(kJoinThreads), 0, st, a)) != cudaSuccess)
            return e;
        li.kernels += 1;
    }
    if (a.weight && !a.weigh) {
        const dim3 g((unsigned)(a.c.B * a.c.H), (unsigned)((a.c.blocks + kWeightBlocks - 1) / kWeightBlocks));
        if ((e = launch_pdl(weight_kernel, g, dim3(kJoinThreads), 0, st, a)) != cudaSuccess)
            return e;
        li.kernels += 1;
    }
    return cudaSuccess;
}

}  // namespace

size_t q8_decode_workspace(const Q8Cache &c, int H, int Tq, int list_n, bool weight) {
    return make_plan(c, H, Tq, list_n, weight).bytes;
}

cudaError_t q8_decode(const Q8Cache &c, const Q8Decode &d, int *err, cudaStream_t st, LaunchInfo &li) {
    const Plan p = make_plan(c, d.H, d.Tq, d.list_n, d.weight != 0);
    DecodeArgs a;
    a.c = c;
    a.q = d.q;
    a.sq = d.sq;
    a.o = d.o;
    a.so = d.so;
    a.lse = d.lse;
    a.lens = d.lens;
    a.list = d.list;
    a.list_n = d.list_n;
    a.H = d.H;
    a.G = d.H / c.H;
    a.Tq = d.Tq;
    a.per_tq = (65536u + d.Tq - 1) / d.Tq;
    a.rows = p.rows;
    a.tiles = p.tiles;
    a.tile_rows = 8 * p.nt;
    a.cluster = p.shares.cluster;
    a.runs = p.shares.runs;
    a.weigh = p.weigh;
    a.qscale = d.scale * kLog2e;
    a.weight = d.weight;
    char *ws = static_cast<char *>(d.workspace);
    a.part.o = reinterpret_cast<float *>(ws + p.o);
    a.part.ml = reinterpret_cast<float2 *>(ws + p.ml);
    a.part.total = d.weight && !p.weigh ? reinterpret_cast<float *>(ws + p.total) : nullptr;
    a.part.lb = reinterpret_cast<float *>(ws + p.lb);
    a.err = err;
#define ATTN_Q8_CASE(DD, NN, CC) \
    if (c.D == DD && p.nt == NN && p.ctas == CC) return launch<DD, NN, CC>(a, p, st, li);
    ATTN_Q8_CASE(32, 1, 3)
    ATTN_Q8_CASE(32, 2, 3)
    ATTN_Q8_CASE(32, 4, 2)
    ATTN_Q8_CASE(32, 4, 3)
    ATTN_Q8_CASE(64, 1, 3)
    ATTN_Q8_CASE(64, 2, 2)
    ATTN_Q8_CASE(64, 2, 3)
    ATTN_Q8_CASE(64, 4, 2)
    ATTN_Q8_CASE(128, 1, 2)
    ATTN_Q8_CASE(128, 1, 3)
    ATTN_Q8_CASE(128, 2, 2)
#undef ATTN_Q8_CASE
    return cudaErrorInvalidValue;
}

}  // namespace attn
