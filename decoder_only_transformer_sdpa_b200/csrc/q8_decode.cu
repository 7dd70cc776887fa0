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
// eight bits of anything down to 2^-31 of it.  P is rounded to f16 (half a
// step: 2^-11, less than the bf16 output's 2^-9) after scaling by 2^14, so
// weights down to 2^-28 of the largest keep that precision.  Sums of P, the
// scores and both accumulators are float32.
//
// What bounds it is the stream of codes, 128 D bytes a block: every warp has a
// ring of its own in shared memory, filled by bulk copies that its first lane
// issues, so a warp never waits for another and some 100 to 190 KB are in
// flight on an SM.  Blocks go to the warps of a row group's CTAs in turn.
// The open block is read in bf16 from the ring of recent positions, 16 tokens
// a warp, with exact products and P as the sum of two bf16 numbers.
#include "q8_cache.cuh"

namespace attn {
namespace {

using namespace sm100;
using namespace q8;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kPShift = 14.f;  // P is held as 2^14 p

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
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
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(a));
    return w;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 w;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(a));
    return w;
}

// Warps of a CTA and stages of a warp's ring, by head size: 192 KB of rings at
// D = 64 and 128, 128 KB at D = 32.
template <int D>
struct Cfg {
    static constexpr int kWarps = D == 128 ? 6 : 8;
    static constexpr int kStages = D == 128 ? 2 : (D == 64 ? 3 : 4);
};

// Layout of the workspace: each CTA's unnormalised output and its running
// maximum (log2 units) and sum per row, then each block's log2-sum per row
// (only when the blocks' weights are kept).
struct Parts {
    float *o;    // [tile][split][rows][D]
    float2 *ml;  // [tile][split][rows]
    float *lb;   // [B * Hkv][R][blocks]
};

template <int D, int NT>
struct Smem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kStage = 2 * kBlock * D;
    static constexpr int kPitch = D + 4;  // rows of partial outputs: four rows apart are on other banks
    // the rings, then (once they are empty) [warp][row][kPitch] partial outputs
    alignas(128) uint8_t ring[Cfg<D>::kWarps][Cfg<D>::kStages][kStage];
    uint64_t full[Cfg<D>::kWarps][Cfg<D>::kStages];
    float m[Cfg<D>::kWarps][kRows], l[Cfg<D>::kWarps][kRows];
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
    int rows;       // rows of a group: G * Tq, or G with lists (a group is then one token)
    int tiles;      // row tiles of a group
    int splits;     // CTAs that share a row tile
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
// Head in the group and token of row `row` of a group.
__device__ __forceinline__ int row_head(const DecodeArgs &a, int row) { return a.list ? row : row / a.Tq; }
__device__ __forceinline__ int row_token(const DecodeArgs &a, const Where &w, int row) {
    return a.list ? w.r0 : row % a.Tq;
}

// Running softmax state of a warp: this lane's rows 2t and 2t + 1 of each row
// tile (t = lane % 4), and O^T with channels 16 i + g, + 8 (g = lane / 4).
template <int D, int NT>
struct State {
    float m[NT][2], l[NT][2];
    float o[D / 16][NT][4];
};

// Folds scores s[i][nt] (log2 units; -inf where masked) of 16 * Tiles tokens
// into the running maximum and replaces them by 2^14 exp2(s - max).  Returns
// the sums of this lane's weights in `sum`.
template <int D, int NT, int Tiles>
__device__ __forceinline__ void softmax_step(State<D, NT> &st, float (&s)[Tiles][NT][4], float (&sum)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float base[2], alpha[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float mx = s[0][nt][x];
#pragma unroll
            for (int i = 0; i < Tiles; ++i) mx = fmaxf(mx, fmaxf(s[i][nt][x], s[i][nt][x + 2]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float m_new = fmaxf(st.m[nt][x], mx);
            const float safe = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet
            alpha[x] = ex2(st.m[nt][x] - safe);
            base[x] = safe - kPShift;
            st.m[nt][x] = m_new;
            sum[nt][x] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < Tiles; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[i][nt][x] = ex2(s[i][nt][x] - base[x & 1]);
                sum[nt][x & 1] += s[i][nt][x];
            }
#pragma unroll
        for (int x = 0; x < 2; ++x) st.l[nt][x] = fmaf(st.l[nt][x], alpha[x], sum[nt][x]);
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) st.o[i][nt][x] *= alpha[x & 1];
        }
    }
}

// One bf16 row chunk of the lane: channels slab * S + (S / 4) t + 0 .. S / 4 - 1.
template <int D>
__device__ __forceinline__ void load_row(uint32_t (&w)[D / 8], const __nv_bfloat16 *row, int t) {
    constexpr int S = slab(D);
#pragma unroll
    for (int i = 0; i < D / 8; i += 4) {  // four words = eight channels
        const int sl = i / (S / 8), in = i % (S / 8);
        const uint4 x = *reinterpret_cast<const uint4 *>(row + sl * S + (S / 4) * t + 2 * in);
        w[i] = x.x;
        w[i + 1] = x.y;
        w[i + 2] = x.z;
        w[i + 3] = x.w;
    }
}

// 16 tokens of the open block, positions p0 .. p0 + 15 of a sequence of length L.
template <int D, int NT>
__device__ __forceinline__ void open_tokens(State<D, NT> &st, const DecodeArgs &a, const Where &w,
                                            const __nv_bfloat16 *(&qrow)[NT], const int (&sees)[NT][2], int p0,
                                            int L, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const __nv_bfloat16 *rk = a.c.recent_k + w.bh * kRing * D, *rv = a.c.recent_v + w.bh * kRing * D;
    float s[1][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[0][nt][0] = s[0][nt][1] = s[0][nt][2] = s[0][nt][3] = 0.f;
    uint32_t k0[D / 8], k1[D / 8];  // tokens p0 + g and p0 + g + 8
#pragma unroll
    for (int i = 0; i < D / 8; ++i) k0[i] = k1[i] = 0;
    if (p0 + g < L) load_row<D>(k0, rk + ((p0 + g) % kRing) * D, t);
    if (p0 + g + 8 < L) load_row<D>(k1, rk + ((p0 + g + 8) % kRing) * D, t);
    // values: the pairs of tokens (2t, 2t + 1) and (2t + 8, 2t + 9) of channels 16 i + g and + 8; rows past the
    // end are not read
    uint32_t va[D / 16][4];
    uint32_t odd = 0;  // an infinity or a NaN among them
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int tok = p0 + 2 * t + (x & 2) * 4, ch = 16 * i + g + (x & 1) * 8;
            uint32_t lo = 0, hi = 0;
            if (tok < L) lo = *reinterpret_cast<const uint16_t *>(rv + (tok % kRing) * D + ch);
            if (tok + 1 < L) hi = *reinterpret_cast<const uint16_t *>(rv + ((tok + 1) % kRing) * D + ch);
            if ((lo & 0x7f80u) == 0x7f80u) {
                odd = 1;
                lo = 0;
            }
            if ((hi & 0x7f80u) == 0x7f80u) {
                odd = 1;
                hi = 0;
            }
            va[i][x] = lo | (hi << 16);
        }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint32_t q[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) q[i] = 0;
        if (qrow[nt]) load_row<D>(q, qrow[nt], t);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint32_t ka[4] = {k0[2 * i], k1[2 * i], k0[2 * i + 1], k1[2 * i + 1]};
            mma_bf16(s[0][nt], ka, q[2 * i], q[2 * i + 1]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int p = p0 + g + (x & 2) * 4;
            s[0][nt][x] = p <= sees[nt][x & 1] ? s[0][nt][x] * a.qscale : -INFINITY;
        }
    }
    float sum[NT][2];
    softmax_step<D, NT, 1>(st, s, sum);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        // P as a bf16 number and what that leaves, another one
        const uint32_t h0 = pack_bf16x2(s[0][nt][0], s[0][nt][1]), h1 = pack_bf16x2(s[0][nt][2], s[0][nt][3]);
        const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&h0));
        const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&h1));
        const uint32_t r0 = pack_bf16x2(s[0][nt][0] - f0.x, s[0][nt][1] - f0.y);
        const uint32_t r1 = pack_bf16x2(s[0][nt][2] - f1.x, s[0][nt][3] - f1.y);
        const uint32_t b0 = transpose8(h0), b1 = transpose8(h1), c0 = transpose8(r0), c1 = transpose8(r1);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            mma_bf16(st.o[i][nt], va[i], b0, b1);
            mma_bf16(st.o[i][nt], va[i], c0, c1);
        }
    }
    if (__any_sync(0xffffffffu, odd != 0)) {
        // Infinities and NaN reach only the rows that see their token: added one by one, never as 0 * inf.
        for (int y = 0; y < 16; ++y) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int src = 4 * (y & 7) + t;
                const float pa = __shfl_sync(0xffffffffu, y < 8 ? s[0][nt][0] : s[0][nt][2], src);
                const float pb = __shfl_sync(0xffffffffu, y < 8 ? s[0][nt][1] : s[0][nt][3], src);
                if (p0 + y < L) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float f = __bfloat162float(rv[((p0 + y) % kRing) * D + 16 * i + g + (x & 2) * 4]);
                            if ((!isfinite(f)) && p0 + y <= sees[nt][x & 1])
                                st.o[i][nt][x] = fmaf((x & 1) ? pb : pa, f, st.o[i][nt][x]);
                        }
                }
            }
        }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * Cfg<D>::kWarps) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using Sm = Smem<D, NT>;
    constexpr int W = Cfg<D>::kWarps, ST = Cfg<D>::kStages, kThreads = 32 * W;
    constexpr int S = slab(D);
    constexpr int kRows = 8 * NT;
    static_assert(sizeof(float) * kRows * Sm::kPitch <= (size_t)ST * Sm::kStage, "partial outputs fit the rings");
    extern __shared__ uint8_t smem_raw[];
    Sm &sm = *reinterpret_cast<Sm *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    volatile int *abort = &sm.abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const unsigned group = blockIdx.x / a.splits;  // (row group, row tile)
    const int split = (int)(blockIdx.x - group * a.splits);
    const Where w = where(a, group);
    if (lane == 0) {
        for (int s = 0; s < ST; ++s) mbar_init(&sm.full[warp][s], 1);
        fence_mbar_init();
    }
    if (tid == 0) sm.abort = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    int L = checked_length(a.lens, w.b, a.c.blocks, a.err);
    if (L < 0) L = 0;

    // ---- this warp's blocks: `first`, + step, ... below `count` (of all closed blocks, or of the list)
    const int closed = L / kBlock;
    const int step = a.splits * W, first = split * W + warp;
    const int count = a.list ? a.list_n : closed;
    const int32_t *list = a.list ? a.list + (w.bh * a.Tq + w.r0) * a.list_n : nullptr;
    const uint8_t *kc = a.c.k_codes + w.bh * a.c.blocks * (long long)(kBlock * D);
    const uint8_t *vc = a.c.v_codes + w.bh * a.c.blocks * (long long)(kBlock * D);
    const float2 *scales = reinterpret_cast<const float2 *>(a.c.scales) + w.bh * a.c.blocks;
    // The block at place i of the list, or -1.  What is not an ascending list of closed blocks ended by -1 is
    // recorded, and the entry skipped.
    auto block_at = [&](int i) -> int {
        if (i >= count) return -1;
        if (!list) return i;
        const int id = list[i];
        if (id < 0) return -1;
        const int before = i > 0 ? list[i - 1] : -1;
        if (id >= closed || id <= before || (i > 0 && before < 0)) {
            if (lane == 0) atomicExch(a.err, kErrLength);
            return -1;
        }
        return id;
    };
    auto issue = [&](int stage, int id) {
        if (lane == 0 && id >= 0) {
            ATTN_DCHECK(id < a.c.blocks, a.err);
            uint8_t *dst = sm.ring[warp][stage];
            mbar_arrive_expect_tx(&sm.full[warp][stage], Sm::kStage);
            bulk_load(dst, kc + (long long)id * (kBlock * D), kBlock * D, &sm.full[warp][stage]);
            bulk_load(dst + kBlock * D, vc + (long long)id * (kBlock * D), kBlock * D, &sm.full[warp][stage]);
        }
    };
    int ids[ST];
    float2 sc[ST];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        ids[s] = block_at(first + s * step);
        issue(s, ids[s]);
        sc[s] = ids[s] >= 0 ? scales[ids[s]] : make_float2(0.f, 0.f);
    }

    // ---- queries: fragments of this lane's row g of each row tile, and the factors of rows 2t, 2t + 1
    uint32_t qf[NT][D / 8];
    const __nv_bfloat16 *qrow[NT];
    float rowf[NT][2];
    int sees[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = w.tile * kRows + nt * 8 + g;
        qrow[nt] = nullptr;
        uint32_t x[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) x[i] = 0;
        if (row < a.rows) {
            qrow[nt] = a.q + (long long)w.b * a.sq.b + (long long)(w.h * a.G + row_head(a, row)) * a.sq.h +
                       (long long)row_token(a, w, row) * a.sq.t;
            load_row<D>(x, qrow[nt], t);
        }
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) mx = __vmaxu2(mx, x[i] & 0x7fff7fffu);
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
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x[i]));
            qf[nt][i] = pack_f16x2(f.x * up, f.y * up);
        }
#pragma unroll
        for (int x2 = 0; x2 < 2; ++x2) {
            rowf[nt][x2] = __shfl_sync(0xffffffffu, down, 4 * (2 * t + x2));
            const int r = w.tile * kRows + nt * 8 + 2 * t + x2;
            sees[nt][x2] = r < a.rows ? L - a.Tq + row_token(a, w, r) : -1;
        }
    }

    State<D, NT> st;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        st.m[nt][0] = st.m[nt][1] = -INFINITY;
        st.l[nt][0] = st.l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[i][nt][0] = st.o[i][nt][1] = st.o[i][nt][2] = st.o[i][nt][3] = 0.f;
    }
    const int all_see = L - a.Tq;  // positions up to here are seen by every query

    // ---- the closed blocks
    bool ok = true;
    uint32_t phase = 0;
    for (int base = first; base < count && ok; base += ST * step) {
#pragma unroll
        for (int s = 0; s < ST; ++s) {
            const int i = base + s * step;
            if (i >= count) break;
            const int id = ids[s];
            if (id >= 0) {
                if (!(ok = mbar_wait_warp(&sm.full[warp][s], phase, a.err, abort))) break;
                const uint32_t kb = smem_u32(sm.ring[warp][s]), vb = kb + kBlock * D;
                // S^T: four tiles of 16 tokens; row y of tile u is token 16 (y >> 1) + 4 u + (y & 1), row y + 8 the
                // token two further, which is the order in which a lane's 16 value bytes pair up below
                float sv[4][NT][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sv[u][nt][0] = sv[u][nt][1] = sv[u][nt][2] = sv[u][nt][3] = 0.f;
                    const int tok = 16 * (g >> 1) + 4 * u + (g & 1);
#pragma unroll
                    for (int sl = 0; sl < D / S; ++sl) {
                        uint32_t r0[S / 16], r1[S / 16];
                        const uint32_t at = kb + sl * (kBlock * S) + tok * S + t * (S / 4);
                        if constexpr (S == 64) {
                            const uint4 x = lds128(at), y = lds128(at + 2 * S);
                            r0[0] = x.x, r0[1] = x.y, r0[2] = x.z, r0[3] = x.w;
                            r1[0] = y.x, r1[1] = y.y, r1[2] = y.z, r1[3] = y.w;
                        } else {
                            const uint2 x = lds64(at), y = lds64(at + 2 * S);
                            r0[0] = x.x, r0[1] = x.y;
                            r1[0] = y.x, r1[1] = y.y;
                        }
#pragma unroll
                        for (int k = 0; k < S / 16; ++k) {
                            const uint32_t ka[4] = {codes_f16x2<0>(r0[k]), codes_f16x2<0>(r1[k]),
                                                    codes_f16x2<1>(r0[k]), codes_f16x2<1>(r1[k])};
                            const int f = 2 * (sl * (S / 16) + k);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_f16(sv[u][nt], ka, qf[nt][f], qf[nt][f + 1]);
                        }
                    }
                }
                const float ks = sc[s].x, vs = sc[s].y;
                const int p0 = id * kBlock;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float f0 = ks * rowf[nt][0], f1 = ks * rowf[nt][1];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int x = 0; x < 4; ++x) sv[u][nt][x] *= (x & 1) ? f1 : f0;
                }
                if (p0 + kBlock - 1 > all_see) {  // only the newest positions are masked
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (p0 + 16 * (g >> 1) + 4 * u + (g & 1) + (x & 2) > sees[nt][x & 1])
                                    sv[u][nt][x] = -INFINITY;
                }
                float sum[NT][2];
                softmax_step<D, NT, 4>(st, sv, sum);
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
                                a.part.lb[(w.bh * a.rows + row) * a.c.blocks + id] =
                                    v == 0.f ? -INFINITY : st.m[nt][x] + log2f(v);
                        }
                }
                uint32_t p[4][NT][2];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        p[u][nt][0] = transpose8(pack_f16x2(sv[u][nt][0], sv[u][nt][1]));
                        p[u][nt][1] = transpose8(pack_f16x2(sv[u][nt][2], sv[u][nt][3]));
                    }
                // O^T: channels 16 c + g and + 8, the lane's 16 tokens 16 t ..
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const uint32_t at = vb + (16 * c + g) * kBlock + 16 * t;
                    const uint4 x = lds128(at), y = lds128(at + 8 * kBlock);
                    const uint32_t r0[4] = {x.x, x.y, x.z, x.w}, r1[4] = {y.x, y.y, y.z, y.w};
                    float acc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t va[4] = {codes_f16x2<0>(r0[u]), codes_f16x2<0>(r1[u]), codes_f16x2<1>(r0[u]),
                                                codes_f16x2<1>(r1[u])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], va, p[u][nt][0], p[u][nt][1]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x2 = 0; x2 < 4; ++x2) st.o[c][nt][x2] = fmaf(vs, acc[nt][x2], st.o[c][nt][x2]);
                }
                __syncwarp();
            }
            // the stage is read: the block ST places on comes in (a skipped place leaves its barrier's phase
            // where it is, so it ends the warp's blocks: lists end at their first -1, and bad entries are errors)
            ids[s] = id >= 0 ? block_at(i + ST * step) : -1;
            issue(s, ids[s]);
            sc[s] = ids[s] >= 0 ? scales[ids[s]] : make_float2(0.f, 0.f);
        }
        phase ^= 1;
    }
    if (!ok) {
        // a wait ran out: this warp's copies in flight land before its shared memory is used again
        if (lane == 0) {
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                if (ids[s] >= 0) mbar_wait_drain(&sm.full[warp][s], phase), mbar_wait_drain(&sm.full[warp][s], phase ^ 1);
            }
        }
        __syncwarp();
    }

    // ---- the open block, 16 tokens a warp, the last warp of the last CTA first
    const int open = L - closed * kBlock;
    for (int u = step - 1 - first; 16 * u < open; u += step)
        open_tokens<D, NT>(st, a, w, qrow, sees, closed * kBlock + 16 * u, L, lane);

    // ---- the warps' results into one
    __syncthreads();  // every ring is empty
    float *part = reinterpret_cast<float *>(&sm.ring[0][0][0]);
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
                part[(warp * kRows + nt * 8 + 2 * t + (x & 1)) * Sm::kPitch + 16 * c + g + (x & 2) * 4] =
                    st.o[c][nt][x];
    }
    __syncthreads();
    const int here = min(kRows, a.rows - w.tile * kRows);
    for (int e = tid; e < here * (D / 4); e += kThreads) {
        const int row = e / (D / 4), ch = 4 * (e % (D / 4));
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int y = 0; y < W; ++y) m = fmaxf(m, sm.m[y][row]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const float safe = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int y = 0; y < W; ++y) {
            const float f = ex2(sm.m[y][row] - safe);
            const float4 x = *reinterpret_cast<const float4 *>(part + (y * kRows + row) * Sm::kPitch + ch);
            l = fmaf(f, sm.l[y][row], l);
            o.x = fmaf(f, x.x, o.x);
            o.y = fmaf(f, x.y, o.y);
            o.z = fmaf(f, x.z, o.z);
            o.w = fmaf(f, x.w, o.w);
        }
        const long long at = ((long long)group * a.splits + split) * kRows + row;
        *reinterpret_cast<float4 *>(a.part.o + at * D + ch) = o;
        if (ch == 0) a.part.ml[at] = make_float2(m, l);
    }
}

// Joins the CTAs of each row tile: o, lse, and with `weight` the blocks'
// attention weights.  One CTA a row tile (and, with weights, kWeightCtas a key
// head in blockIdx.y).
constexpr int kJoinThreads = 128;
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int kRows = 8 * NT;
    const int tid = threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    const unsigned group = blockIdx.x;
    const Where w = where(a, group);
    const int here = min(kRows, a.rows - w.tile * kRows);
    for (int e = tid; e < here * (D / 4); e += kJoinThreads) {
        const int row = e / (D / 4), ch = 4 * (e % (D / 4));
        const long long at = (long long)group * a.splits * kRows + row;
        float m = -INFINITY, l = 0.f;
        for (int y = 0; y < a.splits; ++y) m = fmaxf(m, a.part.ml[at + y * kRows].x);
        const float safe = m == -INFINITY ? 0.f : m;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int y = 0; y < a.splits; ++y) {
            const float2 ml = a.part.ml[at + y * kRows];
            const float4 x = *reinterpret_cast<const float4 *>(a.part.o + (at + y * kRows) * D + ch);
            const float f = ex2(ml.x - safe);
            l = fmaf(f, ml.y, l);
            o.x = fmaf(f, x.x, o.x);
            o.y = fmaf(f, x.y, o.y);
            o.z = fmaf(f, x.z, o.z);
            o.w = fmaf(f, x.w, o.w);
        }
        const int r = w.tile * kRows + row;
        const int head = w.h * a.G + row_head(a, r), tok = row_token(a, w, r);
        const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing seen: zeros
        *reinterpret_cast<uint2 *>(a.o + (long long)w.b * a.so.b + (long long)head * a.so.h +
                                   (long long)tok * a.so.t + ch) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (ch == 0)
            a.lse[((long long)w.b * a.H + head) * a.Tq + tok] =
                l == 0.f ? -INFINITY : (m + (log2f(l) - kPShift)) * kLn2;
    }
}

// weight[j] (+)= sum over rows of exp(block j's log-sum - the row's log-sum).
// blockIdx.x: key head; blockIdx.y: 128 blocks at a time.
template <int NT>
__global__ void __launch_bounds__(kJoinThreads) weight_kernel(const __grid_constant__ DecodeArgs a) {
    constexpr int kRows = 8 * NT;
    extern __shared__ float total[];  // [rows] log2 of each row's sum
    grid_dep_wait();
    grid_dep_launch();
    const long long bh = blockIdx.x;
    const int b = (int)(bh / a.c.H);
    int L = a.lens[b];
    if (L < 0 || L / kBlock > a.c.blocks) L = 0;  // recorded by the attention
    const int closed = L / kBlock;
    if ((int)blockIdx.y * kJoinThreads >= closed) return;
    for (int row = threadIdx.x; row < a.rows; row += kJoinThreads) {
        const long long at = ((bh * a.tiles + row / kRows) * a.splits) * kRows + row % kRows;
        float m = -INFINITY, l = 0.f;
        for (int y = 0; y < a.splits; ++y) m = fmaxf(m, a.part.ml[at + y * kRows].x);
        const float safe = m == -INFINITY ? 0.f : m;
        for (int y = 0; y < a.splits; ++y) {
            const float2 ml = a.part.ml[at + y * kRows];
            l = fmaf(ex2(ml.x - safe), ml.y, l);
        }
        total[row] = l == 0.f ? INFINITY : m + log2f(l);  // a row that sees nothing gives nothing
    }
    __syncthreads();
    const int j = (int)blockIdx.y * kJoinThreads + threadIdx.x;
    if (j >= closed) return;
    float sum = 0.f;
    for (int row = 0; row < a.rows; ++row) sum += ex2(a.part.lb[(bh * a.rows + row) * a.c.blocks + j] - total[row]);
    float *out = a.c.weight + bh * a.c.blocks + j;
    *out = a.weight == 2 ? *out + sum : sum;
}

// CTAs that share a row tile: enough to fill the GPU's 148 SMs, no more than
// give every warp a block.
int splits_for(long long tiles, int D, int blocks) {
    const int warps = D == 128 ? Cfg<128>::kWarps : Cfg<64>::kWarps;
    const long long most = (blocks + warps) / warps;  // the open block is a unit of work too
    long long n = 148 / tiles;
    n = n < 1 ? 1 : n;
    return (int)(n > most ? most : n);
}

struct Plan {
    int rows, nt, tiles, splits;
    long long groups;  // row groups x row tiles
    size_t o, ml, lb, total;
};
Plan make_plan(const Q8Cache &c, int H, int Tq, int list_n, bool lists, bool weight) {
    Plan p;
    const int G = H / c.H;
    p.rows = lists ? G : G * Tq;
    p.nt = p.rows > 8 ? 2 : 1;
    p.tiles = (p.rows + 8 * p.nt - 1) / (8 * p.nt);
    p.groups = (long long)c.B * c.H * (lists ? Tq : 1) * p.tiles;
    p.splits = splits_for(p.groups, c.D, lists ? (list_n < c.blocks ? list_n : c.blocks) : c.blocks);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = (size_t)p.groups * p.splits * 8 * p.nt;
    p.o = 0;
    p.ml = up(rows * c.D * sizeof(float));
    p.lb = p.ml + up(rows * sizeof(float2));
    p.total = p.lb + (weight ? up((size_t)c.B * c.H * p.rows * c.blocks * sizeof(float)) : 0);
    return p;
}

template <int D, int NT>
cudaError_t launch(const DecodeArgs &a, const Plan &p, cudaStream_t st, LaunchInfo &li) {
    int dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const size_t smem = sizeof(Smem<D, NT>) + 128;
    static std::atomic<unsigned long long> smem_set{0};
    if ((e = set_max_smem_once(reinterpret_cast<const void *>(decode_kernel<D, NT>), smem, dev, smem_set)) !=
        cudaSuccess)
        return e;
    const long long grid = p.groups * p.splits;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if ((e = mark_main_start(li, st)) != cudaSuccess) return e;
    if ((e = launch_pdl(decode_kernel<D, NT>, dim3((unsigned)grid), dim3(32 * Cfg<D>::kWarps), smem, st, a)) !=
        cudaSuccess)
        return e;
    if ((e = mark_main_end(li, st)) != cudaSuccess) return e;
    if ((e = launch_pdl(join_kernel<D, NT>, dim3((unsigned)p.groups), dim3(kJoinThreads), 0, st, a)) != cudaSuccess)
        return e;
    li.kernels += 2;
    if (a.weight) {
        const dim3 g((unsigned)(a.c.B * a.c.H), (unsigned)((a.c.blocks + kJoinThreads - 1) / kJoinThreads));
        if ((e = launch_pdl(weight_kernel<NT>, g, dim3(kJoinThreads), a.rows * sizeof(float), st, a)) != cudaSuccess)
            return e;
        li.kernels += 1;
    }
    return cudaSuccess;
}

}  // namespace

size_t q8_decode_workspace(const Q8Cache &c, int H, int Tq, int list_n, bool weight) {
    return make_plan(c, H, Tq, list_n, list_n > 0, weight).total;
}

cudaError_t q8_decode(const Q8Cache &c, const Q8Decode &d, int *err, cudaStream_t st, LaunchInfo &li) {
    const bool lists = d.list != nullptr;
    const Plan p = make_plan(c, d.H, d.Tq, d.list_n, lists, d.weight != 0);
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
    a.rows = p.rows;
    a.tiles = p.tiles;
    a.splits = p.splits;
    a.qscale = d.scale * kLog2e;
    a.weight = d.weight;
    char *ws = static_cast<char *>(d.workspace);
    a.part.o = reinterpret_cast<float *>(ws + p.o);
    a.part.ml = reinterpret_cast<float2 *>(ws + p.ml);
    a.part.lb = reinterpret_cast<float *>(ws + p.lb);
    a.err = err;
#define ATTN_Q8_CASE(DD, NN) \
    if (c.D == DD && p.nt == NN) return launch<DD, NN>(a, p, st, li);
    ATTN_Q8_CASE(32, 1)
    ATTN_Q8_CASE(32, 2)
    ATTN_Q8_CASE(64, 1)
    ATTN_Q8_CASE(64, 2)
    ATTN_Q8_CASE(128, 1)
    ATTN_Q8_CASE(128, 2)
#undef ATTN_Q8_CASE
    return cudaErrorInvalidValue;
}

}  // namespace attn
