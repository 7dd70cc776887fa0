// q8_select.cu -- choosing blocks of the 8-bit cache: by a cheap score for a
// query (which blocks to attend to), and by the attention weight they have
// received (which blocks to keep).
//
// Both come down to the n largest of up to 32768 numbers a head, ties to the
// lowest index, listed in ascending order: one CTA a list holds the numbers'
// order keys in shared memory and finds the n-th largest ten bits at a time,
// from the highest bit in which any two keys differ (a histogram of the keys
// that agree so far; starting at the top bits, which scores of one size share,
// every key would count in one bin).  Up to 256 keys are ranked by comparing each
// with each instead, which has two barriers and not some twelve (choice and decode
// over 128 blocks 10.3 us against 11.3, eviction of 16 blocks and reading 17.7
// against 20.1).
//
// The score of block J for query q is a bound on its keys' products with q,
// with q in 8 bits too: c = rint(127 q / max|q|),
//   dot_J = sum_d max(c_d lo_Jd, c_d hi_Jd)     (whole numbers, exact)
//   score_J = (dot_J * kscale_J) * (max|q| / 127)
// with the smallest and largest key code of each channel, and the largest
// score over the heads of a group.  It reads 2 D bytes a block, 1/64 of it;
// the positive c take `hi` and the negative ones `lo`, so that it is two
// four-way byte products for four channels.  The CTAs of a cluster share a
// list's blocks and write their scores into the first one's shared memory.
#include "q8_cache.cuh"

#include <cooperative_groups.h>

namespace attn {
namespace {

using namespace sm100;
using namespace q8;

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

constexpr int kBits = 10;  // of a pass: two bins a thread
static_assert(1 << kBits == 2 * kThreads, "two bins a thread");

constexpr int kRanked = 256;  // up to so many keys are ranked by comparing each with each

struct SelectSmem {
    alignas(8) uint32_t hist[1 << kBits];
    uint32_t low[kWarps], high[kWarps], sum[kWarps], ties[kWarps];
    uint32_t bin, above, in_bin;
};

// Sum of x over the threads before this one, with `total` over all.
__device__ __forceinline__ uint32_t sum_before(uint32_t x, uint32_t *of_warp, uint32_t &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t upto = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
    }
    if (lane == 31) of_warp[warp] = upto;
    __syncthreads();
    uint32_t before = upto - x;
    total = 0;
#pragma unroll
    for (int y = 0; y < kWarps; ++y) {
        if (y < warp) before += of_warp[y];
        total += of_warp[y];
    }
    return before;
}

// Writes the places of the n largest of key[0 .. count - 1] to list, ascending,
// and -1 behind them up to n.  The whole CTA calls it; keys are complete.
__device__ void largest(const uint32_t *key, int count, int n, int32_t *list, SelectSmem &sm) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (count <= n) {
        for (int i = tid; i < n; i += kThreads) list[i] = i < count ? i : -1;
        return;
    }
    if (count <= kRanked) {
        // ---- few keys: each one's rank, its comparisons shared by the threads of one index
        const int width = count <= kRanked / 2 ? kRanked / 2 : kRanked, parts = kThreads / width;
        const int i = tid % width, per = (count + parts - 1) / parts, j0 = tid / width * per, j1 = min(count, j0 + per);
        const uint32_t mine = i < count ? key[i] : 0u;
        uint32_t rank = 0;
#pragma unroll 8
        for (int j = j0; j < j1; ++j) {
            const uint32_t x = key[j];
            rank += x > mine || (x == mine && j < i);
        }
        sm.hist[tid] = rank;
        __syncthreads();
        for (int y = 1; y < parts; ++y) rank += sm.hist[(tid + y * width) % kThreads];
        const bool in = tid < count && rank < (uint32_t)n;
        const uint32_t together = __ballot_sync(0xffffffffu, in);
        if (lane == 0) sm.sum[warp] = __popc(together);
        __syncthreads();
        uint32_t out = __popc(together & ((1u << lane) - 1u));
        for (int y = 0; y < warp; ++y) out += sm.sum[y];
        if (in) list[out] = tid;
        return;
    }
    // ---- the bits in which keys differ
    uint32_t low = 0xffffffffu, high = 0;
    for (int i = tid; i < count; i += kThreads) {
        low = min(low, key[i]);
        high = max(high, key[i]);
    }
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
        sm.low[warp] = low;
        sm.high[warp] = high;
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kWarps; ++y) {
        low = min(low, sm.low[y]);
        high = max(high, sm.high[y]);
    }
    int bits = 32 - __clz(low ^ high);  // bits not yet known of the n-th largest key
    uint32_t prefix = bits == 32 ? 0u : high >> bits << bits, want = (uint32_t)n;
    while (bits > 0) {
        const int shift = max(0, bits - kBits);
        const uint32_t known = bits == 32 ? 0u : 0xffffffffu << bits;
        *reinterpret_cast<uint2 *>(&sm.hist[2 * tid]) = make_uint2(0u, 0u);
        __syncthreads();
        for (int i = tid; i < count; i += kThreads) {
            const uint32_t x = key[i];
            if ((x & known) == prefix) atomicAdd(&sm.hist[(x & ~known) >> shift], 1u);
        }
        __syncthreads();
        // thread t holds the t-th pair of bins from the top, so that sums run from the highest bin down
        const int pair = kThreads - 1 - tid;
        const uint2 mine = *reinterpret_cast<const uint2 *>(&sm.hist[2 * pair]);
        uint32_t total;
        uint32_t above = sum_before(mine.x + mine.y, sm.sum, total);
        if (above < want && above + mine.y + mine.x >= want) {
            const bool upper = above + mine.y >= want;
            sm.bin = (uint32_t)(2 * pair + upper);
            sm.above = upper ? above : above + mine.y;
            sm.in_bin = upper ? mine.y : mine.x;
        }
        __syncthreads();
        prefix |= sm.bin << shift;
        want -= sm.above;
        bits = shift;
        if (sm.in_bin == want) break;  // all of the bin is in
    }
    // keys from `prefix + 2^bits` on are in, and the first `want` of those from `prefix` on (all of them, where bits > 0)
    const uint32_t span = (1u << bits) - 1u;
    // ---- the list: a thread takes consecutive keys
    const int per = (count + kThreads - 1) / kThreads, i0 = min(count, tid * per), i1 = min(count, i0 + per);
    uint32_t above = 0, equal = 0, all;
    for (int i = i0; i < i1; ++i) {
        const uint32_t x = key[i];
        if (x >= prefix) {
            if (x - prefix <= span)
                ++equal;
            else
                ++above;
        }
    }
    const uint32_t above_before = sum_before(above, sm.sum, all), equal_before = sum_before(equal, sm.ties, all);
    uint32_t out = above_before + min(equal_before, want), seen = equal_before;
    for (int i = i0; i < i1; ++i) {
        const uint32_t x = key[i];
        if (x >= prefix && (x - prefix > span || seen++ < want)) list[out++] = i;
    }
}

// ---- by score.  One cluster a key head and new token.  64 registers a thread, so
// that an SM holds two CTAs (at 84 it held one: 384 lists of 2048 blocks 35.1 us,
// now 28.2).
template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    select_kernel(const Q8Cache c, const __nv_bfloat16 *__restrict__ q, const TStrides sq,
                  const int32_t *__restrict__ lens, int32_t *__restrict__ lists, int n, int G, int Tq, int ctas,
                  int *err) {
    constexpr int kLanes = D / 16;       // lanes of a block, 16 channels each
    constexpr int kAtOnce = 4;           // blocks a lane loads before it computes
    __shared__ SelectSmem sm;
    extern __shared__ uint4 dyn[];
    uint4 *pos = dyn;                                               // [G][D / 16] codes above zero
    uint4 *neg = pos + G * kLanes;                                  // [G][D / 16] codes below zero
    float *qs = reinterpret_cast<float *>(neg + G * kLanes);        // [G] max|q| / 127
    uint32_t *key = reinterpret_cast<uint32_t *>(qs + G);           // [blocks]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned which = blockIdx.x / ctas;
    const int rank = (int)(blockIdx.x - which * ctas);
    const int r = (int)(which % Tq);
    const long long bh = which / Tq;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    // (waited for before another CTA's shared memory is written; nothing is passed on by it)
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    grid_dep_wait();
    grid_dep_launch();
    // ---- this lane's first blocks and query channels are on their way while the length is (within the cache, whatever
    // the length)
    const int part = tid % kLanes;
    constexpr int kRow = kThreads / kLanes;  // blocks of a step
    uint4 lo[kAtOnce], hi[kAtOnce];
    float ks[kAtOnce];
    auto load = [&](int j0, int end) {
#pragma unroll
        for (int y = 0; y < kAtOnce; ++y) {
            const int j = j0 + y * kRow + tid / kLanes;
            lo[y] = hi[y] = make_uint4(0, 0, 0, 0);
            ks[y] = 0.f;
            if (j < end) {
                const long long at = bh * c.blocks + j;
                const uint4 *e = reinterpret_cast<const uint4 *>(c.bounds + at * (2 * D));
                lo[y] = e[part];
                hi[y] = e[kLanes + part];
                ks[y] = c.scales[2 * at];
            }
        }
    };
    const int step = kRow * kAtOnce;
    load(rank * step, c.blocks);
    const int L = max(0, checked_length(lens[b], c.blocks, err));
    if (ctas > 1) asm volatile("barrier.cluster.wait;" ::: "memory");  // the cluster's CTAs have all started
    const int last = L - Tq + r;  // the query's own position
    const int count = last < 0 ? 0 : min(L / kBlock, last / kBlock + 1);
    if (count > n) {  // (the same in all CTAs of the cluster)
        // ---- the queries' codes, a warp a head, four channels a lane
        for (int x = warp; x < G; x += kWarps) {
            uint2 w = make_uint2(0, 0);
            if (lane < D / 4)
                w = *reinterpret_cast<const uint2 *>(q + (long long)b * sq.b + (long long)(h * G + x) * sq.h +
                                                     (long long)r * sq.t + 4 * lane);
            uint32_t m = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
            m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
            const float most = __uint_as_float(m << 16);
            uint32_t p = 0, ng = 0;
            if (m != 0 && m < 0x7f80u) {
                const uint32_t codes = Coder(most)(w.x, w.y);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int code = (int)((codes >> (8 * y)) & 255u) - 128;
                    p |= (uint32_t)(max(code, 0) & 255) << (8 * y);
                    ng |= (uint32_t)(min(code, 0) & 255) << (8 * y);
                }
            }
            if (lane < D / 4) {
                reinterpret_cast<uint32_t *>(pos)[x * (D / 4) + lane] = p;
                reinterpret_cast<uint32_t *>(neg)[x * (D / 4) + lane] = ng;
            }
            if (lane == 0) qs[x] = __fdiv_rn(most, 127.f);  // an infinity or a NaN stays one
        }
        __syncthreads();
        // ---- the scores
        uint32_t *to = ctas > 1 ? cg::this_cluster().map_shared_rank(key, 0) : key;
        for (int j0 = rank * step; j0 < count; j0 += ctas * step) {
            if (j0 != rank * step) load(j0, count);
            float best[kAtOnce];
            bool none[kAtOnce];
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
                best[y] = -INFINITY;
                none[y] = false;
            }
            for (int x = 0; x < G; ++x) {
                const uint4 p = pos[x * kLanes + part], m = neg[x * kLanes + part];
                const float scale = qs[x];
#pragma unroll
                for (int y = 0; y < kAtOnce; ++y) {
                    int dot = __dp4a((int)p.x, (int)hi[y].x, __dp4a((int)m.x, (int)lo[y].x, 0));
                    dot = __dp4a((int)p.y, (int)hi[y].y, __dp4a((int)m.y, (int)lo[y].y, dot));
                    dot = __dp4a((int)p.z, (int)hi[y].z, __dp4a((int)m.z, (int)lo[y].z, dot));
                    dot = __dp4a((int)p.w, (int)hi[y].w, __dp4a((int)m.w, (int)lo[y].w, dot));
#pragma unroll
                    for (int off = 1; off < kLanes; off <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
                    const float score = __fmul_rn(__fmul_rn((float)dot, ks[y]), scale);
                    none[y] = none[y] || score != score;
                    best[y] = fmaxf(best[y], score);
                }
            }
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
                const int j = j0 + y * kRow + tid / kLanes;
                if (part == 0 && j < count) to[j] = none[y] ? kFirst - 1 : order_key(best[y]);
            }
        }
        if (ctas > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    }
    if (rank == 0) largest(key, count, n, lists + (long long)which * n, sm);
}

// What becomes of a sequence of length L (-1: out of range, it stays as it is).
struct Fate {
    int kept, length, odd;  // blocks it keeps, its new length, whether an odd count of blocks goes
};
__device__ __forceinline__ Fate fate_of(int L, int keep) {
    if (L < 0) return Fate{0, -1, 0};
    const int closed = L / kBlock, kept = min(closed, keep);
    return Fate{kept, kept * kBlock + L % kBlock, (closed - kept) & 1};
}

// ---- by weight.  One CTA a key head.  Where the new lengths take the old ones'
// place, `fates` keeps what the kernel that moves the blocks has to know of them.
__global__ void __launch_bounds__(kThreads)
    keep_kernel(const Q8Cache c, const int32_t *__restrict__ lens, int32_t *__restrict__ kept, int keep, int sink,
                int recent, Fate *__restrict__ fates, int *err) {
    __shared__ SelectSmem sm;
    extern __shared__ uint32_t key[];
    const long long bh = blockIdx.x;
    const int b = (int)(bh / c.H);
    grid_dep_wait();
    grid_dep_launch();
    const int L = checked_length(lens[b], c.blocks, err);
    const int closed = L < 0 ? 0 : L / kBlock;
    const float *weight = c.weight + bh * c.blocks;
    if (closed > keep) {
        for (int j = threadIdx.x; j < closed; j += kThreads)
            key[j] = (j < sink || j >= closed - recent) ? kFirst : order_key(weight[j]);
        __syncthreads();
    }
    largest(key, closed, keep, kept + bh * keep, sm);
    if (fates && threadIdx.x == 0) fates[bh] = fate_of(L, keep);
}

// ---- the kept blocks to the front (of the same cache, or of another one).
// A CTA moves one 1 KB slice of each block's codes, in ascending order and with
// all of a round's loads before its stores, so that blocks may move within one
// cache: a block's new place is never behind its old one.  The CTA of the last
// slice moves everything else.
constexpr int kSlice = 1024;
constexpr int kMoveThreads = 256;
constexpr int kAtOnce = kMoveThreads / (kSlice / 16);  // blocks whose slices a CTA moves side by side
constexpr int kRounds = 8;

template <int D>
__global__ void __launch_bounds__(kMoveThreads)
    move_kernel(const Q8Cache c, const Q8Cache d, const int32_t *__restrict__ lens, int32_t *__restrict__ lens_out,
                const int32_t *__restrict__ kept, int keep, const Fate *__restrict__ fates, int chunks, int *err) {
    constexpr int kBytes = kBlock * D;            // codes of a block's keys
    constexpr int kSlices = 2 * kBytes / kSlice;
    const int tid = threadIdx.x;
    const int slice = (int)(blockIdx.x % (kSlices + 1));
    const unsigned rest = blockIdx.x / (kSlices + 1);
    const int chunk = (int)(rest % chunks);
    const long long bh = rest / chunks;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    const bool same = c.k_codes == d.k_codes;
    grid_dep_wait();
    grid_dep_launch();
    const int L = fates ? 0 : lens[b];
    const Fate fate = fates ? fates[bh] : fate_of(L >= 0 && L / kBlock <= c.blocks ? L : -1, keep);
    const int count = fate.kept;
    const int32_t *from = kept + bh * keep;
    // this chunk's blocks: all of them when they move within one cache
    const int per = (min(keep, c.blocks) + chunks - 1) / chunks;
    const int begin = chunk * per, end = min(count, begin + per);
    ATTN_DCHECK(count <= d.blocks && count <= keep && (!same || chunks == 1), err);
    if (slice < kSlices) {
        const bool values = slice >= kSlices / 2;
        const long long off = (long long)(slice % (kSlices / 2)) * kSlice + 16 * (tid % (kSlice / 16));
        const uint8_t *src = (values ? c.v_codes : c.k_codes) + bh * c.blocks * (long long)kBytes + off;
        uint8_t *dst = (values ? d.v_codes : d.k_codes) + bh * d.blocks * (long long)kBytes + off;
        for (int i0 = begin; i0 < end; i0 += kAtOnce * kRounds) {
            uint4 x[kRounds];
#pragma unroll
            for (int y = 0; y < kRounds; ++y) {
                const int i = i0 + y * kAtOnce + tid / (kSlice / 16);
                if (i < end) x[y] = *reinterpret_cast<const uint4 *>(src + (long long)from[i] * kBytes);
            }
            if (same) __syncthreads();
#pragma unroll
            for (int y = 0; y < kRounds; ++y) {
                const int i = i0 + y * kAtOnce + tid / (kSlice / 16);
                if (i < end) *reinterpret_cast<uint4 *>(dst + (long long)i * kBytes) = x[y];
            }
            if (same) __syncthreads();
        }
        return;
    }
    // ---- scales, bounds and weight
    for (int i0 = begin; i0 < end; i0 += kMoveThreads) {
        const int i = i0 + tid;
        float2 s = make_float2(0.f, 0.f);
        float w = 0.f;
        if (i < end) {
            s = reinterpret_cast<const float2 *>(c.scales)[bh * c.blocks + from[i]];
            w = c.weight[bh * c.blocks + from[i]];
        }
        if (same) __syncthreads();
        if (i < end) {
            reinterpret_cast<float2 *>(d.scales)[bh * d.blocks + i] = s;
            if (d.weight) d.weight[bh * d.blocks + i] = w;
        }
        if (same) __syncthreads();
    }
    if (d.bounds) {
        constexpr int kWords = 2 * D / 16;  // 16-byte words of a block's bounds
        for (int e0 = begin * kWords; e0 < end * kWords; e0 += kMoveThreads) {
            const int e = e0 + tid, i = e / kWords;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (e < end * kWords)
                x = reinterpret_cast<const uint4 *>(c.bounds)[(bh * c.blocks + from[i]) * kWords + e % kWords];
            if (same) __syncthreads();
            if (e < end * kWords) reinterpret_cast<uint4 *>(d.bounds)[(bh * d.blocks + i) * kWords + e % kWords] = x;
            if (same) __syncthreads();
        }
    }
    if (chunk != 0) return;
    if (h == 0 && tid == 0) lens_out[b] = fate.length < 0 ? lens[b] : fate.length;
    if (fate.length < 0) return;
    // ---- the ring: position p lies in row p % 128, so its halves change places when an odd count of blocks goes
    if (same && !fate.odd) return;
    constexpr int kChunks = kBlock * D / 8;  // 16-byte chunks of a half
    const int other = fate.odd ? kChunks : 0;
    const uint4 *sk = reinterpret_cast<const uint4 *>(c.recent_k) + bh * 2 * kChunks;
    const uint4 *sv = reinterpret_cast<const uint4 *>(c.recent_v) + bh * 2 * kChunks;
    uint4 *dk = reinterpret_cast<uint4 *>(d.recent_k) + bh * 2 * kChunks;
    uint4 *dv = reinterpret_cast<uint4 *>(d.recent_v) + bh * 2 * kChunks;
    for (int e = tid; e < kChunks; e += kMoveThreads) {  // a thread alone reads and writes both halves' chunk e
        const uint4 k0 = sk[e], k1 = sk[kChunks + e], v0 = sv[e], v1 = sv[kChunks + e];
        dk[other + e] = k0;
        dk[kChunks - other + e] = k1;
        dv[other + e] = v0;
        dv[kChunks - other + e] = v1;
    }
}

}  // namespace

size_t q8_evict_workspace(const Q8Cache &c) { return (size_t)c.B * c.H * sizeof(Fate); }

cudaError_t q8_select(const Q8Cache &c, const __nv_bfloat16 *q, const TStrides &sq, const int32_t *lens,
                      int32_t *list, int list_n, int H, int Tq, int *err, cudaStream_t st, LaunchInfo &li) {
    const int G = H / c.H;
    const long long grid = (long long)c.B * c.H * Tq;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    size_t smem = ((size_t)c.blocks + 2 * (size_t)G * (c.D / 4) + G) * 4;
    // CTAs of a cluster: a step of 512 threads takes 16 D^-1 * 512 * 4 blocks; as many as there are steps, while the
    // GPU's 148 SMs have one for each CTA (an SM holds two, so every cluster finds room at once).  Against clusters
    // that fill two CTAs an SM (us, 148 / 259 CTAs): 96 lists of 2048 blocks 10.2 / 11.4, 64 of 8 heads of 128
    // channels 16.3 / 17.9, 144 10.4 / 10.4, 48 10.7 / 9.2.
    const int step = kThreads / (c.D / 16) * 4;
    int ctas = (int)(148 / grid);
    ctas = ctas > kMaxCluster ? kMaxCluster : ctas < 1 ? 1 : ctas;
    if (ctas > (c.blocks + step - 1) / step) ctas = (c.blocks + step - 1) / step;
    // CTAs fill one SM after another, so where each has one it asks for more than half of the shared memory: a decode
    // that follows starts where the choice leaves room, and else finds its clusters crowded onto the SMs without one
    // (choice and decode of 64 lists of 128 channels 23.9 us, now 21.2; of 96 over up to 2048 blocks 30.7, now 27.6).
    const size_t more_than_half = 120 * 1024;
    if (grid * ctas <= 148 && smem < more_than_half) smem = more_than_half;
    const void *fn = c.D == 32 ? (const void *)select_kernel<32>
                               : c.D == 64 ? (const void *)select_kernel<64> : (const void *)select_kernel<128>;
    int dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    static std::atomic<unsigned long long> smem_set[3];
    const size_t most = ((size_t)kQ8MaxBlocks + 2 * kQ8MaxGroup * (128 / 4) + kQ8MaxGroup) * 4;
    if ((e = set_max_smem_once(fn, most, dev, smem_set[c.D == 32 ? 0 : c.D == 64 ? 1 : 2])) != cudaSuccess) return e;
    if ((e = mark_main_start(li, st)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    if (c.D == 32)
        e = cudaLaunchKernelEx(&cfg, select_kernel<32>, c, q, sq, lens, list, list_n, G, Tq, ctas, err);
    else if (c.D == 64)
        e = cudaLaunchKernelEx(&cfg, select_kernel<64>, c, q, sq, lens, list, list_n, G, Tq, ctas, err);
    else
        e = cudaLaunchKernelEx(&cfg, select_kernel<128>, c, q, sq, lens, list, list_n, G, Tq, ctas, err);
    if (e != cudaSuccess) return e;
    li.kernels += 1;
    return mark_main_end(li, st);
}

cudaError_t q8_evict(const Q8Cache &src, const Q8Cache &dst, const int32_t *lens, int32_t *lens_out, int32_t *kept,
                     int keep, int sink, int recent, void *workspace, int *err, cudaStream_t st, LaunchInfo &li) {
    Fate *fates = lens_out == lens ? static_cast<Fate *>(workspace) : nullptr;
    int dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    static std::atomic<unsigned long long> smem_set{0};
    if ((e = set_max_smem_once(reinterpret_cast<const void *>(keep_kernel), (size_t)kQ8MaxBlocks * 4, dev, smem_set)) !=
        cudaSuccess)
        return e;
    const long long heads = (long long)src.B * src.H;
    const int slices = 2 * kQ8Block * src.D / kSlice + 1;
    // Within one cache a head's blocks move in one run; into another one they
    // are cut into chunks of 32, a round of a CTA's loads.
    const int most = keep < src.blocks ? keep : src.blocks;
    const int chunks = src.k_codes == dst.k_codes ? 1 : (most + kAtOnce * kRounds - 1) / (kAtOnce * kRounds);
    const long long grid = heads * slices * chunks;
    if (heads > 0x7fffffffLL || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if ((e = launch_pdl(keep_kernel, dim3((unsigned)heads), dim3(kThreads), (size_t)src.blocks * 4, st, src, lens, kept,
                        keep, sink, recent, fates, err)) != cudaSuccess)
        return e;
    if ((e = mark_main_start(li, st)) != cudaSuccess) return e;
    const dim3 g((unsigned)grid), t(kMoveThreads);
    if (src.D == 32)
        e = launch_pdl(move_kernel<32>, g, t, 0, st, src, dst, lens, lens_out, kept, keep, fates, chunks, err);
    else if (src.D == 64)
        e = launch_pdl(move_kernel<64>, g, t, 0, st, src, dst, lens, lens_out, kept, keep, fates, chunks, err);
    else
        e = launch_pdl(move_kernel<128>, g, t, 0, st, src, dst, lens, lens_out, kept, keep, fates, chunks, err);
    if (e != cudaSuccess) return e;
    li.kernels += 2;
    return mark_main_end(li, st);
}

}  // namespace attn
