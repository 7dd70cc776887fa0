// q8_select.cu -- choosing blocks of the 8-bit cache: by a cheap score for a
// query (which blocks to attend to), and by the attention weight they have
// received (which blocks to keep).
//
// Both come down to the n largest of up to 32768 numbers a head, ties to the
// lowest index, listed in ascending order: one CTA a list holds the numbers'
// order keys in shared memory and finds the n-th largest by its bytes, from
// the highest one (a histogram of the keys that agree so far).
//
// The score of block J for query q is a bound on its keys' products with q,
// with q in 8 bits too: c = rint(127 q / max|q|),
//   dot_J = sum_d max(c_d lo_Jd, c_d hi_Jd)     (whole numbers, exact)
//   score_J = (dot_J * kscale_J) * (max|q| / 127)
// with the smallest and largest key code of each channel, and the largest
// score over the heads of a group.  It reads 2 D bytes a block, 1/64 of it;
// the positive c take `hi` and the negative ones `lo`, so that it is two
// four-way byte products for four channels.
#include "q8_cache.cuh"

namespace attn {
namespace {

using namespace sm100;
using namespace q8;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct SelectSmem {
    uint32_t hist[256];
    uint32_t warp_sum[kWarps];
    uint32_t bin, above;
    uint32_t above_n[kWarps], equal_n[kWarps];
};

// Writes the places of the n largest of key[0 .. count - 1] to list, ascending,
// and -1 behind them up to n.  The whole CTA calls it; keys are complete.
__device__ void largest(const uint32_t *key, int count, int n, int32_t *list, SelectSmem &sm) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t least = 0, ties = 0xffffffffu;  // keys above `least` are in, and the first `ties` that equal it
    if (count > n) {
        uint32_t prefix = 0, want = (uint32_t)n;
        for (int shift = 24; shift >= 0; shift -= 8) {
            sm.hist[tid] = 0;
            __syncthreads();
            const uint32_t high = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int i = tid; i < count; i += kThreads) {
                const uint32_t x = key[i];
                if ((x & high) == prefix) atomicAdd(&sm.hist[(x >> shift) & 255u], 1u);
            }
            __syncthreads();
            // bin 255 - tid, summed from the highest bin down
            const uint32_t mine = sm.hist[255 - tid];
            uint32_t sum = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += o;
            }
            if (lane == 31) sm.warp_sum[warp] = sum;
            __syncthreads();
            for (int y = 0; y < warp; ++y) sum += sm.warp_sum[y];
            if (sum >= want && sum - mine < want) {
                sm.bin = (uint32_t)(255 - tid);
                sm.above = sum - mine;
            }
            __syncthreads();
            prefix |= sm.bin << shift;
            want -= sm.above;
        }
        least = prefix;
        ties = want;
    }
    // ---- the list, kThreads keys at a time
    uint32_t out = 0, equal_seen = 0;
    for (int base = 0; base < count; base += kThreads) {
        const int i = base + tid;
        const uint32_t x = i < count ? key[i] : 0u;
        const bool all = count <= n;
        const bool above = i < count && (all || x > least), equal = i < count && !all && x == least;
        const uint32_t am = __ballot_sync(0xffffffffu, above), em = __ballot_sync(0xffffffffu, equal);
        __syncthreads();
        if (lane == 0) {
            sm.above_n[warp] = __popc(am);
            sm.equal_n[warp] = __popc(em);
        }
        __syncthreads();
        uint32_t a = 0, e = 0, a_all = 0, e_all = 0;
#pragma unroll
        for (int y = 0; y < kWarps; ++y) {
            if (y < warp) a += sm.above_n[y], e += sm.equal_n[y];
            a_all += sm.above_n[y], e_all += sm.equal_n[y];
        }
        const uint32_t below = (1u << lane) - 1u;
        a += __popc(am & below);
        e += equal_seen + __popc(em & below);  // equal keys before this one
        const uint32_t taken = min(e, ties) - min(equal_seen, ties);  // of those, in this round, that are in
        if (above || (equal && e < ties)) list[out + a + taken] = i;
        out += a_all + (min(equal_seen + e_all, ties) - min(equal_seen, ties));
        equal_seen += e_all;
    }
    for (int i = (int)out + tid; i < n; i += kThreads) list[i] = -1;
}

// ---- by score.  One CTA a key head and new token.
template <int D>
__global__ void __launch_bounds__(kThreads)
    select_kernel(const Q8Cache c, const __nv_bfloat16 *__restrict__ q, const TStrides sq,
                  const int32_t *__restrict__ lens, int32_t *__restrict__ lists, int n, int G, int Tq, int *err) {
    __shared__ SelectSmem sm;
    extern __shared__ uint32_t dyn[];
    uint32_t *key = dyn;                                            // [blocks]
    uint32_t *pos = dyn + (c.blocks + 3) / 4 * 4;                   // [G][D / 4] codes above zero
    uint32_t *neg = pos + G * (D / 4);                              // [G][D / 4] codes below zero
    float *qs = reinterpret_cast<float *>(neg + G * (D / 4));       // [G] max|q| / 127
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = (int)(blockIdx.x % Tq);
    const long long bh = blockIdx.x / Tq;
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    grid_dep_wait();
    grid_dep_launch();
    int L = checked_length(lens, b, c.blocks, err);
    if (L < 0) L = 0;
    const int last = L - Tq + r;  // the query's own position
    const int count = last < 0 ? 0 : min(L / kBlock, last / kBlock + 1);
    int32_t *list = lists + ((long long)blockIdx.x) * n;
    if (count > n) {
        // ---- the queries' codes, a warp a head, four channels a lane
        for (int x = warp; x < G; x += kWarps) {
            uint2 w = make_uint2(0, 0);
            if (lane < D / 4)
                w = *reinterpret_cast<const uint2 *>(q + (long long)b * sq.b + (long long)(h * G + x) * sq.h +
                                                     (long long)r * sq.t + 4 * lane);
            uint32_t m = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
            m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
            const float most = __uint_as_float(m << 16);
            const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.x));
            const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.y));
            const float f[4] = {f0.x, f0.y, f1.x, f1.y};
            uint32_t p = 0, ng = 0;
            if (m != 0 && m < 0x7f80u) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int code = code_number(f[y], most);
                    p |= (uint32_t)(max(code, 0) & 255) << (8 * y);
                    ng |= (uint32_t)(min(code, 0) & 255) << (8 * y);
                }
            }
            if (lane < D / 4) {
                pos[x * (D / 4) + lane] = p;
                neg[x * (D / 4) + lane] = ng;
            }
            if (lane == 0) qs[x] = __fdiv_rn(most, 127.f);  // an infinity or a NaN stays one
        }
        __syncthreads();
        // ---- the scores: D / 16 lanes a block, 16 channels each
        constexpr int kLanes = D / 16;
        const int part = tid % kLanes;
        for (int j0 = 0; j0 < count; j0 += kThreads / kLanes) {
            const int j = j0 + tid / kLanes;
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            float ks = 0.f;
            if (j < count) {
                const long long at = bh * c.blocks + j;
                const uint4 *e = reinterpret_cast<const uint4 *>(c.bounds + at * (2 * D));
                lo = e[part];
                hi = e[kLanes + part];
                ks = c.scales[2 * at];
            }
            const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
            float best = -INFINITY;
            bool none = false;
            for (int x = 0; x < G; ++x) {
                int dot = 0;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    dot = __dp4a((int)pos[x * (D / 4) + 4 * part + y], (int)hw[y], dot);
                    dot = __dp4a((int)neg[x * (D / 4) + 4 * part + y], (int)lw[y], dot);
                }
#pragma unroll
                for (int off = 1; off < kLanes; off <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
                const float score = __fmul_rn(__fmul_rn((float)dot, ks), qs[x]);
                none = none || score != score;
                best = fmaxf(best, score);
            }
            if (part == 0 && j < count) key[j] = none ? kFirst - 1 : order_key(best);
        }
        __syncthreads();
    }
    largest(key, count, n, list, sm);
}

// ---- by weight.  One CTA a key head; `state` takes twice the count of kept
// blocks, plus one if an odd count goes, and the sequence's new length (-1
// where the length is out of range): the lengths themselves may be overwritten
// while the blocks move.
__global__ void __launch_bounds__(kThreads)
    keep_kernel(const Q8Cache c, const int32_t *__restrict__ lens, int32_t *__restrict__ kept, int keep, int sink,
                int recent, int *__restrict__ state, int *err) {
    __shared__ SelectSmem sm;
    extern __shared__ uint32_t key[];
    const long long bh = blockIdx.x;
    const int b = (int)(bh / c.H);
    grid_dep_wait();
    grid_dep_launch();
    const int L = checked_length(lens, b, c.blocks, err);
    const int closed = L < 0 ? 0 : L / kBlock;
    const float *weight = c.weight + bh * c.blocks;
    if (closed > keep) {
        for (int j = threadIdx.x; j < closed; j += kThreads)
            key[j] = (j < sink || j >= closed - recent) ? kFirst : order_key(weight[j]);
        __syncthreads();
    }
    largest(key, closed, keep, kept + bh * keep, sm);
    if (threadIdx.x == 0) {
        const int left = closed < keep ? closed : keep;
        state[2 * bh] = L < 0 ? 0 : 2 * left + ((closed - left) & 1);
        state[2 * bh + 1] = L < 0 ? -1 : left * kBlock + L % kBlock;
    }
}

// ---- the kept blocks to the front (of the same cache, or of another one).
// A CTA moves one 1 KB slice of each block's codes, in ascending order and with
// all of a round's loads before its stores, so that blocks may move within one
// cache: a block's new place is never behind its old one.  The CTA of the last
// slice moves everything else.
constexpr int kSlice = 1024;
constexpr int kAtOnce = kThreads / (kSlice / 16);  // blocks whose slices a CTA moves side by side
constexpr int kRounds = 8;

template <int D>
__global__ void __launch_bounds__(kThreads)
    move_kernel(const Q8Cache c, const Q8Cache d, const int32_t *__restrict__ lens, int32_t *__restrict__ lens_out,
                const int32_t *__restrict__ kept, int keep, const int *__restrict__ state, int chunks, int *err) {
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
    const int count = state[2 * bh] >> 1, length = state[2 * bh + 1];
    const bool odd = state[2 * bh] & 1;
    const int32_t *from = kept + bh * keep;
    // this chunk's blocks: all of them when they move within one cache
    const int per = (keep + chunks - 1) / chunks;
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
    for (int i0 = begin; i0 < end; i0 += kThreads) {
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
        for (int e0 = begin * kWords; e0 < end * kWords; e0 += kThreads) {
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
    if (h == 0 && tid == 0) lens_out[b] = length < 0 ? lens[b] : length;
    if (length < 0) return;
    // ---- the ring: position p lies in row p % 128, so its halves change places when an odd count of blocks goes
    if (same && !odd) return;
    constexpr int kChunks = kBlock * D / 8;  // 16-byte chunks of a half
    const int other = odd ? kChunks : 0;
    const uint4 *sk = reinterpret_cast<const uint4 *>(c.recent_k) + bh * 2 * kChunks;
    const uint4 *sv = reinterpret_cast<const uint4 *>(c.recent_v) + bh * 2 * kChunks;
    uint4 *dk = reinterpret_cast<uint4 *>(d.recent_k) + bh * 2 * kChunks;
    uint4 *dv = reinterpret_cast<uint4 *>(d.recent_v) + bh * 2 * kChunks;
    for (int e = tid; e < kChunks; e += kThreads) {  // a thread alone reads and writes both halves' chunk e
        const uint4 k0 = sk[e], k1 = sk[kChunks + e], v0 = sv[e], v1 = sv[kChunks + e];
        dk[other + e] = k0;
        dk[kChunks - other + e] = k1;
        dv[other + e] = v0;
        dv[kChunks - other + e] = v1;
    }
}

}  // namespace

cudaError_t q8_select(const Q8Cache &c, const __nv_bfloat16 *q, const TStrides &sq, const int32_t *lens,
                      int32_t *list, int list_n, int H, int Tq, int *err, cudaStream_t st, LaunchInfo &li) {
    const int G = H / c.H;
    const long long grid = (long long)c.B * c.H * Tq;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const size_t smem = ((size_t)(c.blocks + 3) / 4 * 4 + 2 * (size_t)G * (c.D / 4) + G) * 4;
    const void *fn = c.D == 32 ? (const void *)select_kernel<32>
                               : c.D == 64 ? (const void *)select_kernel<64> : (const void *)select_kernel<128>;
    int dev = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    static std::atomic<unsigned long long> smem_set[3];
    const size_t most = ((size_t)kQ8MaxBlocks + 2 * kQ8MaxGroup * (128 / 4) + kQ8MaxGroup) * 4;
    if ((e = set_max_smem_once(fn, most, dev, smem_set[c.D == 32 ? 0 : c.D == 64 ? 1 : 2])) != cudaSuccess) return e;
    if ((e = mark_main_start(li, st)) != cudaSuccess) return e;
    const dim3 g((unsigned)grid), t(kThreads);
    if (c.D == 32)
        e = launch_pdl(select_kernel<32>, g, t, smem, st, c, q, sq, lens, list, list_n, G, Tq, err);
    else if (c.D == 64)
        e = launch_pdl(select_kernel<64>, g, t, smem, st, c, q, sq, lens, list, list_n, G, Tq, err);
    else
        e = launch_pdl(select_kernel<128>, g, t, smem, st, c, q, sq, lens, list, list_n, G, Tq, err);
    if (e != cudaSuccess) return e;
    li.kernels += 1;
    return mark_main_end(li, st);
}

cudaError_t q8_evict(const Q8Cache &src, const Q8Cache &dst, const int32_t *lens, int32_t *lens_out, int32_t *kept,
                     int keep, int sink, int recent, int *workspace, int *err, cudaStream_t st, LaunchInfo &li) {
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
    const int chunks = src.k_codes == dst.k_codes ? 1 : (keep + kAtOnce * kRounds - 1) / (kAtOnce * kRounds);
    const long long grid = heads * slices * chunks;
    if (heads > 0x7fffffffLL || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if ((e = launch_pdl(keep_kernel, dim3((unsigned)heads), dim3(kThreads), (size_t)src.blocks * 4, st, src, lens, kept,
                        keep, sink, recent, workspace, err)) != cudaSuccess)
        return e;
    if ((e = mark_main_start(li, st)) != cudaSuccess) return e;
    const dim3 g((unsigned)grid), t(kThreads);
    if (src.D == 32)
        e = launch_pdl(move_kernel<32>, g, t, 0, st, src, dst, lens, lens_out, kept, keep, workspace, chunks, err);
    else if (src.D == 64)
        e = launch_pdl(move_kernel<64>, g, t, 0, st, src, dst, lens, lens_out, kept, keep, workspace, chunks, err);
    else
        e = launch_pdl(move_kernel<128>, g, t, 0, st, src, dst, lens, lens_out, kept, keep, workspace, chunks, err);
    if (e != cudaSuccess) return e;
    li.kernels += 2;
    return mark_main_end(li, st);
}

}  // namespace attn
