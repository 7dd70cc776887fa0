// q8_append.cu -- new tokens into the 8-bit block cache, and the cache's
// contents back out.
//
// Append: sequence b ends up lens[b] tokens long, of which the last new_lens[b]
// are rows 0 .. of k and v.  One CTA takes one block of 64 positions that the
// new tokens touch.  When the block is full it gathers its 64 tokens (those
// that came earlier from the bf16 ring, the others from k and v), finds the
// two maxima, and writes codes, scales and the smallest and largest key code of
// each channel.  The CTA of the oldest touched block, the only one that reads
// the ring, also writes the newest positions into it once it has read.
//
// The work is a stream: 4 D bytes read and 2 D written for a token.
#include "q8_cache.cuh"

namespace attn {
namespace {

using namespace sm100;
using namespace q8;

// Threads of a CTA: four or eight 16-byte chunks each of keys and values a
// thread at D = 64 and 128, since most of a thread's work on two is what goes
// with any number of them (128 threads take 3.2 us less than 256 for 144 heads of
// 1024 tokens at D = 64, now 13.4 us for a floor of 8.6, and 6 us less for 8 heads
// of 16411, 12308 and 8206 tokens at D = 128, now 37.6 us for 34.6).
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of bf16 pairs; NaN stays
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The larger |x| of a pair as its 15 bits, which grow with it; infinities and NaN come out on top.
__device__ __forceinline__ uint32_t top(uint32_t pair) {
    return max(pair & 0x7fffu, (pair >> 16) & 0x7fffu);
}
// Byte y of four words as a word, for y = 0 .. 3.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
    const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
    const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
    w[0] = __byte_perm(a, b, 0x5410);
    w[1] = __byte_perm(a, b, 0x7632);
    w[2] = __byte_perm(c, d, 0x5410);
    w[3] = __byte_perm(c, d, 0x7632);
}

template <int D>
struct AppendSmem {
    // values' codes, [token][channel]; the pad puts tokens eight apart on few banks' distance
    alignas(16) uint8_t v[kBlock][D + 8];
    uint32_t lo[kWarps][D / 2], hi[kWarps][D / 2];  // each warp's smallest and largest keys, bf16 pairs
    uint32_t most[2][kWarps];
};

template <int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const Q8Cache c, const __nv_bfloat16 *__restrict__ k, const TStrides sk,
                  const __nv_bfloat16 *__restrict__ v, const TStrides sv, int n,
                  const int32_t *__restrict__ lens, const int32_t *__restrict__ new_lens, int touched,
                  int *err) {
    constexpr int kChunks = D / 8;                     // 16-byte chunks of a token
    constexpr int kPer = kBlock * kChunks / kThreads;  // chunks of a thread: the same channels of every kStep-th token
    constexpr int kStep = kThreads / kChunks;
    __shared__ AppendSmem<D> sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long bh = blockIdx.x / touched;
    const int j = (int)(blockIdx.x - bh * touched);
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    grid_dep_wait();
    grid_dep_launch();
    const int length = lens[b], m = new_lens ? new_lens[b] : n;
    const int L = checked_length(length, c.blocks, err);
    if (L < 0) return;
    if (m < 0 || m > n || m > L) {
        if (tid == 0) atomicExch(err, kErrLength);
        return;
    }
    if (m == 0) return;
    const int start = L - m;                // position of row 0
    const int block = start / kBlock + j;
    if (block > (L - 1) / kBlock) return;
    const int closed = L / kBlock;
    const __nv_bfloat16 *kr = k + (long long)b * sk.b + (long long)h * sk.h;
    const __nv_bfloat16 *vr = v + (long long)b * sv.b + (long long)h * sv.h;
    __nv_bfloat16 *rk = c.recent_k + bh * kRing * D, *rv = c.recent_v + bh * kRing * D;
    if (block < closed) {
        const int p0 = block * kBlock;
        ATTN_DCHECK(block < c.blocks && p0 + kBlock <= L, err);
        // ---- load
        const int t0 = tid / kChunks, ch = 8 * (tid % kChunks);
        uint4 kx[kPer], vx[kPer];
        if (p0 >= start) {
            const __nv_bfloat16 *ks = kr + (long long)(p0 - start + t0) * sk.t + ch;
            const __nv_bfloat16 *vs = vr + (long long)(p0 - start + t0) * sv.t + ch;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                kx[i] = *reinterpret_cast<const uint4 *>(ks + i * kStep * sk.t);
                vx[i] = *reinterpret_cast<const uint4 *>(vs + i * kStep * sv.t);
            }
        } else {  // some of the tokens came earlier
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int p = p0 + t0 + i * kStep;
                const bool old = p < start;
                kx[i] = *reinterpret_cast<const uint4 *>((old ? rk + (p % kRing) * D : kr + (long long)(p - start) * sk.t) + ch);
                vx[i] = *reinterpret_cast<const uint4 *>((old ? rv + (p % kRing) * D : vr + (long long)(p - start) * sv.t) + ch);
            }
        }
        // ---- the smallest and largest key of each channel, the largest |value|
        uint32_t lo[4] = {kx[0].x, kx[0].y, kx[0].z, kx[0].w}, hi[4] = {kx[0].x, kx[0].y, kx[0].z, kx[0].w};
        uint32_t va = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t kw[4] = {kx[i].x, kx[i].y, kx[i].z, kx[i].w}, vw[4] = {vx[i].x, vx[i].y, vx[i].z, vx[i].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (i > 0) {
                    lo[x] = min2(lo[x], kw[x]);
                    hi[x] = max2(hi[x], kw[x]);
                }
                va = max2(va, vw[x] & 0x7fff7fffu);
            }
        }
        uint32_t mk = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) mk = max(mk, max(top(lo[x]), top(hi[x])));
        mk = __reduce_max_sync(0xffffffffu, mk);
        const uint32_t mv_warp = __reduce_max_sync(0xffffffffu, top(va));
        if (lane == 0) {
            sm.most[0][warp] = mk;
            sm.most[1][warp] = mv_warp;
        }
        // (the lanes of a warp with the same channels)
#pragma unroll
        for (int off = kChunks; off < 32; off <<= 1)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                lo[x] = min2(lo[x], __shfl_xor_sync(0xffffffffu, lo[x], off));
                hi[x] = max2(hi[x], __shfl_xor_sync(0xffffffffu, hi[x], off));
            }
        if (lane < kChunks) {
            *reinterpret_cast<uint4 *>(&sm.lo[warp][4 * lane]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<uint4 *>(&sm.hi[warp][4 * lane]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        }
        __syncthreads();
        uint32_t mv = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mk = max(mk, sm.most[0][w]);
            mv = max(mv, sm.most[1][w]);
        }
        const bool bad_k = mk >= 0x7f80u, bad_v = mv >= 0x7f80u;
        const bool none_k = mk == 0 || bad_k, none_v = mv == 0 || bad_v;  // all codes are 128
        const float most_k = __uint_as_float(mk << 16), most_v = __uint_as_float(mv << 16);
        const Coder code_k(none_k ? 1.f : most_k), code_v(none_v ? 1.f : most_v);
        const long long at = bh * c.blocks + block;
        uint8_t *kc = c.k_codes + at * (kBlock * D), *vc = c.v_codes + at * (kBlock * D);
        // ---- the codes: keys straight to their place, values by way of shared memory
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            uint2 kw = make_uint2(0x80808080u, 0x80808080u), vw = kw;
            if (!none_k) kw = make_uint2(code_k(kx[i].x, kx[i].y), code_k(kx[i].z, kx[i].w));
            if (!none_v) vw = make_uint2(code_v(vx[i].x, vx[i].y), code_v(vx[i].z, vx[i].w));
            *reinterpret_cast<uint2 *>(kc + key_offset<D>(t0 + i * kStep, ch)) = kw;
            *reinterpret_cast<uint2 *>(&sm.v[t0 + i * kStep][ch]) = vw;
        }
        if (c.bounds && tid < D / 2) {
            // the codes grow with the keys, so the outermost keys have the outermost codes
            uint32_t l = sm.lo[0][tid], h = sm.hi[0][tid];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                l = min2(l, sm.lo[w][tid]);
                h = max2(h, sm.hi[w][tid]);
            }
            const uint32_t word = none_k ? 0u : code_k(l, h) ^ 0x80808080u;  // code - 128 as signed bytes
            uint16_t *to = reinterpret_cast<uint16_t *>(c.bounds + at * (2 * D));
            to[tid] = (uint16_t)word;
            to[D / 2 + tid] = (uint16_t)(word >> 16);
        }
        __syncthreads();
        // four channels of eight tokens a thread; eight threads with consecutive tokens fill a channel's 64 bytes
        for (int e = tid; e < 2 * D; e += kThreads) {
            const int t = 8 * (e % 8), c4 = 4 * (e / 8);
            uint32_t w0[4], w1[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                w0[x] = *reinterpret_cast<const uint32_t *>(&sm.v[t + x][c4]);
                w1[x] = *reinterpret_cast<const uint32_t *>(&sm.v[t + 4 + x][c4]);
            }
            transpose4(w0);
            transpose4(w1);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint2 *>(vc + (c4 + x) * kBlock + t) = make_uint2(w0[x], w1[x]);
        }
        if (tid == 0) {
            const float nan = __int_as_float(0x7fffffff);
            reinterpret_cast<float2 *>(c.scales)[at] =
                make_float2(bad_k ? nan : __fdiv_rn(most_k, 127.f), bad_v ? nan : __fdiv_rn(most_v, 127.f));
            if (c.weight) c.weight[at] = 0.f;
        }
    }
    if (j == 0) {
        // ---- the ring: the new positions of the open block and of the block before it (a step can then be
        // taken back, or taken again, over up to 64 tokens)
        __syncthreads();  // the old positions above are read
        const int low = max(start, (closed - 1) * kBlock);
        for (int e = tid; e < (L - low) * kChunks; e += kThreads) {
            const int p = low + e / kChunks, ch = 8 * (e % kChunks);
            ATTN_DCHECK(p >= start && p < L && L - low <= kRing, err);
            *reinterpret_cast<uint4 *>(rk + (p % kRing) * D + ch) =
                *reinterpret_cast<const uint4 *>(kr + (long long)(p - start) * sk.t + ch);
            *reinterpret_cast<uint4 *>(rv + (p % kRing) * D + ch) =
                *reinterpret_cast<const uint4 *>(vr + (long long)(p - start) * sv.t + ch);
        }
    }
}

// ---- read: positions starts[b] .. + n - 1 as they are held, in bf16 (zero
// rows past the end).  One CTA takes one block of 64 positions; the values turn
// over through shared memory.  2 D bytes read and 4 D written for a token: 53.3 us
// for those 36925 tokens of 8 heads of 128 (floor 52.5).
constexpr int kReadThreads = 256;
// A code byte under the exponent of 2^23: the float 2^23 + code; and two of these as held numbers in bf16 (subtracting
// 2^23 + 128 is exact).
__device__ __forceinline__ uint32_t code_float(uint32_t w, int byte) { return __byte_perm(w, 0x4B000000u, 0x7650 | byte); }
__device__ __forceinline__ uint32_t held_pair(uint32_t a, uint32_t b, uint64_t scale) {
    const uint64_t x = f2pack(__uint_as_float(a), __uint_as_float(b));
    const float2 r = f2unpack(fmul2(fadd2(x, f2pack(-8388736.f, -8388736.f)), scale));
    return pack_bf16x2(r.x, r.y);
}
template <int D>
__global__ void __launch_bounds__(kReadThreads)
    read_kernel(const Q8Cache c, const int32_t *__restrict__ lens, const int32_t *__restrict__ starts, int n,
                int touched, __nv_bfloat16 *__restrict__ k, __nv_bfloat16 *__restrict__ v, int *err) {
    constexpr int kChunks = D / 8;
    __shared__ uint32_t sv[D][kBlock / 4 + 1];
    const int tid = threadIdx.x;
    const long long bh = blockIdx.x / touched;
    const int j = (int)(blockIdx.x - bh * touched);
    const int b = (int)(bh / c.H);
    grid_dep_wait();
    grid_dep_launch();
    const int length = lens[b];
    int start = starts ? starts[b] : 0, L = checked_length(length, c.blocks, err);
    if (start < 0) {
        if (tid == 0) atomicExch(err, kErrLength);
        L = -1;
    }
    if (L < 0) L = start = 0;  // zeros
    const long long block = start / kBlock + j;
    const long long p0 = block * kBlock;
    const long long first = p0 > start ? p0 : start;
    const long long last = p0 + kBlock < (long long)start + n ? p0 + kBlock : (long long)start + n;
    if (first >= last) return;
    __nv_bfloat16 *ko = k + bh * n * D, *vo = v + bh * n * D;
    if (block < L / kBlock) {
        const long long at = bh * c.blocks + block;
        const uint8_t *kc = c.k_codes + at * (kBlock * D), *vc = c.v_codes + at * (kBlock * D);
        // all loads first: a CTA's time is their latency
        constexpr int kKeys = kBlock * kChunks / kReadThreads, kValues = (D * (kBlock / 16) + kReadThreads - 1) / kReadThreads;
        auto wanted = [&](int t) { return p0 + t >= first && p0 + t < last; };
        const float2 scale = reinterpret_cast<const float2 *>(c.scales)[at];
        uint4 vw[kValues];
#pragma unroll
        for (int i = 0; i < kValues; ++i) {  // 16 tokens of a channel
            const int e = tid + i * kReadThreads;
            if (e < D * (kBlock / 16)) vw[i] = *reinterpret_cast<const uint4 *>(vc + 16 * e);
        }
        uint2 kw[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {  // eight channels of a token
            const int e = tid + i * kReadThreads, t = e / kChunks, ch = 8 * (e % kChunks);
            if (wanted(t)) kw[i] = *reinterpret_cast<const uint2 *>(kc + key_offset<D>(t, ch));
        }
        const uint64_t ks = f2pack(scale.x, scale.x), vs = f2pack(scale.y, scale.y);
#pragma unroll
        for (int i = 0; i < kValues; ++i) {
            const int e = tid + i * kReadThreads, ch = e / (kBlock / 16), q = 4 * (e % (kBlock / 16));
            if (e < D * (kBlock / 16)) {
                sv[ch][q] = vw[i].x;
                sv[ch][q + 1] = vw[i].y;
                sv[ch][q + 2] = vw[i].z;
                sv[ch][q + 3] = vw[i].w;
            }
        }
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int e = tid + i * kReadThreads, t = e / kChunks, ch = 8 * (e % kChunks);
            if (!wanted(t)) continue;
            const uint2 w = kw[i];
            uint4 r;
            r.x = held_pair(code_float(w.x, 0), code_float(w.x, 1), ks);
            r.y = held_pair(code_float(w.x, 2), code_float(w.x, 3), ks);
            r.z = held_pair(code_float(w.y, 0), code_float(w.y, 1), ks);
            r.w = held_pair(code_float(w.y, 2), code_float(w.y, 3), ks);
            *reinterpret_cast<uint4 *>(ko + (p0 + t - start) * D + ch) = r;
        }
        __syncthreads();
        for (int e = tid; e < (kBlock / 4) * kChunks; e += kReadThreads) {
            const int quad = e / kChunks, ch = 8 * (e % kChunks);
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) w[x] = sv[ch + x][quad];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const long long p = p0 + 4 * quad + y;
                if (p < first || p >= last) continue;
                uint32_t r[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    r[x] = held_pair(code_float(w[2 * x], y), code_float(w[2 * x + 1], y), vs);
                *reinterpret_cast<uint4 *>(vo + (p - start) * D + ch) = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
        return;
    }
    const __nv_bfloat16 *rk = c.recent_k + bh * kRing * D, *rv = c.recent_v + bh * kRing * D;
    for (int e = tid; e < kBlock * kChunks; e += kReadThreads) {
        const int t = e / kChunks, ch = 8 * (e % kChunks);
        const long long p = p0 + t;
        if (p < first || p >= last) continue;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (p < L) {
            x = *reinterpret_cast<const uint4 *>(rk + (p % kRing) * D + ch);
            y = *reinterpret_cast<const uint4 *>(rv + (p % kRing) * D + ch);
        }
        *reinterpret_cast<uint4 *>(ko + (p - start) * D + ch) = x;
        *reinterpret_cast<uint4 *>(vo + (p - start) * D + ch) = y;
    }
}

}  // namespace

cudaError_t q8_append(const Q8Cache &c, const __nv_bfloat16 *k, const TStrides &sk, const __nv_bfloat16 *v,
                      const TStrides &sv, int n, const int32_t *lens, const int32_t *new_lens, int *err,
                      cudaStream_t st, LaunchInfo &li) {
    const int touched = (int)(((long long)n + 2 * kBlock - 2) / kBlock);  // blocks n tokens can lie in
    const long long grid = (long long)c.B * c.H * touched;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaError_t e = mark_main_start(li, st);
    if (e != cudaSuccess) return e;
    const dim3 g((unsigned)grid);
    if (c.D == 32)
        e = launch_pdl(append_kernel<32>, g, dim3(kThreads), 0, st, c, k, sk, v, sv, n, lens, new_lens, touched, err);
    else if (c.D == 64)
        e = launch_pdl(append_kernel<64>, g, dim3(kThreads), 0, st, c, k, sk, v, sv, n, lens, new_lens, touched, err);
    else
        e = launch_pdl(append_kernel<128>, g, dim3(kThreads), 0, st, c, k, sk, v, sv, n, lens, new_lens, touched, err);
    if (e != cudaSuccess) return e;
    li.kernels += 1;
    return mark_main_end(li, st);
}

cudaError_t q8_read(const Q8Cache &c, const int32_t *lens, const int32_t *starts, int n, __nv_bfloat16 *k,
                    __nv_bfloat16 *v, int *err, cudaStream_t st, LaunchInfo &li) {
    const int touched = starts ? (int)(((long long)n + 2 * kBlock - 2) / kBlock) : (int)(((long long)n + kBlock - 1) / kBlock);
    const long long grid = (long long)c.B * c.H * touched;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaError_t e = mark_main_start(li, st);
    if (e != cudaSuccess) return e;
    const dim3 g((unsigned)grid), t(kReadThreads);
    if (c.D == 32)
        e = launch_pdl(read_kernel<32>, g, t, 0, st, c, lens, starts, n, touched, k, v, err);
    else if (c.D == 64)
        e = launch_pdl(read_kernel<64>, g, t, 0, st, c, lens, starts, n, touched, k, v, err);
    else
        e = launch_pdl(read_kernel<128>, g, t, 0, st, c, lens, starts, n, touched, k, v, err);
    if (e != cudaSuccess) return e;
    li.kernels += 1;
    return mark_main_end(li, st);
}

}  // namespace attn
