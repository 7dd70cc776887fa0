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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint32_t code_of(float x, float most) { return (uint32_t)(128 + code_number(x, most)); }

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

template <int D>
struct AppendSmem {
    uint32_t v[D][kBlock / 4 + 1];  // values' codes, four tokens a word
    uint32_t lo[kWarps][D / 4], hi[kWarps][D / 4];
    uint32_t most[2][kWarps];
};

template <int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const Q8Cache c, const __nv_bfloat16 *__restrict__ k, const TStrides sk,
                  const __nv_bfloat16 *__restrict__ v, const TStrides sv, int n,
                  const int32_t *__restrict__ lens, const int32_t *__restrict__ new_lens, int touched,
                  int *err) {
    constexpr int kChunks = D / 8;                         // 16-byte chunks of a token
    constexpr int kPer = kBlock * kChunks / kThreads;      // chunks of a thread
    constexpr int kQuads = (D / 2) * (kBlock / 4) / kThreads;  // (channel pair, four tokens) of a thread
    __shared__ AppendSmem<D> sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long bh = blockIdx.x / touched;
    const int j = (int)(blockIdx.x - bh * touched);
    const int b = (int)(bh / c.H), h = (int)(bh % c.H);
    grid_dep_wait();
    grid_dep_launch();
    const int L = checked_length(lens, b, c.blocks, err);
    if (L < 0) return;
    int m = new_lens ? new_lens[b] : n;
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
        // ---- load: keys by 16-byte chunks of a token, values by channel pairs of four tokens
        uint4 kx[kPer];
        uint32_t vx[kQuads][4];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = tid + i * kThreads, t = e / kChunks, ch = 8 * (e % kChunks);
            const int p = p0 + t;
            const __nv_bfloat16 *src = p < start ? rk + (p % kRing) * D : kr + (long long)(p - start) * sk.t;
            kx[i] = *reinterpret_cast<const uint4 *>(src + ch);
        }
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const int e = tid + i * kThreads, cp = e % (D / 2), quad = e / (D / 2);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int p = p0 + 4 * quad + x;
                const __nv_bfloat16 *src = p < start ? rv + (p % kRing) * D : vr + (long long)(p - start) * sv.t;
                vx[i][x] = *reinterpret_cast<const uint32_t *>(src + 2 * cp);
            }
        }
        // ---- the two maxima, on the bits: |x| as a 15-bit number grows with |x|, and infinities and NaN
        // come out on top
        uint32_t mk = 0, mv = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            mk = abs_max2(abs_max2(abs_max2(abs_max2(mk, kx[i].x), kx[i].y), kx[i].z), kx[i].w);
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) mv = abs_max2(mv, vx[i][x]);
        mk = __reduce_max_sync(0xffffffffu, max(mk & 0xffffu, mk >> 16));
        mv = __reduce_max_sync(0xffffffffu, max(mv & 0xffffu, mv >> 16));
        if (lane == 0) {
            sm.most[0][warp] = mk;
            sm.most[1][warp] = mv;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mk = max(mk, sm.most[0][w]);
            mv = max(mv, sm.most[1][w]);
        }
        const bool bad_k = mk >= 0x7f80u, bad_v = mv >= 0x7f80u;
        const float most_k = __uint_as_float(mk << 16), most_v = __uint_as_float(mv << 16);
        const long long at = bh * c.blocks + block;
        // ---- keys
        uint8_t *kc = c.k_codes + at * (kBlock * D);
        uint32_t lo[2] = {0xffffffffu, 0xffffffffu}, hi[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = tid + i * kThreads, t = e / kChunks, ch = 8 * (e % kChunks);
            const __nv_bfloat162 *x2 = reinterpret_cast<const __nv_bfloat162 *>(&kx[i]);
            uint32_t w[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 f0 = __bfloat1622float2(x2[2 * x]), f1 = __bfloat1622float2(x2[2 * x + 1]);
                w[x] = 0x80808080u;
                if (mk != 0 && !bad_k)
                    w[x] = code_of(f0.x, most_k) | (code_of(f0.y, most_k) << 8) | (code_of(f1.x, most_k) << 16) |
                           (code_of(f1.y, most_k) << 24);
                lo[x] = __vminu4(lo[x], w[x]);
                hi[x] = __vmaxu4(hi[x], w[x]);
            }
            *reinterpret_cast<uint2 *>(kc + key_offset<D>(t, ch)) = make_uint2(w[0], w[1]);
        }
        // a warp's lanes with the same channels, then the warps
#pragma unroll
        for (int off = kChunks; off < 32; off <<= 1)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                lo[x] = __vminu4(lo[x], __shfl_xor_sync(0xffffffffu, lo[x], off));
                hi[x] = __vmaxu4(hi[x], __shfl_xor_sync(0xffffffffu, hi[x], off));
            }
        if (lane < kChunks) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                sm.lo[warp][2 * lane + x] = lo[x];
                sm.hi[warp][2 * lane + x] = hi[x];
            }
        }
        // ---- values: four tokens of a channel a word, turned over in shared memory
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const int e = tid + i * kThreads, cp = e % (D / 2), quad = e / (D / 2);
            uint32_t w0 = 0x80808080u, w1 = 0x80808080u;
            if (mv != 0 && !bad_v) {
                w0 = w1 = 0;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&vx[i][x]));
                    w0 |= code_of(f.x, most_v) << (8 * x);
                    w1 |= code_of(f.y, most_v) << (8 * x);
                }
            }
            sm.v[2 * cp][quad] = w0;
            sm.v[2 * cp + 1][quad] = w1;
        }
        __syncthreads();
        uint8_t *vc = c.v_codes + at * (kBlock * D);
        for (int e = tid; e < D * (kBlock / 16); e += kThreads) {
            const int ch = e / (kBlock / 16), q = 4 * (e % (kBlock / 16));
            *reinterpret_cast<uint4 *>(vc + ch * kBlock + 4 * q) =
                make_uint4(sm.v[ch][q], sm.v[ch][q + 1], sm.v[ch][q + 2], sm.v[ch][q + 3]);
        }
        if (c.bounds && tid < D / 2) {
            const int x = tid % (D / 4);
            const bool high = tid >= D / 4;
            uint32_t r = high ? 0u : 0xffffffffu;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) r = high ? __vmaxu4(r, sm.hi[w][x]) : __vminu4(r, sm.lo[w][x]);
            // code - 128 as a signed byte
            reinterpret_cast<uint32_t *>(c.bounds + at * (2 * D))[(high ? D / 4 : 0) + x] = r ^ 0x80808080u;
        }
        if (tid == 0) {
            const float nan = __int_as_float(0x7fffffff);
            c.scales[2 * at] = bad_k ? nan : __fdiv_rn(most_k, 127.f);
            c.scales[2 * at + 1] = bad_v ? nan : __fdiv_rn(most_v, 127.f);
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
// rows past the end).  One CTA takes one block of 64 positions.
template <int D>
__global__ void __launch_bounds__(kThreads)
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
    int L = checked_length(lens, b, c.blocks, err);
    int start = starts ? starts[b] : 0;
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
        const float ks = c.scales[2 * at], vs = c.scales[2 * at + 1];
        for (int e = tid; e < D * (kBlock / 16); e += kThreads) {
            const int ch = e / (kBlock / 16), q = 4 * (e % (kBlock / 16));
            const uint4 w = *reinterpret_cast<const uint4 *>(vc + ch * kBlock + 4 * q);
            sv[ch][q] = w.x;
            sv[ch][q + 1] = w.y;
            sv[ch][q + 2] = w.z;
            sv[ch][q + 3] = w.w;
        }
        for (int e = tid; e < kBlock * kChunks; e += kThreads) {
            const int t = e / kChunks, ch = 8 * (e % kChunks);
            if (p0 + t < first || p0 + t >= last) continue;
            const uint2 w = *reinterpret_cast<const uint2 *>(kc + key_offset<D>(t, ch));
            uint4 r;
            r.x = pack_bf16x2((int)((w.x & 255) - 128) * ks, (int)(((w.x >> 8) & 255) - 128) * ks);
            r.y = pack_bf16x2((int)(((w.x >> 16) & 255) - 128) * ks, (int)((w.x >> 24) - 128) * ks);
            r.z = pack_bf16x2((int)((w.y & 255) - 128) * ks, (int)(((w.y >> 8) & 255) - 128) * ks);
            r.w = pack_bf16x2((int)(((w.y >> 16) & 255) - 128) * ks, (int)((w.y >> 24) - 128) * ks);
            *reinterpret_cast<uint4 *>(ko + (p0 + t - start) * D + ch) = r;
        }
        __syncthreads();
        for (int e = tid; e < (kBlock / 4) * kChunks; e += kThreads) {
            const int quad = e / kChunks, ch = 8 * (e % kChunks);
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) w[x] = sv[ch + x][quad];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const long long p = p0 + 4 * quad + y;
                if (p < first || p >= last) continue;
                float f[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) f[x] = (int)(((w[x] >> (8 * y)) & 255) - 128) * vs;
                *reinterpret_cast<uint4 *>(vo + (p - start) * D + ch) =
                    make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                               pack_bf16x2(f[6], f[7]));
            }
        }
        return;
    }
    const __nv_bfloat16 *rk = c.recent_k + bh * kRing * D, *rv = c.recent_v + bh * kRing * D;
    for (int e = tid; e < kBlock * kChunks; e += kThreads) {
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
    const dim3 g((unsigned)grid), t(kThreads);
    if (c.D == 32)
        e = launch_pdl(append_kernel<32>, g, t, 0, st, c, k, sk, v, sv, n, lens, new_lens, touched, err);
    else if (c.D == 64)
        e = launch_pdl(append_kernel<64>, g, t, 0, st, c, k, sk, v, sv, n, lens, new_lens, touched, err);
    else
        e = launch_pdl(append_kernel<128>, g, t, 0, st, c, k, sk, v, sv, n, lens, new_lens, touched, err);
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
    const dim3 g((unsigned)grid), t(kThreads);
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
