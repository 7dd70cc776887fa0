// q8_api.cu -- the extern "C" entry points of the 8-bit block cache
// (declared in include/attn.h): argument checks and dispatch to the kernels.
#include "../../include/attn.h"
#include "q8.h"

#include <math.h>

#include <array>

#define ATTN_API extern "C" __attribute__((visibility("default")))

using namespace attn;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A piece of memory (NULL: none) and its bytes.
struct Part {
    const void *at;
    size_t bytes;
};
bool overlap(const Part &a, const Part &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return x && y && x < y + b.bytes && y < x + a.bytes;
}
// A cache's seven parts.
std::array<Part, 7> parts_of(const Q8Cache &c) {
    const size_t heads = (size_t)c.B * c.H, blocks = heads * c.blocks, side = (size_t)kQ8Block * c.D;
    const size_t ring = heads * 2 * side * sizeof(__nv_bfloat16);
    return {{{c.k_codes, blocks * side}, {c.v_codes, blocks * side}, {c.scales, blocks * 8}, {c.bounds, blocks * 2 * c.D},
             {c.weight, blocks * 4}, {c.recent_k, ring}, {c.recent_v, ring}}};
}

bool strides_ok(const attn_strides &x) {
    auto ok = [](int64_t v) { return v > 0 && v % 8 == 0 && v < (1ll << 39); };
    return ok(x.b) && ok(x.h) && ok(x.t);
}

// The strides of a [B, H, T, D] operand, given or contiguous.
int operand(const attn_strides *given, int H, int T, int D, TStrides &out) {
    if (!given) {
        out = TStrides{(long long)H * T * D, (long long)T * D, (long long)D};
        return ATTN_OK;
    }
    if (!strides_ok(*given)) return ATTN_ERR_ALIGN;
    out = TStrides{given->b, given->h, given->t};
    return ATTN_OK;
}

// Checks a cache's sizes alone (what a workspace query needs).
int check_sizes(const attn_q8_cache &c) {
    if (c.B < 1 || c.H < 1 || c.blocks < 1 || c.blocks > kQ8MaxBlocks) return ATTN_ERR_SHAPE;
    if (c.D != 32 && c.D != 64 && c.D != 128) return ATTN_ERR_UNSUPPORTED_D;
    if ((long long)c.B * c.H > 0x7fffffffLL / 64) return ATTN_ERR_SHAPE;
    if ((long double)c.B * c.H * c.blocks * kQ8Block * c.D > (long double)(1ll << 40)) return ATTN_ERR_SHAPE;
    return ATTN_OK;
}

int check_cache(const attn_q8_cache *c, Q8Cache &out) {
    if (!c || !c->k_codes || !c->v_codes || !c->scales || !c->recent_k || !c->recent_v) return ATTN_ERR_NULL;
    const int st = check_sizes(*c);
    if (st != ATTN_OK) return st;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->scales, 8) || !aligned(c->bounds, 16) ||
        !aligned(c->weight, 4) || !aligned(c->recent_k, 16) || !aligned(c->recent_v, 16))
        return ATTN_ERR_ALIGN;
    out.k_codes = static_cast<uint8_t *>(c->k_codes);
    out.v_codes = static_cast<uint8_t *>(c->v_codes);
    out.scales = c->scales;
    out.bounds = static_cast<int8_t *>(c->bounds);
    out.weight = c->weight;
    out.recent_k = static_cast<__nv_bfloat16 *>(c->recent_k);
    out.recent_v = static_cast<__nv_bfloat16 *>(c->recent_v);
    out.B = c->B;
    out.H = c->H;
    out.blocks = c->blocks;
    out.D = c->D;
    return ATTN_OK;
}

int check_queries(const attn_q8_cache &c, int H, int Tq) {
    if (H < 1 || H % c.H != 0 || H / c.H > kQ8MaxGroup) return ATTN_ERR_SHAPE;
    if (Tq < 1 || Tq > ATTN_DECODE_MAX_QUERIES) return ATTN_ERR_SHAPE;
    return ATTN_OK;
}

}  // namespace

ATTN_API int attn_q8_append(const attn_q8_cache *cache, const void *k, const void *v, int n, const int32_t *lens,
                            const int32_t *new_lens, const attn_strides *strides, cudaStream_t stream) {
    LaunchInfo li = take_launch_info();
    if (!k || !v || !lens) return ATTN_ERR_NULL;
    Q8Cache c;
    int st;
    if ((st = check_cache(cache, c)) != ATTN_OK) return st;
    if (n < 1 || (long long)n > (long long)kQ8Block * c.blocks + kQ8Block - 1) return ATTN_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(lens, 4) || !aligned(new_lens, 4)) return ATTN_ERR_ALIGN;
    TStrides sk, sv;
    if ((st = operand(strides, c.H, n, c.D, sk)) != ATTN_OK) return st;
    if ((st = operand(strides ? strides + 1 : nullptr, c.H, n, c.D, sv)) != ATTN_OK) return st;
    int *err = nullptr;
    if ((st = device_setup(&err)) != ATTN_OK) return st;
    return finish(q8_append(c, static_cast<const __nv_bfloat16 *>(k), sk, static_cast<const __nv_bfloat16 *>(v), sv, n,
                            lens, new_lens, err, stream, li),
                  li);
}

ATTN_API int attn_q8_read(const attn_q8_cache *cache, const int32_t *lens, const int32_t *starts, int n, void *k,
                          void *v, cudaStream_t stream) {
    LaunchInfo li = take_launch_info();
    if (!k || !v || !lens) return ATTN_ERR_NULL;
    Q8Cache c;
    int st;
    if ((st = check_cache(cache, c)) != ATTN_OK) return st;
    if (n < 1 || n > kQ8Block * (kQ8MaxBlocks + 1)) return ATTN_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(lens, 4) || !aligned(starts, 4)) return ATTN_ERR_ALIGN;
    int *err = nullptr;
    if ((st = device_setup(&err)) != ATTN_OK) return st;
    return finish(q8_read(c, lens, starts, n, static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v), err,
                          stream, li),
                  li);
}

ATTN_API size_t attn_q8_decode_workspace_bytes(const attn_q8_cache *cache, int H, int Tq,
                                               const attn_q8_decode_options *opts) {
    if (!cache || check_sizes(*cache) != ATTN_OK || check_queries(*cache, H, Tq) != ATTN_OK) return 0;
    if (opts && (opts->blocks_n < 0 || opts->blocks_n > kQ8MaxBlocks)) return 0;
    Q8Cache c{};
    c.B = cache->B;
    c.H = cache->H;
    c.blocks = cache->blocks;
    c.D = cache->D;
    return q8_decode_workspace(c, H, Tq, opts ? opts->blocks_n : 0, opts && opts->weight != ATTN_Q8_WEIGHT_NONE);
}

ATTN_API int attn_q8_decode(const attn_q8_cache *cache, const void *q, void *o, float *lse, const int32_t *lens, int H,
                            int Tq, float scale, const attn_strides *strides, const attn_q8_decode_options *opts,
                            void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    LaunchInfo li = take_launch_info();
    if (!q || !o || !lse || !lens) return ATTN_ERR_NULL;
    Q8Cache c;
    int st;
    if ((st = check_cache(cache, c)) != ATTN_OK) return st;
    if ((st = check_queries(*cache, H, Tq)) != ATTN_OK) return st;
    if (!(isfinite(scale) && scale > 0.f)) return ATTN_ERR_SCALE;
    Q8Decode d{};
    if (opts) {
        if (opts->weight < ATTN_Q8_WEIGHT_NONE || opts->weight > ATTN_Q8_WEIGHT_ADD) return ATTN_ERR_OPTION;
        if ((opts->blocks != nullptr) != (opts->blocks_n > 0) || opts->blocks_n < 0 || opts->blocks_n > kQ8MaxBlocks)
            return ATTN_ERR_OPTION;
        // A block's weight is what all rows give it: with lists, rows differ in what they see.
        if (opts->weight != ATTN_Q8_WEIGHT_NONE && (opts->blocks || !c.weight)) return ATTN_ERR_OPTION;
        if (!aligned(opts->blocks, 4)) return ATTN_ERR_ALIGN;
        d.list = opts->blocks;
        d.list_n = opts->blocks_n;
        d.weight = opts->weight;
    }
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(lens, 4)) return ATTN_ERR_ALIGN;
    if ((st = operand(strides, H, Tq, c.D, d.sq)) != ATTN_OK) return st;
    if ((st = operand(strides ? strides + 1 : nullptr, H, Tq, c.D, d.so)) != ATTN_OK) return st;
    const size_t need = q8_decode_workspace(c, H, Tq, d.list_n, d.weight != 0);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return ATTN_ERR_WORKSPACE;
    int *err = nullptr;
    if ((st = device_setup(&err)) != ATTN_OK) return st;
    d.q = static_cast<const __nv_bfloat16 *>(q);
    d.o = static_cast<__nv_bfloat16 *>(o);
    d.lse = lse;
    d.lens = lens;
    d.H = H;
    d.Tq = Tq;
    d.scale = scale;
    d.workspace = workspace;
    return finish(q8_decode(c, d, err, stream, li), li);
}

ATTN_API int attn_q8_select(const attn_q8_cache *cache, const void *q, const int32_t *lens, int32_t *blocks, int n,
                            int H, int Tq, const attn_strides *strides, cudaStream_t stream) {
    LaunchInfo li = take_launch_info();
    if (!q || !lens || !blocks) return ATTN_ERR_NULL;
    Q8Cache c;
    int st;
    if ((st = check_cache(cache, c)) != ATTN_OK) return st;
    if (!c.bounds) return ATTN_ERR_NULL;
    if ((st = check_queries(*cache, H, Tq)) != ATTN_OK) return st;
    if (n < 1 || n > kQ8MaxBlocks) return ATTN_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(lens, 4) || !aligned(blocks, 4)) return ATTN_ERR_ALIGN;
    TStrides sq;
    if ((st = operand(strides, H, Tq, c.D, sq)) != ATTN_OK) return st;
    int *err = nullptr;
    if ((st = device_setup(&err)) != ATTN_OK) return st;
    return finish(
        q8_select(c, static_cast<const __nv_bfloat16 *>(q), sq, lens, blocks, n, H, Tq, err, stream, li), li);
}

ATTN_API size_t attn_q8_evict_workspace_bytes(const attn_q8_cache *cache) {
    if (!cache || check_sizes(*cache) != ATTN_OK) return 0;
    Q8Cache c{};
    c.B = cache->B;
    c.H = cache->H;
    return (q8_evict_workspace(c) + 255) / 256 * 256;
}

ATTN_API int attn_q8_evict(const attn_q8_cache *cache, const attn_q8_cache *out, const int32_t *lens,
                           int32_t *lens_out, int32_t *kept, int keep, int sink, int recent, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
    LaunchInfo li = take_launch_info();
    if (!lens || !lens_out || !kept) return ATTN_ERR_NULL;
    Q8Cache c, d;
    int st;
    if ((st = check_cache(cache, c)) != ATTN_OK) return st;
    if ((st = check_cache(out, d)) != ATTN_OK) return st;
    if (!c.weight || (d.bounds && !c.bounds)) return ATTN_ERR_NULL;
    if (c.B != d.B || c.H != d.H || c.D != d.D) return ATTN_ERR_SHAPE;
    if (keep < 1 || keep > kQ8MaxBlocks || sink < 0 || recent < 0 || sink > keep || recent > keep - sink)
        return ATTN_ERR_SHAPE;
    if (d.blocks < (keep < c.blocks ? keep : c.blocks)) return ATTN_ERR_SHAPE;
    // One cache, or two that share nothing.
    const bool same[] = {c.k_codes == d.k_codes,   c.v_codes == d.v_codes,   c.scales == d.scales,
                         c.recent_k == d.recent_k, c.recent_v == d.recent_v, c.weight == d.weight};
    for (bool s : same)
        if (s != same[0]) return ATTN_ERR_OPTION;
    if (same[0] && (c.blocks != d.blocks || c.bounds != d.bounds)) return ATTN_ERR_OPTION;
    if (!same[0])
        for (const Part &x : parts_of(c))
            for (const Part &y : parts_of(d))
                if (overlap(x, y)) return ATTN_ERR_OPTION;
    if (!aligned(lens, 4) || !aligned(lens_out, 4) || !aligned(kept, 4)) return ATTN_ERR_ALIGN;
    if (lens_out == lens &&
        (!workspace || workspace_bytes < attn_q8_evict_workspace_bytes(cache) || !aligned(workspace, 256)))
        return ATTN_ERR_WORKSPACE;
    // The lengths are read while the list of kept blocks and the new lengths are written.
    const size_t lens_bytes = (size_t)c.B * 4;
    const Part old_lens{lens, lens_bytes}, new_lens{lens_out, lens_bytes}, list{kept, (size_t)c.B * c.H * keep * 4};
    if ((lens_out != lens && overlap(new_lens, old_lens)) || overlap(list, old_lens) || overlap(list, new_lens))
        return ATTN_ERR_OPTION;
    int *err = nullptr;
    if ((st = device_setup(&err)) != ATTN_OK) return st;
    return finish(q8_evict(c, d, lens, lens_out, kept, keep, sink, recent, workspace, err, stream, li),
                  li);
}
