// q8.h -- declarations of the 8-bit block cache shared by its translation units
// and attn_api.cu (not part of the public ABI; hidden visibility).
#pragma once

#include "internal.h"

namespace attn {

// A sequence length or a block list held on the device is out of range: noted in
// the device error word; the kernel treats the sequence as empty, or skips the
// entry.
constexpr int kErrLength = 5;

// The cache (layout of its parts: q8_cache.cuh).
constexpr int kQ8Block = 64;           // tokens of a block
constexpr int kQ8MaxBlocks = 32768;    // blocks of a sequence
constexpr int kQ8MaxGroup = 64;        // query heads that share a key head
struct Q8Cache {
    uint8_t *k_codes, *v_codes;
    float *scales;
    int8_t *bounds;   // NULL: not kept
    float *weight;    // NULL: not kept
    __nv_bfloat16 *recent_k, *recent_v;
    int B, H, blocks, D;
};
cudaError_t q8_append(const Q8Cache &c, const __nv_bfloat16 *k, const TStrides &sk, const __nv_bfloat16 *v,
                      const TStrides &sv, int n, const int32_t *lens, const int32_t *new_lens, int *err,
                      cudaStream_t st, LaunchInfo &li);
cudaError_t q8_read(const Q8Cache &c, const int32_t *lens, const int32_t *starts, int n, __nv_bfloat16 *k,
                    __nv_bfloat16 *v, int *err, cudaStream_t st, LaunchInfo &li);
struct Q8Decode {
    const __nv_bfloat16 *q;
    TStrides sq;
    __nv_bfloat16 *o;
    TStrides so;
    float *lse;
    const int32_t *lens;
    const int32_t *list;  // [B, Hkv, Tq, list_n] block lists, or NULL
    int list_n;
    int H, Tq;
    float scale;
    int weight;  // 0: not kept, 1: set, 2: add
    void *workspace;
};
// list_n: 0 without lists.
size_t q8_decode_workspace(const Q8Cache &c, int H, int Tq, int list_n, bool weight);
cudaError_t q8_decode(const Q8Cache &c, const Q8Decode &d, int *err, cudaStream_t st, LaunchInfo &li);
cudaError_t q8_select(const Q8Cache &c, const __nv_bfloat16 *q, const TStrides &sq, const int32_t *lens,
                      int32_t *list, int list_n, int H, int Tq, int *err, cudaStream_t st, LaunchInfo &li);
// Workspace of q8_evict, which uses it only where lens_out == lens.
size_t q8_evict_workspace(const Q8Cache &c);
cudaError_t q8_evict(const Q8Cache &src, const Q8Cache &dst, const int32_t *lens, int32_t *lens_out, int32_t *kept,
                     int keep, int sink, int recent, void *workspace, int *err, cudaStream_t st, LaunchInfo &li);

// ---- what every entry point does: the armed events of the call being made,
// the device check with the error word's address, the end of a call.
LaunchInfo take_launch_info();
int device_setup(int **err_addr);
int finish(cudaError_t e, const LaunchInfo &li);

}  // namespace attn
