// Launch parameters of the paged attention kernels, and how a row's visible
// tokens fall into blocks.  Included by the .hip translation units only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bcg_decode.h"

namespace bcg {

constexpr int kMaxSplits = 128;

struct AttnParams {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* table;
    const int32_t* len;
    const int32_t* qoff;
    const float* kscale;
    const float* vscale;
    void* out;
    float* lse;
    float* part_o;      // [splits][tokens * q_heads][head_dim], unnormalised
    float2* part_ml;    // [splits][tokens * q_heads]: running maximum (log2 units) and sum
    int64_t qstride, kps, vps;  // elements
    int rows, tokens, qh, kvh, G, D;
    int ps, shift, maxb, np;    // shift: log2(ps), or -1
    int window, sinks;
    int max_len, max_new, tiles, splits, chunk;  // chunk: blocks of a split
    int columns;        // prompt: of a workgroup
    int waves;          // decode: of a workgroup
    float scale2;       // softmax scale * log2(e)
};

// The visible tokens of queries whose first sees [0, s) and [lo, ..) and whose
// last sees up to hi, as a list of `nb` blocks of T tokens: blocks of the
// sinks first, then those of the window.
struct BlockList {
    int nb1, b0, nb;
    __device__ __forceinline__ int operator()(int v) const { return v < nb1 ? v : v - nb1 + b0; }
};
__device__ __forceinline__ BlockList visible_blocks(int lo, int hi, int sinks, int T) {
    BlockList l;
    l.nb1 = (min(sinks, lo) + T - 1) / T;
    l.b0 = max(lo / T, l.nb1);
    l.nb = l.nb1 + max(0, (hi + T - 1) / T - l.b0);
    return l;
}

template <typename QT, typename KT> hipError_t launch_decode(const AttnParams& p, hipStream_t st);
template <typename QT, typename KT> hipError_t launch_prompt(const AttnParams& p, hipStream_t st);
// Columns (query, head) of one prompt workgroup, for runs of many queries, and
// tokens of its tiles.
template <typename QT, typename KT> int prompt_columns(int head_dim);
template <typename QT, typename KT> int prompt_block(int head_dim);

struct e4m3_t { uint8_t b; };

}  // namespace bcg
