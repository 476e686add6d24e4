// Attention over 4-bit caches: what its kernels share.
#pragma once

#include "kv4.cuh"

namespace qerl {
namespace kv4 {

constexpr int kRows = 8;  // of a row tile

// One kind of segments, prefixes or suffixes (n = 0: there are none).  The rows that share a segment's kv head form row tiles.
struct Side {
    Cache c;
    const int32_t *lens;  // NULL: full
    int n, rows, row_tiles;
    float scale_log2;  // from the products' sum to log2 units
};

// One call as the kernels see it.  Strides of q and out in elements.  A query row is (b, l, h): sequence, new token, query head;
// gs = Hq / Hkv heads share a kv head, G sequences share a prefix.
// A unit is (segment, kv head, row tile); its steps are the segment's key tiles.  All units' steps form a line, prefixes before
// suffixes, which the CTAs share in contiguous ranges of line[0] steps; line[1 + k] is where segment k starts.  Each range in a
// unit leaves a part: o = sum 2^(a - m) v unnormalised (without the cache's factor), m and l = sum 2^(a - m).  Unit u and CTA c
// leave part u + c, which no other pair has: along the line, u or c grows from one part to the next.
struct Call {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse;
    float *part_o;    // [part][kRows][D]
    float2 *part_ml;  // [part][kRows]
    int *line;
    int64_t q_b, q_l, q_h, o_b, o_l, o_h;
    int B, Lq, Hq, Hkv, G, gs, grid;
    Side pre, suf;
};

__device__ __forceinline__ int length(const Side &s, int k) { return s.lens ? max(0, min(s.lens[k], s.c.T)) : s.c.T; }
__device__ __forceinline__ int tiles_of(int len) { return (len + kTok - 1) / kTok; }

// Row r of segment k and kv head hk.
struct Row {
    int b, l, h;
};
__device__ __forceinline__ Row row_of(const Call &a, bool pre, int k, int hk, int r)
{
    const int per = a.Lq * a.gs, bi = r / per, in = r - bi * per, l = in / a.gs;
    return Row{pre ? k * a.G + bi : k, l, hk * a.gs + in - l * a.gs};
}

constexpr float kNone = -3.402823466e+38f;  // m of a part without keys

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace kv4
}  // namespace qerl
