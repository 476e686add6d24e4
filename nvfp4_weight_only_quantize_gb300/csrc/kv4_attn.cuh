// Attention over 4-bit caches: what its kernels share.
#pragma once

#include "kv4.cuh"
#include "prefix_attn.cuh"

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
// suffixes, which the CTAs share in contiguous ranges of line[0] steps; before a unit's steps come line[1] empty ones, and
// line[2 + k] is where segment k starts.  Each range in a
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

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The two scale pairs of a word as fp16 pairs.
__device__ __forceinline__ void scales_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
}

// From the products' sum to log2 units where the row was divided by 2^e.  Not 0, which a masked score of -inf would make NaN (a
// row of zeros has the smallest e), and not inf, which a score of 0 would.  Sums are below 2^20: with the smallest scale
// all scores are 0 within 2^-106.
__device__ __forceinline__ float row_scale(float scale_log2, int e)
{
    return fminf(fmaxf(scale_log2 * pow2f(e), 1.17549435e-38f), 3.402823466e+38f);
}

// The tcgen05 kernel's launch over the sides that `a` gives it.
cudaError_t many_rows(const attn::Args &a, const Side &pre, const Side &suf, int64_t D, cudaStream_t s, bool chain);

}  // namespace kv4
}  // namespace qerl
