// Attention over a shared prefix and per-sequence suffixes: what the kernels share.
#pragma once

#include "common.cuh"

namespace qerl {
namespace attn {

// One call as the kernels see it.  Strides in elements.  A query row is (b, l,
// h): sequence, new token, query head; gs = Hq / Hkv heads share a kv head, G =
// B / n_prefix sequences share a prefix.  Keys of a segment (a prefix or a
// suffix) are cut into chunks; each chunk of a row leaves a part in the
// workspace: o = sum e^(a - m) v unnormalised, m (log2 units) and l = sum e^(a - m).
// Parts of a row: n_pp of the prefix, then n_sp of the suffix.
struct Args {
    const __nv_bfloat16 *q, *kp, *vp, *ks, *vs;
    const int32_t *plen, *slen;  // NULL plen: P everywhere
    __nv_bfloat16 *out;
    float *lse;
    float *part_o;   // [row][part][D]
    float2 *part_ml;  // [row][part]
    int64_t q_b, q_l, q_h, o_b, o_l, o_h;
    int64_t kp_g, kp_t, kp_h, vp_g, vp_t, vp_h;
    int64_t ks_b, ks_t, ks_h, vs_b, vs_t, vs_h;
    int B, Lq, Hq, Hkv, G, gs, n_prefix;
    int P, S;
    int p_chunk, s_chunk, n_pp, n_sp, p_tiles, s_tiles;
    float scale_log2;  // scale * log2(e)
};

constexpr float kNone = -3.402823466e+38f;  // m of a part without keys

__device__ __forceinline__ int prefix_len(const Args &a, int g)
{
    return a.plen ? max(0, min(a.plen[g], a.P)) : a.P;
}
__device__ __forceinline__ int suffix_len(const Args &a, int b) { return max(0, min(a.slen[b], a.S)); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace attn
}  // namespace qerl
