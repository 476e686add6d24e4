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
    int *line;        // the tcgen05 kernel's line: steps per CTA, then where each prefix and each suffix starts
    int64_t q_b, q_l, q_h, o_b, o_l, o_h;
    int64_t kp_g, kp_t, kp_h, vp_g, vp_t, vp_h;
    int64_t ks_b, ks_t, ks_h, vs_b, vs_t, vs_h;
    int B, Lq, Hq, Hkv, G, gs, n_prefix;
    int P, S;
    int p_chunk, s_chunk, n_pp, n_sp, p_tiles, s_tiles;
    int p_tc, s_tc, grid_tc;  // segments that the tcgen05 kernel takes, and its CTAs
    float scale_log2;         // scale * log2(e)
};

constexpr float kNone = -3.402823466e+38f;  // m of a part without keys

__device__ __forceinline__ int prefix_len(const Args &a, int g)
{
    return a.plen ? max(0, min(a.plen[g], a.P)) : a.P;
}
__device__ __forceinline__ int suffix_len(const Args &a, int b) { return max(0, min(a.slen[b], a.S)); }

// The tcgen05 kernel's schedule.  Its work is a line of steps that its CTAs share
// evenly, in contiguous ranges.  The rows of a segment and kv head form tiles of
// 128: two tiles together are a unit whose step is one 128-key tile for both; a
// tile that is left over is a unit whose step is two key tiles, one per half of
// the CTA.  Order: segment (prefixes, then suffixes), kv head, unit.  A unit's
// steps follow kStart empty ones, which stand for what it costs to begin a unit
// (its rows' loads and stores, about as long as three steps).
constexpr int kStart = 3;
struct Units {
    int full, single;  // units of two row tiles; 1 if one tile is left over
    __device__ __forceinline__ explicit Units(int rows)
    {
        const int t = (rows + 127) / 128;
        full = t / 2;
        single = t & 1;
    }
    __device__ __forceinline__ int steps(int key_tiles) const  // of one kv head
    {
        return key_tiles ? full * (kStart + key_tiles) + single * (kStart + (key_tiles + 1) / 2) : 0;
    }
};
__device__ __forceinline__ int key_tiles(int len) { return (len + 127) / 128; }

// Steps of segment k of the line (prefixes, then suffixes).
__device__ __forceinline__ int segment_steps(const Args &a, int k)
{
    const int np = a.p_tc ? a.n_prefix : 0;
    const bool pre = k < np;
    const Units u((pre ? a.G : 1) * a.Lq * a.gs);
    return u.steps(key_tiles(pre ? prefix_len(a, k) : suffix_len(a, k - np))) * a.Hkv;
}
// Steps of the prefixes and of all segments, over a whole warp.  (The host sees to it that the line is shorter than 2^31.)
__device__ __forceinline__ void line_length(const Args &a, int &prefixes, int &total)
{
    const int lane = threadIdx.x % 32, np = a.p_tc ? a.n_prefix : 0, ns = a.s_tc ? a.B : 0;
    int p = 0, s = 0;
    for (int k = lane; k < np; k += 32) p += segment_steps(a, k);
    for (int k = np + lane; k < np + ns; k += 32) s += segment_steps(a, k);
    prefixes = __reduce_add_sync(0xFFFFFFFFu, p);
    total = prefixes + __reduce_add_sync(0xFFFFFFFFu, s);
}
__device__ __forceinline__ int steps_per_cta(const Args &a, int total)
{
    const int n = (total + a.grid_tc - 1) / a.grid_tc;
    return n ? n : 1;
}

// Parts that the tcgen05 kernel left for row r of a segment (the line's k-th) and kv head.
__device__ __forceinline__ int tc_parts(const Args &a, bool pre, int k, int hk, int r, int len)
{
    const int T = key_tiles(len), per_cta = a.line[0], start = a.line[1 + k];
    if (T == 0) return 0;
    const Units u((pre ? a.G : 1) * a.Lq * a.gs);
    const int pair = r / 256;
    const bool single = pair == u.full;
    const int first = start + hk * u.steps(T) + pair * (kStart + T) + kStart, n = single ? (T + 1) / 2 : T;
    return ((first + n - 1) / per_cta - first / per_cta + 1) * (single ? 2 : 1);
}

// Most parts of a row that the tcgen05 kernel leaves: a unit's steps over a CTA's, which are at least the line's length
// over the CTAs (its empty steps, which only lengthen it, left out); of a left-over tile two each.
inline int tc_parts_most(int64_t rows, int64_t len, int64_t Hkv, int64_t ctas)
{
    const int64_t t = (rows + 127) / 128, full = t / 2, T = (len + 127) / 128, half = (T + 1) / 2;
    const auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
    const int64_t pairs = full ? least(T, ctas / (Hkv * full) + 3) : 0;
    const int64_t single = t & 1 ? 2 * least(half, ctas / (Hkv * (full ? full + 1 : 1)) + 3) : 0;
    return (int)(pairs > single ? pairs : single);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Launches the tcgen05 kernel; false where its tensor maps cannot describe the caches (nothing is launched).
bool tc_maps(const Args &a, int64_t D, void *maps);
cudaError_t tc_launch(const Args &a, int64_t D, const void *maps, cudaStream_t s, bool chain);
constexpr size_t kTcMapsBytes = 4 * 128;

}  // namespace attn
}  // namespace qerl
