// The 4-bit cache's own operators: new tokens into it, and its values back.
//
// Append: a block of 16 values w gets the scale s = the smallest E4M3 number that
// is at least amax |w| / (6 f), f the cache's factor, and codes nearest(w / (s f)).
// A CTA takes one tile (32 tokens) of a sequence and head, a warp one block of 16
// dims, a lane one token: eight lanes turn their values' codes by three exchanges
// (halves, bytes, nibbles of words) from one token per lane to eight tokens per
// word.  Words that hold older tokens too are read and merged; no two threads write
// to one word.
// Eight prompts of up to 4001 tokens, 8 heads, D = 128: 58 us (131 MB read, 37 MB
// written, 2.9 TB/s), bound by issue (72 % of the slots, ALU 65 %); reading them back
// 44 us (3.8 TB/s), bound by the queue of shuffles, scales' bytes and stores (its stall is
// the longest, issue 42 %).  D = 64: 27 and 22 us.  A token of each of 64 sequences: 5.8
// and 3.3 us in a graph, the launch and three dependent memory accesses.
#include "kv4.cuh"

#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "fp4_round.cuh"

namespace qerl {
namespace kv4 {
namespace {

struct Tokens {
    const __nv_bfloat16 *k, *v;  // or where read() puts them
    int64_t k_b, k_l, k_h, v_b, v_l, v_h;
    const int32_t *lens, *counts;
    int L;
};

// Sixteen values of a block: their codes (element i in bits 4 i of two words) and the scale's byte.
__device__ __forceinline__ uint2 quantise(const uint4 &u0, const uint4 &u1, float factor, uint32_t &scale, bool &finite)
{
    const uint32_t wd[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
    float w[16], amax = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[2 * i] = bf16lo(wd[i]);
        w[2 * i + 1] = bf16hi(wd[i]);
        top = max(top, max(wd[i] & 0x7FFFu, wd[i] >> 16 & 0x7FFFu));
        amax = fmaxf(amax, fmaxf(fabsf(w[2 * i]), fabsf(w[2 * i + 1])));
    }
    if (top >= 0x7F80u) {
        finite = false;
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = isnan(w[i]) ? 0.0f : fminf(fmaxf(w[i], -FLT_MAX), FLT_MAX);
    }
    scale = e4m3_ceil(__fdiv_rn(amax, __fmul_rn(6.0f, factor)));
    const float unit = __fmul_rn(e4m3_to_float(scale), factor);
    // The quotient by a reciprocal and one correction from the exact remainder, which leaves quotients that are borders exact;
    // the conversion rounds to nearest, ties to the even code, and saturates.
    const float inv = scale ? __fdiv_rn(1.0f, unit) : 0.0f;
    uint32_t code[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        float q[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float q0 = fminf(fmaxf(w[i + e] * inv, -8.0f), 8.0f);  // saturates at 6
            q[e] = fmaf(fmaf(-q0, unit, w[i + e]), inv, q0);
        }
        uint32_t byte;
        asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tmov.b32 %0, {c, 0, 0, 0};\n\t}" : "=r"(byte) : "f"(q[0]), "f"(q[1]));
        code[i / 8] |= byte << (4 * (i % 8));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // zero has one code
        const uint32_t c = code[h], some = (c | c >> 1 | c >> 2) & 0x11111111u;
        code[h] = c & (some * 15u);
    }
    return make_uint2(code[0], code[1]);
}

// Nibble n of lane k's word goes to nibble k of lane n's, among eight lanes.
__device__ __forceinline__ uint32_t turned(uint32_t w)
{
    const int k = threadIdx.x;
    uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 4);
    w = k & 4 ? (w & 0xFFFF0000u) | o >> 16 : (w & 0x0000FFFFu) | o << 16;
    o = __shfl_xor_sync(0xFFFFFFFFu, w, 2);
    w = k & 2 ? (w & 0xFF00FF00u) | (o >> 8 & 0x00FF00FFu) : (w & 0x00FF00FFu) | (o << 8 & 0xFF00FF00u);
    o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
    return k & 1 ? (w & 0xF0F0F0F0u) | (o >> 4 & 0x0F0F0F0Fu) : (w & 0x0F0F0F0Fu) | (o << 4 & 0xF0F0F0F0u);
}

// Tokens [first, first + count) of sequence b are new: their positions, taken into the cache.
__device__ __forceinline__ void span(const Cache &c, const Tokens &t, int b, int &first, int &count)
{
    const int len = max(0, min(t.lens[b], c.T));
    count = t.counts ? max(0, min(t.counts[b], t.L)) : t.L;
    first = len - count;  // may be negative: those tokens are left out
}

template <int D>
__global__ void __launch_bounds__(kTok *Tile<D>::B) append_kernel(const Cache c, const Tokens t, int tiles, unsigned int *err)
{
    using M = Tile<D>;
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.x % c.Hkv, rest = blockIdx.x / c.Hkv, b = rest / tiles;
    int first, count;
    span(c, t, b, first, count);
    const int tile = max(first, 0) / kTok + rest % tiles, base = tile * kTok;
    const int lo = max(first - base, 0), hi = min(first + count - base, kTok);  // the tile's new tokens
    if (lo >= hi) return;
    uint8_t *const to = c.data + b * c.s_n + hk * c.s_h + tile * c.s_t;
    const int key = threadIdx.x % 32, blk = threadIdx.x / 32;
    const bool mine = key >= lo && key < hi;
    uint2 vc = make_uint2(0, 0);
    if (mine) {
        const int l = base + key - first;
        const uint4 *ks = reinterpret_cast<const uint4 *>(t.k + b * t.k_b + l * t.k_l + hk * t.k_h + blk * 16);
        const uint4 *vs = reinterpret_cast<const uint4 *>(t.v + b * t.v_b + l * t.v_l + hk * t.v_h + blk * 16);
        const uint4 k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
        uint32_t sk, sv;
        bool finite = true;
        *reinterpret_cast<uint2 *>(to + M::k_word(key, 2 * blk)) = quantise(k0, k1, c.k_scale, sk, finite);
        vc = quantise(v0, v1, c.v_scale, sv, finite);
        to[M::k_scale(key, blk)] = (uint8_t)sk;
        to[M::v_scale(key, blk)] = (uint8_t)sv;
        if (!finite) latch_error(err, QERL_ERR_NONFINITE);
    }
    __syncwarp();
    // the lane's words: dims blk 16 + key % 8 and 8 more, the eight tokens of key / 8
    const uint32_t words[2] = {turned(vc.x), turned(vc.y)};
    const int from = max(lo - key / 8 * 8, 0), upto = min(hi - key / 8 * 8, 8);
    if (from < upto) {
        const uint32_t mask = (upto == 8 ? 0xFFFFFFFFu : (1u << (4 * upto)) - 1u) & ~((1u << (4 * from)) - 1u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t *const at = reinterpret_cast<uint32_t *>(to + M::v_word(blk * 16 + h * 8 + key % 8, key / 8));
            *at = mask == 0xFFFFFFFFu ? words[h] : (*at & ~mask) | (words[h] & mask);
        }
    }
}

__device__ __forceinline__ uint32_t two(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The values of the last L tokens of each sequence, e2m1 * e4m3 * factor in FP32, rounded to bf16 (exact where the factor is a
// power of two); zeros for tokens before the first.
template <int D>
__global__ void __launch_bounds__(kTok *Tile<D>::B) read_kernel(const Cache c, const Tokens t, int tiles)
{
    using M = Tile<D>;
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.x % c.Hkv, rest = blockIdx.x / c.Hkv, b = rest / tiles;
    const int first = max(0, min(t.lens[b], c.T)) - t.L;
    // tiles of 32 from `first` rounded down, which may lie before the cache
    const int base = (first >= 0 ? first / kTok : -((kTok - 1 - first) / kTok)) * kTok + rest % tiles * kTok;
    const int lo = max(first - base, 0), hi = min(first + t.L - base, kTok);
    if (lo >= hi) return;
    const int key = threadIdx.x % 32, blk = threadIdx.x / 32;
    uint32_t ko[8] = {}, vo[8] = {};
    if (base >= 0) {
        const uint8_t *const from = c.data + b * c.s_n + hk * c.s_h + (base / kTok) * c.s_t;
        const uint2 kc = *reinterpret_cast<const uint2 *>(from + M::k_word(key, 2 * blk));
        uint32_t vc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) vc[h] = turned(*reinterpret_cast<const uint32_t *>(from + M::v_word(blk * 16 + h * 8 + key % 8, key / 8)));
        const float sk = __fmul_rn(e4m3_to_float(from[M::k_scale(key, blk)]), c.k_scale);
        const float sv = __fmul_rn(e4m3_to_float(from[M::v_scale(key, blk)]), c.v_scale);
        const auto values = [](uint32_t w, float f, uint32_t *o) {
            uint32_t v[4];
            codes_f16(w, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
                o[i] = two(x.x * f, x.y * f);
            }
        };
        values(kc.x, sk, ko), values(kc.y, sk, ko + 4);
        values(vc[0], sv, vo), values(vc[1], sv, vo + 4);
    }
    if (key < lo || key >= hi) return;
    const int l = base + key - first;
    uint4 *const k = reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(t.k) + b * t.k_b + l * t.k_l + hk * t.k_h + blk * 16);
    uint4 *const v = reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(t.v) + b * t.v_b + l * t.v_l + hk * t.v_h + blk * 16);
    k[0] = make_uint4(ko[0], ko[1], ko[2], ko[3]), k[1] = make_uint4(ko[4], ko[5], ko[6], ko[7]);
    v[0] = make_uint4(vo[0], vo[1], vo[2], vo[3]), v[1] = make_uint4(vo[4], vo[5], vo[6], vo[7]);
}

qerl_status tokens(const qerl_kv4_cache *c, int64_t L, const void *k, const int64_t *ks, const void *v, const int64_t *vs, const int32_t *lens,
                   const int32_t *counts, Cache &cache, Tokens &t, int64_t &tiles)
{
    if (!k || !v || !ks || !vs || !lens) return QERL_ERR_INVALID_ARG;
    QERL_TRY(check_cache(c, cache));
    if (L < 0 || L > 1 << 30) return QERL_ERR_SHAPE;
    for (int i = 0; i < 3; ++i) {
        if (ks[i] < 0 || vs[i] < 0 || ks[i] > (int64_t(1) << 40) || vs[i] > (int64_t(1) << 40)) return QERL_ERR_SHAPE;
        if (ks[i] % 8 || vs[i] % 8) return QERL_ERR_ALIGN;
    }
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(lens) & 3u) || (reinterpret_cast<uintptr_t>(counts) & 3u))
        return QERL_ERR_ALIGN;
    t = Tokens{static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(v), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
               lens, counts, (int)L};
    tiles = (L + kTok - 2) / kTok + 1;  // L tokens from any place in a tile on
    if (tiles * c->n > 0x7FFFFFFF / c->Hkv) return QERL_ERR_SHAPE;  // 2^55 at most, times Hkv it may pass 64 bits
    return QERL_OK;
}

}  // namespace

qerl_status check_cache(const qerl_kv4_cache *c, Cache &out)
{
    if (!c || !c->data) return QERL_ERR_INVALID_ARG;
    const auto fits = [](float f) { return f >= 1e-30f && f <= 1e30f; };
    if (!fits(c->k_scale) || !fits(c->v_scale)) return QERL_ERR_INVALID_ARG;
    const int64_t big = 1 << 30;
    if (c->n < 1 || c->T < 1 || c->Hkv < 1 || (c->D != 64 && c->D != 128) || c->n > big || c->T > big || c->Hkv > 65536) return QERL_ERR_SHAPE;
    for (int i = 0; i < 3; ++i) {
        if (c->stride[i] < 0 || c->stride[i] > (int64_t(1) << 42)) return QERL_ERR_SHAPE;
        if (c->stride[i] % 16) return QERL_ERR_ALIGN;
    }
    if (!aligned16(c->data)) return QERL_ERR_ALIGN;
    out = Cache{static_cast<uint8_t *>(c->data), c->stride[0], c->stride[1], c->stride[2], (int)c->n, (int)c->T, (int)c->Hkv, c->k_scale, c->v_scale};
    return QERL_OK;
}

}  // namespace kv4
}  // namespace qerl

using namespace qerl;

extern "C" qerl_status qerl_kv4_append(const qerl_kv4_cache *cache, int64_t L, const void *k, const int64_t *k_stride, const void *v,
                                       const int64_t *v_stride, const int32_t *lens, const int32_t *counts, qerl_stream_t stream)
{
    kv4::Cache c;
    kv4::Tokens t;
    int64_t tiles;
    QERL_TRY(kv4::tokens(cache, L, k, k_stride, v, v_stride, lens, counts, c, t, tiles));
    QERL_TRY(check_device());
    if (L == 0) return QERL_OK;
    const dim3 grid((unsigned)(tiles * c.n * c.Hkv));
    const bool chain = g_chain.load() != 0;
    if (cache->D == 128) return launched(launch_k(kv4::append_kernel<128>, grid, dim3(256), 0, as_cuda(stream), chain, c, t, (int)tiles, error_word()));
    return launched(launch_k(kv4::append_kernel<64>, grid, dim3(128), 0, as_cuda(stream), chain, c, t, (int)tiles, error_word()));
}

extern "C" qerl_status qerl_kv4_read(const qerl_kv4_cache *cache, int64_t L, const int32_t *lens, void *k, const int64_t *k_stride, void *v,
                                     const int64_t *v_stride, qerl_stream_t stream)
{
    kv4::Cache c;
    kv4::Tokens t;
    int64_t tiles;
    QERL_TRY(kv4::tokens(cache, L, k, k_stride, v, v_stride, lens, nullptr, c, t, tiles));
    if (kv4::repeated(c.n, L, c.Hkv, k_stride) || kv4::repeated(c.n, L, c.Hkv, v_stride)) return QERL_ERR_SHAPE;
    QERL_TRY(check_device());
    if (L == 0) return QERL_OK;
    const dim3 grid((unsigned)(tiles * c.n * c.Hkv));
    const bool chain = g_chain.load() != 0;
    if (cache->D == 128) return launched(launch_k(kv4::read_kernel<128>, grid, dim3(256), 0, as_cuda(stream), chain, c, t, (int)tiles));
    return launched(launch_k(kv4::read_kernel<64>, grid, dim3(128), 0, as_cuda(stream), chain, c, t, (int)tiles));
}
