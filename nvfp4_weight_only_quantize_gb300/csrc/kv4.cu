// The 4-bit cache's own operators: new tokens into it, and its values back.
//
// Append: a block of 16 values w gets the scale s = the smallest E4M3 number that
// is at least amax |w| / (6 f), f the cache's factor, and codes nearest(w / (s f)).
// A CTA takes one tile (32 tokens) of a sequence and head: one thread per token and
// block quantises 16 keys and 16 values, whose codes then turn through shared
// memory from one token per thread to eight tokens per word.  Words that hold
// older tokens too are read and merged; no two threads write to one word.
// Bound by HBM for prompts (reads 4 D, writes 9/8 D bytes per token and head), by
// the launch for single tokens.
#include "kv4.cuh"

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

// Sixteen values of a block: their codes (element i in bits 4 i) and the scale's byte.
__device__ __forceinline__ uint64_t quantise(const uint4 &u0, const uint4 &u1, float factor, uint32_t &scale, bool &finite)
{
    const uint32_t wd[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
    float w[16], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[2 * i] = bf16lo(wd[i]);
        w[2 * i + 1] = bf16hi(wd[i]);
        finite = finite && (wd[i] & 0x7F80u) != 0x7F80u && (wd[i] & 0x7F800000u) != 0x7F800000u;
        amax = fmaxf(amax, fmaxf(fabsf(w[2 * i]), fabsf(w[2 * i + 1])));
    }
    scale = e4m3_ceil(__fdiv_rn(amax, __fmul_rn(6.0f, factor)));
    const float unit = __fmul_rn(e4m3_to_float(scale), factor);
    uint64_t codes = 0;
    if (scale != 0u) {
#pragma unroll
        for (int i = 0; i < 16; ++i) codes |= (uint64_t)e2m1_code(__fdiv_rn(w[i], unit)) << (4 * i);
    }
    return codes;
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
    __shared__ uint64_t s_v[kTok][M::B];
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.x % c.Hkv, rest = blockIdx.x / c.Hkv, b = rest / tiles;
    int first, count;
    span(c, t, b, first, count);
    const int tile = max(first, 0) / kTok + rest % tiles, base = tile * kTok;
    const int lo = max(first - base, 0), hi = min(first + count - base, kTok);  // the tile's new tokens
    if (lo >= hi) return;
    uint8_t *const to = c.data + b * c.s_n + hk * c.s_h + tile * c.s_t;
    const int key = threadIdx.x / M::B, blk = threadIdx.x % M::B;
    const bool mine = key >= lo && key < hi;
    bool finite = true;
    if (mine) {
        const int l = base + key - first;
        const uint4 *ks = reinterpret_cast<const uint4 *>(t.k + b * t.k_b + l * t.k_l + hk * t.k_h + blk * 16);
        const uint4 *vs = reinterpret_cast<const uint4 *>(t.v + b * t.v_b + l * t.v_l + hk * t.v_h + blk * 16);
        const uint4 k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
        uint32_t sk, sv;
        const uint64_t kc = quantise(k0, k1, c.k_scale, sk, finite);
        s_v[key][blk] = quantise(v0, v1, c.v_scale, sv, finite);
        *reinterpret_cast<uint2 *>(to + M::k_word(key, 2 * blk)) = make_uint2((uint32_t)kc, (uint32_t)(kc >> 32));
        to[M::k_scale(key, blk)] = (uint8_t)sk;
        to[M::v_scale(key, blk)] = (uint8_t)sv;
    }
    if (!finite) latch_error(err, QERL_ERR_NONFINITE);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4 * D / (kTok * M::B); ++j) {
        const int w = j * kTok * M::B + threadIdx.x, q = (w / 4) % 4, d = (w / 128) * 32 + (w % 4) * 8 + (w / 16) % 8;
        if (8 * q + 8 <= lo || 8 * q >= hi) continue;
        uint32_t *const at = reinterpret_cast<uint32_t *>(to + M::VC) + w;
        uint32_t word = 0;
        if (8 * q < lo || 8 * q + 8 > hi) word = *at;
#pragma unroll
        for (int n = 0; n < 8; ++n)
            if (8 * q + n >= lo && 8 * q + n < hi) {
                const uint32_t code = (uint32_t)(s_v[8 * q + n][d / 16] >> (4 * (d % 16))) & 15u;
                word = (word & ~(15u << (4 * n))) | code << (4 * n);
            }
        *at = word;
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
    __shared__ __align__(16) uint8_t s_tile[M::BYTES];
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.x % c.Hkv, rest = blockIdx.x / c.Hkv, b = rest / tiles;
    const int first = max(0, min(t.lens[b], c.T)) - t.L;
    // tiles of 32 from `first` rounded down, which may lie before the cache
    const int base = (first >= 0 ? first / kTok : -((kTok - 1 - first) / kTok)) * kTok + rest % tiles * kTok;
    const int lo = max(first - base, 0), hi = min(first + t.L - base, kTok);
    if (lo >= hi) return;
    if (base >= 0) {
        const uint4 *const from = reinterpret_cast<const uint4 *>(c.data + b * c.s_n + hk * c.s_h + (base / kTok) * c.s_t);
        for (int i = threadIdx.x; i < M::BYTES / 16; i += kTok * M::B) reinterpret_cast<uint4 *>(s_tile)[i] = from[i];
    }
    __syncthreads();
    const int key = threadIdx.x / M::B, blk = threadIdx.x % M::B;
    if (key < lo || key >= hi) return;
    uint32_t ko[8] = {}, vo[8] = {};
    if (base >= 0) {
        const float sk = __fmul_rn(e4m3_to_float(s_tile[M::k_scale(key, blk)]), c.k_scale);
        const float sv = __fmul_rn(e4m3_to_float(s_tile[M::v_scale(key, blk)]), c.v_scale);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(s_tile + M::k_word(key, 2 * blk + h));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ko[4 * h + i] = two(e2m1_to_float(w >> (8 * i) & 15u) * sk, e2m1_to_float(w >> (8 * i + 4) & 15u) * sk);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const auto code = [&](int d) { return *reinterpret_cast<const uint32_t *>(s_tile + M::v_word(d, key / 8)) >> (4 * (key % 8)) & 15u; };
            vo[i] = two(e2m1_to_float(code(blk * 16 + 2 * i)) * sv, e2m1_to_float(code(blk * 16 + 2 * i + 1)) * sv);
        }
    }
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
    if (tiles * c->n * c->Hkv > 0x7FFFFFFF) return QERL_ERR_SHAPE;
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
    QERL_TRY(check_device());
    if (L == 0) return QERL_OK;
    const dim3 grid((unsigned)(tiles * c.n * c.Hkv));
    const bool chain = g_chain.load() != 0;
    if (cache->D == 128) return launched(launch_k(kv4::read_kernel<128>, grid, dim3(256), 0, as_cuda(stream), chain, c, t, (int)tiles));
    return launched(launch_k(kv4::read_kernel<64>, grid, dim3(128), 0, as_cuda(stream), chain, c, t, (int)tiles));
}
