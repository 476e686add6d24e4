// One AdamW step over many tensors (the LoRA adapters), FP32 or 8-bit states.
//
//   g = c grad                      c = min(1, max_norm / |grad|) over all tensors, or 1
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Elementwise and bound by HBM: with a bf16 parameter beside its FP32 master an
// element moves 30 bytes with FP32 states and 18 with 8-bit ones (plus 8/256 of
// scales), for some 100 instructions.  A warp owns one block of 256 elements,
// eight per lane, so every access is a 16-byte vector and a block's largest
// magnitude is one warp reduction; a CTA takes 32 blocks of one tensor.  On 80.7 M
// elements, the norm's read of the FP32 gradients (48 us at the copy rate) among
// it: FP32 states 413 us, 99 % of the measured copy rate; 8-bit states 439 us with
// the 80 us that handing both out in bf16 takes, 72 %: their step issues in 71 % of
// all slots, 100 instructions an element, most of them for the codes.
//
// 8-bit states, per block of 256 with an FP32 scale: m as sign, 3 exponent and 4
// mantissa bits; sqrt(v) (half of v's exponent range) as 3 exponent and 5
// mantissa bits, both with subnormals, and scale = (block's largest) / (largest
// code value).  A code's bits placed at the FP32 mantissa's top are the value
// times 2^-120, subnormals included, so both directions are a shift and two
// multiplies.  Rounding is stochastic: b2 = 0.999 moves sqrt(v) by about 0.0005
// of itself a step, far below half a code step (1/128), so rounding to nearest
// would freeze v within a few steps.  The random bits are Philox4x32-10
// (Salmon et al., SC'11) of (element / 4, tensor, step) under the key `seed`.
// A nonzero sqrt(v) keeps a code of at least 1: zero would leave only eps below m.
//
// Every product, sum, division and root that reaches a code is rounded by itself,
// so the codes do not depend on the compiler's choices.  The packed FP32 pairs
// are all fused multiply-adds with a 1 or a -0 that the compiler cannot see
// (kernel arguments): separate packed products and sums, explicitly rounded as
// they were, came out contracted.
#include <math.h>

#include <new>

#include "common.cuh"

namespace qerl {
namespace {

constexpr int kBlk = 256;             // elements that share a scale
constexpr int kThreads = 256;         // 8 warps
constexpr int kChunkBlks = 32;        // most blocks of a CTA's chunk: 4 per warp
constexpr int kSmallChunkBlks = 8;    // of a plan that leaves SMs idle otherwise: 1 per warp
constexpr int kNormThreads = 256, kNormPerSm = 4;
constexpr int kNormCtasMax = 1024;    // partial sums of the global norm
constexpr float kTopM = 1.9375f, kTopV = 1.96875f;  // largest code values: 2 - 2^-4, 2 - 2^-5
constexpr float kTiny = 7.888609052210118e-31f;     // 2^-100: smaller blocks are stored as zero

// One tensor as the kernels see it.
struct Rec {
    int64_t n;
    void *param;
    float *master;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale;
    double lr_scale, weight_decay;
    int64_t first_blk;  // blocks of the tensors before it
};
struct Chunk {
    uint32_t tensor, blk;  // blocks [blk, blk + the plan's chunk length) of the tensor
};

// Per-step values, rounded once to FP32 from the doubles of the call.
struct Step {
    double lr, lr_bc1;  // lr and lr / (1 - b1^t)
    float b1, c1, b2, c2, rs2, eps;
    uint32_t key0, key1, t;
    float one, nought;  // 1 and -0
    bool tame;          // eps is in the range where the approximate inverse of root + eps is a normal number
    int chunk;          // blocks of a chunk
};

// a b and a + b, each rounded once.
struct Pairs {
    float2 one, nought;
    __device__ __forceinline__ explicit Pairs(const Step &s) : one(make_float2(s.one, s.one)), nought(make_float2(s.nought, s.nought)) {}
    __device__ __forceinline__ float2 mul(float2 a, float2 b) const { return fma2(a, b, nought); }
    __device__ __forceinline__ float2 add(float2 a, float2 b) const { return fma2(a, one, b); }
    __device__ __forceinline__ float2 sub(float2 a, float2 b) const { return fma2(make_float2(-b.x, -b.y), one, a); }
};

__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = 0xD2511F53ull * c.x, p1 = 0xCD9E8D57ull * c.z;
        c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ k0, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k1, (uint32_t)p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

constexpr float kUp = 1.329227995784916e+36f;    // 2^120
constexpr float kDown = 7.52316384526264e-37f;   // 2^-120

// Code of y 2^120 in [0, top], rounded up with the probability of the part it drops.
template <int BITS>
__device__ __forceinline__ uint32_t to_code(float y, uint32_t rnd16)
{
    constexpr int DROP = 23 - BITS;
    const uint32_t u = __float_as_uint(y) + (rnd16 << (DROP - 16)) + (1u << (DROP - 17));
    return min(u >> DROP, (8u << BITS) - 1u);
}

// Eight consecutive elements of a lane, in FP32.
template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t i, int64_t n, bool full, float2 (&o)[4])
{
    if (full) {
        if (BF16) {
            const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
            o[0] = make_float2(bf16lo(a.x), bf16hi(a.x)), o[1] = make_float2(bf16lo(a.y), bf16hi(a.y));
            o[2] = make_float2(bf16lo(a.z), bf16hi(a.z)), o[3] = make_float2(bf16lo(a.w), bf16hi(a.w));
        } else {
            const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
            const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
            o[0] = make_float2(a.x, a.y), o[1] = make_float2(a.z, a.w), o[2] = make_float2(b.x, b.y), o[3] = make_float2(b.z, b.w);
        }
    } else {
        const auto one = [&](int j) {
            return i + j < n ? (BF16 ? bf16f(static_cast<const __nv_bfloat16 *>(p)[i + j]) : static_cast<const float *>(p)[i + j]) : 0.0f;
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = make_float2(one(2 * j), one(2 * j + 1));
    }
}
template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t i, int64_t n, bool full, const float2 (&o)[4])
{
    if (full) {
        if (BF16) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(o[j].x, o[j].y);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
            *reinterpret_cast<float4 *>(static_cast<float *>(p) + i + 4) = make_float4(o[2].x, o[2].y, o[3].x, o[3].y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) {
                const float x = j % 2 ? o[j / 2].y : o[j / 2].x;
                if (BF16)
                    static_cast<__nv_bfloat16 *>(p)[i + j] = __float2bfloat16_rn(x);
                else
                    static_cast<float *>(p)[i + j] = x;
            }
    }
}
__device__ __forceinline__ uint2 load_codes(const void *p, int64_t i, int64_t n, bool full)
{
    const uint8_t *c = static_cast<const uint8_t *>(p);
    if (full) return *reinterpret_cast<const uint2 *>(c + i);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (i + j < n) w[j / 4] |= (uint32_t)c[i + j] << (8 * (j % 4));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(void *p, int64_t i, int64_t n, bool full, const uint32_t (&w)[2])
{
    uint8_t *c = static_cast<uint8_t *>(p);
    if (full) {
        *reinterpret_cast<uint2 *>(c + i) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) c[i + j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
    }
}
// Largest FP32 bit pattern of non-negative values over a warp (a NaN is the largest).
__device__ __forceinline__ float warp_top(float x) { return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x))); }

// Square roots of eight values >= 0, each correctly rounded.  Markstein's scheme
// (IBM Journal of Research and Development 34, 1990): from an approximate inverse
// root, one coupled refinement of root and half inverse root, then the root's
// own residual.  It needs the residuals of v in FP32's normal range; where any of
// the eight is not, all of them go through the library's root.  (Before this and the
// packed pairs, with that one for every value, 80 M elements took 421 us with FP32
// states and 486 us with 8-bit ones, after 416 and 436.)
__device__ __forceinline__ bool roots(const Pairs &X, const float2 (&v)[4], float2 (&root)[4])
{
    bool plain = true;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        plain = plain && (v[j].x == 0.0f || (v[j].x > 1e-24f && v[j].x < 1e30f)) && (v[j].y == 0.0f || (v[j].y > 1e-24f && v[j].y < 1e30f));
    if (plain) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 y;
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(fmaxf(v[j].x, 1e-24f)));
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(fmaxf(v[j].y, 1e-24f)));
            float2 g = X.mul(v[j], y), h = X.mul(make_float2(0.5f, 0.5f), y);
            const float2 r = fma2(make_float2(-g.x, -g.y), h, make_float2(0.5f, 0.5f));
            g = fma2(g, r, g);
            h = fma2(h, r, h);
            root[j] = fma2(fma2(make_float2(-g.x, -g.y), g, v[j]), h, g);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) root[j] = make_float2(__fsqrt_rn(v[j].x), __fsqrt_rn(v[j].y));
    }
    return plain;
}
// a / b; `plain`: b comes from such roots and a tame eps, and the approximate inverse's quotient corrected by its residual
// will do (to a unit, and seldom that much).
__device__ __forceinline__ float2 quotient(const Pairs &X, float2 a, float2 b, bool plain)
{
    if (!plain) return make_float2(__fdiv_rn(a.x, b.x), __fdiv_rn(a.y, b.y));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(b.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(b.y));
    const float2 q = X.mul(a, r);
    return fma2(fma2(make_float2(-q.x, -q.y), b, a), r, q);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float larger(float a, float b)  // of values >= 0; a NaN is the largest
{
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// Magnitudes of bytes j and j + 1 of a word of codes, and a byte's sign.
template <int BITS>
__device__ __forceinline__ uint32_t code_bits(uint32_t w, int j)
{
    const int up = 23 - BITS - 8 * j;
    return (up >= 0 ? w << (up & 31) : w >> (-up & 31)) & (((8u << BITS) - 1u) << (23 - BITS));
}
template <int BITS>
__device__ __forceinline__ float2 code_at(const Pairs &X, uint32_t w, int j)
{
    return X.mul(make_float2(__uint_as_float(code_bits<BITS>(w, j)), __uint_as_float(code_bits<BITS>(w, j + 1))), both(kUp));
}
__device__ __forceinline__ float signed_like(float x, uint32_t w, int j)
{
    return __uint_as_float(__float_as_uint(x) | ((w << (24 - 8 * j)) & 0x80000000u));
}
__device__ __forceinline__ uint32_t signed_code(uint32_t code, float like) { return code | (like < 0.0f && code ? 128u : 0u); }

// A CTA takes one chunk, its warps' blocks side by side.  clip: nullptr, or {c, skip flag} from norm_kernel.
template <bool PB, bool GB, bool S8>
__global__ void __launch_bounds__(kThreads, S8 ? 6 : 3) step_kernel(const Rec *recs, const Chunk *chunks, Step st, const float *clip)
{
    __shared__ float s_lr, s_decay;
    pdl_trigger();
    const Chunk ch = chunks[gridDim.x - 1 - blockIdx.x];  // from the end: what the norm's pass read last is in L2
    const Rec &R = recs[ch.tensor];
    if (threadIdx.x == 0) {
        s_lr = (float)__dmul_rn(st.lr_bc1, R.lr_scale);
        s_decay = (float)__dadd_rn(1.0, -__dmul_rn(__dmul_rn(st.lr, R.lr_scale), R.weight_decay));
    }
    __syncthreads();
    const float step_size = s_lr, decay = s_decay;
    pdl_wait();
    float coef = 1.0f;
    if (clip) {
        if (clip[1] != 0.0f) return;  // the norm is not finite: the step is skipped
        coef = clip[0];
    }
    const int64_t n = R.n;
    const Pairs X(st);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float *const p32 = PB ? R.master : static_cast<float *>(R.param);
    // a block as it lies in memory
    struct Raw {
        float2 g[4], p[4], m[S8 ? 1 : 4], v[S8 ? 1 : 4];
        uint2 cm, cv;
        float ms, vs;
    };
    auto fetch = [&](int b, Raw &r) {
        const int64_t blk = (int64_t)ch.blk + b, i = blk * kBlk + lane * 8;
        if (b >= st.chunk || blk * kBlk >= n) return;
        const bool full = i + 8 <= n;
        load8<GB>(R.grad, i, n, full, r.g);
        load8<false>(p32, i, n, full, r.p);
        if constexpr (S8) {
            r.cm = load_codes(R.m, i, n, full), r.cv = load_codes(R.v, i, n, full);
            r.ms = R.m_scale[blk], r.vs = R.v_scale[blk];
        } else {
            load8<false>(R.m, i, n, full, r.m);
            load8<false>(R.v, i, n, full, r.v);
        }
    };
    // FP32 states: the next block's loads run under this one's arithmetic (417 -> 414 us on 80 M elements); 8-bit states
    // take the registers for twice the warps instead (463 -> 436 us)
    Raw next;
    if (!S8) fetch(warp, next);
    {
        for (int b = warp; b < st.chunk; b += kThreads / 32) {
            const int64_t blk = (int64_t)ch.blk + b;
            if (blk * kBlk >= n) break;
            const int64_t i = blk * kBlk + lane * 8;
            const bool full = i + 8 <= n;
            if (S8) fetch(b, next);
            float2 g[4], p[4], m[4], v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = next.g[j], p[j] = next.p[j];
            if constexpr (S8) {
                const uint2 cm = next.cm, cv = next.cv;
                const float ms = next.ms, vs = next.vs;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t wm = j < 2 ? cm.x : cm.y, wv = j < 2 ? cv.x : cv.y;
                    const int k = 2 * (j % 2);
                    m[j] = X.mul(code_at<4>(X, wm, k), both(ms));
                    m[j] = make_float2(signed_like(m[j].x, wm, k), signed_like(m[j].y, wm, k + 1));
                    v[j] = X.mul(code_at<5>(X, wv, k), both(vs));
                    v[j] = X.mul(v[j], v[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) m[j] = next.m[j], v[j] = next.v[j];
            }
            if (!S8) fetch(b + kThreads / 32, next);
            float2 root[4];
            float mtop = 0.0f, vtop = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 gc = clip ? X.mul(g[j], both(coef)) : g[j];
                m[j] = X.add(X.mul(m[j], both(st.b1)), X.mul(gc, both(st.c1)));
                v[j] = X.add(X.mul(v[j], both(st.b2)), X.mul(X.mul(gc, gc), both(st.c2)));
            }
            const bool plain = roots(X, v, root) && st.tame;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 den = X.add(X.mul(root[j], both(st.rs2)), both(st.eps));
                p[j] = X.add(X.mul(p[j], both(decay)), X.mul(both(-step_size), quotient(X, m[j], den, plain)));
                if (S8) {
                    mtop = larger(mtop, larger(fabsf(m[j].x), fabsf(m[j].y)));
                    vtop = larger(vtop, larger(root[j].x, root[j].y));
                }
            }
            store8<false>(p32, i, n, full, p);
            if (PB) store8<true>(R.param, i, n, full, p);
            if (S8) {
                // scale and inverse of both states, one division each in four lanes; 0 for a block below 2^-100
                mtop = warp_top(mtop);
                vtop = warp_top(vtop);
                const float amax = lane & 1 ? vtop : mtop, most = lane & 1 ? kTopV : kTopM;
                const float quot = amax < kTiny ? 0.0f : __fdiv_rn(lane & 2 ? most : amax, lane & 2 ? amax : most);
                const float sm = __shfl_sync(0xFFFFFFFFu, quot, 0), sv = __shfl_sync(0xFFFFFFFFu, quot, 1);
                const float im = __shfl_sync(0xFFFFFFFFu, quot, 2), iv = __shfl_sync(0xFFFFFFFFu, quot, 3);
                const uint32_t least = iv != 0.0f ? 1u : 0u;
                uint32_t wm[2] = {0, 0}, wv[2] = {0, 0};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint64_t grp = (uint64_t)(i / 4) + q;
                    const uint4 r4 =
                        philox4x32_10(make_uint4((uint32_t)grp, (uint32_t)(grp >> 32), ch.tensor, st.t), st.key0, st.key1);
                    const uint32_t r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const int j = 2 * q + k / 2;
                        const float2 ym = X.mul(X.mul(make_float2(fabsf(m[j].x), fabsf(m[j].y)), both(im)), both(kDown));
                        const float2 yv = X.mul(X.mul(root[j], both(iv)), both(kDown));
                        wm[q] += signed_code(to_code<4>(ym.x, r[k] & 0xFFFFu), m[j].x) << (8 * k);
                        wm[q] += signed_code(to_code<4>(ym.y, r[k + 1] & 0xFFFFu), m[j].y) << (8 * k + 8);
                        wv[q] += max(to_code<5>(yv.x, r[k] >> 16), root[j].x > 0.0f ? least : 0u) << (8 * k);
                        wv[q] += max(to_code<5>(yv.y, r[k + 1] >> 16), root[j].y > 0.0f ? least : 0u) << (8 * k + 8);
                    }
                }
                store_codes(R.m, i, n, full, wm);
                store_codes(R.v, i, n, full, wv);
                if (lane == 0) {
                    R.m_scale[blk] = sm;
                    R.v_scale[blk] = sv;
                }
            } else {
                store8<false>(R.m, i, n, full, m);
                store8<false>(R.v, i, n, full, v);
            }
        }
    }
}

// Global norm of the gradients: sum of squares as an unevaluated pair of floats
// per thread (the product's and the sum's rounding errors are kept: Dekker's and
// Knuth's exact transformations), joined in double in a fixed order, so that the
// norm is the same on every run and right to FP32's last bit, where the elements
// that matter lie between 1e-15 and 1e19 (their squares and the squares' errors are
// FP32 numbers).  The last CTA to arrive joins the partial sums and resets the
// counter.
// out: {c, 1 if the norm is not finite}; norm_out may be null.
template <bool GB>
__global__ void __launch_bounds__(kNormThreads, kNormPerSm)
    norm_kernel(const Rec *recs, const Chunk *chunks, uint32_t n_chunks, Step st, double max_norm, double *partial, unsigned int *arrived,
                float *out, float *norm_out)
{
    __shared__ double s_sum[kNormThreads / 32];
    __shared__ bool s_last;
    pdl_trigger();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    Chunk next = blockIdx.x < n_chunks ? chunks[blockIdx.x] : Chunk{0, 0};  // the table does not change
    pdl_wait();
    const Pairs X(st);
    float2 s = both(0.0f), e = both(0.0f);
    auto two_sum = [&](float2 p, float2 pe) {  // s + e += p + pe
        const float2 t = X.add(s, p), bb = X.sub(t, s);
        e = X.add(e, X.add(pe, X.add(X.sub(s, X.sub(t, bb)), X.sub(p, bb))));
        s = t;
    };
    for (uint32_t k = blockIdx.x; k < n_chunks; k += gridDim.x) {
        const Chunk ch = next;
        if (k + gridDim.x < n_chunks) next = chunks[k + gridDim.x];
        const int64_t n = min(recs[ch.tensor].n, ((int64_t)ch.blk + st.chunk) * kBlk), i0 = ((int64_t)ch.blk + warp) * kBlk + lane * 8;
        const void *grad = recs[ch.tensor].grad;
        constexpr int kEach = kChunkBlks / (kNormThreads / 32), kGap = kNormThreads / 32 * kBlk;
        float2 g[kEach][4];
#pragma unroll
        for (int b = 0; b < kEach; ++b) load8<GB>(grad, i0 + b * kGap, n, i0 + b * kGap + 8 <= n, g[b]);
#pragma unroll
        for (int b = 0; b < kEach; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = g[b][j], p = X.mul(x, x);
                two_sum(p, fma2(x, x, make_float2(-p.x, -p.y)));
            }
    }
    for (int o = 16; o; o >>= 1)
        two_sum(make_float2(__shfl_xor_sync(0xFFFFFFFFu, s.x, o), __shfl_xor_sync(0xFFFFFFFFu, s.y, o)),
                make_float2(__shfl_xor_sync(0xFFFFFFFFu, e.x, o), __shfl_xor_sync(0xFFFFFFFFu, e.y, o)));
    // An overflowed sum leaves NaN in its error term; the sum itself tells.
    const double d = isfinite(s.x + s.y) ? ((double)s.x + (double)s.y) + ((double)e.x + (double)e.y) : (double)s.x + (double)s.y;
    if (lane == 0) s_sum[warp] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < kNormThreads / 32; ++w) t += s_sum[w];
        partial[blockIdx.x] = t;
        __threadfence();
        s_last = atomicAdd(arrived, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double t = 0.0;
    for (unsigned int k = threadIdx.x; k < gridDim.x; k += kNormThreads) t += __ldcg(partial + k);
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if (lane == 0) s_sum[warp] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        double total = 0.0;
        for (int w = 0; w < kNormThreads / 32; ++w) total += s_sum[w];
        const double norm = sqrt(total);
        out[0] = (float)(norm > max_norm ? max_norm / norm : 1.0);
        out[1] = isfinite(norm) ? 0.0f : 1.0f;
        if (norm_out) *norm_out = (float)norm;
        *arrived = 0;
    }
}

// The values the 8-bit codes stand for, every tensor from a multiple of 256 on.
template <bool OB>
__global__ void __launch_bounds__(kThreads) read_kernel(const Rec *recs, const Chunk *chunks, Step st, void *m_out, void *v_out)
{
    pdl_trigger();
    const Chunk ch = chunks[blockIdx.x];
    const Rec &R = recs[ch.tensor];
    pdl_wait();
    const int64_t n = R.n;
    const Pairs X(st);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int b = warp; b < st.chunk; b += kThreads / 32) {
        const int64_t blk = (int64_t)ch.blk + b;
        if (blk * kBlk >= n) break;
        const int64_t i = blk * kBlk + lane * 8, to = R.first_blk * kBlk + i;
        const bool full = i + 8 <= n;
        const uint2 cm = load_codes(R.m, i, n, full), cv = load_codes(R.v, i, n, full);
        const float ms = R.m_scale[blk], vs = R.v_scale[blk];
        float2 m[4], v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t wm = j < 2 ? cm.x : cm.y, wv = j < 2 ? cv.x : cv.y;
            const int k = 2 * (j % 2);
            m[j] = X.mul(code_at<4>(X, wm, k), both(ms));
            m[j] = make_float2(signed_like(m[j].x, wm, k), signed_like(m[j].y, wm, k + 1));
            v[j] = X.mul(code_at<5>(X, wv, k), both(vs));
            v[j] = X.mul(v[j], v[j]);
        }
        store8<OB>(m_out, to, to + n - i, full, m);
        store8<OB>(v_out, to, to + n - i, full, v);
    }
}

size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

struct Layout {
    size_t recs, chunks, partial, clip, counter, total;
    int64_t n_chunks;
    int chunk;  // blocks of one
};

// false: a negative or too large size.
bool layout(const qerl_adamw_tensor *t, int64_t n, Layout &lo)
{
    int64_t blks = 0, chunks = 0;
    for (int64_t k = 0; k < n; ++k) {
        if (t[k].n < 0 || t[k].n > (int64_t(1) << 38)) return false;
        blks += (t[k].n + kBlk - 1) / kBlk;
    }
    // measured on 64 K elements: one block per warp 5 us, four 7 us; on 80 M the longer chunks save table reads
    lo.chunk = blks <= (int64_t)kChunkBlks * 2 * num_sms() ? kSmallChunkBlks : kChunkBlks;
    for (int64_t k = 0; k < n; ++k) chunks += (t[k].n + (int64_t)kBlk * lo.chunk - 1) / ((int64_t)kBlk * lo.chunk);
    if (chunks > 0x3FFFFFFF) return false;
    lo.n_chunks = chunks;
    lo.recs = 0;
    lo.chunks = round256(sizeof(Rec) * (size_t)n);
    lo.partial = lo.chunks + round256(sizeof(Chunk) * (size_t)chunks);
    lo.clip = lo.partial + sizeof(double) * kNormCtasMax;
    lo.counter = lo.clip + 256;
    lo.total = lo.counter + 256;
    return true;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace qerl

using namespace qerl;

struct qerl_adamw {
    Rec *recs;
    Chunk *chunks;
    double *partial;
    float *clip;
    unsigned int *counter;
    uint32_t n_chunks;
    int chunk;
    qerl_adamw_format fmt;
    int device;
};

extern "C" size_t qerl_adamw_ws_bytes(const qerl_adamw_tensor *tensors, int64_t n_tensors)
{
    Layout lo;
    if (!tensors || n_tensors < 1 || n_tensors > (1 << 24) || !layout(tensors, n_tensors, lo)) return 0;
    return lo.total;
}

extern "C" qerl_status qerl_adamw_plan(const qerl_adamw_tensor *tensors, int64_t n_tensors, const qerl_adamw_format *format,
                                       void *ws, size_t ws_bytes, qerl_adamw **plan)
{
    if (!plan) return QERL_ERR_INVALID_ARG;
    *plan = nullptr;
    if (!tensors || !format || n_tensors < 1 || n_tensors > (1 << 24)) return QERL_ERR_INVALID_ARG;
    const auto dtype_ok = [](int d) { return d == QERL_DTYPE_F32 || d == QERL_DTYPE_BF16; };
    if (!dtype_ok(format->param_dtype) || !dtype_ok(format->grad_dtype) || (format->state_bits != 8 && format->state_bits != 32))
        return QERL_ERR_INVALID_ARG;
    const bool pb = format->param_dtype == QERL_DTYPE_BF16, s8 = format->state_bits == 8;
    Layout lo;
    if (!layout(tensors, n_tensors, lo)) return QERL_ERR_SHAPE;
    for (int64_t k = 0; k < n_tensors; ++k) {
        const qerl_adamw_tensor &t = tensors[k];
        if (!isfinite(t.lr_scale) || !isfinite(t.weight_decay)) return QERL_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || pb != (t.master != nullptr) || (s8 && (!t.m_scale || !t.v_scale)))
            return QERL_ERR_INVALID_ARG;
        if (!aligned16(t.param) || !aligned16(t.master) || !aligned16(t.grad) || !aligned16(t.m) || !aligned16(t.v) ||
            (s8 && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))))
            return QERL_ERR_ALIGN;
    }
    if (!ws || ws_bytes < lo.total) return QERL_ERR_WORKSPACE;
    if (!aligned16(ws)) return QERL_ERR_ALIGN;
    QERL_TRY(check_device());

    Rec *recs = new (std::nothrow) Rec[n_tensors];
    Chunk *chunks = new (std::nothrow) Chunk[lo.n_chunks ? lo.n_chunks : 1];
    qerl_adamw *h = new (std::nothrow) qerl_adamw;
    qerl_status st = recs && chunks && h ? QERL_OK : QERL_ERR_HOST_MEMORY;
    if (st == QERL_OK) {
        int64_t c = 0, blk = 0;
        for (int64_t k = 0; k < n_tensors; ++k) {
            const qerl_adamw_tensor &t = tensors[k];
            recs[k] = Rec{t.n, t.param, t.master, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.lr_scale, t.weight_decay, blk};
            const int64_t nb = (t.n + kBlk - 1) / kBlk;
            for (int64_t b = 0; b < nb; b += lo.chunk) chunks[c++] = Chunk{(uint32_t)k, (uint32_t)b};
            blk += nb;
        }
        char *W = static_cast<char *>(ws);
        h->recs = reinterpret_cast<Rec *>(W + lo.recs);
        h->chunks = reinterpret_cast<Chunk *>(W + lo.chunks);
        h->partial = reinterpret_cast<double *>(W + lo.partial);
        h->clip = reinterpret_cast<float *>(W + lo.clip);
        h->counter = reinterpret_cast<unsigned int *>(W + lo.counter);
        h->n_chunks = (uint32_t)lo.n_chunks;
        h->chunk = lo.chunk;
        h->fmt = *format;
        cudaGetDevice(&h->device);
        // Work that is still queued on any stream may write to the workspace's memory on behalf of its last owner (an allocator
        // that orders by stream hands it out at once), and these copies wait for no non-blocking stream by themselves.
        if (cudaDeviceSynchronize() != cudaSuccess ||
            cudaMemcpy(h->recs, recs, sizeof(Rec) * n_tensors, cudaMemcpyHostToDevice) != cudaSuccess ||
            (lo.n_chunks &&
             cudaMemcpy(h->chunks, chunks, sizeof(Chunk) * lo.n_chunks, cudaMemcpyHostToDevice) != cudaSuccess) ||
            cudaMemset(h->counter, 0, 256) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
            st = QERL_ERR_CUDA;
    }
    delete[] recs;
    delete[] chunks;
    if (st != QERL_OK) {
        delete h;
        return st;
    }
    *plan = h;
    return QERL_OK;
}

namespace {
using StepFn = void (*)(const Rec *, const Chunk *, Step, const float *);
StepFn step_fn(bool pb, bool gb, bool s8)
{
    static const StepFn fns[8] = {step_kernel<false, false, false>, step_kernel<false, false, true>, step_kernel<false, true, false>,
                                  step_kernel<false, true, true>,   step_kernel<true, false, false>, step_kernel<true, false, true>,
                                  step_kernel<true, true, false>,   step_kernel<true, true, true>};
    return fns[(pb ? 4 : 0) + (gb ? 2 : 0) + (s8 ? 1 : 0)];
}
}  // namespace

extern "C" qerl_status qerl_adamw_step(const qerl_adamw *h, const qerl_adamw_hyper *hy, float *grad_norm, qerl_stream_t stream)
{
    if (!h || !hy) return QERL_ERR_INVALID_ARG;
    if (hy->step < 1 || hy->step > 0xFFFFFFFFll || !isfinite(hy->lr) || !(hy->beta1 >= 0.0 && hy->beta1 < 1.0) ||
        !(hy->beta2 >= 0.0 && hy->beta2 < 1.0) || !(hy->eps >= 0.0) || !isfinite(hy->eps) || !(hy->max_grad_norm >= 0.0) ||
        (grad_norm && hy->max_grad_norm == 0.0))
        return QERL_ERR_INVALID_ARG;
    if (!aligned(grad_norm, 4)) return QERL_ERR_ALIGN;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QERL_ERR_CUDA;
    if (dev != h->device) return QERL_ERR_INVALID_ARG;
    if (h->n_chunks == 0 && hy->max_grad_norm == 0.0) return QERL_OK;
    Step st = {};
    st.one = 1.0f, st.nought = -0.0f, st.chunk = h->chunk;
    st.lr = hy->lr;
    st.lr_bc1 = hy->lr / (1.0 - pow(hy->beta1, (double)hy->step));
    st.b1 = (float)hy->beta1;
    st.c1 = (float)(1.0 - hy->beta1);
    st.b2 = (float)hy->beta2;
    st.c2 = (float)(1.0 - hy->beta2);
    st.rs2 = (float)(1.0 / sqrt(1.0 - pow(hy->beta2, (double)hy->step)));
    st.eps = (float)hy->eps;
    st.tame = st.eps >= 1e-30f && st.eps <= 1e30f;
    st.key0 = (uint32_t)hy->seed;
    st.key1 = (uint32_t)(hy->seed >> 32);
    st.t = (uint32_t)hy->step;
    const bool gb = h->fmt.grad_dtype == QERL_DTYPE_BF16, chain = g_chain.load() != 0, clip = hy->max_grad_norm > 0.0;
    if (clip) {
        int64_t grid = h->n_chunks ? h->n_chunks : 1;
        if (grid > kNormPerSm * num_sms()) grid = kNormPerSm * num_sms();
        if (grid > kNormCtasMax) grid = kNormCtasMax;
        auto *fn = gb ? norm_kernel<true> : norm_kernel<false>;
        QERL_TRY(launched(launch_k(fn, dim3((unsigned)grid), dim3(kNormThreads), 0, as_cuda(stream), chain, (const Rec *)h->recs,
                                   (const Chunk *)h->chunks, h->n_chunks, st, hy->max_grad_norm, h->partial, h->counter, h->clip,
                                   grad_norm)));
    }
    if (h->n_chunks == 0) return QERL_OK;
    return launched(launch_k(step_fn(h->fmt.param_dtype == QERL_DTYPE_BF16, gb, h->fmt.state_bits == 8), dim3(h->n_chunks),
                             dim3(kThreads), 0, as_cuda(stream), chain, (const Rec *)h->recs, (const Chunk *)h->chunks, st,
                             clip ? (const float *)h->clip : (const float *)nullptr));
}

extern "C" qerl_status qerl_adamw_read_state(const qerl_adamw *h, void *m_out, void *v_out, int out_dtype, qerl_stream_t stream)
{
    if (!h || !m_out || !v_out || (out_dtype != QERL_DTYPE_F32 && out_dtype != QERL_DTYPE_BF16) || h->fmt.state_bits != 8)
        return QERL_ERR_INVALID_ARG;
    if (!aligned16(m_out) || !aligned16(v_out)) return QERL_ERR_ALIGN;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QERL_ERR_CUDA;
    if (dev != h->device) return QERL_ERR_INVALID_ARG;
    if (h->n_chunks == 0) return QERL_OK;
    Step st = {};
    st.one = 1.0f, st.nought = -0.0f, st.chunk = h->chunk;
    auto *fn = out_dtype == QERL_DTYPE_BF16 ? read_kernel<true> : read_kernel<false>;
    return launched(launch_k(fn, dim3(h->n_chunks), dim3(kThreads), 0, as_cuda(stream), g_chain.load() != 0, (const Rec *)h->recs,
                             (const Chunk *)h->chunks, st, m_out, v_out));
}

extern "C" void qerl_adamw_destroy(qerl_adamw *h) { delete h; }
