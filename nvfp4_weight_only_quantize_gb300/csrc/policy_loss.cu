// Clipped policy loss with a KL term from the logits, with the gradient of the
// logits (GRPO and DAPO), and the token log-probabilities alone.
//
// Per token t with logits x [V], chosen id, temperature tau:
//   p = softmax(x / tau),  logp = log p_id,  H = -sum p log p
//   rho = exp(logp - old),  d = ref - logp
//   l = -min(rho A, clip(rho, 1 - lo, 1 + hi) A) + beta (e^d - d - 1),  L = sum_t w_t l_t
//   dL/dlogp = w (beta (1 - e^d) - [not clipped] rho A)
//   dL/dx_j  = dL/dlogp (1[j = id] - p_j) / tau
//
// Bound by HBM: the logits read once and the gradient written once.  The factor
// dL/dlogp needs only its own row's sums, so one pass does both directions: a
// row is held on the chip by a cluster of up to eight CTAs, whose sums meet by warp
// shuffles, shared memory and one exchange through distributed shared memory, and
// the gradient is formed from what was read.  Two kernels:
//   - few or short rows: a cluster per row, the row in registers, (max, sum,
//     entropy sum) per thread.  16 rows of 16000 bf16: 8 us in a graph, of
//     which both launches are the most part;
//   - many long rows: clusters that stay, one CTA per SM, each row's slice copied
//     to a ring in shared memory while the rows before it are worked on.
//     Read and write together, of the measured copy rate: 4096 rows of 131072 bf16,
//     a tenth masked, 330 us (92 %); 1001 rows of 100003 FP32, 30 % masked, 123 us
//     (82 %: 138 of 152 SMs hold clusters of six, and 30 read rows a cluster leave
//     a tail); log-probabilities of 2048 x 131072 bf16 86 us (93 %).
// Rows longer than the cluster's registers or shared memory are read a second time
// (from L2, as a rule).
// Rows may start at any alignment: a row is walked in the aligned 16-byte
// vectors that hold it, whose two end vectors are read and written by element.
#include <float.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace qerl {
namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr int kMaxCluster = 8;
constexpr int kSumThreads = 512;

struct LossArgs {
    const void *x;
    int64_t ld, T, V;
    const void *ids;
    int ids64;
    const float *old_logp, *ref_logp, *adv, *weight;  // old_logp NULL: log-probabilities only
    float c, dc;                                      // log2(e) / tau, and ln 2 times what its rounding left relative to it
    float it, it_rest;                                // 1 / tau
    int far_tau;                                      // every row is taken by its second attempt
    float lo, hi, beta, gscale;                       // 1 - clip_low, 1 + clip_high, beta, grad_scale / tau
    float *logp, *entropy, *terms;                    // terms [T, 3]: w policy, w kl, w clipped
    void *dx;
    int64_t ldd;
    int dx_vec;                                       // the rows of dx start where those of x do, modulo 16 bytes
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Logits below kLow count as kLow; a row whose maximum lies beyond +-kFar is left to the second attempt.  kLow is the
// lower by far, so that a thread without values (all kLow, its maximum taken as -kFar) adds e^(kLow + kFar) = 0.
// That needs (kLow + kFar) / tau to be far below 0, and kLow / tau to be finite: temperatures outside [kTauLow, kTauHigh]
// leave every row to the second attempt.
constexpr float kLow = -1e30f, kFar = 1e29f, kTauLow = 1e-8f, kTauHigh = 1e20f;

__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, int rank, float4 v)
{
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// A 16-byte vector of logits: E values.
template <bool BF16>
struct Vec;
template <>
struct Vec<true> {
    static constexpr int E = 8;
    static constexpr uint32_t kFill = 0xFF80FF80u;  // -inf, -inf
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8])
    {
        f[0] = bf16lo(v.x), f[1] = bf16hi(v.x), f[2] = bf16lo(v.y), f[3] = bf16hi(v.y);
        f[4] = bf16lo(v.z), f[5] = bf16hi(v.z), f[6] = bf16lo(v.w), f[7] = bf16hi(v.w);
    }
    static __device__ __forceinline__ float top(const uint4 &v)  // ignores NaN, as fmaxf does
    {
        const auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // every value at least kLow; NaN stays
    static __device__ __forceinline__ uint4 raised(const uint4 &v)
    {
        const __nv_bfloat162 low = __float2bfloat162_rn(kLow);
        const auto up = [&](uint32_t w) {
            const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&w), low);
            return *reinterpret_cast<const uint32_t *>(&m);
        };
        return make_uint4(up(v.x), up(v.y), up(v.z), up(v.w));
    }
    static __device__ __forceinline__ uint4 without(const uint4 &v, int e)  // element e -inf
    {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j == e / 2) w[j] = e % 2 ? (w[j] & 0xFFFFu) | 0xFF800000u : (w[j] & 0xFFFF0000u) | 0xFF80u;
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float get(const void *p, int64_t i) { return bf16f(static_cast<const __nv_bfloat16 *>(p)[i]); }
    static __device__ __forceinline__ void put(void *p, int64_t i, float v) { static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v); }
};
template <>
struct Vec<false> {
    static constexpr int E = 4;
    static constexpr uint32_t kFill = 0xFF800000u;  // -inf
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[4])
    {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float top(const uint4 &v)
    {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4])
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ uint4 raised(const uint4 &v)
    {
        const auto up = [](uint32_t w) {
            uint32_t m;
            asm("max.NaN.f32 %0, %1, %2;" : "=r"(m) : "r"(w), "r"(__float_as_uint(kLow)));
            return m;
        };
        return make_uint4(up(v.x), up(v.y), up(v.z), up(v.w));
    }
    static __device__ __forceinline__ uint4 without(const uint4 &v, int e)
    {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j == e) w[j] = 0xFF800000u;
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float get(const void *p, int64_t i) { return static_cast<const float *>(p)[i]; }
    static __device__ __forceinline__ void put(void *p, int64_t i, float v) { static_cast<float *>(p)[i] = v; }
};

// Running (max, sum of e^(x - max), sum of e^(x - max) (x - max)), the last in log2 units.
struct Stat {
    float m, z, s;
};
// The statistics relative to the larger maximum M.  A part without values has
// z = s = 0 and m = -FLT_MAX; the clamp keeps 0 * -inf out.
__device__ __forceinline__ Stat moved(const Stat &a, float M, float c)
{
    const float d = fmaxf((a.m - M) * c, -1e4f), f = ex2(d);
    return Stat{M, a.z * f, f * fmaf(a.z, d, a.s)};
}

// The statistics of 2 x o lanes, in all of them.
__device__ __forceinline__ Stat over_warp(Stat t, float c, int o)
{
    float M = t.m;
    for (int k = o; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, k));
    t = moved(t, M, c);
    for (int k = o; k; k >>= 1) {
        t.z += __shfl_xor_sync(0xFFFFFFFFu, t.z, k);
        t.s += __shfl_xor_sync(0xFFFFFFFFu, t.s, k);
    }
    return t;
}

// A row as the aligned vectors that hold it: vector i holds elements [i E - off, i E - off + E).
template <bool BF16>
struct Row {
    using V = Vec<BF16>;
    static constexpr int E = V::E, S = 16 / E;
    const char *x;
    char *dx;
    int off, n, nvec, full0, full1;  // vectors [full0, full1) lie inside the row
    bool dx_vec;
    __device__ __forceinline__ Row(const LossArgs &a, int64_t row)
        : Row(a, static_cast<const char *>(a.x) + row * a.ld * S,
              a.dx ? static_cast<char *>(a.dx) + row * a.ldd * S : nullptr)
    {
    }
    __device__ __forceinline__ Row(const LossArgs &a, const char *x_row, char *dx_row)
    {
        x = x_row;
        dx = dx_row;
        off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / S);
        n = (int)a.V;
        nvec = (off + n + E - 1) / E;
        full0 = off ? 1 : 0;
        full1 = (off + n) / E;
        dx_vec = a.dx_vec != 0;
    }
    __device__ __forceinline__ const uint4 *vec() const { return reinterpret_cast<const uint4 *>(x - off * S); }
    __device__ __forceinline__ bool inside(int i) const { return i >= full0 && i < full1; }
    __device__ __forceinline__ uint4 load_end(int i) const  // an end vector, by element
    {
        uint32_t w[4] = {V::kFill, V::kFill, V::kFill, V::kFill};
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int e = i * E + j - off;
            if (e >= 0 && e < n) {
                if (BF16) {
                    const uint32_t h = reinterpret_cast<const uint16_t *>(x)[e];
                    w[j / 2] = j % 2 ? (w[j / 2] & 0xFFFFu) | h << 16 : (w[j / 2] & 0xFFFF0000u) | h;
                } else {
                    w[j % 4] = reinterpret_cast<const uint32_t *>(x)[e];
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(int i, const float (&f)[E]) const
    {
        if (dx_vec && inside(i)) {
            *reinterpret_cast<uint4 *>(dx + (int64_t)(i * E - off) * S) = V::pack(f);
            return;
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int e = i * E + j - off;
            if (e >= 0 && e < n) V::put(dx, e, f[j]);
        }
    }
};

// What one token brings besides its logits.
struct Token {
    float x_id, w, adv, old_logp, ref;
    int id;
    int takes;
};
template <bool BF16>
__device__ __forceinline__ Token token(const LossArgs &a, int64_t row)
{
    Token t = {};
    const int64_t id = a.ids64 ? static_cast<const int64_t *>(a.ids)[row] : static_cast<const int32_t *>(a.ids)[row];
    t.w = a.weight ? a.weight[row] : 1.0f;
    t.takes = t.w != 0.0f && id >= 0 && id < a.V;
    t.id = t.takes ? (int)id : 0;
    return t;
}
// The rest of it, for a row that takes part.
template <bool BF16>
__device__ __forceinline__ void token_inputs(const LossArgs &a, int64_t row, Token &t)
{
    t.x_id = Vec<BF16>::get(static_cast<const char *>(a.x) + row * a.ld * (16 / Vec<BF16>::E), t.id);
    if (a.old_logp) t.adv = a.adv[row], t.old_logp = a.old_logp[row];
    if (a.ref_logp) t.ref = a.ref_logp[row];
}

// From the row's statistics: its outputs (where `write`), the factor of its
// gradient, 1 - p of the chosen token, and the gradient's weight of e^((x - m) c).
// The statistics leave the chosen token out: with r the others' sum in units of
// its e^x, log p = -log(1 + r), which a sum that holds the 1 would round to
// 2^-24 absolutely, and tokens next to certain have r far below 1.  (The second
// attempt, `plain`, see below, takes them all.)  With mean = sum p y over the row's
// exponents, c's rounding moves ln z by its relative size times mean ln 2, up to
// 1e-6 at exponents of 20: taken back here.
__device__ __forceinline__ float4 factor(const LossArgs &a, int64_t row, const Token &t, const Stat &all, bool plain, bool write)
{
    const bool empty = plain && all.z == 0.0f;  // every logit -inf: no distribution, no part in the loss
    float logp, H, z;
    if (plain) {
        const float lz = logf(all.z);
        z = all.z;
        logp = empty ? -INFINITY : (t.x_id - all.m) * a.c * kLn2 - lz;
        H = empty ? 0.0f : lz - all.s / z * kLn2;
    } else {
        // +inf gives no distribution either: NaN, as NaN does
        const float y = t.x_id <= FLT_MAX ? fmaf(t.x_id, a.c, -all.m * a.c) : NAN;
        const float f = y >= -1.0f ? ex2(-y) : INFINITY, r = all.z * f;
        if (r < 0.5f) {
            const float lz = log1pf(r);
            z = all.z + ex2(y);
            const float mean = f * fmaf(-y, all.z, all.s) / (1.0f + r);
            logp = 0.0f - fmaf(a.dc, mean, lz);
            H = lz - mean * kLn2;
        } else {
            const float e = ex2(y);
            z = all.z + e;
            const float lz = logf(z);
            const float mean = fmaf(e, fmaxf(y, -1e4f), all.s) / z;
            // (x - m) / tau in nats with its rest, and ln z without what rounding m c moved the sums' unit by: y ln 2 would be
            // off by half a last place of y
            const float d = t.x_id - all.m, b = d - t.x_id, rest = (t.x_id - (d - b)) - (all.m + b);
            const float unit = fmaf(all.m, a.c, -all.m * a.c);
            logp = y == -INFINITY ? y : fmaf(d, a.it, fmaf(d, a.it_rest, fmaf(rest, a.it, fmaf(unit, kLn2, fmaf(-a.dc, mean, -lz)))));
            H = lz - mean * kLn2;
        }
    }
    float dlogp = 0.0f;
    if (write) {
        a.logp[row] = logp;
        if (a.entropy) a.entropy[row] = H;
    }
    if (!a.dx && !a.old_logp) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.old_logp) {
        const float A = t.adv, rho = expf(logp - t.old_logp);
        const float d = a.ref_logp ? t.ref - logp : 0.0f, em = expm1f(d);
        // a NaN ratio or advantage is not clipped: it reaches the loss and the gradient
        const bool cut = A >= 0.0f ? rho > a.hi : A < 0.0f && rho < a.lo;
        const float policy = -((cut ? (A >= 0.0f ? a.hi : a.lo) : rho) * A);
        if (!empty) dlogp = t.w * ((a.beta != 0.0f ? -a.beta * em : 0.0f) - (cut ? 0.0f : rho * A));
        if (write) {
            a.terms[3 * row] = empty ? 0.0f : t.w * policy;
            a.terms[3 * row + 1] = empty ? 0.0f : t.w * (em - d);
            a.terms[3 * row + 2] = !empty && cut ? t.w : 0.0f;
        }
    }
    const float coef = dlogp * a.gscale;
    return make_float4(coef, empty ? 0.0f : -expm1f(logp), empty ? 0.0f : -coef / z, 0.0f);
}
__device__ __forceinline__ void no_part(const LossArgs &a, int64_t row)
{
    a.logp[row] = 0.0f;
    if (a.entropy) a.entropy[row] = 0.0f;
    if (a.terms) a.terms[3 * row] = a.terms[3 * row + 1] = a.terms[3 * row + 2] = 0.0f;
}

// A thread's sums in pairs of lanes: y = x c + shift in one rounding with shift =
// -max c, and logits no lower than kLow, so that 0 * -inf never enters s.  Where
// a row's maximum lies beyond +-kFar (a row of the type's lowest values, or all
// -inf) the row is taken again as (x - max) c (`plain`).
struct Sums {
    float2 z, s;
};
template <bool BF16>
__device__ __forceinline__ void add(Sums &t, const uint4 &q, float c, float shift)
{
    constexpr int E = Vec<BF16>::E;
    float f[E];
    Vec<BF16>::unpack(Vec<BF16>::raised(q), f);
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        const float2 y = fma2(make_float2(f[j], f[j + 1]), make_float2(c, c), make_float2(shift, shift));
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        t.z = add2(t.z, e);
        t.s = fma2(e, y, t.s);
    }
}
// The statistics and N vectors more.
template <bool BF16, int N>
__device__ __forceinline__ void add_block(Stat &st, const uint4 (&q)[N], float c)
{
    float m = st.m;
#pragma unroll
    for (int k = 0; k < N; ++k) m = fmaxf(m, Vec<BF16>::top(q[k]));
    st = moved(st, m, c);
    const float shift = -fmaxf(m, -kFar) * c;
    Sums t = {make_float2(st.z, 0.0f), make_float2(st.s, 0.0f)};
#pragma unroll
    for (int k = 0; k < N; ++k) add<BF16>(t, q[k], c, shift);
    st.z = t.z.x + t.z.y;
    st.s = t.s.x + t.s.y;
}
template <bool BF16>
__device__ __forceinline__ void add_plain(Stat &st, const uint4 &q, float c)
{
    st = moved(st, fmaxf(st.m, Vec<BF16>::top(q)), c);
    float f[Vec<BF16>::E];
    Vec<BF16>::unpack(q, f);
#pragma unroll
    for (int j = 0; j < Vec<BF16>::E; ++j) {
        const float y = (f[j] - st.m) * c, e = ex2(y);
        st.z += e;
        st.s = fmaf(e, fmaxf(y, -1e4f), st.s);
    }
}
__device__ __forceinline__ bool far_off(const Stat &t) { return !(fabsf(t.m) < kFar); }

// k e^(x c + shift) of one vector's elements.
template <bool BF16>
__device__ __forceinline__ uint4 scaled(const uint4 &q, float c, float shift, float k)
{
    constexpr int E = Vec<BF16>::E;
    float f[E];
    Vec<BF16>::unpack(q, f);
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        const float2 y = fma2(make_float2(f[j], f[j + 1]), make_float2(c, c), make_float2(shift, shift));
        const float2 g = mul2(make_float2(ex2(y.x), ex2(y.y)), make_float2(k, k));
        f[j] = g.x, f[j + 1] = g.y;
    }
    return Vec<BF16>::pack(f);
}

// The gradient of one vector, k = -factor / z.
template <bool BF16>
__device__ __forceinline__ void grad(const Row<BF16> &r, int i, const uint4 &q, const Stat &all, float c, float k, bool plain)
{
    constexpr int E = Vec<BF16>::E;
    float f[E];
    Vec<BF16>::unpack(q, f);
    if (plain) {
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = ex2((f[j] - all.m) * c) * k;
    } else {
        const float shift = -all.m * c;
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 y = fma2(make_float2(f[j], f[j + 1]), make_float2(c, c), make_float2(shift, shift));
            const float2 g = mul2(make_float2(ex2(y.x), ex2(y.y)), make_float2(k, k));
            f[j] = g.x, f[j + 1] = g.y;
        }
    }
    r.store(i, f);
}

// ------------------------------------------------------------------ few rows or short ones: one cluster per row
// NT threads per CTA; HOLD: a thread's NV vectors stay in registers, else they are read twice.
template <bool BF16, int NT, int NV, bool HOLD>
__global__ void __launch_bounds__(NT, (NV > 4 ? 512 : 1024) / NT) policy_kernel(LossArgs a, int cs)
{
    using V = Vec<BF16>;
    constexpr int E = V::E, NW = NT / 32;
    static_assert(NW <= kMaxCluster, "the warps' statistics are joined in eight lanes");
    __shared__ float4 s_warp[NW];
    __shared__ alignas(16) float4 s_cta[2][kMaxCluster];
    __shared__ float4 s_factor;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t row = blockIdx.x / cs;
    const int rank = blockIdx.x % cs;
    pdl_trigger();
    if (cs > 1) cluster_arrive_relaxed();  // peers' shared memory may be written once all of them run
    pdl_wait();

    const Row<BF16> r(a, row);
    const int per = (r.nvec + cs - 1) / cs, v0 = rank * per, v1 = min(v0 + per, r.nvec);
    const uint4 *xv = r.vec();
    Token tok = token<BF16>(a, row);
    if (!tok.takes) {  // the logits are not read
        const float zero[E] = {};
        if (r.dx)
            for (int i = v0 + tid; i < v1; i += NT) r.store(i, zero);
        if (rank == 0 && tid == 0) no_part(a, row);
        if (cs > 1) cluster_wait();
        return;
    }
    if (tid == 0) token_inputs<BF16>(a, row, tok);  // arrives beside the logits

    const int own = (tok.id + r.off) / E;  // the vector that holds the chosen token
    const bool owner = own >= v0 && own < v1 && (own - v0) % NT == tid;
    const uint4 nothing = make_uint4(V::kFill, V::kFill, V::kFill, V::kFill);
    uint4 hold[NV];
    Stat st = {-FLT_MAX, 0.0f, 0.0f}, all;
    if (HOLD) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = v0 + k * NT + tid;
            hold[k] = nothing;
            if (i < v1 && r.inside(i)) hold[k] = xv[i];
        }
        if (r.full0 || r.full1 < r.nvec) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int i = v0 + k * NT + tid;
                if (i < v1 && !r.inside(i)) hold[k] = r.load_end(i);
            }
        }
        if (owner) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (v0 + k * NT + tid == own) hold[k] = V::without(hold[k], (tok.id + r.off) % E);
        }
        add_block<BF16, NV>(st, hold, a.c);
    } else {
        for (int i = v0 + tid; i < v1; i += NV * NT) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                hold[k] = nothing;
                if (i + k * NT < v1 && r.inside(i + k * NT)) hold[k] = xv[i + k * NT];
            }
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (i + k * NT < v1 && !r.inside(i + k * NT)) hold[k] = r.load_end(i + k * NT);
            if (owner) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (i + k * NT == own) hold[k] = V::without(hold[k], (tok.id + r.off) % E);
            }
            add_block<BF16, NV>(st, hold, a.c);
        }
    }
    // the row's statistics from every thread's, in all threads
    auto join = [&](const Stat &mine, int buf) {
        Stat t = over_warp(mine, a.c, 16);
        if (lane == 0) s_warp[warp] = make_float4(t.m, t.z, t.s, 0.0f);
        __syncthreads();
        if (warp == 0) {
            const float4 q = lane < NW ? s_warp[lane] : make_float4(-FLT_MAX, 0.0f, 0.0f, 0.0f);
            t = over_warp(Stat{q.x, q.y, q.z}, a.c, 4);  // in lanes 0 to 7, which send it
            if (cs > 1) {
                cluster_wait();
                if (lane < cs) st_cluster_v4(ptx::smem_u32(&s_cta[buf][rank]), lane, make_float4(t.m, t.z, t.s, 0.0f));
            } else if (lane == 0) {
                s_cta[buf][0] = make_float4(t.m, t.z, t.s, 0.0f);
            }
        } else if (cs > 1) {
            cluster_wait();
        }
        if (cs > 1) {
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        const float4 q = (lane & 7) < cs ? s_cta[buf][lane & 7] : make_float4(-FLT_MAX, 0.0f, 0.0f, 0.0f);
        return over_warp(Stat{q.x, q.y, q.z}, a.c, 4);
    };
    all = join(st, 0);
    const bool plain = a.far_tau || far_off(all);
    if (plain) {
        if (cs > 1) cluster_arrive();
        st = Stat{-FLT_MAX, 0.0f, 0.0f};
        for (int i = v0 + tid; i < v1; i += NT) add_plain<BF16>(st, r.inside(i) ? xv[i] : r.load_end(i), a.c);
        all = join(st, 1);
    }
    if (tid == 0) s_factor = factor(a, row, tok, all, plain, rank == 0);
    if (!r.dx) return;
    __syncthreads();
    const float coef = s_factor.x, k = s_factor.z;
    if (HOLD && !plain) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = v0 + j * NT + tid;
            if (i < v1) grad<BF16>(r, i, hold[j], all, a.c, k, false);
        }
    } else {
        for (int i = v0 + tid; i < v1; i += NT) grad<BF16>(r, i, r.inside(i) ? xv[i] : r.load_end(i), all, a.c, k, plain);
    }
    if (owner) V::put(r.dx, tok.id, coef * s_factor.y);
}

// ------------------------------------------------------------------ many long rows: a ring of row slices in shared memory
// The others' statistics are taken relative to the chosen token's logit, which the copies bring along: no maximum, and sums
// that only add.  Where their sum reaches kManyTimes (a token some 33 nats below the maximum) or is not finite, the row is
// taken again with its maximum: beyond, the exponents' own rounding grows, and the gradient's factor -coef / z would lose its
// digits among FP32's subnormals (from 75 nats on, at weights that a loss has).
// Persistent clusters, one CTA per SM; a CTA's slice of a row is one bulk copy
// into a stage of its ring.  Three roles run apart, joined by barriers only:
//   - sixteen warps compute: the statistics of row n + depth, then the gradient of
//     row n, so that no one waits for a row's exchange;
//   - one warp joins the warps' statistics and sends them to the cluster's CTAs (a
//     16-byte asynchronous store to each, counted by the receiver's barrier);
//   - one warp receives them and forms the row's factor;
//   - one warp runs ahead with the copies and the tokens' inputs.
// Every wait is bounded: past two seconds the error is latched and the CTA winds up.
constexpr int kRingWarps = 16, kRingThreads = (kRingWarps + 3) * 32, kMaxStages = 6;
constexpr size_t kRingBytes = 204 << 10;
constexpr float kManyTimes = 281474976710656.0f;  // 2^48
// Rows between a row's statistics and its gradient: at most kRows - 1.  Rows whose tokens are in flight: those, the
// stages that the copies may run ahead, and one.
constexpr int kRows = 4, kTokens = 16;
// Buffers of received statistics.  A CTA sends row n + 8 after its own warps took row n + 8 - kRows to its end, so after
// every other CTA sent that row, so after that CTA had received row n + 8 - 2 kRows = n.
constexpr int kMet = 2 * kRows;
static_assert(kTokens >= kRows + kMaxStages + 1, "a token outlives its stage");

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(ptx::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void st_async_v4(void *addr, uint64_t *bar, int rank, float4 v)
{
    uint32_t to, tb;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(ptx::smem_u32(addr)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(tb) : "r"(ptx::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to), "f"(v.x),
                 "f"(v.y), "f"(v.z), "f"(v.w), "r"(tb)
                 : "memory");
}

// A walk over the ring's stages.
struct Stage {
    int st, parity;
    __device__ __forceinline__ void next(int stages)
    {
        if (++st == stages) st = 0, parity ^= 1;
    }
};

// The rows [first, end) of cluster c of n.  A row that takes no part is written but not read, so the rows are shared out by
// what they move (a read and a write cost 16 each, a row itself 1); a row is of the cluster that its middle falls to.
// Against every n-th row, of 1001 rows of 100003 FP32 logits with 30 % masked (the fullest of 15 clusters has some 6 % more
// than the mean there): 135 -> 130 us.  4096 rows of 131072 bf16 with 10 % masked, which every n-th row balances by itself, pay
// for the sums over the weights: 323 -> 327 us.  Masks in long runs would be worse for every n-th row than either.
template <bool BF16>
__device__ __forceinline__ void my_rows(const LossArgs &a, int64_t c, int64_t n, int64_t &first, int64_t &end)
{
    if (!a.weight) {
        first = a.T * c / n, end = a.T * (c + 1) / n;
        return;
    }
    __shared__ int64_t s_cost[kRingThreads / 32];
    __shared__ unsigned int s_before[2];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t per = (a.T + kRingThreads - 1) / kRingThreads;
    const int64_t t0 = min((int64_t)tid * per, a.T), t1 = min(t0 + per, a.T);
    const auto cost = [&](int64_t row) { return (token<BF16>(a, row).takes ? 16 : 0) + (a.dx ? 16 : 0) + 1; };
    int64_t mine = 0;
    for (int64_t t = t0; t < t1; ++t) mine += cost(t);
    int64_t to = mine;  // the costs of the warp's threads up to this one
    for (int o = 1; o < 32; o *= 2) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, to, o);
        if (lane >= o) to += v;
    }
    if (lane == 31) s_cost[warp] = to;
    if (tid < 2) s_before[tid] = 0;
    __syncthreads();
    int64_t all = 0, at = to - mine;
    for (int w = 0; w < kRingThreads / 32; ++w) {
        if (w < warp) at += s_cost[w];
        all += s_cost[w];
    }
    unsigned int before[2] = {0, 0};  // rows of the clusters before this one, and of those up to it
    for (int64_t t = t0; t < t1; ++t) {
        const int k = cost(t);
        const int64_t middle = (2 * at + k) * n;
        before[0] += middle < 2 * all * c;
        before[1] += middle < 2 * all * (c + 1);
        at += k;
    }
    for (int j = 0; j < 2; ++j) {
        const unsigned int sum = __reduce_add_sync(0xFFFFFFFFu, before[j]);
        if (lane == 0) atomicAdd(&s_before[j], sum);
    }
    __syncthreads();
    first = s_before[0], end = s_before[1];
}

template <bool BF16>
__global__ void __launch_bounds__(kRingThreads, 1)
    policy_ring_kernel(LossArgs a, int cs, int stages, int depth, uint32_t stage_bytes, unsigned int *err)
{
    using V = Vec<BF16>;
    constexpr int E = V::E, NT = kRingWarps * 32;
    extern __shared__ __align__(128) uint8_t ring[];
    // a stage's data is there / it may be filled again; row n's statistics (buffers n % kRows): every warp's are there,
    // the row's are; the cluster's; the same for the second attempt
    __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_part[kRows], s_met[kMet], s_ready[kRows], s_part2, s_met2[2],
        s_ready2;
    __shared__ alignas(16) float4 s_cta[kMet][kMaxCluster], s_cta2[2][kMaxCluster];
    __shared__ alignas(16) float2 s_sum[kRows][NT];  // every thread's (z, s)
    __shared__ float4 s_warp[kRingWarps];           // every warp's statistics, second attempt
    __shared__ bool s_plain[kRows];
    __shared__ Token s_tok[kTokens];
    __shared__ Stat s_all[kRows];
    __shared__ float4 s_factor[kRows];
    __shared__ int s_stop;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int rank = blockIdx.x % cs;
    if (tid == 0) {
        for (int k = 0; k < stages; ++k) {
            ptx::mbar_init(&s_full[k], 1);
            ptx::mbar_init(&s_empty[k], kRingWarps);
        }
        for (int k = 0; k < kRows; ++k) {
            ptx::mbar_init(&s_part[k], kRingWarps);
            ptx::mbar_init(&s_ready[k], 2);  // sent, and received
        }
        for (int k = 0; k < kMet; ++k) ptx::mbar_init(&s_met[k], 1);
        for (int k = 0; k < 2; ++k) ptx::mbar_init(&s_met2[k], 1);
        ptx::mbar_init(&s_part2, kRingWarps);
        ptx::mbar_init(&s_ready2, 1);
        s_stop = 0;
        ptx::fence_mbar_init();
    }
    pdl_trigger();
    __syncthreads();
    if (cs > 1) {
        cluster_arrive();
        cluster_wait();
    }
    pdl_wait();
    int64_t first, end;
    my_rows<BF16>(a, blockIdx.x / cs, gridDim.x / cs, first, end);

    const uint64_t limit_ns = 2000000000ull;
    // true for the whole warp, or false for it
    auto wait = [&](uint64_t *bar, int parity) -> bool {
        bool ok = ptx::mbar_try_wait(bar, (uint32_t)parity);
        if (!ok) {
            const uint64_t until = ptx::globaltimer_ns() + limit_ns;
            while (!(ok = ptx::mbar_try_wait_sleep(bar, (uint32_t)parity, 20000u))) {
                if (*reinterpret_cast<volatile int *>(&s_stop)) break;
                if (ptx::globaltimer_ns() > until) {
                    *reinterpret_cast<volatile int *>(&s_stop) = 1;
                    latch_error(err, QERL_ERR_TIMEOUT);
                    break;
                }
            }
        }
        return __all_sync(0xFFFFFFFFu, ok);
    };
    // x / cs for the few 10^4 vectors of a row, without a division's latency at every row (84 us against 88)
    const uint32_t inv_cs = 0xFFFFFFFFu / (uint32_t)cs + 1;
    const auto slice = [&](const Row<BF16> &r, int &v0, int &len) {
        const int per = cs == 1 ? r.nvec : (int)__umulhi((uint32_t)(r.nvec + cs - 1), inv_cs);
        v0 = rank * per;
        len = max(0, min(per, r.nvec - v0));
    };

    // (z, s) over the CTA's threads, in all lanes
    auto of_threads = [&](int buf) {
        const float4 *p = reinterpret_cast<const float4 *>(s_sum[buf]);
        float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < NT / 64; ++k) {
            const float4 q = p[k * 32 + lane];
            t = add2(t, add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
        }
        for (int o = 16; o; o >>= 1) {
            t.x += __shfl_xor_sync(0xFFFFFFFFu, t.x, o);
            t.y += __shfl_xor_sync(0xFFFFFFFFu, t.y, o);
        }
        return t;
    };

    if (warp == kRingWarps) {  // copies
        int n = 0;
        Token tok = {};
        Stage at = {0, 0};
        for (int64_t row = first; row < end; ++row, ++n, at.next(stages)) {
            const int st = at.st;
            if (n % 32 == 0 && row + lane < end) {  // the next 32 rows' tokens, one per lane
                tok = token<BF16>(a, row + lane);
                if (tok.takes) token_inputs<BF16>(a, row + lane, tok);
            }
            __syncwarp();
            const bool takes = __shfl_sync(0xFFFFFFFFu, tok.takes, n % 32) != 0;
            const Row<BF16> r(a, row);
            int v0, len;
            slice(r, v0, len);
            // the row's ends by element: lane 0 the first vector, lane 1 the last
            const int last = r.nvec - 1;
            const bool edge = takes && (lane == 0 ? v0 == 0 && r.full0 : lane == 1 && last >= max(v0, r.full1) && last < v0 + len && (last > 0 || !r.full0));
            uint4 e = make_uint4(0, 0, 0, 0);
            if (edge) e = r.load_end(lane == 0 ? 0 : last);
            __syncwarp();
            if (n >= stages && !wait(&s_empty[st], at.parity ^ 1)) break;
            uint8_t *to = ring + st * stage_bytes;
            const int b0 = max(v0, r.full0), b1 = min(v0 + len, r.full1);
            const uint32_t bytes = takes && b1 > b0 ? (uint32_t)(b1 - b0) * 16u : 0u;
            ptx::fence_proxy_async_smem();  // what was stored into the stage comes before the copy
            if (lane == 0 && bytes) bulk_load(to + (b0 - v0) * 16, r.vec() + b0, bytes, &s_full[st]);
            if (edge) *reinterpret_cast<uint4 *>(to + (lane == 0 ? 0 : last - v0) * 16) = e;
            if (lane == n % 32) s_tok[n % kTokens] = tok;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_expect_tx(&s_full[st], bytes);
            __syncwarp();
        }
        // no copy may be in flight when the CTA ends
        if (lane == 0 && *reinterpret_cast<volatile int *>(&s_stop)) {
            const uint64_t until = ptx::globaltimer_ns() + limit_ns;
            for (int k = max(0, n - stages); k < n; ++k)
                while (!ptx::mbar_try_wait(&s_full[k % stages], (k / stages) & 1) && ptx::globaltimer_ns() < until) {
                }
        }
    } else if (warp == kRingWarps + 1) {  // sends
        int met = 0;
        const int rows = (int)(end - first);
        for (int n = 0; n < rows; ++n) {
            const int buf = n % kRows;
            if (!wait(&s_part[buf], (n / kRows) & 1)) break;
            if (cs > 1 && s_tok[n % kTokens].takes) {
                const float2 t = of_threads(buf);
                if (lane < cs) st_async_v4(&s_cta[met % kMet][rank], &s_met[met % kMet], lane, make_float4(t.x, t.y, 0.0f, 0.0f));
                ++met;
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s_ready[buf]);
            __syncwarp();
        }
    } else if (warp == kRingWarps + 2) {  // receives
        int n = 0, met = 0, again = 0;
        // what CTA lane % 8 sent; false where the wait ran out
        auto receive = [&](const float4 *from, uint64_t *bar, int parity, float4 &q) -> bool {
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)cs * 16u);
            __syncwarp();
            if (!wait(bar, parity)) return false;
            if ((lane & 7) < cs) q = from[lane & 7];
            return true;
        };
        for (int64_t row = first; row < end; ++row, ++n) {
            const int buf = n % kRows;
            const Token &tok = s_tok[n % kTokens];
            if (!wait(&s_part[buf], (n / kRows) & 1)) break;
            if (!tok.takes) {
                if (lane == 0) {
                    if (rank == 0) no_part(a, row);
                    ptx::mbar_arrive(&s_ready[buf]);
                }
                __syncwarp();
                continue;
            }
            float2 z;
            if (cs == 1) {  // launched without a cluster: nothing to exchange, no access to a peer
                z = of_threads(buf);
            } else {
                float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!receive(s_cta[met % kMet], &s_met[met % kMet], (met / kMet) & 1, q)) break;
                z = make_float2(q.x, q.y);
                for (int o = 4; o; o >>= 1) {
                    z.x += __shfl_xor_sync(0xFFFFFFFFu, z.x, o);
                    z.y += __shfl_xor_sync(0xFFFFFFFFu, z.y, o);
                }
            }
            Stat t = {tok.x_id, z.x, z.y};  // of the others
            ++met;
            const bool plain = a.far_tau || far_off(t) || !(t.z < kManyTimes) || !isfinite(t.s);
            if (lane == 0) {
                s_all[buf] = t;
                s_plain[buf] = plain;
                if (!plain) s_factor[buf] = factor(a, row, tok, t, false, rank == 0);
                ptx::mbar_arrive(&s_ready[buf]);
            }
            __syncwarp();
            if (plain) {
                if (!wait(&s_part2, again & 1)) break;
                float4 q = lane < kRingWarps ? s_warp[lane] : make_float4(-FLT_MAX, 0.0f, 0.0f, 0.0f);
                t = over_warp(Stat{q.x, q.y, q.z}, a.c, 16);
                if (cs > 1) {
                    const int k = again & 1;
                    if (lane < cs) st_async_v4(&s_cta2[k][rank], &s_met2[k], lane, make_float4(t.m, t.z, t.s, 0.0f));
                    __syncwarp();
                    q = make_float4(-FLT_MAX, 0.0f, 0.0f, 0.0f);
                    if (!receive(s_cta2[k], &s_met2[k], (again / 2) & 1, q)) break;
                    t = over_warp(Stat{q.x, q.y, q.z}, a.c, 4);
                }
                if (lane == 0) {
                    s_all[buf] = t;
                    s_factor[buf] = factor(a, row, tok, t, true, rank == 0);
                    ptx::mbar_arrive(&s_ready2);
                }
                __syncwarp();
                ++again;
            }
        }
    } else {
        int again = 0;
        const int64_t x_step = a.ld * (16 / E), dx_step = a.ldd * (16 / E);
        const char *x_in = static_cast<const char *>(a.x) + first * a.ld * (16 / E), *x_out = x_in;
        char *dx = a.dx ? static_cast<char *>(a.dx) + first * a.ldd * (16 / E) : nullptr;
        Stage in = {0, 0}, out = {0, 0};
        // row n's statistics
        auto measure = [&](int n) -> bool {
            if (!wait(&s_full[in.st], in.parity)) return false;
            Sums t = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            const Token &tok = s_tok[n % kTokens];
            if (tok.takes) {
                const Row<BF16> r(a, x_in, nullptr);
                int v0, len;
                slice(r, v0, len);
                uint4 *sl = reinterpret_cast<uint4 *>(ring + in.st * stage_bytes);
                const float shift = -tok.x_id * a.c;
                // the chosen token leaves the sums, and the slice (its gradient is written by itself)
                const uint32_t at = (uint32_t)(tok.id + r.off - v0 * E);
                if (at / E % NT == tid && at < (uint32_t)(len * E)) V::put(sl, at, -INFINITY);
                int i = tid;
                for (; i + 3 * NT < len; i += 4 * NT) {
                    const uint4 q[4] = {sl[i], sl[i + NT], sl[i + 2 * NT], sl[i + 3 * NT]};
#pragma unroll
                    for (int k = 0; k < 4; ++k) add<BF16>(t, q[k], a.c, shift);
                }
                for (; i < len; i += NT) add<BF16>(t, sl[i], a.c, shift);
                s_sum[n % kRows][tid] = make_float2(t.z.x + t.z.y, t.s.x + t.s.y);
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s_part[n % kRows]);
            if (!dx && lane == 0) ptx::mbar_arrive(&s_empty[in.st]);  // the gradient alone reads the slice again
            x_in += x_step;
            in.next(stages);
            return true;
        };
        // row n's gradient
        auto finish = [&](int n) -> bool {
            const int buf = n % kRows;
            const Token &tok = s_tok[n % kTokens];
            if (!wait(&s_ready[buf], (n / kRows) & 1)) return false;
            const bool takes = tok.takes != 0;
            const bool plain = takes && s_plain[buf];
            if (dx || plain) {
                const Row<BF16> r(a, x_out, dx);
                int v0, len;
                slice(r, v0, len);
                if (!takes) {
                    const float zero[E] = {};
                    for (int i = tid; i < len; i += NT) r.store(v0 + i, zero);
                } else {
                    if (plain) {
                        Stat mine = {-FLT_MAX, 0.0f, 0.0f};
                        const uint4 *xv = r.vec();
                        for (int i = v0 + tid; i < v0 + len; i += NT) add_plain<BF16>(mine, r.inside(i) ? xv[i] : r.load_end(i), a.c);
                        mine = over_warp(mine, a.c, 16);
                        if (lane == 0) {
                            s_warp[warp] = make_float4(mine.m, mine.z, mine.s, 0.0f);
                            ptx::mbar_arrive(&s_part2);
                        }
                        __syncwarp();
                        if (!wait(&s_ready2, again & 1)) return false;
                        ++again;
                    }
                    if (dx) {
                        const uint4 *sl = reinterpret_cast<const uint4 *>(ring + out.st * stage_bytes);
                        const Stat all = s_all[buf];
                        const float coef = s_factor[buf].x, k = s_factor[buf].z;
                        int i = tid;
                        if (!plain && r.dx_vec) {  // whole vectors, but for the row's ends
                            const int in0 = max(r.full0 - v0, 0), in1 = min(r.full1 - v0, len);
                            uint4 *to = reinterpret_cast<uint4 *>(dx - r.off * (16 / E)) + v0;
                            const float shift = -all.m * a.c;
                            for (i += in0; i + NT < in1; i += 2 * NT) {
                                const uint4 q0 = sl[i], q1 = sl[i + NT];
                                to[i] = scaled<BF16>(q0, a.c, shift, k);
                                to[i + NT] = scaled<BF16>(q1, a.c, shift, k);
                            }
                            if (i < in1) to[i] = scaled<BF16>(sl[i], a.c, shift, k);
                            if (tid < in0) grad<BF16>(r, v0 + tid, sl[tid], all, a.c, k, false);
                            i = in1 + tid;
                        }
                        for (; i < len; i += NT) grad<BF16>(r, v0 + i, sl[i], all, a.c, k, plain);
                        // the chosen token, by the thread that wrote its vector: which one follows from the loops above
                        const int own = (tok.id + r.off) / E - v0;
                        if (own >= 0 && own < len) {
                            const int in0 = max(r.full0 - v0, 0), in1 = min(r.full1 - v0, len);
                            const int by = plain || !r.dx_vec ? own : own < in0 ? own : own < in1 ? own - in0 : own - in1;
                            if (by % NT == tid) V::put(dx, tok.id, coef * s_factor[buf].y);
                        }
                    }
                }
                __syncwarp();
            }
            if (dx) {
                if (lane == 0) ptx::mbar_arrive(&s_empty[out.st]);
                dx += dx_step;
            }
            x_out += x_step;
            out.next(stages);
            return true;
        };
        bool ok = true;
        const int rows = (int)(end - first);
        for (int n = 0; ok && n < rows + depth; ++n) {
            if (n < rows) ok = measure(n);
            if (ok && n >= depth) ok = finish(n - depth);
        }
    }
    __syncwarp();
    if (cs > 1) {  // no CTA ends while another may still write to it
        cluster_arrive();
        cluster_wait();
    }
}

// sums = {loss, policy term, KL term, clipped weight}, in a fixed order and in double.
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const float *terms, int64_t T, float beta, float *sums)
{
    __shared__ double s_part[kSumThreads / 32][3];
    pdl_trigger();
    pdl_wait();
    double v[3] = {0.0, 0.0, 0.0};
    for (int64_t t = threadIdx.x; t < T; t += kSumThreads)
#pragma unroll
        for (int j = 0; j < 3; ++j) v[j] += (double)terms[3 * t + j];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        for (int o = 16; o; o >>= 1) v[j] += __shfl_xor_sync(0xFFFFFFFFu, v[j], o);
        if (threadIdx.x % 32 == 0) s_part[threadIdx.x / 32][j] = v[j];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double t[3] = {0.0, 0.0, 0.0};
        for (int k = 0; k < kSumThreads / 32; ++k)
            for (int j = 0; j < 3; ++j) t[j] += s_part[k][j];
        sums[0] = (float)(t[0] + (beta != 0.0f ? (double)beta * t[1] : 0.0));
        sums[1] = (float)t[0];
        sums[2] = (float)t[1];
        sums[3] = (float)t[2];
    }
}

template <bool BF16, int NT, int NV, bool HOLD>
cudaError_t launch(const LossArgs &a, int cs, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.T * cs));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cs > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cs;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (g_chain.load() != 0) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, policy_kernel<BF16, NT, NV, HOLD>, a, cs);
}

template <bool BF16, int NT>
cudaError_t launch_nv(const LossArgs &a, int cs, int64_t nv, cudaStream_t s)
{
    if (nv <= 1) return launch<BF16, NT, 1, true>(a, cs, s);
    if (nv <= 2) return launch<BF16, NT, 2, true>(a, cs, s);
    if (nv <= 4) return launch<BF16, NT, 4, true>(a, cs, s);
    if (nv <= 8) return launch<BF16, NT, 8, true>(a, cs, s);
    return launch<BF16, NT, 4, false>(a, cs, s);
}

void set_cluster(cudaLaunchConfig_t &cfg, int cs)
{
    cudaLaunchAttribute &at = cfg.attrs[cfg.numAttrs++];
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
}

// Clusters of the ring's kernel that fit at once: fewer than the SMs would hold, since a cluster stays within a GPC, and
// GPCs differ in size.
template <bool BF16>
cudaError_t ring_clusters(int cs, int &most)
{
    static OncePerDevice once;
    cudaError_t e = allow_smem(once, policy_ring_kernel<BF16>, kRingBytes);
    if (e != cudaSuccess) return e;
    static std::atomic<int> fit[kMaxDevices][kMaxCluster + 1];
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev >= kMaxDevices) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    most = fit[dev][cs].load();
    if (most) return cudaSuccess;
    most = num_sms();
    if (cs > 1) {
        cudaLaunchAttribute attr[1];
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms() / cs * cs));
        cfg.blockDim = dim3(kRingThreads);
        cfg.dynamicSmemBytes = kRingBytes;
        cfg.attrs = attr;
        set_cluster(cfg, cs);
        e = cudaOccupancyMaxActiveClusters(&most, policy_ring_kernel<BF16>, &cfg);
        if (e != cudaSuccess) return e;
        if (most < 1) most = 1;
    }
    fit[dev][cs].store(most);
    return cudaSuccess;
}

template <bool BF16>
cudaError_t launch_ring(const LossArgs &a, int cs, int clusters, int stages, size_t slice, cudaStream_t s)
{
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((clusters < a.T ? clusters : a.T) * cs));
    cfg.blockDim = dim3(kRingThreads);
    cfg.dynamicSmemBytes = kRingBytes;  // whatever the slices take: one CTA per SM
    cfg.stream = s;
    cfg.attrs = attrs;
    if (cs > 1) set_cluster(cfg, cs);
    if (g_chain.load() != 0) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    // without a gradient a slice is free after its statistics; with one, half the stages are left to the copies
    const int depth = !a.dx ? kRows - 1 : stages >= 5 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, policy_ring_kernel<BF16>, a, cs, stages, depth, (uint32_t)slice, error_word());
}

// Bytes of a stage: a CTA's slice of a row, to 128.
size_t ring_slice(int64_t nvec, int cs) { return ((size_t)((nvec + cs - 1) / cs) * 16 + 127) & ~size_t(127); }

// Which kernel, and its cluster.  The ring: rows of 16 KB and more, when there
// are more of them than clusters that fit at once; of the clusters whose slices
// leave three stages, else two, the smallest, unless a larger one puts CTAs on a
// sixteenth more SMs (1001 rows of 100003 FP32: 23 clusters of six 123 us, 15 of
// eight, which leave a fourth stage but 32 SMs idle, 130 us).  Otherwise one cluster per row: 128
// threads where eight vectors each hold a row, else 256; the smallest cluster
// whose registers hold a row (eight vectors a thread), then larger ones while
// the launch would leave SMs idle and every CTA keeps a vector for half its
// threads.
template <bool BF16>
qerl_status launch_any(const LossArgs &a, cudaStream_t s)
{
    constexpr int E = Vec<BF16>::E;
    const bool even = aligned16(a.x) && a.ld % E == 0;  // every row starts with a vector
    const int64_t nvec = (a.V + (even ? 0 : E - 1) + E - 1) / E;
    if (nvec >= 1024) {
        for (int least = 3; least >= 2; --least) {
            int best = 0, best_clusters = 0;
            for (int cs = 1; cs <= kMaxCluster; ++cs) {
                int clusters = 0;
                if ((int64_t)(kRingBytes / ring_slice(nvec, cs)) < least || a.T * cs <= num_sms()) continue;
                const cudaError_t e = ring_clusters<BF16>(cs, clusters);
                if (e != cudaSuccess) return QERL_ERR_CUDA;
                if (16 * clusters * cs > 17 * best_clusters * best) best = cs, best_clusters = clusters;
            }
            if (!best) continue;
            const size_t slice = ring_slice(nvec, best);
            const int64_t stages = kRingBytes / slice;
            return launched(launch_ring<BF16>(a, best, best_clusters, stages > kMaxStages ? kMaxStages : (int)stages, slice, s),
                            QERL_KERNEL_LOSS_RING);
        }
    }
    const int nt = nvec <= 128 * 8 ? 128 : 256;
    int cs = 1;
    while (cs < kMaxCluster && nvec > int64_t(nt) * 8 * cs) cs *= 2;
    while (cs < kMaxCluster && a.T * cs * 2 <= num_sms() && nvec >= int64_t(nt) * cs) cs *= 2;
    const int64_t per = (nvec + cs - 1) / cs, nv = (per + nt - 1) / nt;
    return launched(nt == 128 ? launch_nv<BF16, 128>(a, cs, nv, s) : launch_nv<BF16, 256>(a, cs, nv, s), QERL_KERNEL_LOSS_ROW);
}

bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

void set_scale(LossArgs &a, double tau)
{
    const double c = 1.4426950408889634 / tau;
    a.c = (float)c;
    a.dc = (float)((c - (double)a.c) / (double)a.c * 0.69314718055994531);
    a.it = (float)(1.0 / tau);
    a.it_rest = (float)(1.0 / tau - (double)a.it);
    a.far_tau = !(tau >= kTauLow && tau <= kTauHigh);
}

// Checks shared by both entry points, for T >= 1.
qerl_status check(const void *logits, int dtype, int64_t T, int64_t V, int64_t ld, const void *ids, int ids_bits, const float *logp)
{
    if (!logits || !ids || !logp) return QERL_ERR_INVALID_ARG;
    if (ld < V || T > 0x7FFFFFFF / kMaxCluster || V > 0x7FFFFF00 || ld > (int64_t(1) << 40)) return QERL_ERR_SHAPE;
    if (!aligned_to(logits, dtype == QERL_DTYPE_BF16 ? 2 : 4) || !aligned_to(ids, ids_bits / 8)) return QERL_ERR_ALIGN;
    return QERL_OK;
}
bool args_ok(int dtype, int64_t T, int64_t V, int ids_bits, float tau)
{
    return (dtype == QERL_DTYPE_BF16 || dtype == QERL_DTYPE_F32) && (ids_bits == 32 || ids_bits == 64) && T >= 0 && V >= 1 && tau > 1e-30f &&
           tau <= 1e30f;
}

}  // namespace
}  // namespace qerl

using namespace qerl;

extern "C" qerl_status qerl_token_logp(const void *logits, int dtype, int64_t T, int64_t V, int64_t ld, const void *ids, int ids_bits,
                                       const float *weight, float temperature, float *logp, float *entropy, qerl_stream_t stream)
{
    if (!args_ok(dtype, T, V, ids_bits, temperature)) return QERL_ERR_INVALID_ARG;
    if (T == 0) return QERL_OK;
    QERL_TRY(check(logits, dtype, T, V, ld, ids, ids_bits, logp));
    if (!aligned_to(weight, 4) || !aligned_to(logp, 4) || !aligned_to(entropy, 4)) return QERL_ERR_ALIGN;
    QERL_TRY(check_device());
    LossArgs a = {};
    a.x = logits, a.ld = ld, a.T = T, a.V = V, a.ids = ids, a.ids64 = ids_bits == 64, a.weight = weight;
    set_scale(a, temperature);
    a.logp = logp, a.entropy = entropy;
    return dtype == QERL_DTYPE_BF16 ? launch_any<true>(a, as_cuda(stream)) : launch_any<false>(a, as_cuda(stream));
}

extern "C" qerl_status qerl_policy_loss(const void *logits, int dtype, int64_t T, int64_t V, int64_t ld, const void *ids, int ids_bits,
                                        const float *old_logp, const float *ref_logp, const float *adv, const float *weight,
                                        const qerl_policy_opts *opts, float *sums, float *logp, float *entropy, void *dlogits, int64_t ldd,
                                        void *ws, size_t ws_bytes, qerl_stream_t stream)
{
    if (!opts || !sums || !args_ok(dtype, T, V, ids_bits, opts->temperature)) return QERL_ERR_INVALID_ARG;
    if (!(opts->clip_low >= 0.0f && opts->clip_low <= 1.0f) || !(opts->clip_high >= 0.0f && opts->clip_high <= FLT_MAX) ||
        !(opts->beta >= 0.0f && opts->beta <= FLT_MAX) || !(fabsf(opts->grad_scale) <= FLT_MAX) || (opts->beta != 0.0f && !ref_logp && T))
        return QERL_ERR_INVALID_ARG;
    const size_t esize = dtype == QERL_DTYPE_BF16 ? 2 : 4;
    if (T) {
        if (!old_logp || !adv) return QERL_ERR_INVALID_ARG;
        QERL_TRY(check(logits, dtype, T, V, ld, ids, ids_bits, logp));
        if (dlogits) {
            if (ldd < V || ldd > (int64_t(1) << 40)) return QERL_ERR_SHAPE;
            if (!aligned_to(dlogits, esize)) return QERL_ERR_ALIGN;
            // in place is fine; rows that overlap otherwise are not
            const uintptr_t x = reinterpret_cast<uintptr_t>(logits), d = reinterpret_cast<uintptr_t>(dlogits);
            const uint64_t nx = ((uint64_t)(T - 1) * ld + V) * esize, nd = ((uint64_t)(T - 1) * ldd + V) * esize;
            if (!(x == d && ld == ldd) && x < d + nd && d < x + nx) return QERL_ERR_INVALID_ARG;
        }
        const float *const f[] = {old_logp, ref_logp, adv, weight, logp, entropy};
        for (const float *p : f)
            if (!aligned_to(p, 4)) return QERL_ERR_ALIGN;
        if (!ws || ws_bytes < qerl_workspace_bytes(QERL_OP_POLICY_LOSS, T, V, 0, 0)) return QERL_ERR_WORKSPACE;
        if (!aligned16(ws)) return QERL_ERR_ALIGN;
    }
    if (!aligned_to(sums, 4)) return QERL_ERR_ALIGN;
    QERL_TRY(check_device());
    LossArgs a = {};
    a.x = logits, a.ld = ld, a.T = T, a.V = V, a.ids = ids, a.ids64 = ids_bits == 64;
    a.old_logp = old_logp, a.ref_logp = ref_logp, a.adv = adv, a.weight = weight;
    set_scale(a, opts->temperature);
    a.lo = 1.0f - opts->clip_low, a.hi = 1.0f + opts->clip_high, a.beta = opts->beta;
    a.gscale = opts->grad_scale / opts->temperature;
    a.logp = logp, a.entropy = entropy, a.terms = static_cast<float *>(ws), a.dx = dlogits, a.ldd = ldd;
    a.dx_vec = dlogits && ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(dlogits)) & 15u) == 0 &&
               (uint64_t)(ld - ldd) * esize % 16 == 0;
    if (T) QERL_TRY(dtype == QERL_DTYPE_BF16 ? launch_any<true>(a, as_cuda(stream)) : launch_any<false>(a, as_cuda(stream)));
    return launched(launch_k(sum_kernel, dim3(1), dim3(kSumThreads), 0, as_cuda(stream), g_chain.load() != 0, (const float *)a.terms, T,
                             opts->beta, sums));
}
