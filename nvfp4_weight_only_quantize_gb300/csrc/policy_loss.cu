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
// row is split over the CTAs of a cluster, every thread keeps its vectors in
// registers (32 of them at most), the threads' (max, sum, entropy sum) meet by
// warp shuffles, shared memory and one exchange through the cluster's distributed
// shared memory, and the gradient is formed from the registers.  Rows longer
// than a cluster's registers are read a second time (from L2, as a rule).
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
    float c;                                          // log2(e) / tau
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
    {
        x = static_cast<const char *>(a.x) + row * a.ld * S;
        dx = a.dx ? static_cast<char *>(a.dx) + row * a.ldd * S : nullptr;
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
// gradient and 1 - p of the chosen token.  `plain`: see below.
__device__ __forceinline__ float2 factor(const LossArgs &a, int64_t row, const Token &t, const Stat &all, bool plain, bool write)
{
    const bool empty = all.z == 0.0f;  // every logit -inf: no distribution, no part in the loss
    const float lz = logf(all.z);
    const float y_id = plain ? (t.x_id - all.m) * a.c : fmaf(t.x_id, a.c, -all.m * a.c);
    const float logp = empty ? -INFINITY : y_id * kLn2 - lz;
    float dlogp = 0.0f;
    if (write) {
        a.logp[row] = logp;
        if (a.entropy) a.entropy[row] = empty ? 0.0f : lz - all.s / all.z * kLn2;
    }
    if (a.old_logp) {
        const float A = t.adv, rho = expf(logp - t.old_logp);
        const float d = a.ref_logp ? t.ref - logp : 0.0f, em = expm1f(d);
        const bool keeps = A >= 0.0f ? rho <= a.hi : rho >= a.lo;
        const float policy = -fminf(rho * A, fminf(fmaxf(rho, a.lo), a.hi) * A);
        if (!empty) dlogp = t.w * ((a.beta != 0.0f ? -a.beta * em : 0.0f) - (keeps ? rho * A : 0.0f));
        if (write) {
            a.terms[3 * row] = empty ? 0.0f : t.w * policy;
            a.terms[3 * row + 1] = empty ? 0.0f : t.w * (em - d);
            a.terms[3 * row + 2] = empty || keeps ? 0.0f : t.w;
        }
    }
    return make_float2(dlogp * a.gscale, empty ? 0.0f : -expm1f(logp));
}
__device__ __forceinline__ void no_part(const LossArgs &a, int64_t row)
{
    a.logp[row] = 0.0f;
    if (a.entropy) a.entropy[row] = 0.0f;
    if (a.terms) a.terms[3 * row] = a.terms[3 * row + 1] = a.terms[3 * row + 2] = 0.0f;
}

// One vector's part of the statistics, relative to a maximum: y = x c + shift in
// one rounding with shift = -max c.  Where a maximum lies beyond +-1e30 (a row of
// the type's lowest values) that may overflow and leave z = 0; such a row, or
// one that is all -inf, is taken again as (x - max) c (`plain`).
template <bool BF16>
__device__ __forceinline__ void add(Stat &st, const uint4 &q, float c, float shift)
{
    float f[Vec<BF16>::E];
    Vec<BF16>::unpack(q, f);
#pragma unroll
    for (int j = 0; j < Vec<BF16>::E; ++j) {
        const float y = fmaf(f[j], c, shift), e = ex2(y);
        st.z += e;
        st.s = fmaf(e, fmaxf(y, -1e4f), st.s);
    }
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
__device__ __forceinline__ float shift_of(float m, float c) { return -fmaxf(m, -1e30f) * c; }

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
        for (int j = 0; j < E; ++j) f[j] = ex2(fmaf(f[j], c, shift)) * k;
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
    __shared__ float2 s_factor;
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
#pragma unroll
        for (int k = 0; k < NV; ++k) st.m = fmaxf(st.m, V::top(hold[k]));
        const float shift = shift_of(st.m, a.c);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (v0 + k * NT < v1) add<BF16>(st, hold[k], a.c, shift);
    } else {
        for (int i = v0 + tid; i < v1; i += NV * NT) {
            float m = st.m;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                hold[k] = nothing;
                if (i + k * NT < v1 && r.inside(i + k * NT)) hold[k] = xv[i + k * NT];
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (i + k * NT < v1 && !r.inside(i + k * NT)) hold[k] = r.load_end(i + k * NT);
                m = fmaxf(m, V::top(hold[k]));
            }
            st = moved(st, m, a.c);
            const float shift = shift_of(m, a.c);
#pragma unroll
            for (int k = 0; k < NV; ++k) add<BF16>(st, hold[k], a.c, shift);
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
    const bool plain = all.z == 0.0f;
    if (plain) {
        if (cs > 1) cluster_arrive();
        st = Stat{-FLT_MAX, 0.0f, 0.0f};
        for (int i = v0 + tid; i < v1; i += NT) add_plain<BF16>(st, r.inside(i) ? xv[i] : r.load_end(i), a.c);
        all = join(st, 1);
    }
    if (tid == 0) s_factor = factor(a, row, tok, all, plain, rank == 0);
    if (!r.dx) return;
    __syncthreads();
    const float coef = s_factor.x, k = all.z == 0.0f ? 0.0f : -coef / all.z;
    const int own = (tok.id + r.off) / E;  // the vector that holds the chosen token
    if (HOLD && !plain) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = v0 + j * NT + tid;
            if (i < v1) grad<BF16>(r, i, hold[j], all, a.c, k, false);
        }
    } else {
        for (int i = v0 + tid; i < v1; i += NT) grad<BF16>(r, i, r.inside(i) ? xv[i] : r.load_end(i), all, a.c, k, plain);
    }
    if (own >= v0 && own < v1 && (own - v0) % NT == tid) V::put(r.dx, tok.id, coef * s_factor.y);
}

// ------------------------------------------------------------------ many long rows: a ring of row slices in shared memory
// Persistent clusters; a CTA's slice of a row is one bulk copy into a stage of
// its ring, issued by a producer warp that runs ahead of the eight warps that
// compute, so that reading goes on through the exchanges and the writing.  Two
// CTAs share an SM: one computes while the other waits for its cluster.  The
// exchange is a 16-byte asynchronous store to every CTA of the cluster, which
// counts on the receiver's barrier.
constexpr int kRingWarps = 8, kRingThreads = (kRingWarps + 1) * 32, kMaxStages = 3;
static_assert(kRingWarps <= kMaxCluster, "the warps' statistics are joined in eight lanes");
constexpr size_t kRingBytes = 108 << 10;  // of one of two CTAs on an SM

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

template <bool BF16>
__global__ void __launch_bounds__(kRingThreads, 2)
    policy_ring_kernel(LossArgs a, int cs, int stages, uint32_t stage_bytes, unsigned int *err)
{
    using V = Vec<BF16>;
    constexpr int E = V::E, NT = kRingWarps * 32;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_met[2];
    __shared__ alignas(16) float4 s_cta[2][kMaxCluster];
    __shared__ float4 s_warp[kRingWarps];
    __shared__ Token s_tok[kMaxStages];
    __shared__ float2 s_factor;
    __shared__ Stat s_all;
    __shared__ int s_stop;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int rank = blockIdx.x % cs;
    const int64_t first = blockIdx.x / cs, step = gridDim.x / cs;
    if (tid == 0) {
        for (int k = 0; k < stages; ++k) {
            ptx::mbar_init(&s_full[k], 1);
            ptx::mbar_init(&s_empty[k], kRingWarps);
        }
        ptx::mbar_init(&s_met[0], 1);
        ptx::mbar_init(&s_met[1], 1);
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

    // Every wait is bounded: past two seconds the error is latched and the CTA winds up.
    const uint64_t deadline_ns = 2000000000ull;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        const uint64_t until = ptx::globaltimer_ns() + deadline_ns;
        for (;;) {
            if (ptx::mbar_try_wait_sleep(bar, parity, 20000u)) return true;
            if (*reinterpret_cast<volatile int *>(&s_stop)) return false;
            if (ptx::globaltimer_ns() > until) {
                *reinterpret_cast<volatile int *>(&s_stop) = 1;
                latch_error(err, QERL_ERR_TIMEOUT);
                return false;
            }
        }
    };

    if (warp == kRingWarps) {
        int n = 0;
        for (int64_t row = first; row < a.T; row += step, ++n) {
            const int st = n % stages;
            Token tok = token<BF16>(a, row);
            if (tok.takes) token_inputs<BF16>(a, row, tok);
            if (n >= stages && !__all_sync(0xFFFFFFFFu, wait(&s_empty[st], (n / stages - 1) & 1))) break;
            const Row<BF16> r(a, row);
            const int per = (r.nvec + cs - 1) / cs, v0 = rank * per, v1 = min(v0 + per, r.nvec);
            uint8_t *to = ring + st * stage_bytes;
            const int b0 = max(v0, r.full0), b1 = min(v1, r.full1), last = r.nvec - 1;
            if (tok.takes) {  // the row's ends by element
                if (lane == 0 && v0 == 0 && r.full0) *reinterpret_cast<uint4 *>(to) = r.load_end(0);
                if (lane == 1 && last >= max(v0, r.full1) && last < v1 && (last > 0 || !r.full0))
                    *reinterpret_cast<uint4 *>(to + (last - v0) * 16) = r.load_end(last);
            }
            if (lane == 0) s_tok[st] = tok;
            __syncwarp();
            if (lane == 0) {
                const uint32_t bytes = tok.takes && b1 > b0 ? (uint32_t)(b1 - b0) * 16u : 0u;
                ptx::mbar_arrive_expect_tx(&s_full[st], bytes);
                if (bytes) bulk_load(to + (b0 - v0) * 16, r.vec() + b0, bytes, &s_full[st]);
            }
        }
        // no copy may be in flight when the CTA ends
        if (lane == 0 && *reinterpret_cast<volatile int *>(&s_stop)) {
            const uint64_t until = ptx::globaltimer_ns() + deadline_ns;
            for (int k = max(0, n - stages); k < n; ++k)
                while (!ptx::mbar_try_wait(&s_full[k % stages], (k / stages) & 1) && ptx::globaltimer_ns() < until) {
                }
        }
        __syncwarp();
    } else {
        int n = 0, met = 0;
        for (int64_t row = first; row < a.T; row += step, ++n) {
            const int st = n % stages;
            // warps leave the loop together: the barriers below count all of them
            if (!ptx::named_bar_and(2, NT, wait(&s_full[st], (n / stages) & 1))) break;
            const Row<BF16> r(a, row);
            const int per = (r.nvec + cs - 1) / cs, v0 = rank * per, v1 = min(v0 + per, r.nvec), len = max(0, v1 - v0);
            const uint4 *sl = reinterpret_cast<const uint4 *>(ring + st * stage_bytes);
            const int id = s_tok[st].id;
            if (!s_tok[st].takes) {
                const float zero[E] = {};
                if (r.dx)
                    for (int i = tid; i < len; i += NT) r.store(v0 + i, zero);
                if (rank == 0 && tid == 0) no_part(a, row);
            } else {
                Stat mine = {-FLT_MAX, 0.0f, 0.0f};
                const uint4 nothing = make_uint4(V::kFill, V::kFill, V::kFill, V::kFill);
                for (int i = tid; i < len; i += 4 * NT) {
                    uint4 q[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] = i + k * NT < len ? sl[i + k * NT] : nothing;
                    const float m = fmaxf(fmaxf(fmaxf(mine.m, V::top(q[0])), V::top(q[1])), fmaxf(V::top(q[2]), V::top(q[3])));
                    mine = moved(mine, m, a.c);
                    const float shift = shift_of(m, a.c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) add<BF16>(mine, q[k], a.c, shift);
                }
                // Joins every thread's statistics into the row's; its factor follows in the same warp.  False where the
                // cluster's others did not answer in time.
                auto join = [&](Stat t, bool plain) -> bool {
                    const int buf = met & 1;
                    t = over_warp(t, a.c, 16);
                    if (lane == 0) s_warp[warp] = make_float4(t.m, t.z, t.s, 0.0f);
                    ptx::named_bar_sync(1, NT);
                    bool ok = true;
                    if (warp == 0) {
                        float4 q = lane < kRingWarps ? s_warp[lane] : make_float4(-FLT_MAX, 0.0f, 0.0f, 0.0f);
                        t = over_warp(Stat{q.x, q.y, q.z}, a.c, 4);  // in lanes 0 to 7, which send it
                        if (lane == 0) ptx::mbar_arrive_expect_tx(&s_met[buf], (uint32_t)cs * 16u);
                        __syncwarp();
                        if (lane < cs) st_async_v4(&s_cta[buf][rank], &s_met[buf], lane, make_float4(t.m, t.z, t.s, 0.0f));
                        ok = __all_sync(0xFFFFFFFFu, wait(&s_met[buf], (met / 2) & 1));
                        q = ok && (lane & 7) < cs ? s_cta[buf][lane & 7] : make_float4(-FLT_MAX, 0.0f, 0.0f, 0.0f);
                        t = over_warp(Stat{q.x, q.y, q.z}, a.c, 4);
                        if (lane == 0) {
                            s_all = t;
                            if (ok && (t.z != 0.0f || plain)) s_factor = factor(a, row, s_tok[st], t, plain, rank == 0);
                        }
                    }
                    ++met;
                    return ptx::named_bar_and(1, NT, ok);
                };
                bool ok = join(mine, false);
                const bool plain = ok && s_all.z == 0.0f;
                if (plain) {
                    mine = Stat{-FLT_MAX, 0.0f, 0.0f};
                    for (int i = tid; i < len; i += NT) add_plain<BF16>(mine, sl[i], a.c);
                    ok = join(mine, true);
                }
                if (!ok) break;
                if (r.dx) {
                    const Stat all = s_all;
                    const float coef = s_factor.x, one_p = s_factor.y, k = all.z == 0.0f ? 0.0f : -coef / all.z;
#pragma unroll 2
                    for (int i = tid; i < len; i += NT) grad<BF16>(r, v0 + i, sl[i], all, a.c, k, plain);
                    const int own = (id + r.off) / E - v0;  // the vector that holds the chosen token
                    if (own >= 0 && own < len && own % NT == tid) V::put(r.dx, id, coef * one_p);
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s_empty[st]);
        }
        __syncwarp();
    }
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

template <bool BF16>
cudaError_t launch_ring(const LossArgs &a, int cs, int stages, size_t slice, int per_sm, cudaStream_t s)
{
    const size_t smem = stages * slice;
    static const cudaError_t attr =
        cudaFuncSetAttribute(policy_ring_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(2 * kRingBytes));
    if (attr != cudaSuccess) return attr;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kRingThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2];
    int n = 0;
    if (cs > 1) {
        attrs[n].id = cudaLaunchAttributeClusterDimension;
        attrs[n].val.clusterDim.x = (unsigned)cs;
        attrs[n].val.clusterDim.y = attrs[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    // clusters that fit at once (fewer than the SMs would hold: a cluster stays within a GPC)
    static std::atomic<int> fit[2][4];
    std::atomic<int> &known = fit[per_sm - 1][cs == 1 ? 0 : cs == 2 ? 1 : cs == 4 ? 2 : 3];
    int64_t clusters = known.load();
    if (clusters == 0) {
        clusters = (int64_t)per_sm * num_sms();
        if (cs > 1) {
            int most = 0;
            cfg.gridDim = dim3((unsigned)(clusters / cs * cs));
            cfg.dynamicSmemBytes = (3 - per_sm) * kRingBytes;
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&most, policy_ring_kernel<BF16>, &cfg);
            if (e != cudaSuccess) return e;
            clusters = most > 0 ? most : 1;
            cfg.dynamicSmemBytes = smem;
        }
        known.store((int)clusters);
    }
    if (clusters > a.T) clusters = a.T;
    cfg.gridDim = dim3((unsigned)(clusters * cs));
    if (g_chain.load() != 0) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, policy_ring_kernel<BF16>, a, cs, stages, (uint32_t)slice, error_word());
}

// Which kernel, and its cluster.  The ring: rows of 16 KB and more, when there
// are more of them than clusters that fit at once; the smallest cluster whose
// slices leave three stages to each of two CTAs on an SM, else two stages, else
// two stages of one CTA.  Otherwise one cluster per row: 128 threads where eight
// vectors each hold a row, else 256; the smallest cluster whose registers hold
// a row (eight vectors a thread), then larger ones while the launch would leave
// SMs idle and every CTA keeps a vector for half its threads.
template <bool BF16>
cudaError_t launch_any(const LossArgs &a, cudaStream_t s)
{
    constexpr int E = Vec<BF16>::E;
    const bool even = aligned16(a.x) && a.ld % E == 0;  // every row starts with a vector
    const int64_t nvec = (a.V + (even ? 0 : E - 1) + E - 1) / E;
    if (nvec >= 1024) {
        for (int per_sm = 2; per_sm >= 1; --per_sm)
            for (int stages = 3; stages >= 2; --stages)
                for (int cs = 1; cs <= kMaxCluster; cs *= 2) {
                    const size_t slice = ((size_t)((nvec + cs - 1) / cs) * 16 + 127) & ~size_t(127);
                    if (stages * slice <= (3 - per_sm) * kRingBytes && a.T * cs > (int64_t)per_sm * num_sms())
                        return launch_ring<BF16>(a, cs, stages, slice, per_sm, s);
                }
    }
    const int nt = nvec <= 128 * 8 ? 128 : 256;
    int cs = 1;
    while (cs < kMaxCluster && nvec > int64_t(nt) * 8 * cs) cs *= 2;
    while (cs < kMaxCluster && a.T * cs * 2 <= num_sms() && nvec >= int64_t(nt) * cs) cs *= 2;
    const int64_t per = (nvec + cs - 1) / cs, nv = (per + nt - 1) / nt;
    return nt == 128 ? launch_nv<BF16, 128>(a, cs, nv, s) : launch_nv<BF16, 256>(a, cs, nv, s);
}

bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

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
    a.c = (float)(1.4426950408889634 / (double)temperature);
    a.logp = logp, a.entropy = entropy;
    return launched(dtype == QERL_DTYPE_BF16 ? launch_any<true>(a, as_cuda(stream)) : launch_any<false>(a, as_cuda(stream)));
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
    a.c = (float)(1.4426950408889634 / (double)opts->temperature);
    a.lo = 1.0f - opts->clip_low, a.hi = 1.0f + opts->clip_high, a.beta = opts->beta;
    a.gscale = opts->grad_scale / opts->temperature;
    a.logp = logp, a.entropy = entropy, a.terms = static_cast<float *>(ws), a.dx = dlogits, a.ldd = ldd;
    a.dx_vec = dlogits && ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(dlogits)) & 15u) == 0 &&
               (uint64_t)(ld - ldd) * esize % 16 == 0;
    if (T) QERL_TRY(launched(dtype == QERL_DTYPE_BF16 ? launch_any<true>(a, as_cuda(stream)) : launch_any<false>(a, as_cuda(stream))));
    return launched(launch_k(sum_kernel, dim3(1), dim3(kSumThreads), 0, as_cuda(stream), g_chain.load() != 0, (const float *)a.terms, T,
                             opts->beta, sums));
}
