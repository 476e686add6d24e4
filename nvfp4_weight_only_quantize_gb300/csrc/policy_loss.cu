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

// NT threads per CTA; HOLD: a thread's NV vectors stay in registers, else they are read twice.
template <bool BF16, int NT, int NV, bool HOLD>
__global__ void __launch_bounds__(NT, 1024 / NT) policy_kernel(LossArgs a, int cs)
{
    using V = Vec<BF16>;
    constexpr int E = V::E, NW = NT / 32;
    __shared__ float4 s_warp[NW];
    __shared__ alignas(16) float4 s_cta[kMaxCluster];
    __shared__ float s_coef[2];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t row = blockIdx.x / cs;
    const int rank = blockIdx.x % cs;
    pdl_trigger();
    if (cs > 1) cluster_arrive_relaxed();  // peers' shared memory may be written once all of them run
    pdl_wait();

    // the row as aligned vectors: vector i holds elements [i E - off, i E - off + E)
    const char *xr = static_cast<const char *>(a.x) + row * a.ld * (16 / E);
    const int off = (int)((reinterpret_cast<uintptr_t>(xr) & 15u) / (16 / E));
    const int64_t nvec = (off + a.V + E - 1) / E;
    const int64_t per = (nvec + cs - 1) / cs;
    const int64_t v0 = rank * per, v1 = min(v0 + per, nvec);
    const uint4 *xv = reinterpret_cast<const uint4 *>(xr - off * (16 / E));
    char *dr = a.dx ? static_cast<char *>(a.dx) + row * a.ldd * (16 / E) : nullptr;
    auto load = [&](int64_t i) -> uint4 {
        if (i * E >= off && i * E + E <= off + a.V) return xv[i];
        uint32_t w[4] = {V::kFill, V::kFill, V::kFill, V::kFill};
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int64_t e = i * E + j - off;
            if (e >= 0 && e < a.V) {
                if (BF16) {
                    const uint32_t h = reinterpret_cast<const uint16_t *>(xr)[e];
                    w[j / 2] = j % 2 ? (w[j / 2] & 0xFFFFu) | h << 16 : (w[j / 2] & 0xFFFF0000u) | h;
                } else {
                    w[j % 4] = reinterpret_cast<const uint32_t *>(xr)[e];
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    auto store = [&](int64_t i, const float(&f)[E]) {
        if (a.dx_vec && i * E >= off && i * E + E <= off + a.V) {
            *reinterpret_cast<uint4 *>(dr + (i * E - off) * (16 / E)) = V::pack(f);
            return;
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int64_t e = i * E + j - off;
            if (e >= 0 && e < a.V) V::put(dr, e, f[j]);
        }
    };

    const int64_t id = a.ids64 ? static_cast<const int64_t *>(a.ids)[row] : static_cast<const int32_t *>(a.ids)[row];
    const float w = a.weight ? a.weight[row] : 1.0f;
    if (w == 0.0f || id < 0 || id >= a.V) {  // takes no part: the logits are not read
        const float zero[E] = {};
        if (dr)
            for (int64_t i = v0 + tid; i < v1; i += NT) store(i, zero);
        if (rank == 0 && tid == 0) {
            a.logp[row] = 0.0f;
            if (a.entropy) a.entropy[row] = 0.0f;
            if (a.terms) a.terms[3 * row] = a.terms[3 * row + 1] = a.terms[3 * row + 2] = 0.0f;
        }
        if (cs > 1) cluster_wait();
        return;
    }
    const float x_id = V::get(xr, id);

    uint4 hold[NV];
    Stat st = {-FLT_MAX, 0.0f, 0.0f};
    auto add = [&](const uint4 &q) {  // one vector, relative to st.m
        float f[E];
        V::unpack(q, f);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const float y = (f[j] - st.m) * a.c, e = ex2(y);
            st.z += e;
            st.s = fmaf(e, fmaxf(y, -1e4f), st.s);
        }
    };
    auto top = [&](const uint4 &q) {
        float f[E], m = -FLT_MAX;
        V::unpack(q, f);
#pragma unroll
        for (int j = 0; j < E; ++j) m = fmaxf(m, f[j]);
        return m;
    };
    if (HOLD) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t i = v0 + k * NT + tid;
            hold[k] = i < v1 ? load(i) : make_uint4(V::kFill, V::kFill, V::kFill, V::kFill);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) st.m = fmaxf(st.m, top(hold[k]));
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (v0 + k * NT < v1) add(hold[k]);
    } else {
        for (int64_t i = v0 + tid; i < v1; i += NV * NT) {
            float m = st.m;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                hold[k] = i + k * NT < v1 ? load(i + k * NT) : make_uint4(V::kFill, V::kFill, V::kFill, V::kFill);
                m = fmaxf(m, top(hold[k]));
            }
            st = moved(st, m, a.c);
#pragma unroll
            for (int k = 0; k < NV; ++k) add(hold[k]);
        }
    }

    // warp, CTA, cluster
    float M = st.m;
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    st = moved(st, M, a.c);
    for (int o = 16; o; o >>= 1) {
        st.z += __shfl_xor_sync(0xFFFFFFFFu, st.z, o);
        st.s += __shfl_xor_sync(0xFFFFFFFFu, st.s, o);
    }
    if (lane == 0) s_warp[warp] = make_float4(st.m, st.z, st.s, 0.0f);
    __syncthreads();
    if (warp == 0) {
        const float4 q = lane < NW ? s_warp[lane] : make_float4(-FLT_MAX, 0.0f, 0.0f, 0.0f);
        Stat t = {q.x, q.y, q.z};
        M = t.m;
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
        t = moved(t, M, a.c);
        for (int o = 16; o; o >>= 1) {
            t.z += __shfl_xor_sync(0xFFFFFFFFu, t.z, o);
            t.s += __shfl_xor_sync(0xFFFFFFFFu, t.s, o);
        }
        const float4 r = make_float4(t.m, t.z, t.s, 0.0f);
        if (cs == 1) {
            if (lane == 0) s_cta[0] = r;
        }
        if (cs > 1) {
            cluster_wait();
            if (lane < cs) st_cluster_v4(ptx::smem_u32(&s_cta[rank]), lane, r);
        }
    } else if (cs > 1) {
        cluster_wait();
    }
    if (cs > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    Stat all = {-FLT_MAX, 0.0f, 0.0f};
    for (int k = 0; k < cs; ++k) all.m = fmaxf(all.m, s_cta[k].x);
    for (int k = 0; k < cs; ++k) {
        const Stat t = moved(Stat{s_cta[k].x, s_cta[k].y, s_cta[k].z}, all.m, a.c);
        all.z += t.z;
        all.s += t.s;
    }
    if (tid == 0) {
        const bool empty = all.z == 0.0f;  // every logit -inf: no distribution, no part in the loss
        const float lz = logf(all.z);
        const float logp = empty ? -INFINITY : (x_id - all.m) * a.c * kLn2 - lz;
        float dlogp = 0.0f;
        if (rank == 0) {
            a.logp[row] = logp;
            if (a.entropy) a.entropy[row] = empty ? 0.0f : lz - all.s / all.z * kLn2;
        }
        if (a.old_logp) {
            const float A = a.adv[row], rho = expf(logp - a.old_logp[row]);
            const float d = a.ref_logp ? a.ref_logp[row] - logp : 0.0f, em = expm1f(d);
            const bool keeps = A >= 0.0f ? rho <= a.hi : rho >= a.lo;
            const float policy = -fminf(rho * A, fminf(fmaxf(rho, a.lo), a.hi) * A);
            if (!empty) dlogp = w * ((a.beta != 0.0f ? -a.beta * em : 0.0f) - (keeps ? rho * A : 0.0f));
            if (rank == 0) {
                a.terms[3 * row] = empty ? 0.0f : w * policy;
                a.terms[3 * row + 1] = empty ? 0.0f : w * (em - d);
                a.terms[3 * row + 2] = empty || keeps ? 0.0f : w;
            }
        }
        s_coef[0] = dlogp * a.gscale;
        s_coef[1] = empty ? 0.0f : -expm1f(logp);  // 1 - p_id, without cancellation
    }
    if (!dr) return;
    __syncthreads();
    const float coef = s_coef[0], k = all.z == 0.0f ? 0.0f : -coef / all.z;
    const int64_t own = (id + off) / E;  // the vector that holds the chosen token
    auto grad = [&](int64_t i, const uint4 &q) {
        float f[E];
        V::unpack(q, f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = ex2((f[j] - all.m) * a.c) * k;
        store(i, f);
        if (i == own) V::put(dr, id, coef * s_coef[1]);
    };
    if (HOLD) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int64_t i = v0 + n * NT + tid;
            if (i < v1) grad(i, hold[n]);
        }
    } else {
        for (int64_t i = v0 + tid; i < v1; i += NT) grad(i, load(i));
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

// Threads, cluster and vectors per thread of a launch.  128 threads where eight
// vectors each hold a row, else 512; the smallest cluster whose registers hold
// a row (eight vectors a thread), then larger ones while the launch would leave
// SMs idle and every CTA keeps a vector for half its threads.
template <bool BF16>
cudaError_t launch_any(const LossArgs &a, cudaStream_t s)
{
    constexpr int E = Vec<BF16>::E;
    const int64_t nvec = (a.V + E - 1) / E + 1;  // one more where a row starts inside a vector
    const int nt = nvec <= 128 * 8 ? 128 : 512;
    int cs = 1;
    while (cs < kMaxCluster && nvec > int64_t(nt) * 8 * cs) cs *= 2;
    while (cs < kMaxCluster && a.T * cs * 2 <= num_sms() && nvec >= int64_t(nt) * cs) cs *= 2;
    const int64_t per = (nvec + cs - 1) / cs, nv = (per + nt - 1) / nt;
    return nt == 128 ? launch_nv<BF16, 128>(a, cs, nv, s) : launch_nv<BF16, 512>(a, cs, nv, s);
}

bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks shared by both entry points, for T >= 1.
qerl_status check(const void *logits, int dtype, int64_t T, int64_t V, int64_t ld, const void *ids, int ids_bits, const float *logp)
{
    if (!logits || !ids || !logp) return QERL_ERR_INVALID_ARG;
    if (ld < V || T > 0x7FFFFFFF / kMaxCluster || V > (int64_t(1) << 40) || ld > (int64_t(1) << 40)) return QERL_ERR_SHAPE;
    if (!aligned_to(logits, dtype == QERL_DTYPE_BF16 ? 2 : 4) || !aligned_to(ids, ids_bits / 8)) return QERL_ERR_ALIGN;
    return QERL_OK;
}
bool args_ok(int dtype, int64_t T, int64_t V, int ids_bits, float tau)
{
    return (dtype == QERL_DTYPE_BF16 || dtype == QERL_DTYPE_F32) && (ids_bits == 32 || ids_bits == 64) && T >= 0 && V >= 1 && tau > 0.0f &&
           tau <= FLT_MAX;
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
