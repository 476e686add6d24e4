// The next token of every row of logits from a given uniform number.
//
//   p = softmax(x / tau); the tokens in order of (p, then index): kept is the shortest prefix of
//     the first top_k;  those until their sum reaches top_p of the first top_k's;  those with p >= min_p max p
//   id = the first kept token, in order of index, whose sum of kept p up to it exceeds u times that of all;
//   logp = ln p_id,  logq = ln (p_id / sum of kept p).
//
// Which token that is must not depend on rounding, on the number of CTAs or on
// the order of sums: masses e^((x - max) / tau) are held as 64-bit integers (2^42
// for the most probable token), whose sums are exact.  Two ways lead to them:
//   fast   ex2 in FP32, summed over a chunk of 2 KB of the row and then turned to an
//          integer; such sums are off by at most kEps of their value (below);
//   exact  the exponential in pairs of FP32 numbers, good to 2^-40.
// A choice that kEps could change is made again with exact sums.
//
// A row is swept by one CTA, or by a cluster of up to eight where there are few
// rows; the sweeps after the first find it in L2.  Sweeps: the chunks' maxima and
// sums; with a cut, histograms of the order-preserving integer keys of the logits
// below the maximum, refined until the border is a single key (bf16: as a rule the
// first histogram's bins are single keys already, and their masses exact); the
// chunks' sums of what is kept.  At last one chunk is read again for the token.
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace qerl {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCluster = 8;
constexpr int kVec = 4, kChunkVecs = 32 * kVec;  // 16-byte vectors of a lane and of a chunk
constexpr int kBins = 2048, kBinBits = 11;
constexpr int64_t kMaxV = 1 << 20;  // 2^42 times that fits 62 bits
constexpr int kMaxChunks = kMaxV * 4 / (kChunkVecs * 16) + 1;
constexpr int kScale = 42;
// Of a chunk's fast sum: per value 2 roundings of the exponent y, up to 2^-23 |y| ln 2 with c's own (2^-25), where the
// mean of |y| over a chunk is at most log2 1024; ex2.approx 2^-22; some 25 roundings of the sum, 2^-24 each.
constexpr double kEps = 3e-6;

struct Args {
    const void *x;
    int64_t ld, T, V;
    const float *u;
    float tau, top_p, min_p;
    int top_k;
    const float *taus, *top_ps, *min_ps;
    const int32_t *top_ks;
    int64_t *ids;
    float *logp, *logq;
    int cluster;
};

// 2^(j / 64) in two FP32 numbers.
__device__ const float2 kRoots[64] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f}, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f}, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}, {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f},
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Integers in the order of the values, both zeros the same; of bf16 the upper half, the lower is 0.
template <bool BF16>
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) & (BF16 ? 0xFFFF0000u : 0xFFFFFFFFu);
}
template <bool BF16>
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u ? key ^ 0x80000000u : ~key) & (BF16 ? 0xFFFF0000u : 0xFFFFFFFFu));
}

// e^((x - top) / tau) 2^42, c = log2(e) / tau in two FP32 numbers.  With y = (x - top) c in two numbers, k = round(64 y) and
// r = y - k / 64 it is 2^(k / 64) e^(r ln 2); the exponential of |t| < 0.0055 by its series to t^4 / 24.
struct Exp {
    float top, c, c_lo;
    const float2 *roots;
};
__device__ __forceinline__ uint64_t mass(const Exp &e, float x)
{
    const float d = x - e.top, b = d - x, rest = (x - (d - b)) - (e.top + b);
    const float y = d * e.c;
    if (!(y > -60.0f)) return 0;
    const float y_lo = fmaf(d, e.c, -y) + fmaf(d, e.c_lo, rest * e.c);
    const float k = rintf(y * 64.0f), r0 = fmaf(k, -0.015625f, y), r = r0 + y_lo, r_lo = (r0 - r) + y_lo;
    const float t = r * 0x1.62e430p-1f, t_lo = fmaf(r, 0x1.62e430p-1f, -t) + fmaf(r, -0x1.05c610p-29f, r_lo * 0x1.62e430p-1f);
    const float q = t * t * fmaf(t, fmaf(t, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f), s = t_lo + q;
    const float p = t + s, p_lo = (t - p) + s;
    const int n = (int)k;
    const float2 T = e.roots[n & 63];
    const float mid = T.x * p, low = fmaf(T.x, p, -mid) + fmaf(T.x, p_lo, fmaf(T.y, p, T.y));
    const float unit = pow2f(kScale + (n >> 6));
    return (uint64_t)(__float2ll_rn(T.x * unit) + __float2ll_rn(mid * unit) + __float2ll_rn(low * unit));
}

// A row as the aligned 16-byte vectors that hold it; elements outside it read as -inf.
template <bool BF16>
struct Row {
    static constexpr int E = BF16 ? 8 : 4, S = 16 / E;
    const char *x;
    int off, n, nvec;
    __device__ __forceinline__ Row(const Args &a, int64_t row)
    {
        x = static_cast<const char *>(a.x) + row * a.ld * S;
        off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / S);
        n = (int)a.V;
        nvec = (off + n + E - 1) / E;
    }
    __device__ __forceinline__ float at(int e) const
    {
        if (e < 0 || e >= n) return -INFINITY;
        return BF16 ? bf16f(reinterpret_cast<const __nv_bfloat16 *>(x)[e]) : reinterpret_cast<const float *>(x)[e];
    }
    __device__ __forceinline__ uint4 load(int i) const
    {
        constexpr uint32_t fill = BF16 ? 0xFF80FF80u : 0xFF800000u;
        uint32_t w[4] = {fill, fill, fill, fill};
        if (i >= nvec) return make_uint4(fill, fill, fill, fill);
        if (i * E >= off && (i + 1) * E <= off + n) return *(reinterpret_cast<const uint4 *>(x - off * S) + i);
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
    __device__ __forceinline__ bool holds(int i, int j) const { return (uint32_t)(i * E + j - off) < (uint32_t)n; }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[E])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = !BF16 ? __uint_as_float(w[j % 4]) : j % 2 ? bf16hi(w[j / 2]) : bf16lo(w[j / 2]);
    }
};

// What the CTAs of a row share; the first one's copy counts.
struct Shared {
    float2 roots[64];
    float chunk_m[kMaxChunks], chunk_s[kMaxChunks];
    uint64_t chunk[kMaxChunks];  // masses of what is kept
    uint32_t ties[kMaxChunks];   // tokens at the border's key
    uint32_t hist[kBins];      // tokens of a bin
    uint64_t weight[kBins];    // and their masses, where they are asked for
    uint64_t sum;       // of a sweep
    float top;          // the row's maximum
    // the next sweep
    int what;
    uint32_t hi, lo;
    int shift;
    // scratch of the block
    uint64_t w64[kWarps];
    float wf[kWarps];
    uint64_t got64[2];
    uint32_t got32[2];
};
enum { kDone, kHist, kWeigh, kSum, kChunksFast, kChunksExact };

__device__ __forceinline__ uint64_t warp_sum(uint64_t v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Inclusive sums over the block's threads; `all` is the total.
__device__ __forceinline__ uint64_t block_scan(Shared &s, uint64_t v, uint64_t &all)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int o = 1; o < 32; o *= 2) {
        const uint64_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) s.w64[warp] = v;
    __syncthreads();
    uint64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint64_t t = s.w64[w];
        if (w < warp) before += t;
        total += t;
    }
    __syncthreads();
    all = total;
    return before + v;
}

__device__ __forceinline__ uint32_t remote(const void *p, int rank)
{
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(ptx::smem_u32(p)), "r"(rank));
    return to;
}
__device__ __forceinline__ void put(uint32_t to, uint32_t v) { asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "r"(v) : "memory"); }
__device__ __forceinline__ void put64(uint32_t to, uint64_t v) { asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(v) : "memory"); }
__device__ __forceinline__ void add32(uint32_t to, uint32_t v) { asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(to), "r"(v) : "memory"); }
__device__ __forceinline__ void add64(uint32_t to, uint64_t v) { asm volatile("red.shared::cluster.add.u64 [%0], %1;" ::"r"(to), "l"(v) : "memory"); }

template <bool BF16, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Args a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    using R = Row<BF16>;
    constexpr int E = R::E, kUnit = BF16 ? 16 : 0;  // a key's low bits that say nothing
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    int rank = 0, ranks = 1;
    if (CLUSTER) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        ranks = a.cluster;
    }
    const bool lead = rank == 0;
    const auto meet = [&]() {
        if (CLUSTER) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
    };
    if (tid < 64) s.roots[tid] = kRoots[tid];
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0, s.weight[i] = 0;
    if (tid == 0) s.sum = 0;
    if (CLUSTER) meet();  // every CTA of the cluster runs: the first one's memory may be written
    pdl_wait();
    pdl_trigger();

    const int64_t row = blockIdx.x / ranks;
    const R r(a, row);
    const float tau = a.taus ? a.taus[row] : a.tau;
    const int chunks = (r.nvec + kChunkVecs - 1) / kChunkVecs;
    const double c64 = 1.4426950408889634 / (double)tau;
    Exp ex = {0.0f, (float)c64, 0.0f, s.roots};
    ex.c_lo = (float)(c64 - (double)ex.c);
    const bool tau_ok = tau > 1e-30f && tau <= 1e30f;
    if (!tau_ok) {
        if (lead && tid == 0) a.ids[row] = -1, a.logp[row] = a.logq[row] = NAN;
        if (CLUSTER) meet();
        return;
    }

    // ------------------------------------------------------------ chunks' maxima and sums
    for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps) {
        uint4 v[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = r.load(ch * kChunkVecs + j * 32 + lane);
        float m = -FLT_MAX;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            float f[E];
            R::unpack(v[j], f);
#pragma unroll
            for (int e = 0; e < E; ++e) m = fmaxf(m, f[e]);
        }
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float z[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            float f[E];
            R::unpack(v[j], f);
#pragma unroll
            for (int e = 0; e < E; ++e) z[e % 2] += ex2((f[e] - m) * ex.c);  // NaN and +inf leave NaN
        }
        float sum = z[0] + z[1];
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) {
            if (CLUSTER) {
                put(remote(&s.chunk_m[ch], 0), __float_as_uint(m));
                put(remote(&s.chunk_s[ch], 0), __float_as_uint(sum));
            } else {
                s.chunk_m[ch] = m, s.chunk_s[ch] = sum;
            }
        }
    }
    meet();

    // ------------------------------------------------------------ the other CTAs do what the first one asks for
    const auto count_hist = [&](uint32_t hi, uint32_t lo, int shift, bool weigh) {  // and the last bin's fast mass, or all exact
        uint32_t last = 0;
        float z = 0.0f;
        uint64_t zs = 0;
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps) {
            uint4 v[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = r.load(ch * kChunkVecs + j * 32 + lane);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const int i = ch * kChunkVecs + j * 32 + lane;
                const bool whole = i * E >= r.off && (i + 1) * E <= r.off + r.n;
                float f[E];
                R::unpack(v[j], f);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t k = key_of<BF16>(f[e]), bin = (hi - k) >> shift;
                    if (k <= hi && k >= lo && (whole || r.holds(i, e))) {
                        if (weigh) {
                            const uint64_t w = mass(ex, f[e]);
                            if (w) atomicAdd(reinterpret_cast<unsigned long long *>(&s.weight[min(bin, kBins - 1)]), (unsigned long long)w);
                        }
                        if (bin < kBins - 1) {
                            atomicAdd(&s.hist[bin], 1u);
                        } else {
                            ++last;
                            z += ex2((f[e] - ex.top) * ex.c);
                        }
                    }
                }
            }
            zs += (uint64_t)__float2ll_rn(z * pow2f(kScale));
            z = 0.0f;
        }
        last = __reduce_add_sync(0xFFFFFFFFu, last);
        zs = warp_sum(zs);
        if (lane == 0) {
            if (last) atomicAdd(&s.hist[kBins - 1], last);
            if (CLUSTER) {
                add64(remote(&s.sum, 0), zs);
            } else {
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.sum), (unsigned long long)zs);
            }
        }
        if (CLUSTER) {
            __syncthreads();
            if (!lead)
                for (int b = tid; b < kBins; b += kThreads) {
                    const uint32_t n = s.hist[b];
                    if (n) add32(remote(&s.hist[b], 0), n), s.hist[b] = 0;
                    if (weigh) {
                        const uint64_t w = s.weight[b];
                        if (w) add64(remote(&s.weight[b], 0), w), s.weight[b] = 0;
                    }
                }
        }
    };
    const auto sum_exact = [&](uint32_t hi, uint32_t lo) {  // masses of keys in [lo, hi]
        uint64_t z = 0;
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps)
#pragma unroll 1
            for (int j = 0; j < kVec; ++j) {
                float f[E];
                R::unpack(r.load(ch * kChunkVecs + j * 32 + lane), f);
#pragma unroll 1
                for (int e = 0; e < E; ++e) {
                    const uint32_t k = key_of<BF16>(f[e]);
                    if (k >= lo && k <= hi) z += mass(ex, f[e]);
                }
            }
        z = warp_sum(z);
        if (lane == 0) {
            if (CLUSTER) {
                add64(remote(&s.sum, 0), z);
            } else {
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.sum), (unsigned long long)z);
            }
        }
    };
    const auto sum_chunks = [&](uint32_t border, bool exact) {  // keys above the border, and how many are at it
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps) {
            uint4 v[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = r.load(ch * kChunkVecs + j * 32 + lane);
            float z = 0.0f;
            uint64_t z64 = 0;
            uint32_t ties = 0;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const int i = ch * kChunkVecs + j * 32 + lane;
                const bool whole = i * E >= r.off && (i + 1) * E <= r.off + r.n;
                float f[E];
                R::unpack(v[j], f);
                if (exact) {
#pragma unroll 1
                    for (int e = 0; e < E; ++e) {
                        const float x = r.at(i * E + e - r.off);
                        if (key_of<BF16>(x) > border) z64 += mass(ex, x);
                    }
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t k = key_of<BF16>(f[e]);
                    if (!exact) z += k > border ? ex2((f[e] - ex.top) * ex.c) : 0.0f;
                    ties += k == border && (whole || r.holds(i, e));
                }
            }
            ties = __reduce_add_sync(0xFFFFFFFFu, ties);
            if (!exact) {
                for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
                z64 = (uint64_t)__double2ll_rn((double)z * (double)(uint64_t(1) << kScale));
            } else {
                z64 = warp_sum(z64);
            }
            if (lane == 0) {
                if (CLUSTER) {
                    put64(remote(&s.chunk[ch], 0), z64);
                    put(remote(&s.ties[ch], 0), ties);
                } else {
                    s.chunk[ch] = z64, s.ties[ch] = ties;
                }
            }
        }
    };
    const auto sweep = [&]() {
        ex.top = s.top;
        const int what = s.what;
        if (what == kHist || what == kWeigh) count_hist(s.hi, s.lo, s.shift, what == kWeigh);
        if (what == kSum) sum_exact(s.hi, s.lo);
        if (what == kChunksFast || what == kChunksExact) sum_chunks(s.hi, what == kChunksExact);
    };
    if (CLUSTER && !lead) {
        for (;;) {
            meet();  // the order is there
            if (s.what == kDone) break;
            sweep();
            meet();  // and done
        }
        return;
    }
    // One sweep by all of the row's CTAs; called by the first one's threads together.
    const auto ask = [&](int what, uint32_t hi, uint32_t lo, int shift) {
        __syncthreads();
        if (what == kHist || what == kWeigh)
            for (int b = tid; b < kBins; b += kThreads) s.hist[b] = 0, s.weight[b] = 0;
        if (tid == 0) {
            s.sum = 0;
            s.what = what, s.hi = hi, s.lo = lo, s.shift = shift;
        }
        if (CLUSTER && tid > 0 && tid < ranks) {
            put(remote(&s.top, tid), __float_as_uint(ex.top));
            put(remote(&s.hi, tid), hi);
            put(remote(&s.lo, tid), lo);
            put(remote(&s.shift, tid), (uint32_t)shift);
            put(remote(&s.what, tid), (uint32_t)what);
        }
        meet();
        if (what == kDone) return;
        sweep();
        meet();
    };

    // ------------------------------------------------------------ the row's maximum and sum
    float top = -FLT_MAX, bad = 0.0f;
    for (int i = tid; i < chunks; i += kThreads) {
        top = fmaxf(top, s.chunk_m[i]);
        if (isnan(s.chunk_s[i])) bad = 1.0f;
    }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) s.wf[warp] = top;
    const bool any_bad = __syncthreads_or(bad != 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s.wf[w]);
    if (tid == 0) s.top = top;
    ex.top = top;
    uint64_t Z = 0, mine = 0;
    for (int i = tid; i < chunks; i += kThreads) {
        const float t = s.chunk_s[i];
        const uint64_t m = any_bad || t == 0.0f ? 0 : (uint64_t)__double2ll_rn((double)t * (double)mass(ex, s.chunk_m[i]));
        s.chunk[i] = m;
        s.ties[i] = 0;
        mine += m;
    }
    block_scan(s, mine, Z);
    if (any_bad || Z == 0) {  // NaN or +inf among the logits, or nothing but -inf
        if (tid == 0) a.ids[row] = -1, a.logp[row] = a.logq[row] = any_bad ? NAN : -INFINITY;
        ask(kDone, 0, 0, 0);
        return;
    }

    // ------------------------------------------------------------ the border of what is kept
    int k = a.top_ks ? a.top_ks[row] : a.top_k;
    float top_p = a.top_ps ? a.top_ps[row] : a.top_p, min_p = a.min_ps ? a.min_ps[row] : a.min_p;
    if (top_p <= 0.0f) k = 1;
    const bool cut_k = k > 0 && k < r.n, cut_p = top_p > 0.0f && top_p < 1.0f;
    const uint32_t top_key = key_of<BF16>(top);
    uint32_t border = 0;           // keys above it are kept,
    uint32_t keep = 0xFFFFFFFFu;   // and the first `keep` at it
    // The weights of this thread's four bins: tokens, or masses.  Bins of single keys need no sweep of masses; what the last one
    // has then is given.
    const auto weights = [&](bool by_mass, bool weighed, uint32_t hi, int shift, uint64_t last, uint64_t (&w)[4]) -> uint64_t {
        uint64_t sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int b = tid * 4 + j;
            const uint64_t n = s.hist[b];
            w[j] = n;
            if (by_mass && n) w[j] = weighed ? s.weight[b] : b < kBins - 1 ? n * mass(ex, value_of<BF16>(hi - ((uint32_t)b << shift))) : last;
            sum += w[j];
        }
        return sum;
    };
    // The first bin where the sum of weights, `before` it included, reaches `want` (kBins where none does), and the sum before it.
    const auto reach = [&](const uint64_t (&w)[4], uint64_t sum, uint64_t before, uint64_t want, uint64_t &reached) -> uint32_t {
        uint64_t all, at = block_scan(s, sum, all);
        at += before - sum;
        if (tid == 0) s.got32[0] = kBins;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (at < want && at + w[j] >= want) s.got32[0] = tid * 4 + j, s.got64[0] = at;
            at += w[j];
        }
        __syncthreads();
        const uint32_t bin = s.got32[0];
        reached = s.got64[0];
        __syncthreads();
        return bin;
    };
    const auto settle = [&](bool by_mass, uint32_t key, uint64_t n, uint64_t reached, uint64_t want) {
        const uint64_t one = by_mass ? mass(ex, value_of<BF16>(key)) : 1, more = one ? (want - reached + one - 1) / one : n;
        border = key;
        keep = (uint32_t)(more < n ? more : n);
    };
    // The place of the k-th token, or of the first where the sum of masses reaches `want`, by histograms of ever finer bins
    // below the maximum; `first`: the first one is there.  No key below lo counts.
    constexpr int kFirst = BF16 ? 16 : 14;  // fp32: four octaves below the maximum in 2^-9 of the value
    const auto find = [&](bool by_mass, uint64_t want, bool first, uint32_t lo) {
        uint32_t hi = top_key;
        int shift = kFirst;
        uint64_t before = 0;
        for (int turn = 0; turn < 6; ++turn) {  // 2^32 keys, 2^10 bins or more a turn
            const bool weighed = by_mass && shift != kUnit;
            if (!(first && turn == 0)) ask(weighed ? kWeigh : kHist, hi, lo, shift);
            uint64_t w[4], reached;
            const uint64_t sum = weights(by_mass, weighed, hi, shift, uint64_t(1) << 61, w);  // the last bin reaches it if no other does
            const uint32_t bin = reach(w, sum, before, want, reached);
            if (bin >= kBins) return;  // all are kept
            if (shift == kUnit && bin < kBins - 1) {
                settle(by_mass, hi - (bin << shift), s.hist[bin], reached, want);
                return;
            }
            before = reached;
            hi -= bin << shift;
            if (bin < kBins - 1 && hi - lo >= (1u << shift)) lo = hi - ((1u << shift) - 1u);
            const int bits = 32 - __clz(hi - lo);
            shift = max(kUnit, bits < kBinBits ? 0 : bits - kBinBits + 1);  // at most 2^10 bins: no remainder in the last one
        }
    };
    if (cut_k) find(false, (uint64_t)k, false, 0);
    if (cut_p) {
        uint64_t w[4], all, reached;
        const auto wanted = [&](uint64_t z) { return (uint64_t)ceil((double)top_p * (double)z); };
        if (cut_k) {  // the sum of the first k
            uint64_t above = 0;
            if (border != top_key) {
                ask(kSum, 0xFFFFFFFFu, border + (1u << kUnit), 0);
                above = s.sum;
            }
            find(true, wanted(above + keep * mass(ex, value_of<BF16>(border))), false, border);
        } else if (BF16) {
            // Single keys but for the last bin, whose mass is fast: would the choice differ at the ends of what it may be?
            ask(kHist, top_key, 0, kFirst);
            const uint64_t rest = s.sum, sum = weights(true, false, top_key, kFirst, s.sum, w);
            block_scan(s, sum, all);
            const uint64_t off = rest ? (uint64_t)((double)rest * kEps) + 1 : 0;
            const uint32_t bin = reach(w, sum, 0, wanted(all - off), reached);
            bool sure = bin < kBins - 1;
            if (sure) {
                const uint32_t key = top_key - (bin << kFirst);
                settle(true, key, s.hist[bin], reached, wanted(all - off));
                const uint32_t kept = keep;
                if (off) sure = reach(w, sum, 0, wanted(all + off), reached) == bin;
                if (off && sure) {
                    settle(true, key, s.hist[bin], reached, wanted(all + off));
                    sure = keep == kept;
                }
            }
            if (!sure) {
                ask(kSum, 0xFFFFFFFFu, 0, 0);
                Z = s.sum;
                find(true, wanted(Z), false, 0);
            }
        } else {
            ask(kWeigh, top_key, 0, kFirst);
            block_scan(s, weights(true, true, top_key, kFirst, 0, w), Z);
            find(true, wanted(Z), true, 0);
        }
    }
    if (min_p > 0.0f) {
        const double t = (double)top + (double)tau * log((double)fminf(min_p, 1.0f));
        uint32_t least = key_of<false>(__double2float_ru(t));
        // the first bf16 that is as large: their keys end in 0000 above zero and, before the lower half went, in FFFF below
        if (BF16) least = (least & 0x80000000u ? least + 0xFFFFu : least) & 0xFFFF0000u;
        if (least > border) border = least, keep = 0xFFFFFFFFu;
    }
    const bool cut = cut_k || cut_p || min_p > 0.0f;

    // ------------------------------------------------------------ the token
    const float u = fminf(fmaxf(a.u[row], 0.0f), 0.99999994f);  // NaN as 0
    for (int attempt = cut ? 0 : -1; attempt < 2; ++attempt) {
        const bool exact = attempt == 1;
        if (attempt >= 0) {
            if (attempt == 1 || cut) ask(exact ? kChunksExact : kChunksFast, border, 0, 0);
        }
        // ties up to the keep-th; masses up to the target
        uint64_t total = 0, upto_mass = 0;
        const uint64_t tie = cut ? mass(ex, value_of<BF16>(border)) : 0;
        uint64_t seen = 0;
        if (tid == 0) s.got32[0] = 0xFFFFFFFFu;
        uint64_t target = 0;
        // per-thread runs of consecutive chunks
        const int per = (chunks + kThreads - 1) / kThreads, i0 = min(tid * per, chunks), i1 = min(i0 + per, chunks);
        uint64_t nt = 0;
        if (cut || exact) {
            for (int i = i0; i < i1; ++i) nt += s.ties[i];
            uint64_t all;
            seen = block_scan(s, nt, all) - nt;
        }
        uint64_t w = 0, at_tie = seen;
        for (int i = i0; i < i1; ++i) {
            uint64_t m = s.chunk[i];
            if (cut || exact) {
                const uint64_t t = s.ties[i], kept = at_tie >= keep ? 0 : (at_tie + t > keep ? keep - at_tie : t);
                m += kept * (cut ? tie : mass(ex, value_of<BF16>(border)));
                at_tie += t;
            }
            w += m;
        }
        upto_mass = block_scan(s, w, total) - w;
        target = (uint64_t)floor((double)u * (double)total);
        if (target >= total) target = total - 1;
        at_tie = seen;
        uint64_t at = upto_mass;
        for (int i = i0; i < i1; ++i) {
            uint64_t m = s.chunk[i];
            const uint64_t t0 = at_tie;
            if (cut || exact) {
                const uint64_t t = s.ties[i], kept = at_tie >= keep ? 0 : (at_tie + t > keep ? keep - at_tie : t);
                m += kept * (cut ? tie : mass(ex, value_of<BF16>(border)));
                at_tie += t;
            }
            if (at <= target && target < at + m) s.got32[0] = i, s.got64[0] = at, s.got64[1] = t0;
            at += m;
        }
        __syncthreads();
        const int ch = (int)s.got32[0];
        const uint64_t before = s.got64[0], ties_before = s.got64[1];
        __syncthreads();
        if (ch < 0) continue;  // cannot be: total > target
        // that chunk again, consecutive elements a thread
        constexpr int per_thread = kChunkVecs * E / kThreads;
        float f[per_thread];
        uint64_t m[per_thread], t_n = 0;
        const int e0 = ch * kChunkVecs * E + tid * per_thread - r.off;
#pragma unroll
        for (int j = 0; j < per_thread; ++j) {
            f[j] = r.at(e0 + j);
            t_n += cut && e0 + j >= 0 && e0 + j < r.n && key_of<BF16>(f[j]) == border;
        }
        uint64_t all, t_at = 0;
        if (cut) t_at = ties_before + block_scan(s, t_n, all) - t_n;
        uint64_t own = 0;
#pragma unroll
        for (int j = 0; j < per_thread; ++j) {
            const bool in = e0 + j >= 0 && e0 + j < r.n;
            const uint32_t key = key_of<BF16>(f[j]);
            bool kept = in && (!cut || key > border);
            if (cut && in && key == border) kept = t_at++ < keep;
            m[j] = kept ? mass(ex, f[j]) : 0;
            own += m[j];
        }
        uint64_t cum = before + block_scan(s, own, all) - own;
        // how far the fast sums before this chunk and the target may be off
        const uint64_t off = exact ? 0 : (uint64_t)((double)total * kEps) + 2;
        if (tid == 0) s.got32[0] = 0xFFFFFFFFu;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < per_thread; ++j) {
            if (m[j] && cum + off <= target + (cum == 0 ? off : 0) && target + off < cum + m[j]) {
                s.got32[0] = (uint32_t)(e0 + j);
                s.got32[1] = __float_as_uint(f[j]);
            }
            cum += m[j];
        }
        __syncthreads();
        const uint32_t id = s.got32[0];
        if (id != 0xFFFFFFFFu) {
            if (tid == 0) {
                const double y = ((double)__uint_as_float(s.got32[1]) - (double)top) / (double)tau, unit = (double)(uint64_t(1) << kScale);
                a.ids[row] = id;
                a.logp[row] = (float)(y - log((double)Z / unit));
                a.logq[row] = (float)(y - log((double)total / unit));
            }
            break;
        }
        if (attempt == -1) attempt = 0;  // without a cut the chunks' exact sums are next
    }
    ask(kDone, 0, 0, 0);
}

template <bool BF16, bool CLUSTER>
cudaError_t launch(const Args &a, cudaStream_t stream, bool chain)
{
    static OncePerDevice once;
    const auto kernel = sample_kernel<BF16, CLUSTER>;
    cudaError_t e = allow_smem(once, kernel, sizeof(Shared));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.T * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (CLUSTER) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)a.cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (chain) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace
}  // namespace qerl

using namespace qerl;

extern "C" qerl_status qerl_sample(const void *logits, int dtype, int64_t T, int64_t V, int64_t ld, const float *u, const qerl_sample_opts *o,
                                   int64_t *ids, float *logp, float *logq, qerl_stream_t stream)
{
    if ((T != 0 && (!logits || !u || !ids || !logp || !logq)) || !o || (dtype != QERL_DTYPE_F32 && dtype != QERL_DTYPE_BF16)) return QERL_ERR_INVALID_ARG;
    if (T < 0 || V < 1 || ld < V) return QERL_ERR_INVALID_ARG;
    if (!o->temperatures && !(o->temperature > 1e-30f && o->temperature <= 1e30f)) return QERL_ERR_INVALID_ARG;
    if (!o->top_ps && !(o->top_p >= 0.0f && o->top_p <= 1.0f)) return QERL_ERR_INVALID_ARG;
    if (!o->min_ps && !(o->min_p >= 0.0f && o->min_p <= 1.0f)) return QERL_ERR_INVALID_ARG;
    if (!o->top_ks && o->top_k < 0) return QERL_ERR_INVALID_ARG;
    if (V > kMaxV || T > 0x0FFFFFFF || ld > (int64_t(1) << 40)) return QERL_ERR_SHAPE;
    const uintptr_t el = dtype == QERL_DTYPE_BF16 ? 1 : 3;
    const auto at = [](const void *p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) == 0; };
    if (!at(logits, el) || !at(u, 3) || !at(ids, 7) || !at(logp, 3) || !at(logq, 3) || !at(o->temperatures, 3) || !at(o->top_ks, 3) ||
        !at(o->top_ps, 3) || !at(o->min_ps, 3))
        return QERL_ERR_ALIGN;
    QERL_TRY(check_device());
    if (T == 0) return QERL_OK;
    const bool bf16 = dtype == QERL_DTYPE_BF16, chain = g_chain.load() != 0;
    Args a = {logits, ld, T, V, u, o->temperature, o->top_p, o->min_p, o->top_k, o->temperatures, o->top_ps, o->min_ps, o->top_ks, ids, logp, logq, 1};
    // Clusters while the rows alone leave SMs idle (two CTAs each), and no more CTAs than give every warp a chunk.
    const int64_t chunks = (V * (bf16 ? 2 : 4) + kChunkVecs * 16 - 1) / (kChunkVecs * 16);
    while (a.cluster < kMaxCluster && T * a.cluster < num_sms() && chunks > (int64_t)a.cluster * kWarps) a.cluster *= 2;
    if (a.cluster > 1) return launched(bf16 ? launch<true, true>(a, as_cuda(stream), chain) : launch<false, true>(a, as_cuda(stream), chain));
    return launched(bf16 ? launch<true, false>(a, as_cuda(stream), chain) : launch<false, false>(a, as_cuda(stream), chain));
}
