// The next token of every row of logits from a given uniform number.
//
//   p = softmax(x / tau); the tokens in order of (p, then index): kept is the shortest prefix of
//     the first top_k;  those until their sum reaches top_p of the first top_k's;  those with p >= min_p max p
//   id = the first kept token, in order of index, whose sum of kept p up to it exceeds u times that of all;
//   logp = ln p_id,  logq = ln (p_id / sum of kept p).
//
// Which token that is must not depend on rounding, on the number of CTAs or on
// the order of sums: masses e^((x - max) / tau) are held as 64-bit integers (2^42
// for the most probable token), whose sums are exact.  Ways that lead to them:
//   fast   ex2 in FP32, summed over a chunk of 2 KB of the row and then turned to an
//          integer;
//   good   the same with the exponent's rounding taken back, summed as integers;
//   exact  the exponential in pairs of FP32 numbers, good to 2^-40 and one unit.
// The first two are off by at most what is said below, whatever the row holds (equal
// logits are all off the same way).  A choice that this could change is made again with
// good sums, and then with exact ones.
//
// A row is swept by one CTA, or by a cluster of up to eight where there are few
// rows.  The first sweep takes it from HBM: the maximum and the fast sum of each
// chunk.  Without a cut that is enough to know the token's chunk, which is read
// again.  With a cut the first sweep also leaves a sample of the logits, from which
// two thresholds are chosen such that the border of what is kept lies between them,
// with a few thousand tokens at most.  The second sweep (L2; chunks whose maximum
// is below are skipped) lists the tokens between, with their indices, and sums what
// is above by chunk, and below.  The list is sorted and the border found in it with
// exact masses.  top_p compares what is left below the border with 1 - top_p of the
// sum: with top_p near 1 the fast part of that is small.  Where the sample misled,
// or more tokens than the list holds are as good as equal, histograms of the keys
// find the border.
//
// In a graph, over ten inputs each: one row of 131072 bf16 (top-k and top-p) 21 us,
// cluster barriers and dependent steps; 64 rows uncut 14 to 48 us, by how many rows
// need the better sums (their CTAs then work alone); 1024 rows with top-p 0.95, half of
// whose mass is a bulk of tens of thousands of alike tokens: 382 to 484 us, bound by
// issue (70 % of the slots); 257 x 100003 FP32 with every cut 79 to 221 us, the slowest
// rows' latency.  Margins that took errors for independent: 371 to 490 us for the 1024
// rows, and tokens beside the border's.  With histograms of every row's keys in shared
// memory instead of the list: 500 us and 2700 us, atomics on few addresses.
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
constexpr int kMostChunks = kMaxV * 4 / (kChunkVecs * 16) + 2;  // a row may start inside a vector; an even number
constexpr int kScale = 42;
constexpr int kList = 8192, kSamples = 8192;
// What a fast sum may be off by, relative to it.  The exponent y has two roundings of 2^-24 |y| each, 2^-23 ln 2 a value and
// octave.  Weighted by the masses the mean of |y| over n tokens is at most log2 n less the logarithm of their sum (the entropy of
// their shares is at most log2 n).  ex2.approx is off by -1.44e-7 to 1.05e-7 (measured, every float down to -64), and the
// sum of a chunk by seven roundings, as the trees of additions below have them.  These are bounds, not deviations: a row of few
// distinct logits has errors of one sign.
constexpr float kOctave = 8.3e-8f, kFast = 5.7e-7f;
constexpr double kMost = 2.6e-6;  // both over 2^20 tokens
// Of a good sum, with kBias added, ex2.approx's error is what is left; values and the exponent's rounding are summed apart.
constexpr float kGood = 1.3e-7f;
constexpr double kBias = 2e-8;

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
    int cluster, chunks;  // CTAs of a row; chunks that a row may take, wherever it starts
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
    float top, c, c_lo, low;  // low: 200 octaves below 0
    const float2 *roots;
};
// The same in FP32 for a difference d <= 0, 1 for d = 0; NaN stays.
__device__ __forceinline__ float fast(const Exp &e, float d) { return ex2(fmaf(d, e.c, d * e.c_lo)); }
__device__ __forceinline__ uint64_t mass_in_line(const Exp &e, float x)
{
    const float d0 = x - e.top;
    const bool some = d0 * e.c > -60.0f;  // false for NaN
    const float d = some ? d0 : 0.0f, b = d - x, rest = some ? (x - (d - b)) - (e.top + b) : 0.0f;
    const float y = d * e.c;
    const float y_lo = fmaf(d, e.c, -y) + fmaf(d, e.c_lo, rest * e.c);
    const float magic = 12582912.0f, ky = fmaf(y, 64.0f, magic), k = ky - magic, r0 = fmaf(k, -0.015625f, y), r = r0 + y_lo, r_lo = (r0 - r) + y_lo;
    const float t = r * 0x1.62e430p-1f, t_lo = fmaf(r, 0x1.62e430p-1f, -t) + fmaf(r, -0x1.05c610p-29f, r_lo * 0x1.62e430p-1f);
    const float q = t * t * fmaf(t, fmaf(t, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f), s = t_lo + q;
    const float p = t + s, p_lo = (t - p) + s;
    // 2^(k / 64) (1 + p): its first term is an integer of 24 bits times a power of two; the rest, below 2^-7 of it, in two steps
    // of 2^14 and 1, each below 2^22 and rounded by adding 3 * 2^22
    const int n = __float_as_int(ky) - 0x4B400000;
    const float2 T = e.roots[n & 63];
    const int down = -(n >> 6);  // 0 .. 60
    const float unit = pow2f(kScale - down), mid = T.x * p;
    const float low = fmaf(T.x, p, -mid) + fmaf(T.x, p_lo, fmaf(T.y, p, T.y));
    const float coarse = fmaf(mid, unit * 0x1p-14f, magic), a = coarse - magic;
    const float fine = fmaf(low, unit, fmaf(a, -16384.0f, mid * unit)) + magic;
    const uint64_t first = (uint64_t)((__float_as_uint(T.x) & 0x7FFFFFu) | 0x800000u) << (kScale - 23);
    const uint64_t head = (first + ((uint64_t(1) << down) >> 1)) >> down;
    const uint64_t all = head + (int64_t)(__float_as_int(coarse) - 0x4B400000) * 16384 + (int64_t)(__float_as_int(fine) - 0x4B400000);
    return some ? all : 0;
}

// The same as a call, where it is not in a sweep.
__device__ __noinline__ uint64_t mass_call(float x, float top, float c, float c_lo);  // below: the table lies in shared memory
__device__ __forceinline__ uint64_t mass(const Exp &e, float x) { return mass_call(x, e.top, e.c, e.c_lo); }
// The same as fast() of the difference to the maximum, and what the exponent's rounding took from it.
__device__ __forceinline__ float2 good(const Exp &e, float x, bool in)
{
    const float d0 = x - e.top;
    const bool some = in && d0 > e.low;
    const float d = some ? d0 : 0.0f, b = d - x, rest = some ? (x - (d - b)) - (e.top + b) : 0.0f;
    const float y = d * e.c, y_lo = fmaf(d, e.c, -y) + fmaf(d, e.c_lo, rest * e.c), v = some ? ex2(y) : 0.0f;
    return make_float2(v, v * 0x1.62e430p-1f * y_lo);
}
// Sums as trees: log2 E roundings.
template <int E>
__device__ __forceinline__ float tree(float (&g)[E])
{
#pragma unroll
    for (int o = E / 2; o; o /= 2)
#pragma unroll
        for (int e = 0; e < o; ++e) g[e] += g[e + o];
    return g[0];
}

// A row as the aligned 16-byte vectors that hold it; elements outside it read as -inf.
template <bool BF16>
struct Row {
    static constexpr int E = BF16 ? 8 : 4, S = 16 / E;
    const char *x;
    int off, n, nvec;
    __device__ __forceinline__ Row(const char *row, int off_, int n_) : x(row), off(off_), n(n_), nvec((off_ + n_ + E - 1) / E) {}
    __device__ __forceinline__ Row(const Args &a, int64_t row) : Row(static_cast<const char *>(a.x) + row * a.ld * S, 0, (int)a.V)
    {
        off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / S);
        nvec = (off + n + E - 1) / E;
    }
    __device__ __forceinline__ float at(int e) const
    {
        if (!inside(e)) return -INFINITY;
        return BF16 ? bf16f(reinterpret_cast<const __nv_bfloat16 *>(x)[e]) : reinterpret_cast<const float *>(x)[e];
    }
    __device__ __forceinline__ uint4 load(int i) const
    {
        constexpr uint32_t fill = BF16 ? 0xFF80FF80u : 0xFF800000u;
        uint32_t w[4] = {fill, fill, fill, fill};
        if (i >= nvec) return make_uint4(fill, fill, fill, fill);
        if (whole(i)) return *(reinterpret_cast<const uint4 *>(x - off * S) + i);
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
    __device__ __forceinline__ bool whole(int i) const { return i * E >= off && (i + 1) * E <= off + n; }  // vector i
    __device__ __forceinline__ bool inside(int e) const { return e >= 0 && e < n; }
    __device__ __forceinline__ bool holds(int i, int j) const { return inside(i * E + j - off); }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[E])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = !BF16 ? __uint_as_float(w[j % 4]) : j % 2 ? bf16hi(w[j / 2]) : bf16lo(w[j / 2]);
    }
};

// A token's place in the order: larger logits first, equal ones by index.
__device__ __forceinline__ uint64_t place_of(uint32_t key, uint32_t index) { return (uint64_t)~key << 32 | index; }

// What the CTAs of a row share; the first one's copy counts, but for the chunks' maxima, of which each also has its own.
struct Shared {
    float2 roots[64];
    union {
        float sample[kSamples];
        uint64_t list[kList];  // places
    };
    uint64_t small[kThreads];  // those near the border
    uint32_t hist[kBins];    // tokens of a bin
    uint64_t weight[kBins];  // and their masses, where they are asked for
    uint64_t sum, sum_above;  // of a sweep
    uint32_t listed;
    float top;  // the row's maximum
    // the next sweep
    int what;
    uint32_t hi, lo;
    int shift;
    // scratch of the block
    uint64_t w64[kWarps];
    float wf[kWarps];
    uint64_t got64[2];
    uint32_t got32[2], mark[6];
    // and behind it, by chunk: the masses of what is kept, the maximum, the sum, the tokens at the border's key
    static constexpr int kChunkBytes = 8 + 4 + 4 + 4;
};
extern __shared__ __align__(16) uint8_t smem[];

enum { kDone, kHist, kWeigh, kSum, kSumOutside, kBetween, kBetweenSums, kKeptFast, kKeptGood, kKeptExact };

__device__ __forceinline__ uint64_t warp_sum(uint64_t v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __noinline__ uint64_t mass_call(float x, float top, float c, float c_lo)
{
    return mass_in_line(Exp{top, c, c_lo, 0.0f, reinterpret_cast<Shared *>(smem)->roots}, x);
}

// The sum over a warp of numbers up to 32, in units of 2^-42, each rounded to one: in steps of 2^-21 and of a unit.
__device__ __forceinline__ uint64_t warp_fixed(float v)
{
    const uint32_t coarse = __float2uint_rn(v * 0x1p21f);
    const int fine = __float2int_rn(fmaf((float)coarse, -0x1p-21f, v) * 0x1p42f);
    return ((uint64_t)__reduce_add_sync(0xFFFFFFFFu, coarse) << 21) + (int64_t)__reduce_add_sync(0xFFFFFFFFu, fine);
}

struct Scan {
    uint64_t upto, all;
};
__device__ __noinline__ Scan scan_call(uint64_t v)
{
    Shared &s = *reinterpret_cast<Shared *>(smem);
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
    return Scan{before + v, total};
}
// Inclusive sums over the block's threads; `all` is the total.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t &all)
{
    const Scan r = scan_call(v);
    all = r.all;
    return r.upto;
}
__device__ __forceinline__ uint64_t fixed(float v) { return (uint64_t)__float2ll_rn(v * pow2f(kScale)); }  // 2^20 tokens at most

// Shared memory of the row's first CTA.
template <bool CLUSTER>
struct Lead {
    static __device__ __forceinline__ uint32_t remote(const void *p, int rank)
    {
        uint32_t to;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(ptx::smem_u32(p)), "r"(rank));
        return to;
    }
    static __device__ __forceinline__ void put(uint32_t *p, uint32_t v, int rank = 0)
    {
        if (CLUSTER)
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(remote(p, rank)), "r"(v) : "memory");
        else
            *p = v;
    }
    static __device__ __forceinline__ void put(float *p, float v) { put(reinterpret_cast<uint32_t *>(p), __float_as_uint(v)); }
    static __device__ __forceinline__ void put(uint64_t *p, uint64_t v)
    {
        if (CLUSTER)
            asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(remote(p, 0)), "l"(v) : "memory");
        else
            *p = v;
    }
    static __device__ __forceinline__ uint32_t add(uint32_t *p, uint32_t v)
    {
        uint32_t old;
        if (CLUSTER)
            asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(remote(p, 0)), "r"(v) : "memory");
        else
            old = atomicAdd(p, v);
        return old;
    }
    static __device__ __forceinline__ void add(uint64_t *p, uint64_t v)
    {
        if (CLUSTER)
            asm volatile("red.shared::cluster.add.u64 [%0], %1;" ::"r"(remote(p, 0)), "l"(v) : "memory");
        else
            atomicAdd(reinterpret_cast<unsigned long long *>(p), (unsigned long long)v);
    }
};

// The first n <= kThreads entries of s.small in order; returns this thread's.
__device__ __noinline__ uint64_t sort_small(int n)
{
    Shared &s = *reinterpret_cast<Shared *>(smem);
    const int tid = threadIdx.x;
    uint64_t v = tid < n ? s.small[tid] : ~uint64_t(0);
    for (int k = 2; k < 2 * n; k *= 2)
        for (int j = k / 2; j; j /= 2) {
            uint64_t y;
            if (j >= 32) {  // near exchanges stay in a warp
                __syncthreads();
                s.small[tid] = v;
                __syncthreads();
                y = s.small[tid ^ j];
            } else {
                y = __shfl_xor_sync(0xFFFFFFFFu, v, j);
            }
            const bool smaller = ((tid & j) == 0) == ((tid & k) == 0);  // this place gets the smaller one
            if ((y < v) == smaller) v = y;
        }
    __syncthreads();
    return v;
}

// What the first CTA of a row asks all of them for (s.what): one place in the code, with what it needs by value.
template <bool BF16, bool CLUSTER>
__device__ __noinline__ void sweep(const char *x, int off, int n, int chunks, int most_chunks, float c, float c_lo, float low_, int rank, int ranks)
{
    Shared &s = *reinterpret_cast<Shared *>(smem);
    using R = Row<BF16>;
    using L = Lead<CLUSTER>;
    constexpr int E = R::E;
    const auto key_of = [](float v) { return qerl::key_of<BF16>(v); };
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const bool lead = rank == 0;
    const R r(x, off, n);
    const Exp ex = {s.top, c, c_lo, low_, s.roots};
    uint64_t *const s_chunk = reinterpret_cast<uint64_t *>(smem + sizeof(Shared));
    const float *const s_chunk_m = reinterpret_cast<const float *>(s_chunk + most_chunks);
    uint32_t *const s_ties = reinterpret_cast<uint32_t *>(s_chunk + 2 * most_chunks);
    const auto merge_hist = [&]() {
        if (!CLUSTER) return;
        __syncthreads();
        if (!lead)
            for (int b = tid; b < kBins; b += kThreads) {
                const uint32_t n = s.hist[b];
                if (n) L::add(&s.hist[b], n), s.hist[b] = 0;
                const uint64_t w = s.weight[b];
                if (w) L::add(&s.weight[b], w), s.weight[b] = 0;
            }
    };
    // histogram of keys in [lo, hi], the last bin with the rest; and the bins' exact masses
    const auto count_hist = [&](uint32_t hi, uint32_t lo, int shift, bool weigh) {
        uint32_t last = 0;
        uint64_t zs = 0;
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps) {
            if (key_of(s_chunk_m[ch]) < lo) continue;
            uint4 v[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = r.load(ch * kChunkVecs + j * 32 + lane);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const int i = ch * kChunkVecs + j * 32 + lane;
                const bool whole = r.whole(i);
                float f[E];
                R::unpack(v[j], f);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t key = key_of(f[e]), bin = (hi - key) >> shift;
                    if (key <= hi && key >= lo && (whole || r.holds(i, e))) {
                        const uint64_t w = weigh ? mass(ex, f[e]) : 0;
                        if (bin < kBins - 1) {
                            atomicAdd(&s.hist[bin], 1u);
                            if (w) atomicAdd(reinterpret_cast<unsigned long long *>(&s.weight[bin]), (unsigned long long)w);
                        } else {
                            ++last;
                            zs += w;
                        }
                    }
                }
            }
        }
        last = __reduce_add_sync(0xFFFFFFFFu, last);
        if (lane == 0 && last) atomicAdd(&s.hist[kBins - 1], last);
        if (weigh) {
            zs = warp_sum(zs);
            if (lane == 0 && zs) atomicAdd(reinterpret_cast<unsigned long long *>(&s.weight[kBins - 1]), (unsigned long long)zs);
        }
        merge_hist();
    };
    // The good masses of a vector's elements that are in the mask, to z, and of those that are in `also`, to z_also as well; without
    // branches, so that the elements' chains overlap.  Values as integers of 2^-21, what that leaves as integers of 2^-42, both
    // by adding 3 * 2^22; the exponents' part, some 2^-20 of them, beside them.
    const auto add_good = [&](const float (&f)[E], uint32_t in, uint32_t also, uint64_t &z, uint64_t &z_also) {
        const float magic = 12582912.0f;
        uint32_t coarse[2] = {0u - E * 0x4B400000u, 0u - __popc(also) * 0x4B400000u}, fine[2] = {coarse[0], coarse[1]};
        float rest[2] = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 v = good(ex, f[e], in >> e & 1);
            const float c = fmaf(v.x, 0x1p21f, magic), d = fmaf(fmaf(c - magic, -0x1p-21f, v.x), 0x1p42f, magic);
            coarse[0] += __float_as_uint(c), fine[0] += __float_as_uint(d), rest[0] += v.y;
            if (also >> e & 1) coarse[1] += __float_as_uint(c), fine[1] += __float_as_uint(d), rest[1] += v.y;
        }
        const auto all = [&](int i) { return ((uint64_t)coarse[i] << 21) + (int64_t)(int)fine[i] + (int64_t)__float2int_rn(rest[i] * 0x1p42f); };
        z += all(0);
        if (also) z_also += all(1);
    };
    // exact
    const auto add_exact = [&](const float (&f)[E], uint32_t in, uint64_t &z) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint64_t m = mass_in_line(ex, f[e]);
            z += in >> e & 1 ? m : 0;
        }
    };
    const auto sum_again = [&](uint32_t hi, uint32_t lo) {  // exact masses of keys in [lo, hi]
        uint64_t z = 0;
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps) {
            if (key_of(s_chunk_m[ch]) < lo) continue;
#pragma unroll 1
            for (int j = 0; j < kVec; ++j) {
                float f[E];
                R::unpack(r.load(ch * kChunkVecs + j * 32 + lane), f);
                uint32_t in = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) in |= (key_of(f[e]) >= lo && key_of(f[e]) <= hi ? 1u : 0u) << e;
                if (!__any_sync(0xFFFFFFFFu, in)) continue;
                add_exact(f, in, z);
            }
        }
        z = warp_sum(z);
        if (lane == 0) L::add(&s.sum, z);
    };
    const auto sum_outside = [&](float high, float low) {  // good masses outside [low, high], and of those the ones above
        uint64_t z = 0, z_above = 0;
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps)
#pragma unroll 1
            for (int j = 0; j < kVec; ++j) {
                float f[E];
                R::unpack(r.load(ch * kChunkVecs + j * 32 + lane), f);
                uint32_t below = 0, above = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) below |= (f[e] < low ? 1u : 0u) << e, above |= (f[e] > high ? 1u : 0u) << e;
                if (__any_sync(0xFFFFFFFFu, below | above)) add_good(f, below | above, above, z, z_above);
            }
        z = warp_sum(z), z_above = warp_sum(z_above);
        if (lane == 0) L::add(&s.sum, z), L::add(&s.sum_above, z_above);
    };
    // Tokens in [low, high] to the list; with `sums` the fast masses above it by chunk, and below it together.  The chunks that
    // lie below are the first CTA's to add.
    const auto between = [&](float high, float low, bool sums) {
        uint64_t zs = 0;
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps) {
            if (s_chunk_m[ch] < low) continue;
            uint4 v[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = r.load(ch * kChunkVecs + j * 32 + lane);
            float above[E] = {}, below[E] = {};
            uint32_t in = 0;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                float f[E];
                R::unpack(v[j], f);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const bool is_low = f[e] < low, is_high = f[e] > high;
                    if (sums) {
                        const float m = fast(ex, f[e] - ex.top);
                        if (is_low) below[e] += m;
                        if (is_high) above[e] += m;
                    }
                    if (!is_low && !is_high) in |= 1u << (j * E + e);
                }
            }
            if (sums) {
                const uint64_t sum = warp_fixed(tree(above));
                zs += fixed(tree(below));
                if (lane == 0) L::put(&s_chunk[ch], sum);
            }
            if (__any_sync(0xFFFFFFFFu, in)) {
                const uint32_t n = __popc(in);
                uint32_t at = n;
                for (int o = 1; o < 32; o *= 2) {
                    const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, at, o);
                    if (lane >= o) at += t;
                }
                uint32_t base = 0;
                if (lane == 31) base = L::add(&s.listed, at);
                at += __shfl_sync(0xFFFFFFFFu, base, 31) - n;
                for (; in; in &= in - 1, ++at) {
                    const int b = __ffs(in) - 1, e = (ch * kChunkVecs + (b / E) * 32 + lane) * E + b % E - r.off;
                    // outside the row only where low is -inf: the last of all, without mass
                    if (at < kList) L::put(&s.list[at], r.inside(e) ? place_of(key_of(r.at(e)), (uint32_t)e) : ~uint64_t(0) - 1);
                }
            }
        }
        if (sums) {
            zs = warp_sum(zs);
            if (lane == 0) L::add(&s.sum, zs);
        }
    };
    // By chunk: what is above the border, fast, and how many are at it; or what is kept, good or exact, `upto` the last index at the border.
    const auto kept_fast = [&](float border) {
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps) {
            uint64_t sum = 0;
            uint32_t ties = 0;
            if (s_chunk_m[ch] >= border) {
                uint4 v[kVec];
                float above[E] = {};
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[j] = r.load(ch * kChunkVecs + j * 32 + lane);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    float f[E];
                    R::unpack(v[j], f);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        if (f[e] > border) above[e] += fast(ex, f[e] - ex.top);
                        if (f[e] == border) ++ties;  // nothing outside the row unless the border is -inf, where no mass is at it
                    }
                }
                sum = warp_fixed(tree(above));
                ties = __reduce_add_sync(0xFFFFFFFFu, ties);
            }
            if (lane == 0) {
                L::put(&s_chunk[ch], sum);
                L::put(&s_ties[ch], ties);
            }
        }
    };
    const auto kept_again = [&](float border, uint32_t upto, bool exact) {
        for (int ch = rank * kWarps + warp; ch < chunks; ch += ranks * kWarps) {
            uint64_t z = 0;
            if (s_chunk_m[ch] >= border) {
#pragma unroll 1
                for (int j = 0; j < kVec; ++j) {
                    const int i = ch * kChunkVecs + j * 32 + lane;
                    float f[E];
                    R::unpack(r.load(i), f);
                    uint32_t in = 0;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        in |= (f[e] > border || (f[e] == border && (uint32_t)max(i * E + e - r.off, 0) <= upto) ? 1u : 0u) << e;
                    if (!__any_sync(0xFFFFFFFFu, in)) continue;
                    if (exact)
                        add_exact(f, in, z);
                    else
                        add_good(f, in, 0, z, z);
                }
                z = warp_sum(z);
            }
            if (!exact) z += (uint64_t)((float)z * (float)kBias);
            if (lane == 0) L::put(&s_chunk[ch], z);
        }
    };
    const int what = s.what;
    const uint32_t hi = s.hi, lo = s.lo;
    if (what == kHist || what == kWeigh) count_hist(hi, lo, s.shift, what == kWeigh);
    if (what == kSum) sum_again(hi, lo);
    if (what == kSumOutside) sum_outside(__uint_as_float(hi), __uint_as_float(lo));
    if (what == kBetween || what == kBetweenSums) between(__uint_as_float(hi), __uint_as_float(lo), what == kBetweenSums);
    if (what == kKeptFast) kept_fast(__uint_as_float(hi));
    if (what == kKeptExact || what == kKeptGood) kept_again(__uint_as_float(hi), lo, what == kKeptExact);
}

template <bool BF16, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Args a)
{
    Shared &s = *reinterpret_cast<Shared *>(smem);
    using R = Row<BF16>;
    using L = Lead<CLUSTER>;
    constexpr int E = R::E, kUnit = BF16 ? 16 : 0;  // a key's low bits that say nothing
    constexpr int kChunk = kChunkVecs * E;          // tokens of a chunk
    const auto key_of = [](float x) { return qerl::key_of<BF16>(x); };
    const auto value_of = [](uint32_t k) { return qerl::value_of<BF16>(k); };
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
    if (CLUSTER) meet();  // every CTA of the cluster runs: the first one's memory may be written
    pdl_wait();
    pdl_trigger();

    const int64_t row = blockIdx.x / ranks;
    const R r(a, row);
    const float tau = a.taus ? a.taus[row] : a.tau;
    int k = a.top_ks ? a.top_ks[row] : a.top_k;
    const float top_p = a.top_ps ? a.top_ps[row] : a.top_p, min_p = a.min_ps ? a.min_ps[row] : a.min_p;
    if (top_p <= 0.0f) k = 1;
    const bool cut_k = k > 0 && k < r.n, cut_p = top_p > 0.0f && top_p < 1.0f, cut_m = min_p > 0.0f;
    const int chunks = (r.nvec + kChunkVecs - 1) / kChunkVecs;
    uint64_t *const s_chunk = reinterpret_cast<uint64_t *>(smem + sizeof(Shared));
    float *const s_chunk_m = reinterpret_cast<float *>(s_chunk + a.chunks), *const s_chunk_s = s_chunk_m + a.chunks;
    uint32_t *const s_ties = reinterpret_cast<uint32_t *>(s_chunk_s + a.chunks);
    // log2(e) / tau in two numbers; log2(e) = 0x1.715476p+0 + 0x1.4ae0cp-26
    Exp ex = {0.0f, __fdiv_rn(0x1.715476p+0f, tau), 0.0f, -138.0f * tau, s.roots};
    const auto rest_of = [&](float c) { return __fdiv_rn(fmaf(-c, tau, 0x1.715476p+0f) + 0x1.4ae0cp-26f, tau); };
    ex.c_lo = rest_of(ex.c);
    if (!(ex.c_lo > 0.0f)) ex.c = __uint_as_float(__float_as_uint(ex.c) - 1u), ex.c_lo = rest_of(ex.c);  // so that -inf c_lo is -inf
    if (!(tau > 1e-30f && tau <= 1e30f)) {
        if (lead && tid == 0) a.ids[row] = -1, a.logp[row] = a.logq[row] = NAN;
        if (CLUSTER) meet();
        return;
    }

    // ------------------------------------------------------------ chunks' maxima and sums, and a sample
    // two of a lane's tokens, from every chunk or from fewer, so that kSamples hold
    const int every = (chunks + kSamples / 64 - 1) / (kSamples / 64);
    const bool sampled = cut_k || cut_p;
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
            if (sampled && j % 2 == 0 && ch % every == 0) L::put(&s.sample[(ch / every) * 64 + j * 16 + lane], f[E / 2]);
        }
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float z[E] = {};
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            float f[E];
            R::unpack(v[j], f);
#pragma unroll
            for (int e = 0; e < E; ++e) z[e] += fast(ex, f[e] - m);  // NaN and +inf leave NaN
        }
        const float own = tree(z), sum = __any_sync(0xFFFFFFFFu, isnan(own)) ? NAN : (float)warp_fixed(own) * 0x1p-42f;
        if (lane == 0) {
            if (CLUSTER) s_chunk_m[ch] = m;
            L::put(&s_chunk_m[ch], m);
            L::put(&s_chunk_s[ch], sum);
        }
    }
    meet();

    const auto run_sweep = [&]() { sweep<BF16, CLUSTER>(r.x, r.off, r.n, chunks, a.chunks, ex.c, ex.c_lo, ex.low, rank, ranks); };
    if (CLUSTER && !lead) {
        for (;;) {
            meet();  // the order is there
            if (s.what == kDone) break;
            run_sweep();
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
            s.sum = s.sum_above = 0;
            s.listed = 0;
            s.what = what, s.hi = hi, s.lo = lo, s.shift = shift;
        }
        if (CLUSTER && tid > 0 && tid < ranks) {
            L::put(reinterpret_cast<uint32_t *>(&s.top), __float_as_uint(ex.top), tid);
            L::put(&s.hi, hi, tid);
            L::put(&s.lo, lo, tid);
            L::put(reinterpret_cast<uint32_t *>(&s.shift), (uint32_t)shift, tid);
            L::put(reinterpret_cast<uint32_t *>(&s.what), (uint32_t)what, tid);
        }
        meet();
        if (what == kDone) return;
        run_sweep();
        meet();
    };

    // ------------------------------------------------------------ the row's maximum and sum
    float top = -FLT_MAX, bad = 0.0f;
    for (int i = tid; i < chunks; i += kThreads) {
        top = fmaxf(top, s_chunk_m[i]);
        if (isnan(s_chunk_s[i])) bad = 1.0f;
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
        const float t = s_chunk_s[i];
        const uint64_t m = any_bad || t == 0.0f ? 0 : (uint64_t)__double2ll_rn((double)t * (double)mass(ex, s_chunk_m[i]));
        s_chunk[i] = m;
        mine += m;
    }
    block_scan(mine, Z);
    if (any_bad || Z == 0) {  // NaN or +inf among the logits, or nothing but -inf
        if (tid == 0) a.ids[row] = -1, a.logp[row] = a.logq[row] = any_bad ? NAN : -INFINITY;
        ask(kDone, 0, 0, 0);
        return;
    }
    const uint32_t top_key = key_of(top);
    uint32_t least = 0;  // the smallest key that min_p keeps
    if (cut_m) {
        least = qerl::key_of<false>(__double2float_ru((double)top + (double)tau * log((double)fminf(min_p, 1.0f))));
        // the first bf16 that is as large: their keys end in 0000 above zero and, before the lower half went, in FFFF below
        if (BF16) least = (least & 0x80000000u ? least + 0xFFFFu : least) & 0xFFFF0000u;
    }

    // What a fast sum of the row's may be off by: |y| counts from the row's maximum, in the first sweep from the chunk's.
    const auto off_fast = [&](uint64_t z) -> float {
        const float octaves = __log2f((float)r.n) + (float)kScale - __log2f((float)z), most = sampled || cut_m ? 64.0f : __log2f((float)kChunk);
        return z ? (float)z * fmaf(kOctave, fminf(fmaxf(octaves, 0.0f), most), kFast) : 0.0f;
    };
    const uint64_t units = (uint64_t)chunks * kChunk + 1024;  // and every sum for roundings to units, less than one a token

    // ------------------------------------------------------------ the border of what is kept, by a list
    uint64_t last = ~uint64_t(0);  // the last place that is kept
    bool found = !sampled && !cut_m, fast = found;  // `fast`: the chunks' masses are
    const auto wanted = [&](uint64_t z) { return (uint64_t)ceil((double)top_p * (double)z); };
    if (sampled) {
        // Thresholds from a histogram in 32nds of an octave below the maximum; the last bin has no mass.  For the first k tokens: of
        // the chunks' maxima, k of which are k tokens, or, where there are too few chunks, of the sample.  For top_p: of the
        // sample, by what it puts below.
        const bool by_max = cut_k && 2 * (int64_t)k <= chunks;
        const int n_sample = by_max ? chunks : (chunks + every - 1) / every * 64;
        const float step = 32.0f * ex.c, W = by_max ? 1.0f : (float)(kChunk * every) / 64.0f;
        for (int i = tid; i < n_sample; i += kThreads) {
            const float x = by_max ? s_chunk_m[i] : s.sample[i], y = (top - x) * step;
            if (y < kBins - 1.0f)
                atomicAdd(&s.hist[(int)y], 1u);
        }
        if (tid < 6) s.mark[tid] = kBins;
        __syncthreads();
        uint64_t cnt = 0, below = 0, all_cnt, all_mass = 0;
        float squares = 0.0f;
        uint32_t n[4];
        uint64_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int b = tid * 4 + j;
            n[j] = s.hist[b];
            m[j] = 0;
            if (!cut_k && n[j] && b < kBins - 1) {
                const float e = ex2((float)(2 * b + 1) * (-1.0f / 64.0f));
                m[j] = fixed((float)n[j] * e);
                squares += (float)n[j] * e * e;
            }
            cnt += n[j], below += m[j];
        }
        uint64_t at_cnt = block_scan(cnt, all_cnt) - cnt, at_mass = 0;
        if (!cut_k) {
            at_mass = block_scan(below, all_mass) - below;
            // the sum of squares of the masses from this thread's bins on: the variance of what the sample puts below
            for (int o = 1; o < 32; o *= 2) {
                const float t = __shfl_down_sync(0xFFFFFFFFu, squares, o);
                if (lane + o < 32) squares += t;
            }
            if (lane == 0) s.wf[warp] = squares;
            __syncthreads();
            for (int w = warp + 1; w < kWarps; ++w) squares += s.wf[w];
        }
        const float sigma = W * sqrtf(squares) * pow2f(kScale), rest = (1.0f - top_p) * (float)Z, need = by_max ? (float)k : (float)k + 8.0f * sqrtf(W * (float)k) + 6.0f * W;
        // of bin b on: enough tokens in the bins up to b; or little enough below them; or surely too much
        const auto marks = [&](uint64_t c, uint64_t at) -> uint32_t {
            const float left = W * (float)(all_mass - at), upto = W * (float)c;
            if (cut_k) return upto >= need ? 2 : 0;
            // A list of all that is above has to be generous: what stands out is not in the sample.  Where the border lies among
            // many alike, the sample knows what is below it within its own deviation.
            return (left + 3.0f * sigma <= 0.25f * rest && upto <= 0.6f * kList ? 1 : 0) | (left + 3.0f * sigma <= 0.99f * rest ? 2 : 0) |
                   (left - 3.0f * sigma < 1.01f * rest ? 4 : 0) | (upto > 1000.0f ? 8 : 0) | (left + 2.0f * sigma <= 0.997f * rest ? 16 : 0) |
                   (left - 2.0f * sigma < 1.003f * rest ? 32 : 0);
        };
        uint64_t c = at_cnt, at = at_mass;
        uint32_t first[6] = {kBins, kBins, kBins, kBins, kBins, kBins};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t b = tid * 4 + j;
            c += n[j], at += m[j];
            const uint32_t now = marks(c, at);
#pragma unroll
            for (int i = 0; i < 6; ++i)
                if (now >> i & 1) first[i] = min(first[i], b);
        }
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            const uint32_t b = __reduce_min_sync(0xFFFFFFFFu, first[i]);
            if (lane == 0 && b < kBins) atomicMin(&s.mark[i], b);
        }
        __syncthreads();
        const bool all_listed = cut_k || s.mark[0] < kBins;
        // all that is above: down to where there are a thousand, or further
        uint32_t b_low = cut_k || !all_listed ? s.mark[1] : max(s.mark[0], min(s.mark[3], kBins - 1u) - 1u), b_high = all_listed ? 0 : s.mark[2] % kBins;
        const uint32_t narrow[2] = {s.mark[4], s.mark[5] % kBins};
        const auto tokens_between = [&](uint32_t from, uint32_t to) -> float {  // in the bins up to b_low, less those before b_high
            __syncthreads();
            if (tid < 2) s.got64[tid] = 0;
            __syncthreads();
            uint64_t c = at_cnt;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t b = tid * 4 + j;
                c += n[j];
                if (b == min(to, kBins - 1u)) s.got64[0] = c;
                if (b + 1 == from) s.got64[1] = c;
            }
            __syncthreads();
            return W * (float)(s.got64[0] - s.got64[1]);
        };
        bool try_list = tokens_between(b_high, b_low) <= 0.8f * kList;
        if (!try_list && !all_listed) {  // nearer thresholds, which miss the border more often
            b_low = narrow[0], b_high = narrow[1];
            try_list = tokens_between(b_high, b_low) <= 0.8f * kList;
        }
        // fewer than k within 64 octaves: what lies below has no mass
        float low = top - (float)min(b_low + 1, kBins - 1u) / step, high = b_high ? top - (float)b_high / step : INFINITY;
        if (r.n <= kThreads || (r.n <= kList && !try_list)) try_list = true, low = -INFINITY, high = INFINITY;
        if (BF16) low = __bfloat162float(__float2bfloat16_rd(low)), high = __bfloat162float(__float2bfloat16_ru(high));
        const auto skipped_below = [&](float bound) -> uint64_t {  // fast masses of the chunks that the sweep skips
            uint64_t sum = 0, all;
            for (int i = tid; i < chunks; i += kThreads)
                if (s_chunk_m[i] < bound) sum += s_chunk[i];
            block_scan(sum, all);
            return all;
        };
        if (cut_m && least > key_of(high)) try_list = false;  // min_p's border is the one, as a rule
        if (try_list) {
            const bool sums = !cut_k;
            const uint64_t skipped = sums ? skipped_below(low) : 0;
            for (int i = tid; i < chunks; i += kThreads) s_chunk[i] = 0;
            for (int i = tid; i < kBins; i += kThreads) s.weight[i] = 0;
            uint64_t below = 0, above = 0, held = 0, t;
            ask(sums ? kBetweenSums : kBetween, __float_as_uint(high), __float_as_uint(low), 0);
            const uint32_t listed = s.listed;
            below = skipped + s.sum;
            if (listed <= kList && listed > 0) {
                const auto mass_at = [&](uint64_t place) { return mass(ex, value_of(~(uint32_t)(place >> 32))); };
                // Longer lists than a thread's entry each: in bins of keys, of which those near the border are gathered.
                const bool binned = listed > kThreads;
                const uint32_t spread = top_key - key_of(low);
                const int shift = max(kUnit, 32 - __clz(spread) - kBinBits);
                const auto bin_of = [&](uint64_t place) { return min((top_key - ~(uint32_t)(place >> 32)) >> shift, kBins - 1u); };
                if (binned) {
                    __syncthreads();
                    for (int b = tid; b < kBins; b += kThreads) s.hist[b] = 0;
                    __syncthreads();
                    for (int i = tid; i < (int)listed; i += kThreads) {
                        const uint64_t place = s.list[i], w = mass_at(place);
                        atomicAdd(&s.hist[bin_of(place)], 1u);
                        if (w && shift > kUnit) atomicAdd(reinterpret_cast<unsigned long long *>(&s.weight[bin_of(place)]), (unsigned long long)w);
                        held += w;
                    }
                } else {
                    uint64_t place = 0;
                    if (tid < (int)listed) held = mass_at(place = s.list[tid]);
                    s.small[tid] = place;
                }
                t = held;
                block_scan(t, held);
                // The first entries up to which the tokens, or masses, reach `from` and `to`; with the mass up to the first.
                int sorted = 0;
                uint64_t own = 0, mass_before = 0, count_before = 0;
                const auto pick = [&](bool by_mass, uint64_t from, uint64_t to, uint64_t &place0, uint64_t &place1, uint64_t &upto) -> bool {
                    if (binned) {
                        uint64_t w[4], c[4], sum = 0, count = 0, all;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int b = tid * 4 + j;
                            c[j] = s.hist[b];
                            w[j] = shift > kUnit ? s.weight[b] : c[j] ? c[j] * mass(ex, value_of(top_key - ((uint32_t)b << shift))) : 0;  // one key a bin
                            sum += w[j], count += c[j];
                        }
                        uint64_t at_m = block_scan(sum, all) - sum, at_c = block_scan(count, all) - count;
                        if (tid < 2) s.got32[tid] = kBins;
                        if (tid == 2) s.listed = 0;
                        __syncthreads();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t at = by_mass ? at_m : at_c, add = by_mass ? w[j] : c[j];
                            if (at < from && at + add >= from) s.got32[0] = tid * 4 + j, s.got64[0] = at_m, s.got64[1] = at_c;
                            if (at < to && at + add >= to) s.got32[1] = tid * 4 + j;
                            at_m += w[j], at_c += c[j];
                        }
                        __syncthreads();
                        const uint32_t b0 = s.got32[0], b1 = s.got32[1];
                        mass_before = s.got64[0], count_before = s.got64[1];
                        if (b0 >= kBins || b1 >= kBins) return false;
                        for (int i = tid; i < (int)listed; i += kThreads) {
                            const uint64_t place = s.list[i];
                            if (bin_of(place) >= b0 && bin_of(place) <= b1) {
                                const uint32_t to_ = atomicAdd(&s.listed, 1u);
                                if (to_ < kThreads) s.small[to_] = place;
                            }
                        }
                        __syncthreads();
                        sorted = 0;
                        if (s.listed > kThreads) return false;  // as good as equal ones
                    }
                    const int n_small = binned ? (int)s.listed : (int)listed;
                    if (!sorted) {
                        own = sort_small(n_small);
                        sorted = 1;
                    }
                    const uint64_t m = tid < n_small ? mass_at(own) : 0;
                    uint64_t all, at_m = mass_before + block_scan(m, all);
                    const uint64_t at = by_mass ? at_m : count_before + tid + 1, before = at - (by_mass ? m : 1);
                    if (tid < 2) s.got64[tid] = 0;
                    __syncthreads();
                    if (tid < n_small && before < from && at >= from) s.got64[0] = own, s.sum = at_m;
                    if (tid < n_small && before < to && at >= to) s.got64[1] = own;
                    __syncthreads();
                    place0 = s.got64[0], place1 = s.got64[1], upto = s.sum;
                    __syncthreads();
                    return place0 != 0 && place1 != 0;
                };
                bool kept = false;
                uint64_t border = 0, other, upto;
                if (cut_k) {
                    const uint64_t few = min((uint32_t)k, listed);
                    kept = (listed >= (uint32_t)k || b_low >= kBins - 1) && pick(false, few, few, border, other, upto);
                    if (kept && cut_p) {
                        const uint64_t want = wanted(upto);  // of the sum of the first k
                        kept = pick(true, want, want, border, other, upto);
                    }
                } else {
                    uint64_t part = 0;
                    for (int i = tid; i < chunks; i += kThreads) part += s_chunk[i];
                    block_scan(part, above);
                    // The border is the first token after which at most 1 - top_p of the sum is left.  The fast sums may move that by
                    // `off`: is it the same token at either end?
                    const auto again = [&](bool exact) {
                        if (exact) {
                            const auto sum = [&](uint64_t &v, uint32_t hi, uint32_t lo) {
                                if (!v) return;
                                ask(kSum, hi, lo, 0);
                                v = s.sum;
                            };
                            sum(below, key_of(low) - (1u << kUnit), 0);
                            sum(above, 0xFFFFFFFFu, key_of(high) + (1u << kUnit));
                        } else {
                            ask(kSumOutside, __float_as_uint(high), __float_as_uint(low), 0);
                            above = s.sum_above, below = s.sum - above;
                            above += (uint64_t)((float)above * (float)kBias), below += (uint64_t)((float)below * (float)kBias);
                        }
                        Z = above + held + below;
                    };
                    const auto choose = [&](bool good) -> bool {
                        const double in_list = (double)(held + below), leaves = (1.0 - (double)top_p) * (double)(above + held + below);
                        const double off = (double)((1.0f - top_p) * (good ? kGood * (float)above : off_fast(above)) +
                                                    top_p * (good ? kGood * (float)below : off_fast(below))) + (double)units;
                        if (!(in_list - leaves > off && in_list - leaves + off <= (double)held)) return false;
                        return pick(true, (uint64_t)ceil(in_list - leaves - off), (uint64_t)ceil(in_list - leaves + off), border, other, upto);
                    };
                    if ((above | below) == 0) {
                        kept = pick(true, wanted(held), wanted(held), border, other, upto);
                    } else {
                        kept = choose(false);
                        if (kept && border != other) {
                            again(false);
                            kept = choose(true);
                        }
                        if (kept && border != other) {  // by what is reached
                            again(true);
                            const uint64_t want = wanted(Z);
                            kept = want > above && pick(true, want - above, want - above, border, other, upto);
                        }
                    }
                }
                if (kept) {
                    last = border;
                    if (cut_m) last = min(last, place_of(least, 0xFFFFFFFFu));
                    // what min_p leaves has to end in the list
                    found = high == INFINITY || last >= place_of(key_of(high), 0);
                    fast = high != INFINITY;
                    __syncthreads();
                    if (found) {
                        // What is kept of the list, in halves of 21 bits, so that a chunk's sums fit 32; the chunks' first sums are
                        // not needed any more.
                        uint32_t *const s_high = reinterpret_cast<uint32_t *>(s_chunk_s);
                        for (int i = tid; i < chunks; i += kThreads) s_ties[i] = s_high[i] = 0;
                        __syncthreads();
                        for (int i = tid; i < (int)listed; i += kThreads) {
                            const uint64_t place = s.list[i];
                            if (place <= last) {
                                const uint64_t m = mass_at(place);
                                const int ch = ((int)(uint32_t)place + r.off) / kChunk;
                                if (m) atomicAdd(&s_ties[ch], (uint32_t)m & 0x1FFFFFu), atomicAdd(&s_high[ch], (uint32_t)(m >> 21));
                            }
                        }
                        __syncthreads();
                        for (int i = tid; i < chunks; i += kThreads) s_chunk[i] += ((uint64_t)s_high[i] << 21) + s_ties[i];
                    }
                    __syncthreads();
                }
            }
        }
    }

    // ------------------------------------------------------------ or by histograms
    if (!found) {
        uint32_t border = key_of(-INFINITY), keep = 0xFFFFFFFFu;  // keys above the border are kept, and the first `keep` at it
        // The weights of this thread's four bins: tokens, or masses.  Bins of single keys need no sweep of masses; what the last one
        // has then is given.
        const auto weights = [&](bool by_mass, bool weighed, uint32_t hi, int shift, uint64_t (&w)[4]) -> uint64_t {
            uint64_t sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int b = tid * 4 + j;
                const uint64_t n = s.hist[b];
                w[j] = n;
                if (by_mass && n) w[j] = weighed ? s.weight[b] : b < kBins - 1 ? n * mass(ex, value_of(hi - ((uint32_t)b << shift))) : uint64_t(1) << 61;
                sum += w[j];
            }
            return sum;
        };
        // The place of the k-th token, or of the first where the sum of masses reaches `want`, by histograms of ever finer bins
        // below the maximum.  No key below lo counts.
        constexpr int kFirst = BF16 ? 16 : 14;  // fp32: four octaves below the maximum in 2^-9 of the value
        const auto find = [&](bool by_mass, uint64_t want, uint32_t lo) {
            uint32_t hi = top_key;
            int shift = kFirst;
            uint64_t before = 0;
            for (int turn = 0; turn < 6; ++turn) {  // 2^32 keys, 2^10 bins or more a turn
                const bool weighed = by_mass && shift != kUnit;
                ask(weighed ? kWeigh : kHist, hi, lo, shift);
                uint64_t w[4], all;
                const uint64_t sum = weights(by_mass, weighed, hi, shift, w);  // the last bin reaches it if no other does
                uint64_t at = before + block_scan(sum, all) - sum;
                if (tid == 0) s.got32[0] = kBins;
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (at < want && at + w[j] >= want) s.got32[0] = tid * 4 + j, s.got64[0] = at;
                    at += w[j];
                }
                __syncthreads();
                const uint32_t bin = s.got32[0];
                const uint64_t reached = s.got64[0];
                __syncthreads();
                if (bin >= kBins) return;  // all are kept
                if (shift == kUnit && bin < kBins - 1) {
                    border = hi - (bin << shift);
                    const uint64_t one = by_mass ? mass(ex, value_of(border)) : 1, n = s.hist[bin];
                    const uint64_t more = one ? (want - reached + one - 1) / one : n;
                    keep = (uint32_t)(more < n ? more : n);
                    return;
                }
                before = reached;
                hi -= bin << shift;
                if (bin < kBins - 1 && hi - lo >= (1u << shift)) lo = hi - ((1u << shift) - 1u);
                const int bits = 32 - __clz(hi - lo);
                shift = max(kUnit, bits < kBinBits ? 0 : bits - kBinBits + 1);  // at most 2^10 bins: no remainder in the last one
            }
        };
        bool by_least = !sampled;
        if (cut_m && cut_p && !cut_k) {  // does min_p leave less than top_p?
            ask(kKeptFast, __float_as_uint(value_of(least)), 0, 0);
            uint64_t sum = 0, all;
            for (int i = tid; i < chunks; i += kThreads) sum += s_chunk[i] + s_ties[i] * mass(ex, value_of(least));
            block_scan(sum, all);
            by_least = (double)all * (1.0 + kMost) < (double)top_p * (double)Z * (1.0 - kMost);
        }
        if (cut_k && !by_least) find(false, (uint64_t)k, 0);
        if (cut_p && !by_least) {
            uint64_t sum = 0;
            if (cut_k) {  // of the first k
                if (border != top_key) {
                    ask(kSum, 0xFFFFFFFFu, border + (1u << kUnit), 0);
                    sum = s.sum;
                }
                sum += keep * mass(ex, value_of(border));
            } else {
                ask(kSum, 0xFFFFFFFFu, 0, 0);
                sum = Z = s.sum;
            }
            find(true, wanted(sum), border);
        }
        if (cut_m && least > border) border = least, keep = 0xFFFFFFFFu;
        // what is above it by chunk, and the chunk of the last that is kept at it
        ask(kKeptFast, __float_as_uint(value_of(border)), 0, 0);
        const uint64_t tie = mass(ex, value_of(border));
        const int per = (chunks + kThreads - 1) / kThreads, i0 = min(tid * per, chunks), i1 = min(i0 + per, chunks);
        uint64_t n = 0, all;
        for (int i = i0; i < i1; ++i) n += s_ties[i];
        if (tid == 0) s.got32[0] = 0xFFFFFFFFu;
        uint64_t at = block_scan(n, all) - n;
        for (int i = i0; i < i1; ++i) {
            const uint64_t t = s_ties[i], kept = at >= keep ? 0 : (at + t > keep ? keep - at : t);
            s_chunk[i] += kept * tie;
            if (at < keep && at + t >= keep) s.got32[0] = i, s.got32[1] = (uint32_t)(keep - at);
            at += t;
        }
        __syncthreads();
        const int ch = (int)s.got32[0];
        const uint32_t nth = s.got32[1];
        uint32_t index = 0xFFFFFFFFu;
        if (ch >= 0) {  // the index of its nth
            constexpr int per_thread = kChunk / kThreads;
            const int e0 = ch * kChunk + tid * per_thread - r.off;
            uint64_t ties = 0;
            for (int j = 0; j < per_thread; ++j) ties += r.inside(e0 + j) && r.at(e0 + j) == value_of(border);
            uint64_t seen = block_scan(ties, all) - ties;
            for (int j = 0; j < per_thread; ++j)
                if (r.inside(e0 + j) && r.at(e0 + j) == value_of(border) && ++seen == nth) s.got32[0] = (uint32_t)(e0 + j);
            __syncthreads();
            index = s.got32[0];
        }
        last = place_of(border, index);
        fast = true;
        __syncthreads();
    }

    // ------------------------------------------------------------ the token
    const float u = fminf(fmaxf(a.u[row], 0.0f), 0.99999994f);  // NaN as 0
    const uint32_t u_bits = __float_as_uint(u);
    const uint64_t u_m = u_bits >> 23 ? (u_bits & 0x7FFFFFu) | 0x800000u : 0;  // below 2^-126 as 0
    const int u_e = 150 - (int)(u_bits >> 23);  // 24 or more
    const uint32_t last_key = ~(uint32_t)(last >> 32), last_index = (uint32_t)last;
    for (int level = fast ? 0 : 2;;) {  // of the chunks' sums
        const int per = (chunks + kThreads - 1) / kThreads, i0 = min(tid * per, chunks), i1 = min(i0 + per, chunks);
        uint64_t w = 0, total = 0;
        for (int i = i0; i < i1; ++i) w += s_chunk[i];
        uint64_t at = block_scan(w, total) - w;
        // floor(u total), u = u_m 2^-u_e
        const uint64_t high_part = __umul64hi(total, u_m), low_part = total * u_m;
        const uint64_t target = u_e < 64 ? low_part >> u_e | high_part << (64 - u_e) : u_e < 128 ? high_part >> (u_e - 64) : 0;
        for (int i = i0; i < i1; ++i) {
            const uint64_t m = s_chunk[i];
            if (at <= target && target < at + m) s.got32[0] = i, s.got64[0] = at;
            at += m;
        }
        __syncthreads();
        const int ch = (int)s.got32[0];
        const uint64_t before = s.got64[0];
        __syncthreads();
        if (tid == 0) s.got32[0] = 0xFFFFFFFFu;
        // that chunk again, consecutive tokens a thread
        constexpr int per_thread = kChunk / kThreads;
        float f[per_thread];
        uint64_t m[per_thread], own = 0, all;
        const int e0 = ch * kChunk + tid * per_thread - r.off;
#pragma unroll
        for (int j = 0; j < per_thread; ++j) {
            f[j] = r.at(e0 + j);
            const uint32_t key = key_of(f[j]);
            const bool kept = key > last_key || (key == last_key && (uint32_t)max(e0 + j, 0) <= last_index);
            m[j] = kept ? mass(ex, f[j]) : 0;  // 0 outside the row, which reads as -inf
            own += m[j];
        }
        uint64_t cum = before + block_scan(own, all) - own;
        // how far the sum before this chunk less the target, u times it and the sum from here on, may be off
        const auto off_of = [&](uint64_t z) -> float { return level ? kGood * (float)z : off_fast(z); };
        const uint64_t off = level < 2 ? (uint64_t)((1.0f - u) * off_of(before) + u * off_of(total - before)) + units : 0;
#pragma unroll
        for (int j = 0; j < per_thread; ++j) {
            if (m[j] && (cum == 0 || cum + off <= target) && target + off < cum + m[j]) {
                s.got32[0] = (uint32_t)(e0 + j);
                s.got32[1] = __float_as_uint(f[j]);
            }
            cum += m[j];
        }
        __syncthreads();
        const uint32_t id = s.got32[0];
        if (id != 0xFFFFFFFFu || level == 2) {
            if (tid == 0) {
                // the sums less the most probable token's, which is 1
                const float y = (__uint_as_float(s.got32[1]) - top) / tau;
                const auto log_of = [](uint64_t z) { return log1pf((float)(int64_t)(z - (uint64_t(1) << kScale)) * pow2f(-kScale)); };
                a.ids[row] = id;
                a.logp[row] = y - log_of(Z);
                a.logq[row] = y - log_of(total);
            }
            break;
        }
        ++level;
        ask(level == 1 ? kKeptGood : kKeptExact, last == ~uint64_t(0) ? 0xFF800000u : __float_as_uint(value_of(last_key)), last_index, 0);
    }
    ask(kDone, 0, 0, 0);
}

template <bool BF16, bool CLUSTER>
cudaError_t launch(const Args &a, cudaStream_t stream, bool chain)
{
    static OncePerDevice once;
    const auto kernel = sample_kernel<BF16, CLUSTER>;
    cudaError_t e = allow_smem(once, kernel, sizeof(Shared) + kMostChunks * Shared::kChunkBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.T * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared) + a.chunks * Shared::kChunkBytes;
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
    Args a = {logits, ld, T, V, u, o->temperature, o->top_p, o->min_p, o->top_k, o->temperatures, o->top_ps, o->min_ps, o->top_ks, ids, logp, logq, 1, 0};
    // Clusters while the rows alone leave SMs idle (two CTAs each), and no more CTAs than give every warp a chunk.
    const int64_t chunks = (V * (bf16 ? 2 : 4) + 14 + kChunkVecs * 16 - 1) / (kChunkVecs * 16);
    a.chunks = (int)chunks + (int)(chunks & 1);
    while (a.cluster < kMaxCluster && T * a.cluster < num_sms() && chunks > (int64_t)a.cluster * kWarps) a.cluster *= 2;
    if (a.cluster > 1) return launched(bf16 ? launch<true, true>(a, as_cuda(stream), chain) : launch<false, true>(a, as_cuda(stream), chain));
    return launched(bf16 ? launch<true, false>(a, as_cuda(stream), chain) : launch<false, false>(a, as_cuda(stream), chain));
}
