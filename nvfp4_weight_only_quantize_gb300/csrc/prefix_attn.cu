// Attention of a batch whose sequences share long prefixes (the prompt of a
// group of sampled answers): every query row sees its group's prefix and, causally,
// its own sequence's suffix, in one softmax.
//
//   a_k = scale q . k_k,  lse = log sum_k e^(a_k),  out = sum_k e^(a_k - lse) v_k
//
// The prefix's keys and values are read once for all the group's sequences: their
// query rows share its tiles.  Segments are cut along the keys into chunks that
// run side by side; each leaves (o, m, l) in the workspace and a second kernel
// joins a row's parts.
//
// Bound by HBM where the suffixes are most of the keys (rows16_kernel: each is read
// by one CTA, for its up to 16 rows), by the tensor cores and shared memory where
// many rows share a prefix (the tcgen05 kernel), by latency below some 10 us.
// 64 sequences of up to 4096 own tokens, 40 / 8 heads, D = 128: 100 us, 82 % of
// the measured copy rate.  Eight of a group of 512 + 1024 keys 11 us; one
// sequence over 512 keys 9 us a call, 6 us in a graph.
#include <float.h>
#include <math.h>

#include "prefix_attn.cuh"
#include "sm100_ptx.cuh"

namespace qerl {
namespace attn {
namespace {

// ------------------------------------------------------------------ chunks of up to 16 rows
constexpr int kWarps = 4;    // a warp takes every fourth 16-key tile of the chunk
constexpr int kStages = 2;   // tile buffers per warp (a tile's load is issued after the products of the one before it)
constexpr int kTile = 16;

template <int D>
constexpr int smem_bytes()
{
    return kWarps * kStages * kTile * D * 2 * 2;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool take)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One CTA: up to 16 query rows that share a kv head, one chunk of a segment's
// keys.  Each warp streams its own 16-key tiles through a ring of cp.async
// stages (no barrier between warps until the end) and keeps its own softmax
// statistics; the warps' results are joined in shared memory.
// Probabilities are rounded to bf16 for the second product, as its operands are
// bf16; their sum l stays in FP32.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) rows16_kernel(const Args a, int prefix_items, int beside_tc)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    // Beside the tcgen05 kernel, whose CTAs let this one start once all work before both has finished, there is nothing to
    // wait for here; the kernel that joins the parts waits for both, because this one's last CTA waits at its end.
    if (!beside_tc) pdl_wait();
    beside_tc = beside_tc && blockIdx.x == gridDim.x - 1;
    pdl_trigger();
    // which rows, which keys
    int item = blockIdx.x;
    const bool pre = item < prefix_items;
    if (!pre) item -= prefix_items;
    const int n_parts = pre ? a.n_pp : a.n_sp, tiles = pre ? a.p_tiles : a.s_tiles;
    const int part = item % n_parts;
    int rest = item / n_parts;
    const int tile = rest % tiles;
    rest /= tiles;
    const int hk = rest % a.Hkv, seg = rest / a.Hkv;  // seg: group or sequence
    const int len = pre ? prefix_len(a, seg) : suffix_len(a, seg);
    const int k_lo = part * (pre ? a.p_chunk : a.s_chunk);
    if (k_lo >= len) {
        if (beside_tc) pdl_wait();
        return;
    }
    const int k_hi = min(len, k_lo + (pre ? a.p_chunk : a.s_chunk));
    const int n_rows = (pre ? a.G : 1) * a.Lq * a.gs;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t tk = pre ? a.kp_t : a.ks_t, tv = pre ? a.vp_t : a.vs_t;
    const __nv_bfloat16 *K = pre ? a.kp + seg * a.kp_g + hk * a.kp_h : a.ks + seg * a.ks_b + hk * a.ks_h;
    const __nv_bfloat16 *V = pre ? a.vp + seg * a.vp_g + hk * a.vp_h : a.vs + seg * a.vs_b + hk * a.vs_h;

    constexpr int CH = D / 8;                 // 16-byte chunks per key row
    constexpr int STAGE = kTile * D * 2 * 2;  // K tile, V tile
    const uint32_t ring = ptx::smem_u32(smem) + warp * kStages * STAGE;
    const int n_tiles = (k_hi - k_lo + kTile - 1) / kTile;
    const int mine = n_tiles > warp ? (n_tiles - warp + kWarps - 1) / kWarps : 0;
    auto fetch = [&](int j) {
        if (j < mine) {
            const int k0 = k_lo + (j * kWarps + warp) * kTile;
            const uint32_t to = ring + (j % kStages) * STAGE;
#pragma unroll
            for (int c = 0; c < kTile * CH / 32; ++c) {
                const int idx = c * 32 + lane, r = idx / CH, ch = idx % CH;
                const bool in = k0 + r < k_hi;
                const int64_t tok = in ? k0 + r : k_lo;
                const uint32_t at = to + r * D * 2 + ((ch ^ (r & 7)) * 16);
                cp16(at, K + tok * tk + ch * 8, in);
                cp16(at + kTile * D * 2, V + tok * tv + ch * 8, in);
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) fetch(j);

    // query rows lane / 4 and lane / 4 + 8 of the tile
    auto row_of = [&](int r, int &b, int &l, int &h) {
        const int rr = tile * 16 + r;
        const int bi = rr / (a.Lq * a.gs), in = rr % (a.Lq * a.gs);
        b = pre ? seg * a.G + bi : seg;
        l = in / a.gs;
        h = hk * a.gs + in % a.gs;
        return rr < n_rows;
    };
    uint32_t qf[D / 16][4];
    int limit[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        int b, l, h;
        const bool ok = row_of(lane / 4 + 8 * half, b, l, h);
        limit[half] = pre ? len : len - a.Lq + 1 + l;
        const __nv_bfloat16 *q = a.q + b * a.q_b + l * a.q_l + h * a.q_h + (lane % 4) * 2;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            qf[s][half] = ok ? *reinterpret_cast<const uint32_t *>(q + s * 16) : 0u;
            qf[s][half + 2] = ok ? *reinterpret_cast<const uint32_t *>(q + s * 16 + 8) : 0u;
        }
    }

    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    float m[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};
    for (int j = 0; j < mine; ++j) {
        cp_wait<kStages - 2>();
        __syncwarp();
        const uint32_t kt = ring + (j % kStages) * STAGE, vt = kt + kTile * D * 2;
        float s[2][4] = {};
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            const int key = (lane / 16) * 8 + lane % 8, ch = d * 2 + ((lane / 8) & 1);
            uint32_t b[4];
            ldsm4(kt + key * D * 2 + ((ch ^ (key & 7)) * 16), b);
            mma(s[0], qf[d], b[0], b[1]);
            mma(s[1], qf[d], b[2], b[3]);
        }
        const int k0 = k_lo + (j * kWarps + warp) * kTile + (lane % 4) * 2;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float x[4], top = kNone;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int k = k0 + (c / 2) * 8 + c % 2;
                x[c] = k < min(limit[half], k_hi) ? s[c / 2][half * 2 + c % 2] * a.scale_log2 : -INFINITY;
                top = fmaxf(top, x[c]);
            }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const float to = fmaxf(m[half], top), f = ex2(m[half] - to);
            m[half] = to;
            l[half] *= f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[c] = ex2(x[c] - to);
                l[half] += x[c];
                s[c / 2][half * 2 + c % 2] = x[c];
            }
            if (__any_sync(0xFFFFFFFFu, f != 1.0f)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) o[n][half * 2] *= f, o[n][half * 2 + 1] *= f;
            }
        }
        const uint32_t p[4] = {pack2(s[0][0], s[0][1]), pack2(s[0][2], s[0][3]), pack2(s[1][0], s[1][1]), pack2(s[1][2], s[1][3])};
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            const int key = ((lane / 8) & 1) * 8 + lane % 8, ch = n * 2 + lane / 16;
            uint32_t b[4];
            ldsm4_t(vt + key * D * 2 + ((ch ^ (key & 7)) * 16), b);
            mma(o[2 * n], p, b[0], b[1]);
            mma(o[2 * n + 1], p, b[2], b[3]);
        }
        __syncwarp();
        fetch(j + kStages - 1);
    }
    cp_wait<0>();
    __syncthreads();

    // join the warps: [warp][row][D] and [warp][row] (m, l) in the ring's memory
    float *so = reinterpret_cast<float *>(smem);
    float2 *sml = reinterpret_cast<float2 *>(smem + kWarps * 16 * D * 4);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 1);
        l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 2);
        const int r = lane / 4 + 8 * half;
        if (lane % 4 == 0) sml[warp * 16 + r] = make_float2(m[half], l[half]);
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2 *>(so + (warp * 16 + r) * D + n * 8 + (lane % 4) * 2) =
                make_float2(o[n][half * 2], o[n][half * 2 + 1]);
    }
    __syncthreads();
    const int parts = a.n_pp + a.n_sp;
    for (int r = warp; r < 16; r += kWarps) {
        int b, li, h;
        if (!row_of(r, b, li, h)) break;
        float M = kNone, w[kWarps], L = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) M = fmaxf(M, sml[k * 16 + r].x);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            w[k] = ex2(sml[k * 16 + r].x - M);
            L = fmaf(w[k], sml[k * 16 + r].y, L);
        }
        const int64_t at = (((int64_t)b * a.Lq + li) * a.Hq + h) * parts + (pre ? 0 : a.n_pp) + part;
        for (int d = lane; d < D; d += 32) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) t = fmaf(w[k], so[(k * 16 + r) * D + d], t);
            a.part_o[at * D + d] = t;
        }
        if (lane == 0) a.part_ml[at] = make_float2(M, L);
    }
    if (beside_tc) pdl_wait();
}

// ------------------------------------------------------------------ joining a row's parts
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

// The products of a tile run over keys that some of its rows do not see, with weight 0, and 0 times an Inf or NaN of V is NaN.
// Over a warp, for a row whose sum is not finite while it has such keys (the new tokens after its own): where one of those
// values is not finite, the columns that are not are summed again over the keys that the row sees.
template <int D>
__device__ __forceinline__ void sum_again(const Args &a, int b, int l, int h, int plen, int slen, float M, float (&acc)[D / 32])
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x % 32, hk = h / a.gs, g = b / a.G, sees = max(0, slen - a.Lq + 1 + l);
    const auto pair = [](const __nv_bfloat16 *p, int e) { return *reinterpret_cast<const uint32_t *>(p + e); };
    const __nv_bfloat16 *vs = a.vs + b * a.vs_b + hk * a.vs_h + lane * E;
    bool bad = false;
    for (int k = sees; k < slen; ++k)
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const uint32_t v = pair(vs + k * a.vs_t, e);
            bad = bad || !isfinite(bf16lo(v)) || !isfinite(bf16hi(v));
        }
    if (!__any_sync(0xFFFFFFFFu, bad)) return;
    float x[E], sum[E] = {};
    const __nv_bfloat16 *q = a.q + b * a.q_b + l * a.q_l + h * a.q_h + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) x[e] = bf16lo(pair(q, e)) * a.scale_log2, x[e + 1] = bf16hi(pair(q, e)) * a.scale_log2;
    const auto add = [&](const __nv_bfloat16 *k, const __nv_bfloat16 *v, int64_t k_t, int64_t v_t, int n) {
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < E; e += 2) s = fmaf(x[e], bf16lo(pair(k + t * k_t, e)), fmaf(x[e + 1], bf16hi(pair(k + t * k_t, e)), s));
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            const float w = ex2(s - M);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                sum[e] = fmaf(w, bf16lo(pair(v + t * v_t, e)), sum[e]);
                sum[e + 1] = fmaf(w, bf16hi(pair(v + t * v_t, e)), sum[e + 1]);
            }
        }
    };
    add(a.kp + g * a.kp_g + hk * a.kp_h + lane * E, a.vp + g * a.vp_g + hk * a.vp_h + lane * E, a.kp_t, a.vp_t, plen);
    add(a.ks + b * a.ks_b + hk * a.ks_h + lane * E, vs, a.ks_t, a.vs_t, min(sees, slen));
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (!isfinite(acc[e])) acc[e] = sum[e];
}

// W warps per query row (each takes every W-th part); the parts
// that exist follow from the lengths.
template <int D, int W>
__global__ void __launch_bounds__(128) join_kernel(const Args a)
{
    constexpr int E = D / 32, RB = 4 / W, NB = W == 1 ? 4 : 8;  // columns of a lane; rows of a block; parts in flight
    __shared__ float s_o[W > 1 ? 4 : 1][W > 1 ? D : 1];
    __shared__ float2 s_ml[4];
    pdl_trigger();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, share = warp % W;
    const int row = blockIdx.x * RB + warp / W;
    const bool live = row < a.B * a.Lq * a.Hq;
    const int h = row % a.Hq, bl = row / a.Hq, l = bl % a.Lq, b = live ? bl / a.Lq : 0, g = b / a.G;
    // the kernels before this one let it start after all work before the call: the lengths are there
    const int plen = a.n_pp ? prefix_len(a, g) : 0, slen = a.n_sp ? suffix_len(a, b) : 0;
    const int hk = h / a.gs, hi = h - hk * a.gs;
    pdl_wait();
    const int np = a.p_tc ? tc_parts(a, true, g, hk, ((b - g * a.G) * a.Lq + l) * a.gs + hi, plen)
                          : a.n_pp ? (plen + a.p_chunk - 1) / a.p_chunk : 0;
    const int ns = a.s_tc ? tc_parts(a, false, (a.p_tc ? a.n_prefix : 0) + b, hk, l * a.gs + hi, slen)
                          : a.n_sp ? (slen + a.s_chunk - 1) / a.s_chunk : 0;
    const int n = live ? np + ns : 0;
    const int64_t base = (int64_t)row * (a.n_pp + a.n_sp);
    const auto at = [&](int k) { return base + (k < np ? k : a.n_pp + k - np); };
    float M = kNone, L = 0.0f, acc[E] = {};
    for (int k0 = share; k0 < n; k0 += NB * W) {
        float2 ml[NB];
        float v[NB][E];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int k = k0 + j * W;
            ml[j] = make_float2(kNone, 0.0f);
            if (k < n) {
                ml[j] = a.part_ml[at(k)];
                const float *p = a.part_o + at(k) * D + lane * E;
                if (E == 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(p);
                    v[j][0] = q.x, v[j][1] = q.y, v[j][E - 2] = q.z, v[j][E - 1] = q.w;
                } else {
                    const float2 q = *reinterpret_cast<const float2 *>(p);
                    v[j][0] = q.x, v[j][1] = q.y;
                }
            }
        }
        float to = M;
#pragma unroll
        for (int j = 0; j < NB; ++j) to = fmaxf(to, ml[j].x);
        const float f = ex2(M - to);
        M = to;
        L *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const bool none = ml[j].y == 0.0f && ml[j].x == kNone;  // no part, or one that saw no key and may have left no o
            const float w = none ? 0.0f : ex2(ml[j].x - M);
            L = fmaf(w, ml[j].y, L);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(w, none ? 0.0f : v[j][e], acc[e]);
        }
    }
    if (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
        if (lane == 0) s_ml[warp] = make_float2(M, L);
        __syncthreads();
        if (share) return;
#pragma unroll
        for (int k = 1; k < W; ++k) M = fmaxf(M, s_ml[warp + k].x);
        L = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float w = ex2(s_ml[warp + k].x - M);
            L = fmaf(w, s_ml[warp + k].y, L);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(w, s_o[warp + k][lane * E + e], acc[e]);
        }
    }
    if (!live) return;
    if (a.Lq > 1) {
        bool finite = true;
#pragma unroll
        for (int e = 0; e < E; ++e) finite = finite && isfinite(acc[e]);
        if (!__all_sync(0xFFFFFFFFu, finite) && l + 1 < a.Lq && isfinite(L)) sum_again<D>(a, b, l, h, plen, slen, M, acc);
    }
    const float inv = L == 0.0f ? 0.0f : __fdividef(1.0f, L);  // a row that sees no key: zeros, lse -inf
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + b * a.o_b + l * a.o_l + h * a.o_h + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = pack2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && a.lse) a.lse[row] = L == 0.0f ? -INFINITY : (float)((double)M * 0.6931471805599453 + (double)logf(L));
}

int ceil_div(int64_t x, int64_t y) { return (int)((x + y - 1) / y); }

// Most parts of a row that the tcgen05 kernel leaves: a unit's steps over a CTA's, which are at least the line's length
// over the CTAs (its empty steps, which only lengthen it, left out); of a left-over tile two each.
int tc_parts_most(int64_t rows, int64_t len, int64_t Hkv, int64_t ctas)
{
    const int64_t t = (rows + 127) / 128, full = t / 2, T = (len + 127) / 128, half = (T + 1) / 2;
    const auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
    const int64_t pairs = full ? least(T, ctas / (Hkv * full) + 3) : 0;
    const int64_t single = t & 1 ? 2 * least(half, ctas / (Hkv * (full ? full + 1 : 1)) + 3) : 0;
    return (int)(pairs > single ? pairs : single);
}

// Kernels, chunk lengths, tiles and parts of a call; false where a size is not covered.
// A segment of more than 16 rows goes to tcgen05 where that is quicker.  What was measured: a step of its line takes
// about 2 us and a CTA about 8 us besides; the other kernel reads every key once per 16 rows, at some 5 TB/s from L2.
// Chunks of the other kernel: about six CTAs per SM over all rows and keys, 64 to 1024 keys each.  Measured on 64 answers
// of up to 4096 tokens: 256 keys 131 us, 512 108 us, 1024 99 us, 2048 109 us (too few to even the SMs out).
bool shape(const qerl_prefix_attn_dims *d, Args &a, bool tc)
{
    if (d->B < 1 || d->Lq < 1 || d->Hq < 1 || d->Hkv < 1 || d->n_prefix < 1 || d->P < 0 || d->S < 0) return false;
    if ((d->D != 64 && d->D != 128) || d->Hq % d->Hkv || d->B % d->n_prefix) return false;
    const int64_t big = 1 << 30;
    if (d->B > big || d->Lq > big || d->Hq > 65536 || d->P > big || d->S > big || d->B * d->Lq > big / d->Hq) return false;
    a.B = (int)d->B, a.Lq = (int)d->Lq, a.Hq = (int)d->Hq, a.Hkv = (int)d->Hkv, a.n_prefix = (int)d->n_prefix;
    a.G = a.B / a.n_prefix, a.gs = a.Hq / a.Hkv, a.P = (int)d->P, a.S = (int)d->S;
    const int64_t pr = (int64_t)a.G * a.Lq * a.gs, sr = (int64_t)a.Lq * a.gs;
    a.p_tiles = ceil_div(pr, 16), a.s_tiles = ceil_div(sr, 16);
    a.grid_tc = num_sms();
    const auto quicker = [&](int64_t rows, int64_t len, int64_t segments) {
        const int64_t steps = segments * a.Hkv * (rows / 256 + 1) * ((len + 127) / 128);
        const double tc_us = 8.0 + 2.0 * (double)((steps + a.grid_tc - 1) / a.grid_tc);
        return rows > 16 && len >= 128 && tc_us * 5e6 < (double)(segments * a.Hkv * ((rows + 15) / 16) * len) * (double)(d->D * 4);
    };
    a.p_tc = tc && quicker(pr, a.P, a.n_prefix);
    a.s_tc = tc && quicker(sr, a.S, a.B);
    if (a.p_tc && !a.s_tc) {
        // The prefixes on tcgen05 leave SMs to the suffixes, which then run beside them: an SM takes 2 us per step, or reads
        // 50 bytes per ns.  As many as make the later of the two end soonest, against one after the other.
        // The suffixes are taken as half full, which a rollout's caches are on average (the host does not know the lengths).
        // 64 sequences, 28 / 4 heads, 16384 + up to 999 keys, the caches 2, 50 and 100 % full: 42, 44, 56 us; taken as full
        // 48, 51, 56 us, as 30 % full 40, 47, 57 us.
        const double steps = (double)a.n_prefix * a.Hkv * (pr / 256 + 1) * ((a.P + 127) / 128);
        const double bytes = 0.5 * (double)a.B * a.Hkv * a.S * (double)(d->D * 4);
        const int sms = num_sms();
        double best = 2.0 * ceil(steps / sms) + bytes / 6.0e6;
        for (int n = sms - 4; n >= sms / 2; n -= 4) {
            const double t = 2.0 * ceil(steps / n), u = bytes / ((sms - n) * 50.0e3), later = t > u ? t : u;
            if (later < best) best = later, a.grid_tc = n;
        }
    }
    if ((a.p_tc ? (pr / 256 + 1) * (a.P / 128 + 4) * a.Hkv * a.n_prefix : 0) + (a.s_tc ? (sr / 256 + 1) * (a.S / 128 + 4) * a.Hkv * a.B : 0) > big)
        a.p_tc = a.s_tc = 0;  // more steps than the kernel counts
    const int64_t up = a.p_tc ? 0 : (int64_t)a.n_prefix * a.Hkv * a.p_tiles, us = a.s_tc ? 0 : (int64_t)a.B * a.Hkv * a.s_tiles;
    const int64_t want = (up * a.P + us * a.S) / (6 * num_sms());
    int64_t chunk = (want + 63) / 64 * 64;
    chunk = chunk < 64 ? 64 : chunk > 1024 ? 1024 : chunk;
    a.p_chunk = a.s_chunk = (int)chunk;
    a.n_pp = a.p_tc ? tc_parts_most(pr, a.P, a.Hkv, a.grid_tc) : ceil_div(a.P, chunk);
    a.n_sp = a.s_tc ? tc_parts_most(sr, a.S, a.Hkv, a.grid_tc) : ceil_div(a.S, chunk);
    return up * a.n_pp + us * a.n_sp < 0x7FFFFFFF;
}
size_t round256(size_t b) { return (b + 255) & ~size_t(255); }
size_t ml_bytes(const Args &a) { return round256((size_t)a.B * a.Lq * a.Hq * (a.n_pp + a.n_sp) * sizeof(float2)); }
size_t line_bytes(const Args &a) { return round256((size_t)(1 + a.n_prefix + a.B) * sizeof(int)); }
size_t ws_total(const Args &a, int64_t D)
{
    return ml_bytes(a) + line_bytes(a) + (size_t)a.B * a.Lq * a.Hq * (a.n_pp + a.n_sp) * D * sizeof(float);
}

template <int D>
qerl_status run(const Args &a, const void *maps, cudaStream_t s)
{
    const bool chain = g_chain.load() != 0, tc = a.p_tc || a.s_tc;
    if (tc) QERL_TRY(launched(tc_launch(a, D, maps, s, chain), QERL_KERNEL_ATTN_ROWS128));
    const int64_t pi = a.p_tc ? 0 : (int64_t)a.n_prefix * a.Hkv * a.p_tiles * a.n_pp,
                  si = a.s_tc ? 0 : (int64_t)a.B * a.Hkv * a.s_tiles * a.n_sp;
    if (pi + si > 0) {
        static OncePerDevice once;
        if (allow_smem(once, rows16_kernel<D>, smem_bytes<D>()) != cudaSuccess) return QERL_ERR_CUDA;
        QERL_TRY(launched(launch_k(rows16_kernel<D>, dim3((unsigned)(pi + si)), dim3(kWarps * 32), smem_bytes<D>(), s, chain, a, (int)pi,
                                   tc && chain ? 1 : 0),
                          QERL_KERNEL_ATTN_ROWS16));
    }
    // a warp per row where its parts fit one batch or the rows fill the SMs, else four
    const int rows = a.B * a.Lq * a.Hq;
    if (a.n_pp + a.n_sp <= 8 || rows > 32 * num_sms())
        return launched(launch_k(join_kernel<D, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, chain, a));
    return launched(launch_k(join_kernel<D, 4>, dim3((unsigned)rows), dim3(128), 0, s, chain, a));
}

}  // namespace
}  // namespace attn
}  // namespace qerl

using namespace qerl;

extern "C" size_t qerl_prefix_attention_ws_bytes(const qerl_prefix_attn_dims *dims)
{
    attn::Args a = {}, b = {};  // with tcgen05, and without where the caches' strides fit no tensor map
    if (!dims || !attn::shape(dims, a, true) || !attn::shape(dims, b, false)) return 0;
    const size_t n = attn::ws_total(a, dims->D), m = attn::ws_total(b, dims->D);
    return n > m ? n : m ? m : 256;
}

extern "C" qerl_status qerl_prefix_attention(const qerl_prefix_attn_dims *d, const void *q, const void *k_prefix, const void *v_prefix,
                                             const int32_t *prefix_lens, const void *k_suffix, const void *v_suffix,
                                             const int32_t *suffix_lens, float scale, void *out, float *lse, void *ws, size_t ws_bytes,
                                             qerl_stream_t stream)
{
    if (!d || !q || !out || !(scale > 0.0f) || !(scale <= FLT_MAX)) return QERL_ERR_INVALID_ARG;
    attn::Args a = {};
    if (!attn::shape(d, a, true)) return QERL_ERR_SHAPE;
    if ((a.P && (!k_prefix || !v_prefix)) || (a.S && (!k_suffix || !v_suffix || !suffix_lens))) return QERL_ERR_INVALID_ARG;
    const int64_t *const strides[] = {d->q_stride, d->out_stride, d->k_prefix_stride, d->v_prefix_stride, d->k_suffix_stride, d->v_suffix_stride};
    for (int t = 0; t < 6; ++t)
        for (int k = 0; k < 3; ++k) {
            if (strides[t][k] < 0 || strides[t][k] > (int64_t(1) << 40)) return QERL_ERR_SHAPE;
            if (strides[t][k] % 8) return QERL_ERR_ALIGN;
        }
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_prefix) || !aligned16(v_prefix) || !aligned16(k_suffix) || !aligned16(v_suffix) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(prefix_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(suffix_lens) & 3u))
        return QERL_ERR_ALIGN;
    if (!ws || ws_bytes < qerl_prefix_attention_ws_bytes(d)) return QERL_ERR_WORKSPACE;
    if (!aligned16(ws)) return QERL_ERR_ALIGN;
    QERL_TRY(check_device());
    const auto bf = [](const void *p) { return static_cast<const __nv_bfloat16 *>(p); };
    a.q = bf(q), a.kp = bf(k_prefix), a.vp = bf(v_prefix), a.ks = bf(k_suffix), a.vs = bf(v_suffix);
    a.plen = prefix_lens, a.slen = suffix_lens;
    a.out = static_cast<__nv_bfloat16 *>(out), a.lse = lse;
    a.q_b = d->q_stride[0], a.q_l = d->q_stride[1], a.q_h = d->q_stride[2];
    a.o_b = d->out_stride[0], a.o_l = d->out_stride[1], a.o_h = d->out_stride[2];
    a.kp_g = d->k_prefix_stride[0], a.kp_t = d->k_prefix_stride[1], a.kp_h = d->k_prefix_stride[2];
    a.vp_g = d->v_prefix_stride[0], a.vp_t = d->v_prefix_stride[1], a.vp_h = d->v_prefix_stride[2];
    a.ks_b = d->k_suffix_stride[0], a.ks_t = d->k_suffix_stride[1], a.ks_h = d->k_suffix_stride[2];
    a.vs_b = d->v_suffix_stride[0], a.vs_t = d->v_suffix_stride[1], a.vs_h = d->v_suffix_stride[2];
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    alignas(64) char maps[attn::kTcMapsBytes];
    if ((a.p_tc || a.s_tc) && !attn::tc_maps(a, d->D, maps)) attn::shape(d, a, false);
    a.part_ml = static_cast<float2 *>(ws);
    a.line = reinterpret_cast<int *>(static_cast<char *>(ws) + attn::ml_bytes(a));
    a.part_o = reinterpret_cast<float *>(static_cast<char *>(ws) + attn::ml_bytes(a) + attn::line_bytes(a));
    return d->D == 128 ? attn::run<128>(a, maps, as_cuda(stream)) : attn::run<64>(a, maps, as_cuda(stream));
}
