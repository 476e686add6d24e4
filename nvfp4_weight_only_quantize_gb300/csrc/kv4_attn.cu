// Attention over 4-bit caches: prefixes that groups of sequences share, and every
// sequence's own tokens, in one softmax.
//
//   a_k = scale q . k_k,  lse = log sum_k e^(a_k),  out = sum_k e^(a_k - lse) v_k
//
// A warp takes whole tiles of 32 keys, which bulk copies bring to its own ring in
// shared memory, and multiplies them as the m operand of mma.sync, so that the
// query rows, few in decoding, are the narrow side (8 columns) and nothing is
// padded to 16:
//   S^T = K Q^T     K as fp16, code times scale, which is exact there; Q as fp16 after
//                   a power of two per row that brings its largest element to [1, 2):
//                   elements down to 2^-17 of that stay exact, smaller ones are off by
//                   2^-25 of it, as a sum of FP32 products is anyway;
//   P = 2^(S c - m) per column, rounded to fp16 and turned (movmatrix): between 2^8 and
//                   2^15 for the largest, so that keys of up to 15 nats less keep all of
//                   fp16's digits;
//   O^T += V^T P    V as fp16, code times scale, exact.  (Scales that multiply P instead,
//                   half as many products, leave fp16's smallest numbers where values are
//                   small against the cache's factor: 11 % off under a key 14 nats above.)
// m is raised only when a column's maximum outgrows it by 2^15.
//
// The work is one line of steps (kv4_attn.cuh) that 608 CTAs of four warps share, four
// on an SM, so that long and short sequences fill the SMs alike.  Rows are tiled by
// eight whatever their number: tiles of 16 in one warp took three times as long as
// two of eight (213 registers, half the warps).
// Bound by HBM in long caches (two sequences of 2 M tokens: 395 us, 6.1 TB/s, 92 % of
// the copy rate) and by its start, the join and uneven CTAs in shorter ones: some 4 us
// before the first tile and 4 us after the last.  In a graph, 28 / 4 heads, D = 128: two
// sequences of 131072 and 81007 tokens 31 us (122 MB); one sequence over 513 keys 7.8
// us; 64 of up to 4096 tokens, 40 / 8 heads, with prefixes of 512: 52 to 59 us over three
// orders of their lengths (51 to 59 with scales on P); the same at D = 64 without
// prefixes, all of 4096: 44 us, 3.4 TB/s.  Issue slots 58 % used, tensor pipe 19 %.  With
// the keys in bf16 by bit fields, three CTAs an SM, a tile took 703 instructions and a long
// cache read at 5.35 TB/s.
// Rows of a segment beyond 16 go to kv4_attn_tc.cu where that is quicker.
#include "kv4_attn.cuh"

#include <float.h>
#include <math.h>

#include "sm100_ptx.cuh"

namespace qerl {
namespace kv4 {
namespace {

using namespace ptx;

constexpr int kWarps = 4, kStages = 2, kPerSm = 4;
constexpr int kStart = 2;  // empty steps before a unit's
constexpr float kHead = 8.0f, kRoom = 15.0f;  // m is set kHead below a maximum, and raised above kRoom
constexpr uint64_t kLimitNs = 2000000000ull;

template <int D>
struct Smem {
    static constexpr int RING = kWarps * kStages * Tile<D>::BYTES, ROW = D + 4;  // padded: the warps' rows meet without bank conflicts
    static constexpr int O = RING, ML = O + kWarps * kRows * ROW * 4, Q = ML + kWarps * kRows * 8, TOTAL = Q + kRows * D * 2;
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t turned(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// Where a warp stands on its CTA's range of the line.
struct Place {
    int seg, unit, T, i0, i1, take, left, off;  // segment, unit in it, its tiles, the range of them, its steps and all to the end, tiles before it
};
__device__ __forceinline__ int seg_tiles(const Call &a, int k)
{
    return tiles_of(k < a.pre.n ? length(a.pre, k) : length(a.suf, k - a.pre.n));
}
__device__ __forceinline__ int seg_units(const Call &a, int k) { return a.Hkv * (k < a.pre.n ? a.pre.row_tiles : a.suf.row_tiles); }
// The next unit of which the CTA has tiles.
__device__ __forceinline__ bool next_unit(const Call &a, int start, Place &p)
{
    p.off += p.i1 - p.i0;
    p.left -= p.take;
    if (p.left <= start) return false;
    if (++p.unit == seg_units(a, p.seg)) {
        p.unit = 0;
        do p.T = seg_tiles(a, ++p.seg);
        while (p.T == 0);
    }
    p.take = min(p.T + start, p.left);
    p.i0 = 0;
    p.i1 = p.take - start;
    return true;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, kPerSm) rows_kernel(const __grid_constant__ Call a, int beside, unsigned int *err)
{
    using M = Tile<D>;
    using S = Smem<D>;
    constexpr int MT = D / 16, KW = D / 32, R = kRows;  // row tiles of O^T; key words of a lane; query rows
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_full[kWarps][kStages];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, q = lane % 4;
    if (threadIdx.x == 0) {
        for (int k = 0; k < kWarps * kStages; ++k) mbar_init(&s_full[0][0] + k, 1);
        fence_mbar_init();
    }
    // Beside the tcgen05 kernel, whose CTAs let this one start once all work before both has finished, there is nothing to wait
    // for; its last CTA waits at its end, so that the join, which waits for this kernel, has both.
    if (!beside) pdl_wait();
    pdl_trigger();
    __syncthreads();

    const int segs = a.pre.n + a.suf.n;
    constexpr int kHeld = 4;  // 32 segments each whose tiles stay in a register
    int tiles[kHeld], total = 0, units = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) tiles[i] = i * 32 + lane < segs ? seg_tiles(a, i * 32 + lane) : 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (tiles[i]) units += seg_units(a, i * 32 + lane), total += tiles[i] * seg_units(a, i * 32 + lane);
    for (int k = kHeld * 32 + lane; k < segs; k += 32) {
        const int T = seg_tiles(a, k);
        if (T) units += seg_units(a, k), total += T * seg_units(a, k);
    }
    total = __reduce_add_sync(0xFFFFFFFFu, total);
    units = __reduce_add_sync(0xFFFFFFFFu, units);
    // What it costs to begin a unit counts as empty steps before its own, where that matters.
    const int start = total >= 16 * a.grid ? kStart : 0;
    total += units * start;
    const int per = max((total + a.grid - 1) / a.grid, 1);
    const int begin = min((int64_t)blockIdx.x * per, (int64_t)total), end = min(begin + per, total);
    Place at = {};
    int before = 0;
    const auto segments = [&](int k0, int T) {  // 32 of them
        const int k = k0 + lane, steps = T ? (T + start) * seg_units(a, k) : 0;
        int sum = steps;
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        const int from = before + sum - steps;
        if (blockIdx.x == 0 && warp == 0) {
            if (k < segs) a.line[2 + k] = from;
            if (k == 0) a.line[0] = per, a.line[1] = start;
        }
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, begin >= from && begin < before + sum);
        if (here) {
            const int src = __ffs(here) - 1;
            at.seg = k0 + src;
            at.T = __shfl_sync(0xFFFFFFFFu, T, src);
            const int in = begin - __shfl_sync(0xFFFFFFFFu, from, src);
            at.unit = in / (at.T + start);
            const int into = in - at.unit * (at.T + start);
            at.left = end - begin;
            at.take = min(at.T + start - into, at.left);
            at.i0 = max(into - start, 0);
            at.i1 = max(into + at.take - start, 0);
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (i * 32 < segs) segments(i * 32, tiles[i]);
    for (int k0 = kHeld * 32; k0 < segs; k0 += 32) segments(k0, k0 + lane < segs ? seg_tiles(a, k0 + lane) : 0);
    if (begin < end && at.i0 < at.i1) {  // a range of empty steps alone has no tile
        uint8_t *const ring = smem + warp * kStages * M::BYTES;
        // the first of this warp's tiles from i0 on: every fourth step of the CTA's range
        const auto first = [&](const Place &p) { return p.i0 + ((warp - p.off) & (kWarps - 1)); };
        Place ahead = at;
        int fi = first(ahead), fetched = 0, used = 0;
        bool more = true, dead = false;
        const auto fetch = [&]() {
            while (more && fi >= ahead.i1) {
                more = next_unit(a, start, ahead);
                if (more) fi = first(ahead);
            }
            if (!more || dead) return;
            const int st = fetched % kStages;
            if (lane == 0) {
                mbar_arrive_expect_tx(&s_full[warp][st], M::BYTES);
                const bool pre = ahead.seg < a.pre.n;
                const Cache &c = pre ? a.pre.c : a.suf.c;
                const int k = pre ? ahead.seg : ahead.seg - a.pre.n, hk = ahead.unit / (pre ? a.pre.row_tiles : a.suf.row_tiles);
                bulk_load(ring + st * M::BYTES, c.data + k * c.s_n + hk * c.s_h + fi * c.s_t, M::BYTES, &s_full[warp][st]);
            }
            ++fetched;
            fi += kWarps;
        };
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) fetch();

        // A unit's query rows come to shared memory while the parts of the unit before it are summed.
        const auto fetch_q = [&](const Place &p) {
            const bool pre = p.seg < a.pre.n;
            const Side &s = pre ? a.pre : a.suf;
            const int seg = pre ? p.seg : p.seg - a.pre.n, hk = p.unit / s.row_tiles, tile = p.unit - hk * s.row_tiles;
            for (int i = threadIdx.x; i < R * (D / 8); i += kWarps * 32) {
                const int n = i / (D / 8), ch = i % (D / 8), rr = tile * R + n;
                const Row w = row_of(a, pre, seg, hk, min(rr, s.rows - 1));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem + S::Q + (n * (D / 8) + (ch ^ (n & 7))) * 16)),
                             "l"(a.q + w.b * a.q_b + w.l * a.q_l + w.h * a.q_h + ch * 8), "r"(rr < s.rows ? 16 : 0)
                             : "memory");
            }
        };
        fetch_q(at);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        for (bool go = true; go;) {
            const bool pre = at.seg < a.pre.n;
            const Side &s = pre ? a.pre : a.suf;
            const int seg = pre ? at.seg : at.seg - a.pre.n, len = length(s, seg), hk = at.unit / s.row_tiles, tile = at.unit - hk * s.row_tiles;
            // Q^T: lane (r, q) holds dims D / 4 q .. of row r, four of them a step
            uint32_t qf[D / 16][2];
            int limit[2];
            float scale[2];  // to log2 units
            uint4 v[D / 32];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                v[i] = ld_shared_v4(smem_u32(smem + S::Q + (r * (D / 8) + ((q * (D / 32) + i) ^ r)) * 16));
                const auto mag = [](uint32_t x) { return max(x & 0x7FFFu, x >> 16 & 0x7FFFu); };
                top = max(max(top, max(mag(v[i].x), mag(v[i].y))), max(mag(v[i].z), mag(v[i].w)));
            }
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int e = min(max((int)(top >> 7) - 127, -126), 126);  // the largest element's exponent; Inf and NaN stay what they are
            const float down = pow2f(-e);
            const auto half = [&](uint32_t x) { return f16x2(bf16lo(x) * down, bf16hi(x) * down); };
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                qf[2 * i][0] = half(v[i].x), qf[2 * i][1] = half(v[i].y);
                qf[2 * i + 1][0] = half(v[i].z), qf[2 * i + 1][1] = half(v[i].w);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                limit[k] = pre ? len : len - a.Lq + 1 + row_of(a, pre, seg, hk, tile * R + 2 * q + k).l;
                scale[k] = row_scale(s.scale_log2, __shfl_sync(0xFFFFFFFFu, e, (2 * q + k) * 4));
            }
            const int all_see = pre ? len : len - a.Lq + 1;  // keys that every row sees
            float o[MT][4], m[2], l[2];
            m[0] = m[1] = kNone;
            l[0] = l[1] = 0.0f;
#pragma unroll
            for (int t = 0; t < MT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.0f;
            for (int i = first(at); i < at.i1; i += kWarps) {
                const int st = used % kStages;
                if (!dead) {
                    bool ok = false;
                    for (int k = 0; k < 64 && !ok; ++k) ok = mbar_try_wait(&s_full[warp][st], (used / kStages) & 1);
                    if (!ok) {
                        const uint64_t until = globaltimer_ns() + kLimitNs;
                        while (!(ok = mbar_try_wait_sleep(&s_full[warp][st], (used / kStages) & 1, 20000u)))
                            if (globaltimer_ns() > until) break;
                    }
                    dead = !__all_sync(0xFFFFFFFFu, ok);
                    if (dead && lane == 0) latch_error(err, QERL_ERR_TIMEOUT);
                }
                if (dead) break;
                ++used;
                fetch();
                uint8_t *const tl = ring + st * M::BYTES;
                const uint32_t tb = smem_u32(tl);
                const int k0 = i * kTok;
                if (k0 + kTok > len) {  // what lies past the segment may be anything: its scales become 0
                    for (int e = lane; e < 4 * MT; e += 32) {
                        const int keys = max(0, min(8, len - k0 - 8 * (e / MT)));
                        uint64_t *const p = reinterpret_cast<uint64_t *>(tl + M::VS) + e;
                        *p = keys == 8 ? *p : *p & ((uint64_t(1) << (8 * keys)) - 1);
                    }
                    fence_proxy_async_smem();  // before the next copy into this place
                    __syncwarp();
                }
                // S^T: column c (16 keys) in turn
                float x[2][4];
                uint32_t ks[4];  // the lane's key scales, a pair of blocks of token e each (D = 64: of one block, of two tokens)
                if (D == 128) {
                    uint32_t w0, w1;
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(tb + M::KS + lane * 8) : "memory");
                    scales_f16(w0, ks[0], ks[1]);
                    scales_f16(w1, ks[2], ks[3]);
                } else {
                    scales_f16(ld_shared_u32(tb + M::KS + lane * 4), ks[0], ks[1]);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t kw[2][KW], f[2][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t from = tb + M::KC + (8 * (r / 2) + 4 * c + r % 2 + 2 * h) * (D / 2) + q * (D / 8);
                        if (D == 128) {
                            const uint4 v = ld_shared_v4(from);
                            kw[h][0] = v.x, kw[h][1] = v.y, kw[h][KW - 2] = v.z, kw[h][KW - 1] = v.w;
                            f[h][0] = prmt(ks[2 * c + h], 0, 0x1010), f[h][1] = prmt(ks[2 * c + h], 0, 0x3232);
                        } else {
                            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(kw[h][0]), "=r"(kw[h][1]) : "r"(from) : "memory");
                            f[h][0] = prmt(ks[c], 0, h ? 0x3232 : 0x1010);
                        }
                    }
                    x[c][0] = x[c][1] = x[c][2] = x[c][3] = 0.0f;
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        uint32_t k0w[4], k1w[4];
                        codes_f16(kw[0][w], k0w);
                        codes_f16(kw[1][w], k1w);
#pragma unroll
                        for (int i = 0; i < 4; ++i) k0w[i] = f16x2_mul(k0w[i], f[0][w / 2]), k1w[i] = f16x2_mul(k1w[i], f[1][w / 2]);
                        mma_f16(x[c], k0w[0], k1w[0], k0w[1], k1w[1], qf[2 * w][0], qf[2 * w][1]);
                        mma_f16(x[c], k0w[2], k1w[2], k0w[3], k1w[3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
                    }
                }
                if (k0 + kTok > all_see) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (k0 + 8 * (r / 2) + 4 * c + r % 2 + 2 * (e / 2) >= limit[e % 2]) x[c][e] = -INFINITY;
                }
                uint32_t p[2][2];
                float top[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    top[e] = fmaxf(fmaxf(fmaxf(x[0][e], x[0][e + 2]), fmaxf(x[1][e], x[1][e + 2])), kNone) * scale[e];
                if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kRoom || top[1] > m[1] + kRoom)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int k = 4; k < 32; k *= 2) top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], k));
                        const float to = top[e] > m[e] + kRoom ? top[e] - kHead : m[e], f = ex2(m[e] - to);
                        m[e] = to;
                        l[e] *= f;
#pragma unroll
                        for (int t = 0; t < MT; ++t) o[t][e] *= f, o[t][e + 2] *= f;
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[c][e] = ex2(fmaf(x[c][e], scale[e % 2], -m[e % 2]));
                        l[e % 2] += x[c][e];
                    }
                    p[c][0] = turned(f16x2(x[c][0], x[c][1]));
                    p[c][1] = turned(f16x2(x[c][2], x[c][3]));
                }
                // O^T: lane (r, q) holds keys 8 q .. 8 q + 7 of dims r and r + 8 of a row tile
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint4 w = ld_shared_v4(tb + M::VC + (j * 32 + lane) * 16), sc = ld_shared_v4(tb + M::VS + (q * MT + 2 * j) * 8);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        uint32_t v0[4], v1[4], f[4];  // a pair of keys each
                        codes_f16(t ? w.z : w.x, v0);
                        codes_f16(t ? w.w : w.y, v1);
                        scales_f16(t ? sc.z : sc.x, f[0], f[1]);
                        scales_f16(t ? sc.w : sc.y, f[2], f[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v0[i] = f16x2_mul(v0[i], f[i]), v1[i] = f16x2_mul(v1[i], f[i]);
#pragma unroll
                        for (int c = 0; c < 2; ++c) mma_f16(o[2 * j + t], v0[2 * c], v1[2 * c], v0[2 * c + 1], v1[2 * c + 1], p[c][0], p[c][1]);
                    }
                }
                __syncwarp();  // the place is free for the copy that the next turn issues
            }
            // the warps' sums meet
            float *const so = reinterpret_cast<float *>(smem + S::O);
            float2 *const sml = reinterpret_cast<float2 *>(smem + S::ML);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int k = 4; k < 32; k *= 2) l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], k);
                const int row = warp * R + 2 * q + e;
                if (r == 0) sml[row] = make_float2(m[e], l[e]);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    so[row * S::ROW + t * 16 + r] = o[t][e];
                    so[row * S::ROW + t * 16 + r + 8] = o[t][e + 2];
                }
            }
            __syncthreads();
            const int64_t part = (int64_t)(pre ? 0 : a.pre.n * a.Hkv * a.pre.row_tiles) + (int64_t)seg * a.Hkv * s.row_tiles + at.unit + blockIdx.x;
            go = next_unit(a, start, at);
            if (go) fetch_q(at);
            for (int row = warp; row < R; row += kWarps) {
                float M_ = kNone, L = 0.0f, w[kWarps];
#pragma unroll
                for (int k = 0; k < kWarps; ++k) M_ = fmaxf(M_, sml[k * R + row].x);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    w[k] = ex2(sml[k * R + row].x - M_);
                    L = fmaf(w[k], sml[k * R + row].y, L);
                }
                if (lane < D / 4) {
                    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int k = 0; k < kWarps; ++k) {
                        const float4 v = *reinterpret_cast<const float4 *>(so + (k * R + row) * S::ROW + lane * 4);
                        t.x = fmaf(w[k], v.x, t.x), t.y = fmaf(w[k], v.y, t.y), t.z = fmaf(w[k], v.z, t.z), t.w = fmaf(w[k], v.w, t.w);
                    }
                    *reinterpret_cast<float4 *>(a.part_o + (part * R + row) * D + lane * 4) = t;
                }
                if (lane == 0) a.part_ml[part * R + row] = make_float2(M_, L);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
        }
        if (dead) {  // no copy may be in flight when the CTA ends
            const uint64_t until = globaltimer_ns() + kLimitNs;
            for (int k = used; k < fetched; ++k)
                while (!mbar_try_wait(&s_full[warp][k % kStages], (k / kStages) & 1) && globaltimer_ns() < until) {
                }
            __syncwarp();
        }
    }
    if (beside && blockIdx.x == gridDim.x - 1) pdl_wait();
}

// ------------------------------------------------------------------ joining a row's parts
struct Parts {
    const float *o;
    const float2 *ml;
    int n;
    int64_t step;  // from part to part, in rows
    float v_scale;
};
__device__ __forceinline__ Parts parts_of(const Call &a, const attn::Args &tc, bool pre, int k, int hk, int r, int64_t row, int len, int D)
{
    const Side &s = pre ? a.pre : a.suf;
    Parts p = {};
    const int T = tiles_of(len);
    if (T == 0) return p;
    p.v_scale = s.c.v_scale;
    if (pre ? tc.p_tc : tc.s_tc) {
        const int64_t at = row * (tc.n_pp + tc.n_sp) + (pre ? 0 : tc.n_pp);
        p.n = attn::tc_parts(tc, pre, k + (pre || !tc.p_tc ? 0 : tc.n_prefix), hk, r, len);
        p.o = tc.part_o + at * D;
        p.ml = tc.part_ml + at;
        p.step = 1;
        return p;
    }
    const int per = a.line[0], empty = a.line[1], tile = r / kRows, u = hk * s.row_tiles + tile;
    const int start = a.line[2 + k + (pre ? 0 : a.pre.n)] + u * (T + empty) + empty;
    const int c0 = start / per;
    const int64_t at = ((pre ? 0 : (int64_t)a.pre.n * a.Hkv * a.pre.row_tiles) + (int64_t)k * a.Hkv * s.row_tiles + u + c0) * kRows + r % kRows;
    p.n = (start + T - 1) / per - c0 + 1;
    p.o = a.part_o + at * D;
    p.ml = a.part_ml + at;
    p.step = kRows;
    return p;
}

// W warps per query row, each takes every W-th part; in a fixed order, so that results repeat.
template <int D, int W>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128) join_kernel(const __grid_constant__ Call a, const __grid_constant__ attn::Args tc)
{
    constexpr int E = D / 32, RB = W > 4 ? 1 : 4 / W, NB = 4;  // columns of a lane; rows of a block; parts in flight
    __shared__ float s_o[RB * W][W > 1 ? D : 1];
    __shared__ float2 s_ml[RB * W];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, share = warp % W;
    const int row = blockIdx.x * RB + warp / W;
    const bool live = row < a.B * a.Lq * a.Hq;
    const int h = row % a.Hq, bl = row / a.Hq, l = bl % a.Lq, b = live ? bl / a.Lq : 0, g = b / a.G;
    const int hk = h / a.gs, hi = h - hk * a.gs;
    // the kernel before this one lets it start after all work before the call: the lengths are there
    const int tp = live && (a.pre.n || tc.p_tc) ? length(a.pre, g) : 0, ts = live && (a.suf.n || tc.s_tc) ? length(a.suf, b) : 0;
    pdl_wait();
    pdl_trigger();
    const Parts pp = parts_of(a, tc, true, g, hk, ((b - g * a.G) * a.Lq + l) * a.gs + hi, row, tp, D);
    const Parts ps = parts_of(a, tc, false, b, hk, l * a.gs + hi, row, ts, D);
    const int n = pp.n + ps.n;
    // Sums of values without the factor are below 2^57 (2^30 keys); so that they stay finite with one of up to 2^100, 2^40 comes last.
    const bool large = fmaxf(pp.v_scale, ps.v_scale) >= 1.0f;
    const float down = large ? 0x1p-40f : 1.0f, up = large ? 0x1p40f : 1.0f, p_scale = pp.v_scale * down, s_scale = ps.v_scale * down;
    float M = kNone, L = 0.0f, acc[E] = {};
    for (int k0 = share; k0 < n; k0 += NB * W) {
        float2 ml[NB];
        float v[NB][E];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int k = k0 + j * W;
            ml[j] = make_float2(kNone, 0.0f);
            if (k < n) {
                const Parts &p = k < pp.n ? pp : ps;
                const int64_t at = (k < pp.n ? k : k - pp.n) * p.step;
                ml[j] = p.ml[at];
                const float *o = p.o + at * D + lane * E;
                if (E == 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(o);
                    v[j][0] = t.x, v[j][1] = t.y, v[j][E - 2] = t.z, v[j][E - 1] = t.w;
                } else {
                    const float2 t = *reinterpret_cast<const float2 *>(o);
                    v[j][0] = t.x, v[j][1] = t.y;
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
            const bool none = ml[j].x == kNone && ml[j].y == 0.0f;
            const float w = none ? 0.0f : ex2(ml[j].x - M), wv = w * (k0 + j * W < pp.n ? p_scale : s_scale);
            L = fmaf(w, ml[j].y, L);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wv, none ? 0.0f : v[j][e], acc[e]);
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
    const float inv = L == 0.0f ? 0.0f : __fdividef(1.0f, L);  // a row that sees no key: zeros, lse -inf
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + b * a.o_b + l * a.o_l + h * a.o_h + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(acc[e] * inv * up, acc[e + 1] * inv * up);
        out[e / 2] = *reinterpret_cast<const uint32_t *>(&t);
    }
    if (lane == 0 && a.lse) a.lse[row] = L == 0.0f ? -INFINITY : (float)((double)M * 0.6931471805599453 + (double)logf(L));
}

// ------------------------------------------------------------------ host side
int ceil_div(int64_t x, int64_t y) { return (int)((x + y - 1) / y); }
size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

int64_t units_of(const Call &a) { return ((int64_t)a.pre.n * a.pre.row_tiles + (int64_t)a.suf.n * a.suf.row_tiles) * a.Hkv; }
size_t ml_bytes(const Call &a) { return round256((size_t)(units_of(a) + a.grid) * kRows * sizeof(float2)); }
size_t line_bytes(const Call &a) { return round256((size_t)(2 + a.pre.n + a.suf.n) * sizeof(int)); }
size_t rows_bytes(const Call &a, int64_t D)
{
    return a.grid ? ml_bytes(a) + line_bytes(a) + round256((size_t)(units_of(a) + a.grid) * kRows * D * sizeof(float)) : 0;
}
size_t tc_rows(const attn::Args &t) { return (size_t)t.B * t.Lq * t.Hq * (t.n_pp + t.n_sp); }
size_t tc_ml_bytes(const attn::Args &t) { return round256(tc_rows(t) * sizeof(float2)); }
size_t tc_line_bytes(const attn::Args &t) { return round256((size_t)(1 + t.n_prefix + t.B) * sizeof(int)); }

template <int D>
qerl_status run(const Call &a, const attn::Args &tc, cudaStream_t st)
{
    const bool chain = g_chain.load() != 0, many = tc.p_tc || tc.s_tc;
    if (many) QERL_TRY(launched(many_rows(tc, a.pre, a.suf, D, st, chain), QERL_KERNEL_KV4_ROWS128));
    if (a.grid) {
        static OncePerDevice once;
        if (allow_smem(once, rows_kernel<D>, Smem<D>::TOTAL) != cudaSuccess) return QERL_ERR_CUDA;
        QERL_TRY(launched(launch_k(rows_kernel<D>, dim3((unsigned)a.grid), dim3(kWarps * 32), Smem<D>::TOTAL, st, chain, a, many && chain ? 1 : 0,
                                   error_word()),
                          QERL_KERNEL_KV4_ROWS8));
    }
    // warps per row: one where the rows fill the SMs or have few parts, sixteen where there are many
    const int64_t rows = (int64_t)a.B * a.Lq * a.Hq, parts = (a.pre.n != 0) + (a.suf.n != 0) + (a.grid ? 2 * a.grid / units_of(a) : 0) + tc.n_pp + tc.n_sp;
    if (parts <= 8 || rows > 32 * num_sms())
        return launched(launch_k(join_kernel<D, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, chain, a, tc));
    if (parts <= 24 || rows > 4 * num_sms()) return launched(launch_k(join_kernel<D, 4>, dim3((unsigned)rows), dim3(128), 0, st, chain, a, tc));
    return launched(launch_k(join_kernel<D, 16>, dim3((unsigned)rows), dim3(512), 0, st, chain, a, tc));
}

// The call's sizes and the workspace it needs.
qerl_status shape(const qerl_kv4_attn_dims *d, const qerl_kv4_cache *prefix, const qerl_kv4_cache *suffix, Call &a, attn::Args &tc, size_t &bytes)
{
    if (!d || (!prefix && !suffix)) return QERL_ERR_INVALID_ARG;
    if (prefix) QERL_TRY(check_cache(prefix, a.pre.c));
    if (suffix) QERL_TRY(check_cache(suffix, a.suf.c));
    const int64_t big = 1 << 30, Hkv = (prefix ? prefix : suffix)->Hkv, D = (prefix ? prefix : suffix)->D;
    if (d->B < 1 || d->Lq < 1 || d->Hq < 1 || d->B > big || d->Lq > big || d->Hq > 65536 || d->Hq % Hkv || d->B * d->Lq > big / d->Hq)
        return QERL_ERR_SHAPE;
    if (prefix && d->B % prefix->n) return QERL_ERR_SHAPE;
    if (suffix && (suffix->n != d->B || suffix->Hkv != Hkv || suffix->D != D)) return QERL_ERR_SHAPE;
    a.B = (int)d->B, a.Lq = (int)d->Lq, a.Hq = (int)d->Hq, a.Hkv = (int)Hkv, a.gs = (int)(d->Hq / Hkv), a.G = prefix ? (int)(d->B / prefix->n) : 1;
    a.pre.n = prefix ? (int)prefix->n : 0, a.suf.n = suffix ? a.B : 0;
    a.pre.rows = a.G * a.Lq * a.gs, a.suf.rows = a.Lq * a.gs;
    a.pre.row_tiles = ceil_div(a.pre.rows, kRows), a.suf.row_tiles = ceil_div(a.suf.rows, kRows);
    const int64_t pre = (int64_t)a.pre.n * a.pre.row_tiles * a.Hkv, suf = (int64_t)a.suf.n * a.suf.row_tiles * a.Hkv;
    if (pre > big || suf > big || pre + suf > big) return QERL_ERR_SHAPE;
    const int64_t pt = prefix ? (prefix->T + kTok - 1) / kTok : 0, st = suffix ? (suffix->T + kTok - 1) / kTok : 0;
    if ((pt && pre > big / pt) || (st && suf > big / st) || (pre + suf) * kStart + pre * pt + suf * st > big) return QERL_ERR_SHAPE;
    // A kind of segments goes to the tcgen05 kernel where that is quicker: a step of its line (256 rows, 128 keys) takes about 2 us
    // on a CTA, one of this file's (8 rows, 32 keys) 1 ns over all SMs.
    const int sms = num_sms();
    const auto steps_of = [&](int64_t n, int64_t rows, int64_t T) { return n * Hkv * (rows / 256 + 1) * ((T + 127) / 128); };
    const auto quicker = [&](int64_t n, int64_t rows, int64_t T, int64_t steps8) {
        const int64_t steps = steps_of(n, rows, T);
        return n && rows > 16 && T >= 128 && steps + 4 * n * Hkv * (rows / 256 + 1) < big && 8.0 + 2.0 * (double)((steps + sms - 1) / sms) < 1e-3 * (double)steps8;
    };
    tc.p_tc = quicker(a.pre.n, a.pre.rows, prefix ? prefix->T : 0, pre * pt);
    tc.s_tc = quicker(a.suf.n, a.suf.rows, suffix ? suffix->T : 0, suf * st);
    tc.grid_tc = sms;
    int free_sms = sms;
    if (tc.p_tc && !tc.s_tc && suffix) {
        // The prefixes leave SMs to the own tokens, as many as make the later of the two end soonest; the caches half full, which
        // they are on average in a rollout (an SM reads some 40 bytes per ns).
        const double steps = (double)steps_of(a.pre.n, a.pre.rows, prefix->T), bytes8 = 0.5 * (double)(suf * st) * 36.0 * (double)D;
        double best = 2.0 * ceil(steps / sms) + bytes8 / 6.0e6;
        for (int n = sms - 4; n >= sms / 2; n -= 4) {
            const double t = 2.0 * ceil(steps / n), u = bytes8 / ((sms - n) * 40.0e3), later = t > u ? t : u;
            if (later < best) best = later, tc.grid_tc = n, free_sms = sms - n;
        }
    }
    if (tc.p_tc || tc.s_tc) {
        tc.B = a.B, tc.Lq = a.Lq, tc.Hq = a.Hq, tc.Hkv = a.Hkv, tc.G = a.G, tc.gs = a.gs, tc.n_prefix = prefix ? a.pre.n : 1;
        tc.P = prefix ? (int)prefix->T : 0, tc.S = suffix ? (int)suffix->T : 0;
        tc.n_pp = tc.p_tc ? attn::tc_parts_most(a.pre.rows, prefix->T, Hkv, tc.grid_tc) : 0;
        tc.n_sp = tc.s_tc ? attn::tc_parts_most(a.suf.rows, suffix->T, Hkv, tc.grid_tc) : 0;
    }
    // the rest
    if (tc.p_tc) a.pre.n = 0;
    if (tc.s_tc) a.suf.n = 0;
    const int64_t most = (int64_t)free_sms * kPerSm, want = (a.pre.n ? pre * pt : 0) + (a.suf.n ? suf * st : 0);
    a.grid = (int)(want < most ? want : most);
    bytes = rows_bytes(a, D) + tc_ml_bytes(tc) + tc_line_bytes(tc) + tc_rows(tc) * D * sizeof(float);
    return QERL_OK;
}

}  // namespace
}  // namespace kv4
}  // namespace qerl

using namespace qerl;

extern "C" size_t qerl_kv4_attention_ws_bytes(const qerl_kv4_attn_dims *d, const qerl_kv4_cache *prefix, const qerl_kv4_cache *suffix)
{
    kv4::Call a = {};
    attn::Args tc = {};
    size_t bytes = 0;
    return kv4::shape(d, prefix, suffix, a, tc, bytes) == QERL_OK ? bytes : 0;
}

extern "C" qerl_status qerl_kv4_attention(const qerl_kv4_attn_dims *d, const void *q, const qerl_kv4_cache *prefix, const int32_t *prefix_lens,
                                          const qerl_kv4_cache *suffix, const int32_t *suffix_lens, float scale, void *out, float *lse, void *ws,
                                          size_t ws_bytes, qerl_stream_t stream)
{
    if (!d || !q || !out || !(scale > 0.0f) || !(scale <= FLT_MAX) || (suffix && !suffix_lens)) return QERL_ERR_INVALID_ARG;
    kv4::Call a = {};
    attn::Args tc = {};
    size_t need = 0;
    QERL_TRY(kv4::shape(d, prefix, suffix, a, tc, need));
    for (int i = 0; i < 3; ++i) {
        if (d->q_stride[i] < 0 || d->out_stride[i] < 0 || d->q_stride[i] > (int64_t(1) << 40) || d->out_stride[i] > (int64_t(1) << 40))
            return QERL_ERR_SHAPE;
        if (d->q_stride[i] % 8 || d->out_stride[i] % 8) return QERL_ERR_ALIGN;
    }
    if (kv4::repeated(d->B, d->Lq, d->Hq, d->out_stride)) return QERL_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(prefix_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(suffix_lens) & 3u))
        return QERL_ERR_ALIGN;
    for (kv4::Side *s : {&a.pre, &a.suf})
        if (s->c.data) {
            const double c = (double)scale * s->c.k_scale * 1.4426950408889634;
            if (!(c >= FLT_MIN && c <= FLT_MAX)) return QERL_ERR_INVALID_ARG;
            s->scale_log2 = (float)c;
        }
    if (!ws || ws_bytes < need) return QERL_ERR_WORKSPACE;
    if (!aligned16(ws)) return QERL_ERR_ALIGN;
    QERL_TRY(check_device());
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.out = static_cast<__nv_bfloat16 *>(out), a.lse = lse;
    a.q_b = d->q_stride[0], a.q_l = d->q_stride[1], a.q_h = d->q_stride[2];
    a.o_b = d->out_stride[0], a.o_l = d->out_stride[1], a.o_h = d->out_stride[2];
    const int64_t D = (prefix ? prefix : suffix)->D;
    a.pre.lens = prefix_lens, a.suf.lens = suffix_lens;
    char *const to = static_cast<char *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(to);
    a.line = reinterpret_cast<int *>(to + kv4::ml_bytes(a));
    a.part_o = reinterpret_cast<float *>(to + kv4::ml_bytes(a) + kv4::line_bytes(a));
    char *const tc_to = to + kv4::rows_bytes(a, D);
    tc.part_ml = reinterpret_cast<float2 *>(tc_to);
    tc.line = reinterpret_cast<int *>(tc_to + kv4::tc_ml_bytes(tc));
    tc.part_o = reinterpret_cast<float *>(tc_to + kv4::tc_ml_bytes(tc) + kv4::tc_line_bytes(tc));
    tc.q = a.q, tc.q_b = a.q_b, tc.q_l = a.q_l, tc.q_h = a.q_h;
    tc.plen = prefix_lens, tc.slen = suffix_lens;
    return D == 128 ? kv4::run<128>(a, tc, as_cuda(stream)) : kv4::run<64>(a, tc, as_cuda(stream));
}
