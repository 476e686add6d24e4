// Attention parts of many query rows on tcgen05 (see prefix_attn.cuh for the
// schedule and the parts).
//
// A CTA works on two row tiles of 128 (or on two key tiles of one row tile) at a
// time, so that the tensor core multiplies for one while the other is in its
// softmax.  Warps 0-3 and 4-7: the softmax of the two, one thread per row; warps
// 8 and 9: TMA loads of the key and the value tiles (one instruction a tile: some
// 130 ns each, which with four per 64 keys had been what bounded a step); warps
// 10 and 11: the MMAs of the two.
// Per half and 64 keys of a tile:
//     S = Q K^T     Q, K in shared memory (K-major), S in TMEM, FP32
//     P = 2^(S c - m)  read from TMEM, written back as bf16 over S
//     O += P V      P from TMEM, V as it lies in the cache (MN-major), O in TMEM
// There are two S of 64 keys per half, so that the next one is there when a
// softmax ends.  m is raised only when a row's maximum outgrows it by 2^8 (the
// weights stay below 2^8 and are normalised in the end all the same), so O is
// rescaled rarely.  S and P share columns: the Q K^T that overwrites a P is issued
// once its P V has completed.
// Shared memory (D = 128): Q 64 KB, five K and five V tiles of 64 keys, 16 KB each.
// A tile's load has to hide behind the four before it.
// What bounds it: a step (two row tiles, 128 keys: 17 MFLOP) takes 1.9 us, 69 % of
// the measured bf16 rate.  For 64 keys of a half Q K^T takes 389 clocks (its 6 KB of operands per
// instruction are all of shared memory's rate) and P V 260, measured alone; both
// halves and the tiles' arrival in shared memory come to some 0.78 of the 0.95 us.
// One S with two P instead, so that Q K^T waits for no P V, took as long.  A unit's
// rows cost about 6 us besides (loads of Q, first S, stores of O).
// 28 query heads of 64 sequences over a prefix of 16384 keys: 11 steps on each of 96
// CTAs; with the suffixes, on the other SMs meanwhile, and the join (8 us) 45 us.
// 129 tokens of eight sequences, 16 heads, over 4001 keys and their own: 18 steps a
// CTA, its starts among them, 54 us, and 14 for the join of 2 to 5 parts a row.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "prefix_attn.cuh"
#include "sm100_ptx.cuh"

namespace qerl {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // linear_tc.cu

namespace attn {
namespace {

using namespace ptx;

struct Maps {
    CUtensorMap kp, vp, ks, vs;
};
static_assert(sizeof(CUtensorMap) == 128, "");
static_assert(sizeof(Maps) == kTcMapsBytes, "");

constexpr int kThreads = 384, kTmaWarp = 8, kMmaWarp = 10;  // and the warp after each
constexpr int kStages = 5;  // tiles of 64 keys: K and V each

__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w, int v)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
template <int D>
struct Smem {
    static constexpr int SUB = D / 64;             // 64-element column blocks of a tile
    static constexpr int TILE = SUB * 128 * 128;   // bytes of 128 query rows
    static constexpr int KV = SUB * 64 * 128;      // bytes of 64 keys
    static constexpr int Q = 0, K = 2 * TILE, V = K + kStages * KV, TOTAL = V + kStages * KV;
};

// A contiguous range of steps inside one unit.
struct Seg {
    bool pre, single;
    int seg, hk, pair, len, tile0, part;
    int next;    // where the next range starts
    int n0, n1;  // tiles of the two halves
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) rows128_kernel(const __grid_constant__ Maps maps, const Args a, unsigned int *err)
{
    using M = Smem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // the swizzled tiles' alignment
    __shared__ uint64_t b_q[2], b_kfull[kStages], b_kempty[kStages], b_vfull[kStages], b_vempty[kStages], b_s[2][2], b_p[2][2], b_o[2], b_done[2], b_end;
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int k = 0; k < kStages; ++k) {
            mbar_init(&b_kfull[k], 1);
            mbar_init(&b_kempty[k], 2);  // both MMA warps
            mbar_init(&b_vfull[k], 1);
            mbar_init(&b_vempty[k], 2);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&b_q[h], 128);
            for (int k = 0; k < 2; ++k) {
                mbar_init(&b_s[h][k], 1);
                mbar_init(&b_p[h][k], 128);
            }
            mbar_init(&b_o[h], 1);
            mbar_init(&b_done[h], 1);
        }
        mbar_init(&b_end, 2);
        s_stop = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    pdl_trigger();  // a chained successor finds everything before this kernel finished

    // Every wait is bounded: past two seconds the error is latched and the CTA winds up.
    const uint64_t limit_ns = 2000000000ull;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        bool ok = false;
        for (int k = 0; k < 32 && !ok; ++k) ok = mbar_try_wait(bar, parity & 1u);  // the usual case never looks at the clock
        if (!ok) {
            const uint64_t until = globaltimer_ns() + limit_ns;
            while (!(ok = mbar_try_wait_sleep(bar, parity & 1u, 20000u))) {
                if (*reinterpret_cast<volatile int *>(&s_stop)) break;
                if (globaltimer_ns() > until) {
                    *reinterpret_cast<volatile int *>(&s_stop) = 1;
                    latch_error(err, QERL_ERR_TIMEOUT);
                    break;
                }
            }
        }
        return __all_sync(0xFFFFFFFFu, ok);
    };

    int before, total;
    line_length(a, before, total);  // before: the prefixes' steps
    const int per_cta = steps_per_cta(a, total);
    if (blockIdx.x == 0 && warp == 0) {  // for the kernel that joins the parts
        if (lane == 0) a.line[0] = per_cta;
        int at = 0;
        const int segs = (a.p_tc ? a.n_prefix : 0) + (a.s_tc ? a.B : 0);
        for (int k0 = 0; k0 < segs; k0 += 32) {
            const int n = k0 + lane < segs ? segment_steps(a, k0 + lane) : 0;
            int sum = n;
            for (int o = 1; o < 32; o *= 2) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += v;
            }
            if (k0 + lane < segs) a.line[1 + k0 + lane] = at + sum - n;
            at += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
    }
    const int begin = min((int)blockIdx.x * per_cta, total), end = min(begin + per_cta, total);
    const Units up(a.G * a.Lq * a.gs), us(a.Lq * a.gs);
    // the range of steps at `pos` that lies in one unit
    auto locate = [&](int pos) -> Seg {
        Seg s;
        s.pre = pos < before;
        int at = s.pre ? 0 : before;
        const Units &u = s.pre ? up : us;
        int n = 0;
        for (s.seg = 0;; ++s.seg, at += n) {
            s.len = s.pre ? prefix_len(a, s.seg) : suffix_len(a, s.seg);
            n = u.steps(key_tiles(s.len)) * a.Hkv;
            if (pos < at + n) break;
        }
        const int T = key_tiles(s.len);
        const int per_head = u.steps(T);
        s.hk = (pos - at) / per_head;
        at += s.hk * per_head;
        s.pair = min(u.full, (pos - at) / (kStart + T));
        s.single = s.pair == u.full;
        at += s.pair * (kStart + T) + kStart;
        const int unit = s.single ? (T + 1) / 2 : T, first = max(pos - at, 0);
        s.next = min(at + unit, end);
        const int steps = max(s.next - at - first, 0);  // none where the range ends among the empty steps
        s.part = (at + first) / per_cta - at / per_cta;
        if (s.single) {  // half h takes tiles 2 (first + i) + h
            s.tile0 = 2 * first;
            s.n0 = steps;
            s.n1 = min(steps, (T - s.tile0) / 2);
        } else {
            s.tile0 = first;
            s.n0 = s.n1 = steps;
        }
        return s;
    };

    if (warp == kTmaWarp || warp == kTmaWarp + 1) {
        const bool keys = warp == kTmaWarp;
        uint64_t *const full = keys ? b_kfull : b_vfull, *const empty = keys ? b_kempty : b_vempty;
        uint8_t *const ring = smem + (keys ? M::K : M::V);
        uint32_t it = 0;
        bool ok = true;
        for (int pos = begin; ok && pos < end;) {
            const Seg s = locate(pos);
            const int tiles = 2 * (s.single ? s.n0 + s.n1 : s.n0);
            const CUtensorMap *map = s.pre ? (keys ? &maps.kp : &maps.vp) : keys ? &maps.ks : &maps.vs;
            for (int t = 0; t < tiles; ++t, ++it) {
                const uint32_t st = it % kStages, round = it / kStages;
                if (round > 0 && !(ok = wait(&empty[st], round - 1))) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&full[st], M::KV);
                    tma_load_5d(ring + st * M::KV, map, &full[st], 0, s.tile0 * 128 + t * 64, 0, s.hk, s.seg);
                }
                __syncwarp();
            }
            pos = s.next;
        }
        // no load may be in flight when the CTA ends
        if (*reinterpret_cast<volatile int *>(&s_stop)) {
            const uint64_t until = globaltimer_ns() + limit_ns;
            for (uint32_t k = it > kStages ? it - kStages : 0; k < it; ++k)
                while (!mbar_try_wait(&full[k % kStages], (k / kStages) & 1u) && globaltimer_ns() < until) {
                }
        }
        __syncwarp();
    } else if (warp >= kMmaWarp) {
        const int h = warp - kMmaWarp;
        const uint32_t id_qk = idesc_bf16_f32(128, 64), id_pv = idesc_bf16_f32(128, D) | (1u << 16);  // V is MN-major
        const uint32_t d_s = tmem + h * 256, d_o = d_s + 128;
        const uint64_t q_desc = desc_kmajor_sw128(smem_u32(smem + M::Q + h * M::TILE)), k_desc = desc_kmajor_sw128(smem_u32(smem + M::K)),
                       v_desc = desc_mnmajor_sw128(smem_u32(smem + M::V), 8192, 1024);
        uint32_t tc = 0;           // tiles of 128 keys in earlier segments
        uint32_t kn = 0, vn = 0;   // K and V tiles passed: every one of both, so that no phase of a barrier goes unseen
        uint32_t qn = 0, pn = 0;   // Q tiles and P V products so far
        bool ok = true;
        for (int pos = begin; ok && pos < end;) {
            const Seg s = locate(pos);
            pos = s.next;
            const int n = 2 * (h ? s.n1 : s.n0);  // S of 64 keys
            const uint32_t t0 = tc + (s.single ? h : 0), dt = s.single ? 2 : 1;
            tc += (uint32_t)(s.single ? s.n0 + s.n1 : s.n0);
            // the tiles before `to` that only the other half uses
            auto pass = [&](uint64_t *full, uint64_t *empty, uint32_t &seen, uint32_t to) -> bool {
                for (; seen < to; ++seen) {
                    if (!wait(&full[seen % kStages], seen / kStages)) return false;
                    if (elect_one()) mbar_arrive(&empty[seen % kStages]);
                    __syncwarp();
                }
                return true;
            };
            if (n == 0) {
                ok = pass(b_kfull, b_kempty, kn, 2 * tc) && pass(b_vfull, b_vempty, vn, 2 * tc);
                continue;
            }
            if (!(ok = wait(&b_q[h], qn++))) break;
            auto qk = [&](int j) -> bool {
                const uint32_t half = j & 1, t = 2 * (t0 + (j / 2) * dt) + half, st = t % kStages;
                if (!pass(b_kfull, b_kempty, kn, t) || !wait(&b_kfull[st], t / kStages)) return false;
                ++kn;
                tc_fence_after();
                const uint64_t bd = k_desc + st * (uint32_t)(M::KV >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_bf16(d_s + half * 64, q_desc + (uint64_t)((kk / 4) * (16384 >> 4) + 2 * (kk % 4)),
                                  bd + (uint64_t)((kk / 4) * (8192 >> 4) + 2 * (kk % 4)), id_qk, kk > 0);
                    umma_commit(&b_s[h][half]);
                    umma_commit(&b_kempty[st]);
                }
                __syncwarp();
                return true;
            };
            ok = qk(0) && qk(1);
            for (int j = 0; ok && j < n; ++j) {
                const uint32_t half = j & 1, t = 2 * (t0 + (j / 2) * dt) + half, st = t % kStages;
                if (!(ok = pass(b_vfull, b_vempty, vn, t) && wait(&b_vfull[st], t / kStages))) break;
                ++vn;
                if (!(ok = wait(&b_p[h][half], pn / 2))) break;  // pn is even at the start of a segment
                ++pn;
                tc_fence_after();
                const uint64_t vd = v_desc + st * (uint32_t)(M::KV >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // 16 keys: two 8-row groups of every column block
                        umma_bf16_ts(d_o, d_s + half * 64 + 8 * kk, vd + (uint64_t)(kk * (2048 >> 4)), id_pv, j > 0 || kk > 0);
                    umma_commit(&b_o[h]);
                    if (j + 1 == n) umma_commit(&b_done[h]);
                    umma_commit(&b_vempty[st]);
                }
                __syncwarp();
                if (j + 2 < n) ok = wait(&b_o[h], pn - 1) && qk(j + 2);  // this P is read: its S may be overwritten
            }
            ok = ok && pass(b_kfull, b_kempty, kn, 2 * tc) && pass(b_vfull, b_vempty, vn, 2 * tc);
        }
        // every product issued has completed before TMEM is freed
        if (elect_one()) umma_commit(&b_end);
        __syncwarp();
    } else {
        const int h = warp / 4, t = tid % 128;  // half, row
        const uint32_t tm = tmem + h * 256 + ((uint32_t)((warp % 4) * 32) << 16);
        uint32_t sn = 0, units = 0;  // S and units so far
        uint32_t vc = 0, vnext = 0;  // value tiles of earlier segments
        bool ok = true;
        for (int pos = begin; ok && pos < end;) {
            const Seg s = locate(pos);
            pos = s.next;
            vc = vnext;
            vnext += (uint32_t)(s.single ? s.n0 + s.n1 : s.n0);
            const int n = 2 * (h ? s.n1 : s.n0), R = (s.pre ? a.G : 1) * a.Lq * a.gs;
            if (s.n0 == 0) continue;
            const int rr = (s.single ? 2 * s.pair : 2 * s.pair + h) * 128 + t, rows_b = a.Lq * a.gs;
            const bool mine = rr < R;
            const int bi = rr / rows_b, in = rr - bi * rows_b, l = in / a.gs;
            const int b = s.pre ? s.seg * a.G + bi : s.seg, head = s.hk * a.gs + in - l * a.gs;
            const int64_t at = (((int64_t)b * a.Lq + l) * a.Hq + head) * (a.n_pp + a.n_sp) + (s.pre ? 0 : a.n_pp) +
                               (s.single ? 2 * s.part + h : s.part);
            if (n == 0) {  // the odd half of a single key tile
                if (mine) a.part_ml[at] = make_float2(kNone, 0.0f);
                continue;
            }
            // this half's query rows; the last product that read the old rows has completed (b_s)
            constexpr int CH = D / 8, RI = 32 / CH;  // 16-byte chunks of a row; rows per access
            const uint32_t qs = smem_u32(smem + M::Q + h * M::TILE);
            const int64_t q_at = mine ? b * a.q_b + l * a.q_l + head * a.q_h : -1;
            {
                uint4 v[CH];
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int64_t from = __shfl_sync(0xFFFFFFFFu, q_at, i * RI + lane / CH);
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (from >= 0) v[i] = *reinterpret_cast<const uint4 *>(a.q + from + (lane % CH) * 8);
                }
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int r = (warp % 4) * 32 + i * RI + lane / CH, c = lane % CH;
                    st_shared_v4(qs + (c / 8) * 16384 + r * 128 + (((c % 8) ^ (r & 7)) << 4), v[i].x, v[i].y, v[i].z, v[i].w);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&b_q[h]);

            const int limit = s.pre ? s.len : s.len - a.Lq + 1 + l;
            const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
            float m = kNone, sum = 0.0f;
            for (int j = 0; j < n; ++j, ++sn) {
                const int half = j & 1, kt = (s.tile0 + (s.single ? 2 * (j / 2) + h : j / 2)) * 128;  // S of the tile; the tile's first key
                const int k0 = kt + half * 64;
                const uint32_t ts = tm + half * 64;
                if (!(ok = wait(&b_s[h][half], sn / 2))) break;  // sn is even at the start of a segment
                tc_fence_after();
                uint32_t x[64];
                tmem_ld32(ts, x);
                tmem_ld32(ts + 32, x + 32);
                tmem_wait_ld();
                if (k0 + 64 > limit) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (k0 + c >= limit) x[c] = 0xFF800000u;
                }
                __syncwarp();
                float top = kNone, top1 = kNone;
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    top = fmaxf(top, __uint_as_float(x[c]));
                    top1 = fmaxf(top1, __uint_as_float(x[c + 1]));
                }
                top = fmaxf(top, top1);
                top = top == kNone ? kNone : top * a.scale_log2;
                const bool raise = top > m + 8.0f;
                const float to = raise ? top : m, f = raise ? ex2(m - top) : 1.0f;
                if (j > 0 && __any_sync(0xFFFFFFFFu, raise)) {
                    if (!(ok = wait(&b_o[h], sn - 1))) break;  // O is still
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 8) {
                        uint32_t o[8];
                        tmem_ld8(tm + 128 + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st8(tm + 128 + c, o);
                    }
                }
                m = to;
                sum *= f;
                float2 add = make_float2(0.0f, 0.0f), add1 = add;
                const float2 minus = make_float2(-m, -m);
                uint32_t p[32];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 y0 = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale2, minus);
                    const float2 y1 = fma2(make_float2(__uint_as_float(x[2 * e + 2]), __uint_as_float(x[2 * e + 3])), scale2, minus);
                    const float2 p0 = make_float2(ex2(y0.x), ex2(y0.y)), p1 = make_float2(ex2(y1.x), ex2(y1.y));
                    add = add2(add, p0);
                    add1 = add2(add1, p1);
                    const __nv_bfloat162 b0 = __floats2bfloat162_rn(p0.x, p0.y), b1 = __floats2bfloat162_rn(p1.x, p1.y);
                    p[e] = *reinterpret_cast<const uint32_t *>(&b0);
                    p[e + 1] = *reinterpret_cast<const uint32_t *>(&b1);
                }
                tmem_st32(ts, p);
                add = add2(add, add1);
                sum += add.x + add.y;
                if (k0 + 64 > s.len) {  // what the cache holds past the segment must not reach O, not even as 0 * NaN
                    const uint32_t vt = 2 * (vc + (uint32_t)(s.single ? 2 * (j / 2) + h : j / 2)) + half, st = vt % kStages;
                    if (!(ok = wait(&b_vfull[st], vt / kStages))) break;
                    if (k0 + t % 64 >= s.len)  // two threads per key
                        for (int c = 0; c < D / 16; ++c)
                            st_shared_v4(smem_u32(smem + M::V + st * M::KV) + (D == 128 ? t / 64 : 0) * 8192 + (t % 64) * 128 +
                                             (D == 128 ? c : (t / 64) * (D / 16) + c) * 16,
                                         0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&b_p[h][half]);
            }
            if (ok) ok = wait(&b_done[h], units++);  // not b_o, which may be one product behind or, with both done, past it
            tc_fence_after();
            // O's rows through this half's Q tile (read for the last time), which holds D / 2 columns of all of them, so that a
            // row leaves in whole pieces: row r's 16-byte chunk c lies at chunk c ^ (r % OC)
            constexpr int OC = D / 8, RO = 32 / OC;  // chunks of a piece; rows per access
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += D / 2) {
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(tm + 128 + c0 + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        st_shared_v4(qs + t * (OC * 16) + (((c / 4 + e) ^ (t % OC)) << 4), o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
                __syncwarp();
#pragma unroll 8
                for (int i = 0; i < OC; ++i) {
                    const int from = i * RO + lane / OC, r = (warp % 4) * 32 + from;
                    const int64_t to = __shfl_sync(0xFFFFFFFFu, mine ? at : (int64_t)-1, from);
                    const uint4 v = ld_shared_v4(qs + r * (OC * 16) + (((lane % OC) ^ (r % OC)) << 4));
                    if (to >= 0) *reinterpret_cast<uint4 *>(a.part_o + to * D + c0 + (lane % OC) * 4) = v;
                }
                __syncwarp();
            }
            if (mine) a.part_ml[at] = make_float2(m, sum);
            tc_fence_before();
            // the next rows of Q go where other warps' O may still lie; the half's warps leave together
            ok = named_bar_and(1 + h, 128, ok);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        const uint64_t until = globaltimer_ns() + limit_ns;
        while (!mbar_try_wait(&b_end, 0) && globaltimer_ns() < until) {
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The cache [segments, T, Hkv, D] as (64 columns, token, column block, kv head, segment): a box of 64 tokens of one head
// lands as D / 64 blocks of 64 tokens x 64 columns.
bool make_map(CUtensorMap *m, const void *base, int64_t D, int64_t Hkv, int64_t T, int64_t n, int64_t s_h, int64_t s_t, int64_t s_n)
{
    const auto fn = encode_fn();
    if (!fn) return false;
    const auto bytes = [](int64_t stride, int64_t size) { return (cuuint64_t)(size == 1 ? 128 : stride * 2); };  // unused: any
    const cuuint64_t dims[5] = {64, (cuuint64_t)T, (cuuint64_t)(D / 64), (cuuint64_t)Hkv, (cuuint64_t)n};
    const cuuint64_t strides[4] = {bytes(s_t, T), 128, bytes(s_h, Hkv), bytes(s_n, n)};
    const cuuint32_t box[5] = {64, 64, (cuuint32_t)(D / 64), 1, 1}, es[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const Args &a, const Maps &maps, cudaStream_t s, bool chain)
{
    constexpr size_t smem = Smem<D>::TOTAL + 1024;
    static OncePerDevice once;
    const cudaError_t e = allow_smem(once, rows128_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    return launch_k(rows128_kernel<D>, dim3((unsigned)a.grid_tc), dim3(kThreads), smem, s, chain, maps, a, error_word());
}

}  // namespace

bool tc_maps(const Args &a, int64_t D, void *out)
{
    Maps *m = static_cast<Maps *>(out);
    return (!a.p_tc || (make_map(&m->kp, a.kp, D, a.Hkv, a.P, a.n_prefix, a.kp_h, a.kp_t, a.kp_g) &&
                        make_map(&m->vp, a.vp, D, a.Hkv, a.P, a.n_prefix, a.vp_h, a.vp_t, a.vp_g))) &&
           (!a.s_tc || (make_map(&m->ks, a.ks, D, a.Hkv, a.S, a.B, a.ks_h, a.ks_t, a.ks_b) &&
                        make_map(&m->vs, a.vs, D, a.Hkv, a.S, a.B, a.vs_h, a.vs_t, a.vs_b)));
}

cudaError_t tc_launch(const Args &a, int64_t D, const void *maps, cudaStream_t s, bool chain)
{
    const Maps &m = *static_cast<const Maps *>(maps);
    return D == 128 ? launch<128>(a, m, s, chain) : launch<64>(a, m, s, chain);
}

}  // namespace attn
}  // namespace qerl
