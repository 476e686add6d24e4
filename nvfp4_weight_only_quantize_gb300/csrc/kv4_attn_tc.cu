// Attention parts of many query rows over 4-bit caches on tcgen05: the schedule,
// the parts and the softmax of the bf16 kernel (prefix_attn.cuh, prefix_attn_tc.cu),
// with warps that dequantise where that one has TMA loads.
//
// Warps 0-3 and 4-7: the softmax of the two halves, one thread per row; 8 and 9 write
// the keys, 10 and 11 the values of a tile of 64 (a cache tile of 32 tokens each); 12
// and 13 the MMAs of the two halves.
//   Q     bf16 -> fp16 after a power of two per row (as in kv4_attn.cu), once per unit;
//   K, V  code times scale in fp16, exact; the next tile's codes are in registers
//         before the last one's are written;
//   V     K-major, its transpose as the cache holds it: eight tokens of a dim are a
//         16-byte piece of a row of the swizzled tile;
//   P     fp16, between 2^8 and 2^15 for a row's largest, so that keys of up to 15 nats less keep all of fp16's digits.
// 129 tokens of eight sequences, 16 heads, over a prefix of 4001 keys and their own: 72 us
// with the join (the tiles of eight rows: 405 us); 28 heads of 64 sequences over 16384
// keys, the own tokens beside it, 51 to 56 us (126 us).  Tensor pipe 22 % over the run, issue
// 34 %: a step's softmax, products and the arrival of its operands follow one another as
// in the bf16 kernel; HBM is idle (6 MB).  As many new tokens as keys: eight sequences of
// 1000, 16 heads, 178 us (140 at D = 64), one of 4000, 28 heads, 318 us; every key tile runs
// for every row tile, twice what the rows see.
#include <cuda.h>

#include "kv4_attn.cuh"
#include "prefix_attn.cuh"
#include "sm100_ptx.cuh"

namespace qerl {
namespace kv4 {
namespace {

using namespace ptx;
using attn::Args;
using attn::key_tiles;
using attn::kStart;
using attn::line_length;
using attn::prefix_len;
using attn::segment_steps;
using attn::steps_per_cta;
using attn::suffix_len;
using attn::Units;

constexpr int kThreads = 448, kProducer = 8, kMmaWarp = 12;  // the MMA warps are two
constexpr int kStages = 4;  // tiles of 64 keys: K and V each
constexpr float kHead = 8.0f, kRoom = 15.0f;  // m is set kHead below a maximum, and raised above kRoom

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
// A and B fp16, D FP32, both K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

// The raw share of a lane in a cache tile, and where it goes.  Nothing of a tile past the segment is read.
template <int D>
struct RawK {  // keys 8 i + lane % 8, dims D / 4 q .., q = lane / 8
    static constexpr int W = D / 32;
    uint32_t w[4][W], s[4];
    __device__ __forceinline__ void load(const uint8_t *tile)
    {
        const int lane = threadIdx.x % 32, q = lane / 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = 8 * i + lane % 8;
            if (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4 *>(tile + Tile<D>::k_word(key, 4 * q));
                w[i][0] = v.x, w[i][1] = v.y, w[i][W - 2] = v.z, w[i][W - 1] = v.w;
                s[i] = *reinterpret_cast<const uint16_t *>(tile + Tile<D>::k_scale(key, 2 * q));
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(tile + Tile<D>::k_word(key, 2 * q));
                w[i][0] = v.x, w[i][1] = v.y;
                s[i] = tile[Tile<D>::k_scale(key, q)];
            }
        }
    }
    __device__ __forceinline__ void store(uint32_t to, int half) const  // rows of 64 dims, blocks of 64 rows
    {
        const int lane = threadIdx.x % 32, q = lane / 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = half * 32 + 8 * i + lane % 8;
            uint32_t s0, s1;
            scales_f16(s[i], s0, s1);
#pragma unroll
            for (int x = 0; x < W; ++x) {
                uint32_t v[4];
                codes_f16(w[i][x], v);
                const uint32_t f = prmt(s0, 0, x < 2 ? 0x1010 : 0x3232);
                const int c = q * W + x;
                st_shared_v4(to + (c / 8) * 8192 + row * 128 + (((c % 8) ^ (row & 7)) << 4), f16x2_mul(v[0], f), f16x2_mul(v[1], f), f16x2_mul(v[2], f),
                             f16x2_mul(v[3], f));
            }
        }
    }
};
template <int D>
struct RawV {  // tokens 8 q .. of dims 32 j + 8 i + r; a quarter of a warp has q = 0 .. 3 and r, r + 4: eight pieces, eight banks
    static constexpr int J = D / 32;
    uint4 w[J], s[J];
    static __device__ __forceinline__ int r() { return ((threadIdx.x >> 2) & 1) * 4 + threadIdx.x % 32 / 8; }
    __device__ __forceinline__ void load(const uint8_t *tile)
    {
        const int q = threadIdx.x % 4;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            w[j] = *reinterpret_cast<const uint4 *>(tile + Tile<D>::VC + (j * 32 + r() * 4 + q) * 16);
            s[j] = *reinterpret_cast<const uint4 *>(tile + Tile<D>::VS + (q * (D / 16) + 2 * j) * 8);
        }
    }
    // rows of 64 tokens; `keys` of the tile's 32 are the segment's: the others' scales may be anything, and become 0
    __device__ __forceinline__ void store(uint32_t to, int half, int keys) const
    {
        const int q = threadIdx.x % 4, n = max(0, min(8, keys - 8 * q));
        const uint64_t mask = n == 8 ? ~uint64_t(0) : (uint64_t(1) << (8 * n)) - 1;
        const uint32_t m0 = (uint32_t)mask, m1 = (uint32_t)(mask >> 32);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t word[4] = {w[j].x, w[j].y, w[j].z, w[j].w}, scale[4] = {s[j].x & m0, s[j].y & m1, s[j].z & m0, s[j].w & m1};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t v[4], f[4];
                codes_f16(word[i], v);
                scales_f16(scale[i / 2 * 2], f[0], f[1]);
                scales_f16(scale[i / 2 * 2 + 1], f[2], f[3]);
                const int d = j * 32 + 8 * i + r(), c = half * 4 + q;
                st_shared_v4(to + d * 128 + ((c ^ (d & 7)) << 4), f16x2_mul(v[0], f[0]), f16x2_mul(v[1], f[1]), f16x2_mul(v[2], f[2]), f16x2_mul(v[3], f[3]));
            }
        }
    }
};

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
__global__ void __launch_bounds__(kThreads, 1) many_rows_kernel(const __grid_constant__ Args a, const __grid_constant__ Cache pre_cache, const __grid_constant__ Cache suf_cache, float pre_scale,
                     float suf_scale, unsigned int *err)
{
    using M = Smem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // the swizzled tiles' alignment
    __shared__ uint64_t b_q[2], b_kfull[kStages], b_kempty[kStages], b_vfull[kStages], b_vempty[kStages], b_s[2][2], b_p[2][2], b_o[2], b_done[2], b_end;
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    __shared__ int s_up[2][128];  // the power of two that a row of Q was divided by
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int k = 0; k < kStages; ++k) {
            mbar_init(&b_kfull[k], 2);  // both producer warps
            mbar_init(&b_kempty[k], 2);  // both MMA warps
            mbar_init(&b_vfull[k], 2);
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

    if (warp >= kProducer && warp < kMmaWarp) {
        const bool keys = warp < kProducer + 2;
        const int half = warp % 2;  // which cache tile of the two
        uint64_t *const full = keys ? b_kfull : b_vfull, *const empty = keys ? b_kempty : b_vempty;
        uint8_t *const ring = smem + (keys ? M::K : M::V);
        Seg s = {};
        int t = -1, tiles = 0, pos = begin;
        // the next tile of 64 keys, over the CTA's ranges
        const auto next = [&]() -> bool {
            for (++t; t >= tiles; t = 0) {
                if (pos >= end) return false;
                s = locate(pos);
                pos = s.next;
                tiles = 2 * (s.single ? s.n0 + s.n1 : s.n0);
            }
            return true;
        };
        const auto source = [&]() -> const uint8_t * {
            const Cache &c = s.pre ? pre_cache : suf_cache;
            return c.data + s.seg * c.s_n + s.hk * c.s_h + (s.tile0 * 4 + t * 2 + half) * c.s_t;
        };
        const auto left = [&]() { return s.len - (s.tile0 * 128 + t * 64 + half * 32); };  // keys of the segment from this cache tile on
        const auto run = [&](auto raw, auto write) {
            bool more = next();
            int n = more ? left() : 0;
            if (n > 0) raw.load(source());
            for (uint32_t it = 0; more; ++it) {
                const uint32_t st = it % kStages, round = it / kStages;
                if (round > 0 && !wait(&empty[st], round - 1)) break;
                write(raw, smem_u32(ring + st * M::KV), n);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[st]);
                more = next();
                n = more ? left() : 0;
                if (n > 0) raw.load(source());
            }
        };
        if (keys) {
            RawK<D> raw = {};
            run(raw, [&](const RawK<D> &r, uint32_t to, int) { r.store(to, half); });  // keys past the segment are masked in S
        } else {
            RawV<D> raw = {};
            run(raw, [&](const RawV<D> &r, uint32_t to, int n) { r.store(to, half, n); });
        }
    } else if (warp >= kMmaWarp) {
        const int h = warp - kMmaWarp;
        const uint32_t id_qk = idesc_f16_f32(128, 64), id_pv = idesc_f16_f32(128, D);
        const uint32_t d_s = tmem + h * 256, d_o = d_s + 128;
        const uint64_t q_desc = desc_kmajor_sw128(smem_u32(smem + M::Q + h * M::TILE)), k_desc = desc_kmajor_sw128(smem_u32(smem + M::K)),
                       v_desc = desc_kmajor_sw128(smem_u32(smem + M::V));
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
                    for (int kk = 0; kk < 4; ++kk)  // 16 keys
                        umma_bf16_ts(d_o, d_s + half * 64 + 8 * kk, vd + (uint64_t)(2 * kk), id_pv, j > 0 || kk > 0);
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
        bool ok = true;
        for (int pos = begin; ok && pos < end;) {
            const Seg s = locate(pos);
            pos = s.next;
            const int n = 2 * (h ? s.n1 : s.n0), R = (s.pre ? a.G : 1) * a.Lq * a.gs;
            if (s.n0 == 0) continue;
            const int rr = (s.single ? 2 * s.pair : 2 * s.pair + h) * 128 + t, rows_b = a.Lq * a.gs;
            const bool mine = rr < R;
            const int bi = rr / rows_b, in = rr - bi * rows_b, l = in / a.gs;
            const int b = s.pre ? s.seg * a.G + bi : s.seg, head = s.hk * a.gs + in - l * a.gs;
            const int64_t at = (((int64_t)b * a.Lq + l) * a.Hq + head) * (a.n_pp + a.n_sp) + (s.pre ? 0 : a.n_pp) +
                               (s.single ? 2 * s.part + h : s.part);
            if (n == 0) {  // the odd half of a single key tile
                if (mine) a.part_ml[at] = make_float2(attn::kNone, 0.0f);
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
                    const auto mag = [](uint32_t x) { return max(x & 0x7FFFu, x >> 16 & 0x7FFFu); };
                    uint32_t top = max(max(mag(v[i].x), mag(v[i].y)), max(mag(v[i].z), mag(v[i].w)));
#pragma unroll
                    for (int o = 1; o < CH; o *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    const int e = min(max((int)(top >> 7) - 127, -126), 126);  // the row's largest exponent
                    const float down = pow2f(-e);
                    const auto pair = [&](uint32_t x) { return f16x2(bf16lo(x) * down, bf16hi(x) * down); };
                    st_shared_v4(qs + (c / 8) * 16384 + r * 128 + (((c % 8) ^ (r & 7)) << 4), pair(v[i].x), pair(v[i].y), pair(v[i].z), pair(v[i].w));
                    if (c == 0) s_up[h][r] = e;
                }
                __syncwarp();
            }
            fence_proxy_async_smem();
            mbar_arrive(&b_q[h]);

            const int limit = s.pre ? s.len : s.len - a.Lq + 1 + l;
            const float scale = row_scale(s.pre ? pre_scale : suf_scale, s_up[h][t]);
            const float2 scale2 = make_float2(scale, scale);
            float m = attn::kNone, sum = 0.0f;
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
                float top = attn::kNone, top1 = attn::kNone;
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    top = fmaxf(top, __uint_as_float(x[c]));
                    top1 = fmaxf(top1, __uint_as_float(x[c + 1]));
                }
                top = fmaxf(top, top1);
                top = top == attn::kNone ? attn::kNone : top * scale;
                const bool raise = top > m + kRoom;
                const float to = raise ? top - kHead : m, f = raise ? attn::ex2(m - to) : 1.0f;
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
                    const float2 p0 = make_float2(attn::ex2(y0.x), attn::ex2(y0.y)), p1 = make_float2(attn::ex2(y1.x), attn::ex2(y1.y));
                    add = add2(add, p0);
                    add1 = add2(add1, p1);
                    p[e] = f16x2(p0.x, p0.y);
                    p[e + 1] = f16x2(p1.x, p1.y);
                }
                tmem_st32(ts, p);
                add = add2(add, add1);
                sum += add.x + add.y;
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

template <int D>
cudaError_t launch(const Args &a, const Side &pre, const Side &suf, cudaStream_t s, bool chain)
{
    constexpr size_t smem = Smem<D>::TOTAL + 1024;
    static OncePerDevice once;
    const cudaError_t e = allow_smem(once, many_rows_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    return launch_k(many_rows_kernel<D>, dim3((unsigned)a.grid_tc), dim3(kThreads), smem, s, chain, a, pre.c, suf.c, pre.scale_log2, suf.scale_log2,
                    error_word());
}

}  // namespace

cudaError_t many_rows(const Args &a, const Side &pre, const Side &suf, int64_t D, cudaStream_t s, bool chain)
{
    return D == 128 ? launch<128>(a, pre, suf, s, chain) : launch<64>(a, pre, suf, s, chain);
}

}  // namespace kv4
}  // namespace qerl
