// The 4-bit key/value cache: keys and values in NVFP4 (E2M1 codes, an E4M3 scale
// per 16 values along the head, one fixed FP32 factor per cache).
//
// A tile holds 32 tokens of one sequence and kv head in 36 D bytes, in one piece,
// so that one bulk copy brings it to shared memory:
//   keys' codes    [32 tokens][D / 2], the even dim of a pair in the low nibble;
//   values' codes  16 D bytes: a word holds eight tokens of one dim (token 8 q + n
//                  in nibble n), because the second product sums over tokens;
//   keys' scales   2 D bytes,  values' scales 2 D bytes.
// Codes and scales lie in the order in which the lanes of a warp take them for
// the tensor core's fragments (lane = 4 r + q): 16 bytes a lane, no bank conflict.
#pragma once

#include "common.cuh"

namespace qerl {
namespace kv4 {

constexpr int kTok = 32;  // tokens of a tile

struct Cache {
    uint8_t *data;
    int64_t s_n, s_h, s_t;  // bytes from sequence to sequence, head to head, tile to tile
    int n, T, Hkv;
    float k_scale, v_scale;
};

template <int D>
struct Tile {
    static constexpr int B = D / 16;  // blocks of a token
    static constexpr int KC = 0, VC = kTok * D / 2, KS = 2 * VC, VS = KS + kTok * B, BYTES = VS + kTok * B;
    // offset of the key word that holds dims 8 w .. 8 w + 7 of token t
    static __device__ __forceinline__ int k_word(int t, int w) { return KC + t * (D / 2) + w * 4; }
    // Offset of the key scale of token t, block b.  Lane (r, q) multiplies tokens 8 (r / 2) + r % 2 + 2 e, e = 0..3, and dims
    // from D / 4 q on.
    static __device__ __forceinline__ int k_scale(int t, int b)
    {
        constexpr int per = D / 64;  // blocks of a lane
        const int r = 2 * (t / 8) + t % 2, e = (t % 8) / 2;
        return KS + ((r * 4 + b / per) * 4 + e) * per + b % per;
    }
    // offset of the word of dim d, tokens 8 q .. 8 q + 7: sixteen dims are a row tile of the product, two of them a 16-byte piece
    static __device__ __forceinline__ int v_word(int d, int q)
    {
        return VC + (((d / 32) * 32 + (d % 8) * 4 + q) * 4 + (d % 32) / 8) * 4;
    }
    static __device__ __forceinline__ int v_scale(int t, int b) { return VS + ((t / 8) * B + b) * 8 + t % 8; }
};

// The four code pairs of a word as fp16 pairs.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&o)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

// What the entry points share: the cache's description checked and taken over.
qerl_status check_cache(const qerl_kv4_cache *c, Cache &out);
// Whether an output of sizes a, b, c along its strides has elements at one address.
inline bool repeated(int64_t a, int64_t b, int64_t c, const int64_t *stride)
{
    return (a > 1 && stride[0] == 0) || (b > 1 && stride[1] == 0) || (c > 1 && stride[2] == 0);
}

}  // namespace kv4
}  // namespace qerl
