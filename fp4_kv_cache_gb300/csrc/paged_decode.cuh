// paged_decode.cuh -- cache rows to bf16, for the paged cache's read and attention.
//
// Decoding a 4-bit code: bits s e e m of a code placed as bf16's sign, two exponent and one
// mantissa bit are the code's value x 2^-126 (subnormals included), so one bf16 product with
// 2^126 x scale gives the exact value (E4M3 codes: x 2^-120).  To save shifts the two values of a
// register are nibbles k and k + 4 of a word: eight channels come in the order 0 4 1 5 2 6 3 7.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "paged.cuh"

namespace csa2 {

// Factors that put a code from the low bits of a half word (from bits 4-7) in its place; see decode.
constexpr uint32_t kCodeAt0 = (1u << 12) + (1u << 6), kCodeAt4 = (1u << 8) + (1u << 2);

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t half)
{
    const __nv_bfloat16 h = __ushort_as_bfloat16((unsigned short)half);
    return __halves2bfloat162(h, h);
}
__device__ __forceinline__ uint32_t mul2(uint32_t v, __nv_bfloat162 m)
{
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v), m);
    return *reinterpret_cast<const uint32_t *>(&x);
}

// N x 8 channels of a row as they lie in the cache, and their scale bytes (NVFP4: two for 32
// channels).  N = 4: a scale block of 32 channels; N = 2: half of one.
template <int FMT, int N>
struct Raw {
    static constexpr int kWords = N * (FMT == CSA2P_BF16 ? 4 : FMT == CSA2P_MXFP8 ? 2 : 1);
    uint32_t w[kWords];
    uint32_t sb;
};

// Bytes of n channels' codes.
template <int FMT>
__device__ __forceinline__ constexpr int code_bytes(int n)
{
    return FMT == CSA2P_BF16 ? 2 * n : FMT == CSA2P_MXFP8 ? n : n / 2;
}

// The 8 N channels whose codes and scale begin there.
template <int FMT, int N>
__device__ __forceinline__ void load_raw(Raw<FMT, N> &r, const uint8_t *codes, const uint8_t *scale)
{
    constexpr int kW = Raw<FMT, N>::kWords;
    if (kW == 2) {
        const uint2 a = *reinterpret_cast<const uint2 *>(codes);
        r.w[0] = a.x;
        r.w[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < kW / 4; ++i) {
            const uint4 a = reinterpret_cast<const uint4 *>(codes)[i];
            r.w[(4 * i) % kW] = a.x;
            r.w[(4 * i + 1) % kW] = a.y;
            r.w[(4 * i + 2) % kW] = a.z;
            r.w[(4 * i + 3) % kW] = a.w;
        }
    }
    if (FMT == CSA2P_BF16) r.sb = 0;
    else if (FMT == CSA2P_NVFP4_E4M3_16 && N == 4) r.sb = *reinterpret_cast<const uint16_t *>(scale);
    else r.sb = *scale;
}
template <int FMT, int N>
__device__ __forceinline__ void zero_raw(Raw<FMT, N> &r)
{
#pragma unroll
    for (int i = 0; i < Raw<FMT, N>::kWords; ++i) r.w[i] = 0u;
    r.sb = FMT == CSA2P_NVFP4_E4M3_16 ? 0u : 127u;
}
// Swaps the two halves of the channels, when `swap`.
template <int FMT, int N>
__device__ __forceinline__ void swap_raw(Raw<FMT, N> &r, bool swap)
{
    constexpr int kH = Raw<FMT, N>::kWords / 2;
#pragma unroll
    for (int i = 0; i < kH; ++i) {
        const uint32_t a = r.w[i], b = r.w[i + kH];
        r.w[i] = swap ? b : a;
        r.w[i + kH] = swap ? a : b;
    }
    if (FMT == CSA2P_NVFP4_E4M3_16 && N == 4) r.sb = swap ? prmt(r.sb, 0u, 0x4401u) : r.sb;
}

// Whether decode is not enough: something is not finite, or one factor cannot hold the scale.
template <int FMT, int N>
__device__ __forceinline__ bool special(const Raw<FMT, N> &r)
{
    constexpr int kW = Raw<FMT, N>::kWords;
    uint32_t e = 0;
    if (FMT == CSA2P_BF16) {
#pragma unroll
        for (int i = 0; i < kW; ++i) e |= (r.w[i] & 0x7f807f80u) + 0x00800080u;
        return (e & 0x80008000u) != 0;
    }
    if (FMT == CSA2P_MXFP8) {
#pragma unroll
        for (int i = 0; i < kW; ++i) e |= (r.w[i] & 0x7f7f7f7fu) + 0x01010101u;
        return (e & 0x80808080u) != 0 || r.sb > 134u;
    }
    if (FMT == CSA2P_NVFP4_E4M3_16) return (((r.sb & 0x7f7fu) + 0x0101u) & 0x8080u) != 0;
    return r.sb > 128u;
}

// N 16-byte pieces (eight channels each, in the order 0 4 1 5 2 6 3 7) of bf16, nothing special
// among them.
//
// 4-bit codes: n = two codes, one in the low bits of each half of a word; n x (2^12 + 2^6) has the
// sign bit in its place and the other three in theirs, with nothing carried between, and one mask
// keeps those.  With the codes 4 bits higher the factor is 2^8 + 2^2.  (The logic unit is what
// bounds the staging; products go to the other one.  The factors come as parameters so that they
// stay products.)
template <int FMT, int N>
__device__ __forceinline__ void decode(const Raw<FMT, N> &r, uint32_t (&v)[4 * N], uint32_t f0, uint32_t f4)
{
    constexpr int kW = Raw<FMT, N>::kWords;
    if (FMT == CSA2P_BF16) {
#pragma unroll
        for (int h = 0; h < N; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[4 * h + 2 * k] = prmt(r.w[(4 * h + k) % kW], r.w[(4 * h + k + 2) % kW], 0x5410u);
                v[4 * h + 2 * k + 1] = prmt(r.w[(4 * h + k) % kW], r.w[(4 * h + k + 2) % kW], 0x7632u);
            }
    } else if (FMT == CSA2P_MXFP8) {
        // code bits as bf16 bits: value x 2^-120; x 2^(120 + sb - 127)
        const __nv_bfloat162 m = bf2((min(r.sb, 134u) + 120u) << 7);
#pragma unroll
        for (int h = 0; h < N; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = prmt(r.w[(2 * h) % kW], r.w[(2 * h + 1) % kW], 0x4400u + 0x1111u * k);
                v[4 * h + k] = mul2((a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), m);
            }
    } else {
        constexpr bool nv = FMT == CSA2P_NVFP4_E4M3_16;
        // E8M0: x 2^(126 + sb - 127); E4M3: x 2^126, then the scale (both products exact)
        const uint32_t mb = nv ? 253u * 0x00800080u : (min(r.sb, 128u) + 126u) * 0x00800080u;
        const __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162 *>(&mb);
#pragma unroll
        for (int h = 0; h < N; ++h) {
            const uint32_t w = r.w[h % kW], z = w >> 8;
            v[4 * h] = mul2(((w & 0x000f000fu) * f0) & 0x81c081c0u, m);
            v[4 * h + 1] = mul2(((w & 0x00f000f0u) * f4) & 0x81c081c0u, m);
            v[4 * h + 2] = mul2(((z & 0x000f000fu) * f0) & 0x81c081c0u, m);
            v[4 * h + 3] = mul2(((z & 0x00f000f0u) * f4) & 0x81c081c0u, m);
        }
        if (nv) {
#pragma unroll
            for (int h = 0; h < N; h += 2) {             // 16 channels share a scale
                const uint32_t sb = r.sb >> (4 * h), bits = ((sb & 0x80u) << 8) | ((sb & 0x7fu) << 4);   // the scale x 2^-120
                const uint32_t sc = mul2(bits | (bits << 16), bf2(247u << 7));
#pragma unroll
                for (int i = 0; i < 8; ++i) v[4 * h + i] = mul2(v[4 * h + i], *reinterpret_cast<const __nv_bfloat162 *>(&sc));
            }
        }
    }
}

// Mends what decode made of special channels, where it has been stored (piece i at column
// col0 ^ 16 i): the rest of the scale in a second product.  Channels that are not finite become
// zeros, and the answer is true; scale bytes that could take a value past float32 (no quantised row
// has them) count as not finite.
template <int FMT, int N>
__device__ __forceinline__ bool mend(const Raw<FMT, N> &r, uint8_t *u, int col0)
{
    constexpr uint32_t held = FMT == CSA2P_MXFP8 ? 134u : 128u, most = FMT == CSA2P_MXFP8 ? 246u : 252u;
    bool bad = true;
    if (FMT == CSA2P_MXFP4) bad = r.sb > most;
    if (FMT == CSA2P_MXFP8) {
        uint32_t e = 0;
#pragma unroll
        for (int i = 0; i < Raw<FMT, N>::kWords; ++i) e |= (r.w[i] & 0x7f7f7f7fu) + 0x01010101u;
        bad = (e & 0x80808080u) != 0 || r.sb > most;
    }
    const __nv_bfloat162 rest = bf2((max(r.sb, held) - held + 127u) << 7);
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        uint4 *p = reinterpret_cast<uint4 *>(u + (col0 ^ (16 * i)));
        const uint4 v = *p;
        *p = bad ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(mul2(v.x, rest), mul2(v.y, rest), mul2(v.z, rest), mul2(v.w, rest));
    }
    return bad;
}

} // namespace csa2
