// widen.cuh -- block-scaled codes to bf16 pairs, for products with bf16 activations.
//
// A code's bits are a bf16 value up to a power of two once its exponent and mantissa fields
// are shifted to bf16's: E2M1's two exponent bits and one mantissa bit to bits 8..6 give the
// value times 2^-126, E4M3's to bits 10..4 times 2^-120, E5M2's to bits 11..5 times 2^-112
// (subnormal codes land on subnormal bf16 values: the same linear spacing). One packed
// multiplication by the block scale times that power is then exact: at most 2 + 4 (E2M1 under
// E4M3 scales), 4 or 7 significant bits of bf16's 8. INT8 codes are assembled as 128 + (q &
// 127), from which 128 or 256 is subtracted.
//
// 32 codes of a row are widened at a time (one MX block, two NV blocks).
#pragma once

#include "common.cuh"

namespace bq {

__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// 2^(byte - 127) as a bf16 pair.
__device__ __forceinline__ uint32_t bf2_exp(uint32_t byte) { return (byte ? byte << 7 : 0x40u) * 0x00010001u; }

// Bits of 32 codes as 32-bit words, and the words' raw pairs: raw[0] = (e0, e4), raw[1] =
// (e1, e5), raw[2] = (e2, e6), raw[3] = (e3, e7) of an FP4 word's elements, raw[0] = (e0, e2),
// raw[1] = (e1, e3) of an 8-bit word's. NV values carry a factor 2^-8 (NV_OUT undoes it on the
// finished sums), which keeps their one multiplier inside bf16's range.
template <int FMT, bool NV>
struct Widen {
    static constexpr int WORDS = Fmt<FMT>::four ? 4 : 8;
    static constexpr int RAW = Fmt<FMT>::four ? 4 : 2;          // pairs of a word
    // exponent of the raw bits' missing factor (2^-OFF times the value), and the largest UE8M0
    // byte for which 2^OFF times the scale is a bf16 value
    static constexpr uint32_t OFF = FMT == BQ_FP4_E2M1 ? 126u : FMT == BQ_FP8_E4M3 ? 120u : FMT == BQ_FP8_E5M2 ? 112u : 0u;
    static constexpr uint32_t LIMIT = 254u - OFF;

    static __device__ __forceinline__ void raw(uint32_t v, uint32_t (&r)[RAW])
    {
        if constexpr (FMT == BQ_FP4_E2M1) {
            // a nibble times 2^6 + 2^12 (or 2^2 + 2^8 from bits 4..7) has its magnitude at bits
            // 8..6 and its sign at bit 15, without carries: one multiplication on the FMA pipe
            // and one mask instead of two shifts and two masks
            const uint32_t s = v >> 8;
            r[0] = ((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
            r[1] = ((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
            r[2] = ((s & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
            r[3] = ((s & 0x00F000F0u) * 0x0104u) & 0x81C081C0u;
        } else if constexpr (FMT == BQ_FP8_E4M3) {
            r[0] = ((v << 4) & 0x07F007F0u) | ((v << 8) & 0x80008000u);
            r[1] = ((v >> 4) & 0x07F007F0u) | (v & 0x80008000u);
        } else if constexpr (FMT == BQ_FP8_E5M2) {
            r[0] = ((v << 5) & 0x0FE00FE0u) | ((v << 8) & 0x80008000u);
            r[1] = ((v >> 3) & 0x0FE00FE0u) | (v & 0x80008000u);
        } else {
            const uint32_t s = v >> 8;
            r[0] = bf2_sub((v & 0x007F007Fu) | 0x43004300u, (v & 0x00800080u) | 0x43004300u);
            r[1] = bf2_sub((s & 0x007F007Fu) | 0x43004300u, (s & 0x00800080u) | 0x43004300u);
        }
    }

    // Whether a block's scale and the missing factor are one multiplier.
    static __device__ __forceinline__ bool fits(uint32_t scale) { return OFF == 0 || NV || scale <= LIMIT; }

    // FP8 codes that are no numbers (E4M3: S.1111.111, E5M2: exponent 31) come from NaN in what
    // was quantized. Whether w has none: the addition flips bit 7 of such a byte, and of no other
    // below the first one. (Looking costs the weight gradient 6 % at 4096 tokens x 11008 x 4096,
    // 285 to 301 us, however it is spelt, and 10 % when it is done after the widening.)
    static constexpr bool HAS_NAN = FMT == BQ_FP8_E4M3 || FMT == BQ_FP8_E5M2;
    static constexpr uint32_t BEYOND = FMT == BQ_FP8_E4M3 ? 0x01010101u : 0x04040404u;

    static __device__ __forceinline__ bool numbers(const uint32_t (&w)[WORDS])
    {
        uint32_t any = 0;
        if constexpr (HAS_NAN) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) any |= (w[i] + BEYOND) ^ w[i];
        }
        return (any & 0x80808080u) == 0u;
    }

    // The raw pairs of all words times their blocks' scales. scale: the MX byte, or the two NV
    // bytes (first block's low). one: fits(scale) and numbers(w), or false for any (a warp decides
    // for all its lanes).
    static __device__ __forceinline__ void pairs(const uint32_t (&w)[WORDS], uint32_t scale, bool one,
                                                 uint32_t (&p)[WORDS * RAW])
    {
        if (NV || one) {
            uint32_t m[2];
            if constexpr (NV) {
                // E4M3 bits as bf16: s 2^-120; times 2^119 twice: s 2^118, which times 2^-126 leaves 2^-8
                const uint32_t b = ((scale & 0xFFu) << 4) | ((scale & 0xFF00u) << 12);
                const uint32_t s2 = bf2_mul(bf2_mul(b, 0x7B007B00u), 0x7B007B00u);
                m[0] = __byte_perm(s2, s2, 0x1010);
                m[1] = __byte_perm(s2, s2, 0x3232);
            } else {
                m[0] = m[1] = OFF ? (scale + OFF) * 0x00800080u : bf2_exp(scale);
            }
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                uint32_t r[RAW];
                raw(w[i], r);
#pragma unroll
                for (int j = 0; j < RAW; ++j) p[i * RAW + j] = bf2_mul(r[j], m[i >= WORDS / 2]);
            }
        } else {
            // the missing power and the scale one after the other
            const uint32_t off = (127u + OFF) * 0x00800080u, e = bf2_exp(scale);
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                uint32_t r[RAW];
                raw(w[i], r);
#pragma unroll
                for (int j = 0; j < RAW; ++j) p[i * RAW + j] = bf2_mul(bf2_mul(r[j], off), e);
                if constexpr (HAS_NAN) {
                    // bit 7 of a byte: no number, NaN. All exponent bits make the value Inf or NaN
                    constexpr uint32_t above_inf = FMT == BQ_FP8_E4M3 ? 0x01010101u : 0x03030303u;
                    const uint32_t mag = w[i] & 0x7F7F7F7Fu, s = mag + BEYOND, n = mag + above_inf;
                    p[i * RAW] |= (s & 0x00800080u) * 0xFFu | (n & 0x00800080u) >> 1;
                    p[i * RAW + 1] |= ((s >> 8) & 0x00800080u) * 0xFFu | ((n >> 8) & 0x00800080u) >> 1;
                }
            }
        }
    }

    // Pairs in element order: q[i] = (e[2 i], e[2 i + 1]).
    static __device__ __forceinline__ void in_order(const uint32_t (&p)[WORDS * RAW], uint32_t (&q)[16])
    {
        if constexpr (Fmt<FMT>::four) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[4 * i] = __byte_perm(p[4 * i], p[4 * i + 1], 0x5410);
                q[4 * i + 1] = __byte_perm(p[4 * i + 2], p[4 * i + 3], 0x5410);
                q[4 * i + 2] = __byte_perm(p[4 * i], p[4 * i + 1], 0x7632);
                q[4 * i + 3] = __byte_perm(p[4 * i + 2], p[4 * i + 3], 0x7632);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                q[2 * i] = __byte_perm(p[2 * i], p[2 * i + 1], 0x5410);
                q[2 * i + 1] = __byte_perm(p[2 * i], p[2 * i + 1], 0x7632);
            }
        }
    }
};

constexpr float NV_OUT = 256.0f;

}  // namespace bq
