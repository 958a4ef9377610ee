// Rows of the quantized key-value cache: a head row of D channels of one token is held as
//   int8: codes c = rint(x * fp32(127 / m)), one fp32 scale s = fp32(m / 127), m = max(max|x|, 2^-100);
//   fp4:  E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) of x / s, half to even and at most 6, with
//         one scale s = 2^e per 32 channels, held as the byte e + 127: the smallest e with 6 * 2^e >= max|x|, kept
//         where every value is exact and finite in the element type.
// A row (fp4: 32 channels) that is not finite has codes 0 and a NaN scale (byte 255): it reads as NaN.
#pragma once

#include "decode_core.h"

namespace w4a4 {

// exponent bytes that a scale is kept between: 0.5 * 2^lo is the type's smallest number or above it, 6 * 2^hi
// below its largest (bf16's lower end is far above its smallest number, which matrix products may flush)
template <int DT> struct Fp4Range { static constexpr int LO = 127 - 23, HI = 127 + 13; };
template <> struct Fp4Range<W4A4_BF16> { static constexpr int LO = 127 - 100, HI = 127 + 125; };

template <int CTRL> __device__ __forceinline__ uint32_t dpp_max(uint32_t x)
{
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true));
}

// Maximum over LH neighbouring lanes (a power of two, 4 to 32), in every lane.
template <int LH> __device__ __forceinline__ uint32_t max_lanes(uint32_t x)
{
    x = dpp_max<0xB1>(x);
    x = dpp_max<0x4E>(x);
    if (LH >= 8) x = dpp_max<0x141>(x);
    if (LH >= 16) x = dpp_max<0x140>(x);
    if (LH >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = max((uint32_t)p[0], (uint32_t)p[1]);
    }
    return x;
}

// magnitude bits of the largest of eight packed 16-bit elements
__device__ __forceinline__ uint32_t max_abs8(const u4_t &x)
{
    typedef uint16_t s2_t __attribute__((ext_vector_type(2)));
    s2_t m = __builtin_bit_cast(s2_t, x[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(s2_t, x[i] & 0x7FFF7FFFu));
    return max((uint32_t)m.x, (uint32_t)m.y);
}

// byte I of c becomes the codes of two packed 16-bit elements over s, half to even and at most 6 (gfx950's own
// conversion)
template <int DT, int I> __device__ __forceinline__ uint32_t narrow4(uint32_t c, uint32_t x, float s)
{
    if constexpr (DT == W4A4_BF16)
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(b2_t, x), s, I);
    else
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(h2_t, x), s, I);
}

// Codes of a lane's eight channels (two dwords in int8, one in fp4) and the scale of its head or block, which
// every lane of it gets. LH lanes hold a head; lanes past its last channel repeat others or hold zeros.
template <int F> struct QuantRun {
    uint32_t codes[F == W4A4_KV_INT8 ? 2 : 1];
    uint32_t scale;  // fp32 bits, or the exponent byte
};

template <int DT, int F, int LH> __device__ __forceinline__ QuantRun<F> quant_run(const u4_t &x)
{
#pragma clang fp contract(off)
    constexpr uint32_t ONES = DT == W4A4_BF16 ? 0x7F80u : 0x7C00u;
    QuantRun<F> q;
    const uint32_t top = max_lanes<F == W4A4_KV_INT8 ? LH : 4>(max_abs8(x));
    const bool finite = top < ONES;
    const float m = unpack16<DT>(top).x;
    if constexpr (F == W4A4_KV_INT8) {
        const float mm = fmaxf(m, 0x1p-100f), r = 127.0f / mm;
        q.scale = finite ? __builtin_bit_cast(uint32_t, mm / 127.0f) : 0x7FC00000u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f2_t f = unpack16<DT>(x[2 * h + i]);
                // adding 1.5 * 2^23 leaves rint of the rounded product in the low bits. The product is rounded by
                // itself, so that one that is half an integer in exact arithmetic is one here, too, and goes to even
                // whichever way r was rounded.
                const float px = f.x * r, py = f.y * r;
                c[2 * i] = __builtin_bit_cast(uint32_t, px + 12582912.0f);
                c[2 * i + 1] = __builtin_bit_cast(uint32_t, py + 12582912.0f);
            }
            const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u);
            const uint32_t hi = __builtin_amdgcn_perm(c[3], c[2], 0x04000C0Cu);
            q.codes[h] = finite ? lo | hi : 0u;
        }
    } else {
        const uint32_t up = ((__builtin_bit_cast(uint32_t, m) + 0x3FFFFFu) >> 23);  // above 1.5 * 2^n: the next n
        const int e = min(max((int)up - 2, Fp4Range<DT>::LO), Fp4Range<DT>::HI);
        const float s = __builtin_bit_cast(float, (uint32_t)e << 23);
        uint32_t c = 0;
        c = narrow4<DT, 0>(c, x[0], s);
        c = narrow4<DT, 1>(c, x[1], s);
        c = narrow4<DT, 2>(c, x[2], s);
        c = narrow4<DT, 3>(c, x[3], s);
        q.codes[0] = finite ? c : 0u;
        q.scale = finite ? (uint32_t)e : 255u;
    }
    return q;
}

// Place of one token in the cache: page < 0: not kept.
struct KvSlot {
    int64_t page;
    int at;  // offset inside the page
};

__device__ __forceinline__ KvSlot kv_slot(const KvPages &c, int64_t s)
{
    if (s < 0 || s >= (int64_t)c.num_pages * c.page_size) return {-1, 0};
    return {s >> c.page_shift, (int)(s & (c.page_size - 1))};
}

// The run of channels d .. d + 7 of head h into the arrays of keys or of values. `first`: this lane is the one
// that writes the scale of its head or block.
template <int F>
__device__ __forceinline__ void quant_store(const KvPages &c, uint8_t *codes, void *scale, const KvSlot &s, int h, int D,
                                            int d, const QuantRun<F> &q)
{
    const int64_t row = (int64_t)h * c.page_size + s.at;
    if constexpr (F == W4A4_KV_INT8) {
        *reinterpret_cast<u2_t *>(codes + s.page * c.page_stride + row * D + d) = u2_t{q.codes[0], q.codes[1]};
        if (d == 0) reinterpret_cast<uint32_t *>(scale)[s.page * c.scale_stride + row] = q.scale;
    } else {
        *reinterpret_cast<uint32_t *>(codes + s.page * c.page_stride + row * (D / 2) + d / 2) = q.codes[0];
        if (d % 32 == 0)
            reinterpret_cast<uint8_t *>(scale)[s.page * c.scale_stride +
                                               ((int64_t)h * (D / 32) + d / 32) * c.page_size + s.at] = (uint8_t)q.scale;
    }
}

}  // namespace w4a4
