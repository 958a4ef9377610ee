// Device helpers shared by the kernels of the single-token path: 16-bit packing, reductions over lanes, the
// tiles of a sequence's visible keys and the 16 x 16 x 32 matrix product.
#pragma once

#include "w4a4_internal.h"

namespace w4a4 {

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef __bf16 b8_t __attribute__((ext_vector_type(8)));
typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

// two fp32 values rounded to the 16-bit type, low value first, and back
template <int DT> __device__ __forceinline__ uint32_t pack16(float a, float b)
{
    if constexpr (DT == W4A4_BF16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2_t{a, b}, b2_t));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2_t{a, b}, h2_t));
}

template <int DT> __device__ __forceinline__ f2_t unpack16(uint32_t w)
{
    if constexpr (DT == W4A4_BF16)
        return f2_t{__builtin_bit_cast(float, w << 16), __builtin_bit_cast(float, w & 0xFFFF0000u)};
    else
        return __builtin_convertvector(__builtin_bit_cast(h2_t, w), f2_t);
}

// Eight consecutive 16-bit elements from and to any element's address: the hardware's vector accesses
// take them all.
typedef uint32_t any4_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t any2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef float anyf4_t __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ u4_t load8_any(const uint16_t *p) { return *reinterpret_cast<const any4_t *>(p); }
__device__ __forceinline__ void store8_any(uint16_t *p, const u4_t &v) { *reinterpret_cast<any4_t *>(p) = v; }

// Sum over LH neighbouring lanes (a power of two), in every lane.
template <int CTRL> __device__ __forceinline__ float dpp_add(float x)
{
    const int y = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true);
    return x + __builtin_bit_cast(float, y);
}

template <int LH> __device__ __forceinline__ float sum_lanes(float x)
{
    x = dpp_add<0xB1>(x);                       // quad_perm: lane ^ 1
    x = dpp_add<0x4E>(x);                       // quad_perm: lane ^ 2
    if (LH >= 8) x = dpp_add<0x141>(x);         // row_half_mirror: the other quad of eight
    if (LH >= 16) x = dpp_add<0x140>(x);        // row_mirror: the other half of sixteen
    if (LH >= 32) {
        const uint32_t u = __builtin_bit_cast(uint32_t, x);
        const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        x = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
    }
    if (LH >= 64) {
        const uint32_t u = __builtin_bit_cast(uint32_t, x);
        const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        x = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
    }
    return x;
}

// Tiles of 32 keys that hold something visible: tiles [0, ns) and from w0 on, T in all.
struct AttnTiles {
    int ns, w0, T;
    bool over;  // longer than the table can say: poisoned, one logical tile
};

__device__ __forceinline__ AttnTiles attn_tiles(int n, const AttnArgs &a)
{
    AttnTiles t{0, 0, 0, false};
    if (n <= 0) return t;
    if ((int64_t)n > (int64_t)a.table_width * a.page_size) {
        t.over = true;
        t.T = 1;
        return t;
    }
    const int all = (int)(((int64_t)n + 31) >> 5);
    if (a.window > 0 && (int64_t)n > (int64_t)a.window + a.sinks) {
        t.ns = (a.sinks + 31) >> 5;
        t.w0 = max((n - a.window) >> 5, t.ns);
    }
    t.T = t.ns + all - t.w0;
    return t;
}

template <int DT> __device__ __forceinline__ f4_t mma32(const u4_t &a, const u4_t &b, const f4_t &c)
{
    if constexpr (DT == W4A4_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a),
                                                      __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8_t, a),
                                                       __builtin_bit_cast(b8_t, b), c, 0, 0, 0);
}

// combine the four 16-lane groups of a wave: every lane gets the result over lanes l, l^16, l^32, l^48
template <typename F> __device__ __forceinline__ float across_groups(float x, F f)
{
    uint32_t u = __builtin_bit_cast(uint32_t, x);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = f(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
    u = __builtin_bit_cast(uint32_t, x);
    auto b = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return f(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}

constexpr int ATTN_WAVES = 4;   // waves of a workgroup, or one where there is little to do
constexpr int ATTN_PAD = 4;     // floats between the heads' rows in LDS, against bank conflicts

// Orders one wave's LDS writes and reads of other lanes' data (the hardware keeps a wave's LDS accesses in order; this
// keeps the compiler from moving them).
__device__ __forceinline__ void lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// N dwords from a 4-byte aligned address
template <int N> struct __attribute__((aligned(4))) DwordRun {
    uint32_t v[N];
};

}  // namespace w4a4
