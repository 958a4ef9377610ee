// One tile of 32 keys and their values in a wave's registers, from a 16-bit or a quantized cache, and the products
// that attention makes of it:
//  - scores^T (16 keys x 16 query rows, twice) = K (A operand, rows straight from the cache) . q^T;
//  - out^T (16 channels x 16 query rows per product) += V^T (A operand) . p (B operand).
// The scores' result layout already is the B operand of a 32-key product if key 4 g + e (e < 4) of the first and of
// the second half of the tile are its k = 8 g + e and 8 g + 4 + e. A lane loads VE neighbouring channels of those
// eight keys and pairs them up; nothing passes through LDS.
// Codes become matrix operands in registers, exactly:
//  - int8: the codes themselves, as 16-bit numbers. A key's scale multiplies its scores and a value's scale its
//    weight, so that neither is rounded; the second product is bf16 for either element type, for weights times scales
//    need fp32's range.
//  - fp4: gfx950's conversion with a scale, whose results are exact in the element type.
#pragma once

#include "kv_quant.h"

namespace w4a4 {

template <int D, int F> struct KvShape {
    static constexpr int ROW = F == W4A4_KV_16BIT ? 2 * D : F == W4A4_KV_INT8 ? D : D / 2;  // bytes of a row
    // keys: NL loads of KW bytes per lane, NR runs of eight channels (RB bytes) in each; load l of lane g starts at
    // byte (4 l + g) KW of the row, so that four lanes read neighbouring bytes
    static constexpr int KW = ROW % 64 == 0 ? 16 : ROW % 32 == 0 ? 8 : 4;
    static constexpr int NL = ROW / (4 * KW), RB = F == W4A4_KV_16BIT ? 16 : F == W4A4_KV_INT8 ? 8 : 4, NR = KW / RB;
    static constexpr int KJ = NL * NR;  // products over D
    // values: VE channels per lane, a power of two where they are codes (lanes past D hold nothing)
    static constexpr int VE = F == W4A4_KV_16BIT ? D / 16 : D <= 64 ? 4 : D <= 128 ? 8 : 16;
    static constexpr int VB = VE * ROW / D;  // bytes
    static_assert(KJ == D / 32 && VE % 2 == 0);
    // first channel of product j's run of lane g
    static __device__ __forceinline__ int channel(int j, int g) { return ((4 * (j / NR) + g) * KW + j % NR * RB) * D / ROW; }
};

// Where a tile's two halves of 16 keys are: page number and first key inside it (both uniform).
struct KvPlace {
    int key0;
    int64_t page[2];
    int at[2];
};

template <int DT, int D, int F> struct KvTile {
    typedef KvShape<D, F> S;
    static constexpr int PDT = F == W4A4_KV_INT8 ? W4A4_BF16 : DT;  // type of the second product
    struct __attribute__((aligned(4))) KRun { uint32_t w[S::KW / 4]; };
    struct __attribute__((aligned(S::VB < 4 ? 2 : 4))) VRun { uint16_t w[S::VB / 2]; };
    typedef typename std::conditional<S::VB == 2, uint16_t, DwordRun<(S::VB + 3) / 4>>::type VLoad;
    KRun k[2][S::NL];
    VLoad v[8];
    float4 ks[2], vs[2];                // int8: scales of keys 4 g + e
    uint32_t kb[2][S::NL], vb[2];       // fp4: a key's scale byte, the value scale bytes of keys 4 g + e

    __device__ __forceinline__ void load(const KvPages &c, const KvPlace &p, int kvh, int lane)
    {
        const int r = lane & 15, g = lane >> 4;
        const uint32_t koff = r * S::ROW + g * S::KW;
        const uint32_t vch = S::VE * r < D ? S::VE * r : 0, voff = 4 * g * S::ROW + vch * S::ROW / D;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int64_t row = (int64_t)kvh * c.page_size + p.at[hf];
            const uint8_t *kp = c.k + p.page[hf] * c.page_stride + row * S::ROW;
#pragma unroll
            for (int l = 0; l < S::NL; ++l)
                k[hf][l] = *reinterpret_cast<const KRun *>(kp + l * 4 * S::KW + koff);
            if constexpr (F == W4A4_KV_INT8)
                ks[hf] = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(c.k_scale) +
                                                          p.page[hf] * c.scale_stride + row)[g];
            if constexpr (F == W4A4_KV_FP4) {
                const uint8_t *sp = reinterpret_cast<const uint8_t *>(c.k_scale) + p.page[hf] * c.scale_stride +
                                    ((int64_t)kvh * (D / 32)) * c.page_size + p.at[hf];
#pragma unroll
                for (int l = 0; l < S::NL; ++l) kb[hf][l] = sp[S::channel(l * S::NR, g) / 32 * c.page_size + r];
            }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int64_t row = (int64_t)kvh * c.page_size + p.at[hf];
            const uint8_t *vp = c.v + p.page[hf] * c.page_stride + row * S::ROW;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * hf + e] = *reinterpret_cast<const VLoad *>(vp + e * S::ROW + voff);
            if constexpr (F == W4A4_KV_INT8)
                vs[hf] = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(c.v_scale) +
                                                          p.page[hf] * c.scale_stride + row)[g];
            if constexpr (F == W4A4_KV_FP4)
                vb[hf] = *reinterpret_cast<const uint32_t *>(
                    reinterpret_cast<const uint8_t *>(c.v_scale) + p.page[hf] * c.scale_stride +
                    ((int64_t)kvh * (D / 32) + vch / 32) * c.page_size + p.at[hf] + 4 * g);
        }
    }

    static __device__ __forceinline__ float byte_scale(uint32_t b) { return __builtin_bit_cast(float, b << 23); }
    static __device__ __forceinline__ float code8(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }
    template <int I> static __device__ __forceinline__ uint32_t widen4(uint32_t w, float s)
    {
        if constexpr (DT == W4A4_BF16)
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, I));
        else
            return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, I));
    }

    // A operand of product j of half hf: eight channels of key r
    __device__ __forceinline__ u4_t key(int hf, int j) const
    {
        const uint32_t *w = k[hf][j / S::NR].w + j % S::NR * (S::RB / 4);
        if constexpr (F == W4A4_KV_16BIT) {
            return u4_t{w[0], w[1], w[2], w[3]};
        } else if constexpr (F == W4A4_KV_FP4) {
            const float s = byte_scale(kb[hf][j / S::NR]);
            return u4_t{widen4<0>(w[0], s), widen4<1>(w[0], s), widen4<2>(w[0], s), widen4<3>(w[0], s)};
        } else {
            u4_t o;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (DT == W4A4_F16) {  // 0x6400 | u is 1024 + u; u = code + 128
                    const uint32_t u = w[h] ^ 0x80808080u;
                    const h2_t b = {(_Float16)1152.0f, (_Float16)1152.0f};
                    o[2 * h] = __builtin_bit_cast(
                        uint32_t, __builtin_bit_cast(h2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - b);
                    o[2 * h + 1] = __builtin_bit_cast(
                        uint32_t, __builtin_bit_cast(h2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - b);
                } else {
                    o[2 * h] = pack16<DT>(code8(w[h], 0), code8(w[h], 1));
                    o[2 * h + 1] = pack16<DT>(code8(w[h], 2), code8(w[h], 3));
                }
            }
            return o;
        }
    }

    __device__ __forceinline__ uint32_t vword(int e, int i) const  // dword i of key e's run
    {
        if constexpr (S::VB == 2) return v[e];
        else return v[e].v[i];
    }

    // what is not visible must not count, whatever it holds: ok bit e of the lane's eight keys
    __device__ __forceinline__ void hide_values(const bool (&ok)[8])
    {
        if constexpr (F == W4A4_KV_16BIT) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int i = 0; i < S::VB / 4; ++i) v[e].v[i] = ok[e] ? v[e].v[i] : 0u;
        } else if constexpr (F == W4A4_KV_FP4) {  // any code is finite: the scale becomes 1
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t m = 0xFFu << (8 * (e % 4));
                vb[e / 4] = ok[e] ? vb[e / 4] : (vb[e / 4] & ~m) | (m & 0x7F7F7F7Fu);
            }
        } else {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                vs[hf].x = ok[4 * hf] ? vs[hf].x : 0.0f;
                vs[hf].y = ok[4 * hf + 1] ? vs[hf].y : 0.0f;
                vs[hf].z = ok[4 * hf + 2] ? vs[hf].z : 0.0f;
                vs[hf].w = ok[4 * hf + 3] ? vs[hf].w : 0.0f;
            }
        }
    }

    // A operands of the lane's channels 2 i and 2 i + 1: their eight keys
    __device__ __forceinline__ void values(int i, u4_t &even, u4_t &odd) const
    {
        if constexpr (F == W4A4_KV_INT8) {
            const int w = i / 2, b = i % 2 * 2;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                even[e] = pack16<PDT>(code8(vword(2 * e, w), b), code8(vword(2 * e + 1, w), b));
                odd[e] = pack16<PDT>(code8(vword(2 * e, w), b + 1), code8(vword(2 * e + 1, w), b + 1));
            }
        } else {
            uint32_t x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (F == W4A4_KV_16BIT) {
                    x[e] = vword(e, i);
                } else {
                    const float s = byte_scale((vb[e / 4] >> (8 * (e % 4))) & 0xFFu);
                    const uint32_t w = vword(e, i / 4);
                    x[e] = i % 4 == 0 ? widen4<0>(w, s) : i % 4 == 1 ? widen4<1>(w, s) : i % 4 == 2 ? widen4<2>(w, s)
                                                                                                    : widen4<3>(w, s);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                even[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], 0x05040100u);
                odd[e] = __builtin_amdgcn_perm(x[2 * e + 1], x[2 * e], 0x07060302u);
            }
        }
    }
};

// Running softmax of RT tiles of 16 query rows (lane r: row r of each) over tiles of keys.
template <int DT, int D, int F, int RT> struct AttnRows {
    typedef KvShape<D, F> S;
    typedef KvTile<DT, D, F> Tile;
    static constexpr int PDT = Tile::PDT;
    // p is held times 2^14 in fp16, so that what the two parts drop is 2^-38 of the largest
    static constexpr float OFF = PDT == W4A4_F16 ? 14.0f : 0.0f;
    u4_t q[RT][S::KJ];
    f4_t acc[RT][S::VE];
    float mx[RT], sum[RT];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
#pragma unroll
            for (int i = 0; i < S::VE; ++i) acc[t][i] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
            mx[t] = -INFINITY;
            sum[t] = 0.0f;
        }
    }

    __device__ __forceinline__ void load_q(int t, const uint16_t *row, int g)
    {
#pragma unroll
        for (int j = 0; j < S::KJ; ++j) q[t][j] = load8_any(row + S::channel(j, g));
    }

    // whole: every key is visible; else ok says which of the lane's are
    __device__ __forceinline__ void add(Tile &tile, bool whole, const bool (&ok)[8], float scale_log2)
    {
        f4_t s[RT][2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int t = 0; t < RT; ++t) s[t][hf] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < S::KJ; ++j) {
                const u4_t k = tile.key(hf, j);
#pragma unroll
                for (int t = 0; t < RT; ++t) s[t][hf] = mma32<DT>(k, q[t][j], s[t][hf]);
            }
        }
        float kscale[8], vscale[8];
        if constexpr (F == W4A4_KV_INT8) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float4 a = tile.ks[hf];
                kscale[4 * hf] = a.x * scale_log2;
                kscale[4 * hf + 1] = a.y * scale_log2;
                kscale[4 * hf + 2] = a.z * scale_log2;
                kscale[4 * hf + 3] = a.w * scale_log2;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) kscale[e] = scale_log2;
        }
        if (!whole) tile.hide_values(ok);
        if constexpr (F == W4A4_KV_INT8) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float4 a = tile.vs[hf];
                vscale[4 * hf] = a.x;
                vscale[4 * hf + 1] = a.y;
                vscale[4 * hf + 2] = a.z;
                vscale[4 * hf + 3] = a.w;
            }
        }
        u4_t hi[RT], lo[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = s[t][e / 4][e % 4] * kscale[e];
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = ok[e] ? p[e] : -INFINITY;
            }
            float top = p[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, p[e]);
            top = across_groups(top, [](float x, float y) { return fmaxf(x, y); });
            if (__any(top > mx[t])) {
                const float to = fmaxf(mx[t], top), f = to > mx[t] ? __builtin_amdgcn_exp2f(mx[t] - to) : 1.0f;
#pragma unroll
                for (int i = 0; i < S::VE; ++i) acc[t][i] *= f;
                sum[t] *= f;
                mx[t] = to;
            }
            const float from = (mx[t] == -INFINITY ? 0.0f : mx[t]) - OFF;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float x = __builtin_amdgcn_exp2f(p[e] - from), y = __builtin_amdgcn_exp2f(p[e + 1] - from);
                sum[t] += x + y;
                if constexpr (F == W4A4_KV_INT8) {
                    x *= vscale[e];
                    y *= vscale[e + 1];
                }
                hi[t][e / 2] = pack16<PDT>(x, y);
                const f2_t h = unpack16<PDT>(hi[t][e / 2]);
                lo[t][e / 2] = pack16<PDT>(x - h.x, y - h.y);
            }
        }
#pragma unroll
        for (int i = 0; i < S::VE / 2; ++i) {
            u4_t even, odd;
            tile.values(i, even, odd);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                acc[t][2 * i] = mma32<PDT>(even, lo[t], acc[t][2 * i]);
                acc[t][2 * i + 1] = mma32<PDT>(odd, lo[t], acc[t][2 * i + 1]);
                acc[t][2 * i] = mma32<PDT>(even, hi[t], acc[t][2 * i]);
                acc[t][2 * i + 1] = mma32<PDT>(odd, hi[t], acc[t][2 * i + 1]);
            }
        }
    }

    __device__ __forceinline__ float total(int t) const
    {
        return across_groups(sum[t], [](float x, float y) { return x + y; });
    }
};

}  // namespace w4a4
