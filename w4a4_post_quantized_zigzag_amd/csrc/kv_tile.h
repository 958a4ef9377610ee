// One tile of 32 keys and their values in a wave's registers, from a 16-bit or a quantized cache, and the products
// that attention makes of it:
//  - scores^T (16 keys x 16 query rows, twice) = K (A operand) . q^T;
//  - out^T (16 channels x 16 query rows per product) += V^T (A operand) . p (B operand).
// The scores' result layout already is the B operand of a 32-key product if key 4 g + e (e < 4) of the first and of
// the second half of the tile are its k = 8 g + e and 8 g + 4 + e. A lane loads VE neighbouring channels of those
// eight keys and pairs them up. K's operand wants neighbouring lanes in neighbouring keys, a cache line each: its rows are
// loaded as they lie and pass through LDS (KvStage; two long fp4 contexts 62.9 -> 52.7 us with it and the one look at the
// page table below).
// Codes become matrix operands in registers, exactly:
//  - int8: the codes themselves, as 16-bit numbers. A key's scale multiplies its scores and a value's scale its
//    weight, so that neither is rounded; the second product is bf16 for either element type, for weights times scales
//    need fp32's range.
//  - fp4: gfx950's conversion with a scale, whose results are exact in the element type.
#pragma once

#include <type_traits>

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

// Where a tile's two halves of 16 keys are: bytes from the start of the keys' (and the values') codes to the head's row of
// the half's first key, elements from the start of the scales to its first scale; all uniform.
struct KvPlace {
    int key0;
    int64_t codes[2], scales[2];
};

// The places of up to 64 tiles, a lane each: one look at the page table for all of them, and no scalar load, whose wait
// is a wait for everything, between the tiles' own loads.
struct KvPlaces {
    int key0;
    int64_t codes[2], scales[2];

    // This lane's tile starts at key `first` of a sequence of n keys, of which those from `from` on and the first `sinks`
    // are visible. A half without a visible key may have no page any more and reads the other half's. A page that does
    // not exist reads page 0 and sets bad.
    template <int D, int F>
    __device__ __forceinline__ void look_up(const KvPages &c, const int32_t *table, int first, int n, int from, int sinks,
                                            int kvh, bool &bad)
    {
        constexpr int ROW = F == W4A4_KV_16BIT ? 2 * D : F == W4A4_KV_INT8 ? D : D / 2, GROUPS = F == W4A4_KV_FP4 ? D / 32 : 1;
        key0 = first;
        bool any[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int lo = first + 16 * hf;
            any[hf] = lo < n && (min(lo + 15, n - 1) >= from || lo < sinks);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int lo = first + 16 * (any[hf] ? hf : 1 - hf);
            int pid = table[lo >> c.page_shift];
            if ((unsigned)pid >= (unsigned)c.num_pages) {
                bad = true;
                pid = 0;
            }
            const int at = lo & (c.page_size - 1);
            codes[hf] = pid * c.page_stride + ((int64_t)kvh * c.page_size + at) * ROW;
            scales[hf] = pid * c.scale_stride + (int64_t)kvh * GROUPS * c.page_size + at;
        }
    }
    static __device__ __forceinline__ int64_t lane(int64_t x, int i)
    {
        return (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)x, i) | (int64_t)__builtin_amdgcn_readlane((int)(x >> 32), i) << 32;
    }
    template <int F> __device__ __forceinline__ KvPlace get(int i) const
    {
        KvPlace p;
        p.key0 = __builtin_amdgcn_readlane(key0, i);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            p.codes[hf] = lane(codes[hf], i);
            p.scales[hf] = F == W4A4_KV_16BIT ? 0 : lane(scales[hf], i);
        }
        return p;
    }
};

// A tile's rows of keys or of values on their way through LDS, where THREADS threads put them as they lie in memory,
// 16 bytes each: loaded row by row from 16 keys at a time, as the matrix operand wants them, they would touch a line
// per lane, and the number of lines touched, not the bytes, would be what bounds the kernel. Rows are padded to an odd
// number of 16-byte slots, so that 16 rows are read without bank conflicts.
template <int D, int F, int THREADS> struct KvStage {
    static constexpr int CH = KvShape<D, F>::ROW / 16, ROW = (CH | 1) * 16, BYTES = 32 * ROW;
    static constexpr int ITEMS = 32 * CH, NI = (ITEMS + THREADS - 1) / THREADS;
    u4_t x[NI];

    __device__ __forceinline__ void load(const uint8_t *codes, const KvPlace &p, int tid)
    {
        const uint8_t *b0 = codes + p.codes[0], *b1 = codes + p.codes[1];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = min(i * THREADS + tid, ITEMS - 1);
            if ((i + 1) * THREADS <= ITEMS / 2) x[i] = *reinterpret_cast<const u4_t *>(b0 + at * 16u);
            else if (i * THREADS >= ITEMS / 2) x[i] = *reinterpret_cast<const u4_t *>(b1 + (at - ITEMS / 2) * 16u);
            else x[i] = *reinterpret_cast<const u4_t *>((at < ITEMS / 2 ? b0 : b1) + (at < ITEMS / 2 ? at : at - ITEMS / 2) * 16u);
        }
    }
    __device__ __forceinline__ void commit(uint8_t *lds, int tid) const
    {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = i * THREADS + tid;
            if (ITEMS % THREADS == 0 || at < ITEMS)
                *reinterpret_cast<u4_t *>(lds + at / CH * ROW + at % CH * 16) = x[i];
        }
    }
    // keys from `live` on become zeros
    __device__ __forceinline__ void commit(uint8_t *lds, int tid, int live)
    {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if ((i * THREADS + tid) / CH >= live) x[i] = u4_t{0, 0, 0, 0};
        commit(lds, tid);
    }
};

template <int DT, int D, int F> struct KvTile {
    typedef KvShape<D, F> S;
    static constexpr int PDT = F == W4A4_KV_INT8 ? W4A4_BF16 : DT;  // type of the second product
    struct __attribute__((aligned(4))) KRun { uint32_t w[S::KW / 4]; };
    typedef typename std::conditional<S::VB == 2, uint16_t, DwordRun<(S::VB + 3) / 4>>::type VLoad;
    KRun k[2][S::NL];
    VLoad v[8];
    float4 ks[2], vs[2];                // int8: scales of keys 4 g + e
    uint32_t kb[2][S::NL], vb[2];       // fp4: a key's scale byte, the value scale bytes of keys 4 g + e

    // keys from rows that a KvStage has put into LDS
    __device__ __forceinline__ void keys_from(const uint8_t *lds, int lane)
    {
        const int r = lane & 15, g = lane >> 4;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int l = 0; l < S::NL; ++l) {
                typedef typename std::conditional<S::KW == 16, u4_t, typename std::conditional<S::KW == 8, u2_t, uint32_t>::type>::type run_t;
                const run_t w = *reinterpret_cast<const run_t *>(lds + (16 * hf + r) * KvStage<D, F, 64>::ROW + (4 * l + g) * S::KW);
                k[hf][l] = __builtin_bit_cast(KRun, w);
            }
    }
    __device__ __forceinline__ void values_from(const uint8_t *lds, int lane)
    {
        const int r = lane & 15, g = lane >> 4, vch = S::VE * r < D ? S::VE * r : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint8_t *p = lds + (16 * (e / 4) + 4 * g + e % 4) * KvStage<D, F, 64>::ROW + vch * S::ROW / D;
            if constexpr (S::VB == 2) {
                v[e] = *reinterpret_cast<const uint16_t *>(p);
            } else if constexpr (S::VB % 16 == 0) {
#pragma unroll
                for (int i = 0; i < S::VB / 16; ++i) {
                    const u4_t w = reinterpret_cast<const u4_t *>(p)[i];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[e].v[4 * i + q] = w[q];
                }
            } else {
#pragma unroll
                for (int i = 0; i < S::VB / 4; ++i) v[e].v[i] = reinterpret_cast<const uint32_t *>(p)[i];
            }
        }
    }

    // KEYS: the codes of keys, too
    template <bool KEYS> __device__ __forceinline__ void load(const KvPages &c, const KvPlace &p, int lane)
    {
        const int r = lane & 15, g = lane >> 4;
        const uint32_t koff = r * S::ROW + g * S::KW;
        const uint32_t vch = S::VE * r < D ? S::VE * r : 0, voff = 4 * g * S::ROW + vch * S::ROW / D;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            if constexpr (KEYS)
#pragma unroll
                for (int l = 0; l < S::NL; ++l)
                    k[hf][l] = *reinterpret_cast<const KRun *>(c.k + p.codes[hf] + l * 4 * S::KW + koff);
            if constexpr (F == W4A4_KV_INT8)
                ks[hf] = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(c.k_scale) + p.scales[hf])[g];
            if constexpr (F == W4A4_KV_FP4) {
                const uint8_t *sp = reinterpret_cast<const uint8_t *>(c.k_scale) + p.scales[hf];
#pragma unroll
                for (int l = 0; l < S::NL; ++l) kb[hf][l] = sp[(uint32_t)(S::channel(l * S::NR, g) / 32 * c.page_size + r)];
            }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const uint8_t *vp = c.v + p.codes[hf];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * hf + e] = *reinterpret_cast<const VLoad *>(vp + e * S::ROW + voff);
            if constexpr (F == W4A4_KV_INT8)
                vs[hf] = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(c.v_scale) + p.scales[hf])[g];
            if constexpr (F == W4A4_KV_FP4)
                vb[hf] = *reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(c.v_scale) + p.scales[hf] +
                                                             (uint32_t)(vch / 32 * c.page_size + 4 * g));
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

    // what is not visible must not count, whatever it holds
    __device__ __forceinline__ void hide(const bool (&ok)[8])
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
                ks[hf].x = ok[4 * hf] ? ks[hf].x : 1.0f;
                ks[hf].y = ok[4 * hf + 1] ? ks[hf].y : 1.0f;
                ks[hf].z = ok[4 * hf + 2] ? ks[hf].z : 1.0f;
                ks[hf].w = ok[4 * hf + 3] ? ks[hf].w : 1.0f;
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
    // p is held times 2^14 in fp16, so that what the two parts drop is 2^-38 of the largest; it stays below 2^(14 + SLACK)
    static constexpr float OFF = PDT == W4A4_F16 ? 14.0f : 0.0f, SLACK = PDT == W4A4_F16 ? 1.0f : 8.0f;
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

    // The call's scale as add() takes it. 0 becomes the smallest normal number, which makes every weight 1 as well and
    // still leaves a hidden key's -inf one.
    static __device__ __forceinline__ float scale_of(const AttnArgs &a) { return fmaxf(fabsf(a.scale_log2), 0x1p-126f); }
    // flip: that scale is negative; the queries take its sign
    __device__ __forceinline__ void load_q(int t, const uint16_t *row, int g, bool flip)
    {
#pragma unroll
        for (int j = 0; j < S::KJ; ++j) {
            q[t][j] = load8_any(row + S::channel(j, g));
            if (flip) q[t][j] ^= u4_t{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
        }
    }

    // whole: every key is visible; else seen(e) says whether the lane's key e is, and what the others hold must not count
    // (HIDE: it may be anything, else zeros). scale > 0, times log2 e.
    template <bool HIDE, typename Seen>
    __device__ __forceinline__ void add(Tile &tile, bool whole, Seen seen, float scale)
    {
        f4_t s[RT][2];
#pragma unroll
        for (int t = 0; t < RT; ++t) s[t][0] = s[t][1] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < S::KJ; ++j)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const u4_t k = tile.key(hf, j);
#pragma unroll
                for (int t = 0; t < RT; ++t) s[t][hf] = mma32<DT>(k, q[t][j], s[t][hf]);
            }
        if (!whole) {
            asm volatile("");  // a branch that most tiles skip, not 40 selects for all of them
            bool ok[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) ok[e] = seen(e);
            if constexpr (HIDE) tile.hide(ok);
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e) s[t][e / 4][e % 4] = ok[e] ? s[t][e / 4][e % 4] : -INFINITY;
        }
        // int8: the scores' scales differ from key to key; else one scale goes into the exponent's FMA
        constexpr bool EACH = F == W4A4_KV_INT8;
        float kscale[8], vscale[8];
        if constexpr (EACH) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float4 a = tile.ks[hf], b = tile.vs[hf];
                kscale[4 * hf] = a.x * scale;
                kscale[4 * hf + 1] = a.y * scale;
                kscale[4 * hf + 2] = a.z * scale;
                kscale[4 * hf + 3] = a.w * scale;
                vscale[4 * hf] = b.x;
                vscale[4 * hf + 1] = b.y;
                vscale[4 * hf + 2] = b.z;
                vscale[4 * hf + 3] = b.w;
            }
        }
        float p[RT][8], top[RT];
        bool grown = false;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[t][e] = s[t][e / 4][e % 4];
                if constexpr (EACH) p[t][e] *= kscale[e];
            }
            top[t] = p[t][0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top[t] = fmaxf(top[t], p[t][e]);
            top[t] = across_groups(top[t], [](float x, float y) { return fmaxf(x, y); });
            if constexpr (!EACH) top[t] *= scale;
            grown = grown || top[t] > mx[t] + SLACK;
        }
        // The reference is moved only when a maximum has grown by more than 2^SLACK: sums and results are then relative
        // to one that is at most so much too small, and most tiles leave the results alone.
        if (__any(grown)) {
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const float to = fmaxf(mx[t], top[t]), f = to > mx[t] ? __builtin_amdgcn_exp2f(mx[t] - to) : 1.0f;
#pragma unroll
                for (int i = 0; i < S::VE; ++i) acc[t][i] *= f;
                sum[t] *= f;
                mx[t] = to;
            }
        }
        u4_t hi[RT], lo[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const float from = (mx[t] == -INFINITY ? 0.0f : mx[t]) - OFF;
            auto weight = [&](int e) {
                return __builtin_amdgcn_exp2f(EACH ? p[t][e] - from : fmaf(p[t][e], scale, -from));
            };
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float x = weight(e), y = weight(e + 1);
                sum[t] += x + y;
                if constexpr (EACH) {
                    x *= vscale[e];
                    y *= vscale[e + 1];
                }
                const uint32_t w = pack16<PDT>(x, y);
                hi[t][e / 2] = w;
                const f2_t h = unpack16<PDT>(w);
                lo[t][e / 2] = pack16<PDT>(x - h.x, y - h.y);
            }
        }
        u4_t v[S::VE];
#pragma unroll
        for (int i = 0; i < S::VE / 2; ++i) tile.values(i, v[2 * i], v[2 * i + 1]);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
#pragma unroll
            for (int i = 0; i < S::VE; ++i) acc[t][i] = mma32<PDT>(v[i], lo[t], acc[t][i]);
#pragma unroll
            for (int i = 0; i < S::VE; ++i) acc[t][i] = mma32<PDT>(v[i], hi[t], acc[t][i]);
        }
    }

    __device__ __forceinline__ float total(int t) const
    {
        return across_groups(sum[t], [](float x, float y) { return x + y; });
    }
};

}  // namespace w4a4
