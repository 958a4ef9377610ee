// Linears with group-scaled 4-bit weights and 16-bit (or fp32) activations:
//   y[m][n] = sum_g s[g][n] * sum_{k in group g} x[m][k] c[n][k],   codes c in [-8, 7].
//
// The call is bound by the weight bytes: one or a few tokens read N K / 2 bytes of codes once.
//  - Weights are laid out once, offline, as tiles of 16 rows x 128 k (1 KB): one wave reads one tile
//    with one 16-byte load per lane, fully contiguous, and the tile is already the B operand of
//    four v_mfma_f32_16x16x32 (lane (g, r): row r, dword j = the run of eight k at 32 j + 8 g).
//  - The codes are widened to the activation's 16-bit type in registers (exact: |c| <= 8) and the
//    matrix cores form the products and the sums in fp32. 16 activation rows cost no more than one,
//    and the sum over k needs no cross-lane step.
//  - With the activations as the A operand, a lane's four results share the output channel, so one
//    group scale per lane is folded in (fp32 FMA) after each group's exact-product partial sum.
//  - The waves of a workgroup share one tile of 16 channels and split K; their partial sums meet in
//    LDS in a fixed order, so results do not depend on timing.
#include <algorithm>

#include "w4a4_internal.h"

namespace w4a4 {

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef __bf16 b8_t __attribute__((ext_vector_type(8)));
typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

// ---- widening eight codes (one dword, offset-binary nibbles) -----------------------------------
// Nibble position p < 4 holds k = 2p of its run and p >= 4 holds k = 2 (p - 4) + 1, so that the two
// halves of (w >> 4 i) & 0x000F000F are neighbours in k.

// fp16: 0x6400 | u is 1024 + u exactly; subtracting 1032 leaves the code u - 8.
__device__ __forceinline__ u4_t widen_f16(uint32_t w)
{
    u4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t t = ((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
        const h2_t h = __builtin_bit_cast(h2_t, t) - h2_t{(_Float16)1032.0f, (_Float16)1032.0f};
        r[i] = __builtin_bit_cast(uint32_t, h);
    }
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2_t{a, b}, b2_t));
}

// bf16: v_cvt_off_f32_i4 turns a two's-complement nibble into code / 16, exact in bf16 as well; the
// factor 16 is folded into the group scale.
__device__ __forceinline__ u4_t widen_bf16(uint32_t w)
{
    const uint32_t a = w ^ 0x88888888u, b = a >> 4;
    auto c = [](uint32_t v) { return __builtin_amdgcn_cvt_off_f32_i4((int)v); };
    u4_t r;
    r[0] = pack_bf16(c(a), c(a >> 16));
    r[1] = pack_bf16(c(b), c(b >> 16));
    r[2] = pack_bf16(c(a >> 8), c(a >> 24));
    r[3] = pack_bf16(c(b >> 8), c(b >> 24));
    return r;
}

// ---- activation operands -----------------------------------------------------------------------
// Eight consecutive k of one row as PARTS 16-bit operands. fp32 activations are cut into three bf16
// parts by truncation, x = p0 + p1 + p2 exactly (8 bits each), so their products are exact too.
template <int DT> struct ActOf;
template <> struct ActOf<W4A4_F16> { typedef uint16_t raw; static constexpr int PARTS = 1; };
template <> struct ActOf<W4A4_BF16> { typedef uint16_t raw; static constexpr int PARTS = 1; };
template <> struct ActOf<W4A4_F32> { typedef uint32_t raw; static constexpr int PARTS = 3; };

template <int DT> struct ActRun {
    u4_t v[DT == W4A4_F32 ? 2 : 1];
};

template <int DT, bool VEC>
__device__ __forceinline__ ActRun<DT> load_run(const typename ActOf<DT>::raw *__restrict__ p)
{
    ActRun<DT> r;
    if (VEC) {
        const u4_t *q = reinterpret_cast<const u4_t *>(p);
        r.v[0] = q[0];
        if constexpr (DT == W4A4_F32) r.v[1] = q[1];
    } else if constexpr (DT == W4A4_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i / 4][i % 4] = p[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[0][i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    }
    return r;
}

template <int DT> __device__ __forceinline__ void act_parts(const ActRun<DT> &x, u4_t (&p)[ActOf<DT>::PARTS])
{
    if constexpr (DT != W4A4_F32) {
        p[0] = x.v[0];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[2][3];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t bits = x.v[i / 2][2 * (i % 2) + e];
                const float f = __builtin_bit_cast(float, bits);
                const bool fin = (bits & 0x7F800000u) != 0x7F800000u;
                const bool nan = !fin && (bits & 0x007FFFFFu) != 0;
                // an infinity or NaN stays whole in the first part
                h[e][0] = (bits & 0xFFFF0000u) | (nan ? 0x00400000u : 0u);
                const float r1 = fin ? f - __builtin_bit_cast(float, h[e][0]) : 0.0f;
                h[e][1] = __builtin_bit_cast(uint32_t, r1) & 0xFFFF0000u;
                h[e][2] = __builtin_bit_cast(uint32_t, r1 - __builtin_bit_cast(float, h[e][1]));
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) p[q][i] = (h[0][q] >> 16) | (h[1][q] & 0xFFFF0000u);
        }
    }
}

template <int DT> __device__ __forceinline__ f4_t mma(const u4_t &a, const u4_t &b, const f4_t &c)
{
    if constexpr (DT == W4A4_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a),
                                                      __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8_t, a),
                                                       __builtin_bit_cast(b8_t, b), c, 0, 0, 0);
}

struct W4gArgs {
    const void *X;
    int64_t ldx;
    const uint8_t *wt;
    const uint16_t *w_scale;
    int M, K, N, gshift;  // group = 32 << gshift
    uint16_t *Y;
    int64_t ldy;
    int epilogue;
    const uint16_t *residual;
    int64_t ldr;
};

__device__ __forceinline__ float gelu_f32(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

template <int DT> __device__ __forceinline__ float load_y(uint16_t h)
{
    if constexpr (DT == W4A4_BF16) return __builtin_bit_cast(float, (uint32_t)h << 16);
    else return __half2float(__ushort_as_half(h));
}

template <int DT> __device__ __forceinline__ uint16_t store_y(float v)
{
    if constexpr (DT == W4A4_BF16) return (uint16_t)pack_bf16(v, 0.0f);
    else return __half_as_ushort(__float2half_rn(v));
}

// Orders one wave's LDS writes and reads of other lanes' data (the hardware keeps a wave's LDS accesses
// in order; this keeps the compiler from moving them).
__device__ __forceinline__ void turn_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// One workgroup: 16 output channels (blockIdx.x) of 16 MT rows (blockIdx.y), its waves splitting the
// 128-k stages round-robin. GS groups per stage (1 for group >= 128). U stages are in flight per
// wave: all their loads are issued before the first is used.
//
// The matrix operand wants neighbouring lanes in neighbouring rows; loading the activations that way
// touches 64 cache lines per instruction. A wave therefore loads each row's 256 bytes of a stage with
// 16 neighbouring lanes and turns the 16 x 128 tile in its own corner of LDS (no barrier), where run c
// of row r sits in slot c ^ r so that both sides are free of bank conflicts.
// Q: quads of rows that a tile has at most (1 for M <= 4, so that its loads need no registers for more).
template <int DT, int MT, int Q, int GS, bool VEC, int U, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void k_gemv_w4g(const W4gArgs a)
{
    typedef typename ActOf<DT>::raw raw;
    constexpr int P = ActOf<DT>::PARTS;
    // per wave: the tile in turn [P][16][16 slots] of 16 bytes; afterwards [waves][MT][4][64] floats
    extern __shared__ u4_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int nt = blockIdx.x, m0 = blockIdx.y * (16 * MT);
    const int stages = (a.K + 127) >> 7, ngroups = a.K >> (5 + a.gshift);
    const int ns = min(nt * 16 + r, a.N - 1);
    u4_t *turn = lds + wave * (P * 256);

    const uint8_t *wp = a.wt + ((int64_t)nt * stages * 64 + lane) * 16;
    const uint16_t *sp = a.w_scale + ns;
    // as loader: lane (g, r) holds run r of rows 4 q + g
    const raw *xp = reinterpret_cast<const raw *>(a.X) + (int64_t)(m0 + g) * a.ldx + 8 * r;
    const int rows = a.M - m0 - g;  // row 16 t + 4 q + g exists if 16 t + 4 q < rows

    f4_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};

    for (int s0 = wave; s0 < stages; s0 += waves * U) {
        u4_t w[U];
        uint16_t sc[U][GS];
        ActRun<DT> x[U][MT][Q];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = min(s0 + u * waves, stages - 1);
            w[u] = __builtin_nontemporal_load(reinterpret_cast<const u4_t *>(wp + (int64_t)s * 1024));
#pragma unroll
            for (int q = 0; q < GS; ++q) {
                const int grp = GS == 1 ? (s * 4) >> a.gshift : s * GS + q;
                sc[u][q] = sp[(int64_t)min(grp, ngroups - 1) * a.N];
            }
            const bool in = s * 128 + 8 * r < a.K;  // runs past K (the last stage) are not used
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < Q; ++q)
                    if (in && 16 * t + 4 * q < rows)
                        x[u][t][q] = load_run<DT, VEC>(xp + (int64_t)(16 * t + 4 * q) * a.ldx + s * 128);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * waves;
            if (u > 0 && s >= stages) break;
            u4_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = DT == W4A4_F16 ? widen_f16(w[u][j]) : widen_bf16(w[u][j]);
            float f[GS];
#pragma unroll
            for (int q = 0; q < GS; ++q)
                f[q] = __half2float(__ushort_as_half(sc[u][q])) * (DT == W4A4_F16 ? 1.0f : 16.0f);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                // rows past M leave what the slot held: their results are not stored
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    u4_t p[P];
                    act_parts<DT>(x[u][t][q], p);
#pragma unroll
                    for (int i = 0; i < P; ++i) turn[(i * 16 + 4 * q + g) * 16 + (r ^ (4 * q + g))] = p[i];
                }
                turn_fence();
                f4_t part;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (s * 128 + 32 * j >= a.K) break;  // nothing there
                    if (j % (4 / GS) == 0) part = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = P - 1; i >= 0; --i)
                        part = mma<DT>(turn[(i * 16 + r) * 16 + ((4 * j + g) ^ r)], b[j], part);
                    if (GS > 1 && (j + 1) % (4 / GS) == 0) acc[t] += part * f[j * GS / 4];
                }
                turn_fence();
                if (GS == 1) acc[t] += part * f[0];
            }
        }
    }

    float *red = reinterpret_cast<float *>(lds);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[((wave * MT + t) * 4 + i) * 64 + lane] = acc[t][i];
    __syncthreads();
    for (int e = tid; e < MT * 256; e += blockDim.x) {
        const int l = e & 63, i = (e >> 6) & 3, t = e >> 8;
        const int m = m0 + 16 * t + 4 * (l >> 4) + i, col = nt * 16 + (l & 15);
        if (m >= a.M || col >= a.N) continue;
        float y = 0.0f;
        for (int v = 0; v < waves; ++v) y += red[v * (MT * 256) + e];
        if (a.epilogue == W4A4_EPI_GELU) y = gelu_f32(y);
        else if (a.epilogue == W4A4_EPI_RESIDUAL) y += load_y<DT>(a.residual[(int64_t)m * a.ldr + col]);
        a.Y[(int64_t)m * a.ldy + col] = store_y<DT>(y);
    }
}

template <int DT, int MT, int Q, int GS, bool VEC>
static int run_gemv(const W4gArgs &a, hipStream_t s)
{
    constexpr int U = DT == W4A4_F32 ? (Q == 1 ? 2 : 1) : Q == 1 ? 4 : MT == 1 ? 2 : 1;
    constexpr int MAXW = MT == 1 && DT != W4A4_F32 ? 16 : 8;  // at most 96 KB of LDS
    const int tiles = (a.N + 15) / 16, rows = (a.M + 16 * MT - 1) / (16 * MT);
    const int stages = (a.K + 127) / 128;
    int waves = 1;
    while (waves < MAXW && waves * 2 <= stages && (waves < 4 || (int64_t)tiles * rows * waves < 4096)) waves *= 2;
    const size_t lds = (size_t)waves * 1024 * std::max(4 * ActOf<DT>::PARTS, MT);
    const auto kernel = k_gemv_w4g<DT, MT, Q, GS, VEC, U, MAXW>;
    if (int rc = ensure_dynamic_lds(reinterpret_cast<const void *>(kernel), lds, "gemv_w4g")) return rc;
    hipLaunchKernelGGL(kernel, dim3(tiles, rows), dim3(64 * waves), lds, s, a);
    return check_launch("gemv_w4g");
}

template <int DT, int MT, int Q>
static int pick_group(const W4gArgs &a, hipStream_t s)
{
    const size_t eb = sizeof(typename ActOf<DT>::raw);
    const bool vec = (uintptr_t)a.X % 16 == 0 && (a.ldx * eb) % 16 == 0;
    if (a.gshift == 0) return vec ? run_gemv<DT, MT, Q, 4, true>(a, s) : run_gemv<DT, MT, Q, 4, false>(a, s);
    if (a.gshift == 1) return vec ? run_gemv<DT, MT, Q, 2, true>(a, s) : run_gemv<DT, MT, Q, 2, false>(a, s);
    return vec ? run_gemv<DT, MT, Q, 1, true>(a, s) : run_gemv<DT, MT, Q, 1, false>(a, s);
}

template <int DT> static int pick_rows(const W4gArgs &a, hipStream_t s)
{
    if (a.M <= 4) return pick_group<DT, 1, 1>(a, s);
    if (a.M <= 16) return pick_group<DT, 1, 4>(a, s);
    if (a.M <= 32) return pick_group<DT, 2, 4>(a, s);
    return pick_group<DT, 4, 4>(a, s);
}

int launch_gemv_w4g(const void *X, int x_dtype, int M, int K, int64_t ldx, const uint8_t *wt,
                    const uint16_t *w_scale, int gshift, int N, uint16_t *Y, int64_t ldy, int epilogue,
                    const uint16_t *residual, int64_t ldr, hipStream_t s)
{
    const W4gArgs a{X, ldx, wt, w_scale, M, K, N, gshift, Y, ldy, epilogue, residual, ldr};
    switch (x_dtype) {
    case W4A4_F16: return pick_rows<W4A4_F16>(a, s);
    case W4A4_BF16: return pick_rows<W4A4_BF16>(a, s);
    default: return pick_rows<W4A4_F32>(a, s);
    }
}

// ---- weight operand -----------------------------------------------------------------------------
// Dword of the eight offset-binary codes u[0..7] of a run, and where the run of row n, k = 8 kr sits.
__device__ __forceinline__ uint32_t pack_run(const uint32_t (&u)[8])
{
    return u[0] | (u[2] << 4) | (u[4] << 8) | (u[6] << 12) | (u[1] << 16) | (u[3] << 20) |
           (u[5] << 24) | (u[7] << 28);
}

__device__ __forceinline__ int64_t run_index(int n, int kr, int stages)
{
    const int s = kr >> 4, j = (kr >> 2) & 3, g = kr & 3;
    return (((int64_t)(n >> 4) * stages + s) * 64 + g * 16 + (n & 15)) * 4 + j;
}

// Round to nearest per group. A workgroup takes 16 rows x 256 k, 16 threads per row with 16 k each, so
// a group is 2, 4, 8 or 16 neighbouring threads.
__global__ __launch_bounds__(256) void k_pack_w4g(const void *__restrict__ W, int wdt, int N, int K,
                                                  int64_t ldw, int gshift, uint32_t *__restrict__ wt,
                                                  uint16_t *__restrict__ w_scale)
{
    const int r = threadIdx.x >> 4, p = threadIdx.x & 15;
    const int n = blockIdx.x * 16 + r, k0 = blockIdx.y * 256 + p * 16;
    const int stages = (K + 127) >> 7;
    float w[16], mx = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        w[i] = 0.0f;
        if (n < N && k0 + i < K) {
            const int64_t at = (int64_t)n * ldw + k0 + i;
            w[i] = wdt == W4A4_BF16
                       ? __builtin_bit_cast(float, (uint32_t)reinterpret_cast<const uint16_t *>(W)[at] << 16)
                       : load_as_f32(W, wdt, at);
        }
        mx = fmaxf(mx, fabsf(w[i]));
    }
    for (int off = 1; off < (2 << gshift); off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 16));
    // fp16 scale: zero groups get 1; a maximum whose seventh leaves fp16's range takes its end
    uint16_t bits = __half_as_ushort(__float2half_rn(fminf(mx / 7.0f, 65504.0f)));
    if (bits == 0) bits = mx == 0.0f ? 0x3C00 : 0x0001;
    const float s = __half2float(__ushort_as_half(bits));
    if (n < N && k0 < K && (k0 & ((32 << gshift) - 1)) == 0)
        w_scale[(int64_t)(k0 >> (5 + gshift)) * N + n] = bits;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = (uint32_t)((int)fminf(fmaxf(rintf(w[8 * h + i] / s), -8.0f), 7.0f) + 8);
        const int kr = (k0 >> 3) + h;
        if (kr < stages * 16) wt[run_index(n, kr, stages)] = pack_run(u);
    }
}

// Packed int4 codes [N][K / 2] (two's complement, low nibble = even k) -> the tiled operand.
__global__ __launch_bounds__(256) void k_codes_to_w4g(const uint8_t *__restrict__ codes, int N, int K,
                                                      uint32_t *__restrict__ wt, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= total) return;
    const int stages = (K + 127) >> 7;
    const int kr = (int)(id % (stages * 16)), n = (int)(id / (stages * 16));
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = (n < N && kr * 8 < K) ? codes[(int64_t)n * (K / 2) + kr * 4 + i] : 0u;
        u[2 * i] = (b & 15u) ^ 8u;
        u[2 * i + 1] = (b >> 4) ^ 8u;
    }
    wt[run_index(n, kr, stages)] = pack_run(u);
}

int launch_pack_w4g(const void *W, int wdt, int N, int K, int64_t ldw, int gshift, uint8_t *wt,
                    uint16_t *w_scale, hipStream_t s)
{
    hipLaunchKernelGGL(k_pack_w4g, dim3((N + 15) / 16, (K + 255) / 256), dim3(256), 0, s, W, wdt, N, K,
                       ldw, gshift, reinterpret_cast<uint32_t *>(wt), w_scale);
    return check_launch("pack_weights_w4g");
}

int launch_codes_to_w4g(const uint8_t *codes, int N, int K, uint8_t *wt, hipStream_t s)
{
    const int64_t total = (int64_t)((N + 15) / 16 * 16) * ((K + 127) / 128 * 16);
    hipLaunchKernelGGL(k_codes_to_w4g, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s, codes, N,
                       K, reinterpret_cast<uint32_t *>(wt), total);
    return check_launch("codes_to_w4g");
}

}  // namespace w4a4
