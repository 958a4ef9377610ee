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
// Measured: one bf16 token, 2048x16384, group 64, 6.2 us and eight fp16 tokens, 16384x2048, group 128, 7.2 us, of
// which 1.7 us are the launch and 2.1 us the bare reading of the 17 MB from the last-level cache (in a graph over 24
// weights, 430 MB, which that cache does not hold, a call takes 6.5 and 7.5 us, with three 6.8 and 7.9); 50 tokens,
// 1024x4099, group 32, 5.6 us.
#include <algorithm>
#include <type_traits>

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

// fp16: with u in the low four bits of the mantissa, 0x6400 | u is 1024 + u; in the next four, 0x5400 |
// 16 u is 64 + u, which saves the shift. Subtracting 1032 or 72 leaves the code u - 8, all exactly. The
// or-mask is kept in a register: v_and_or_b32 takes one scalar constant only.
__device__ __forceinline__ u4_t widen_f16(uint32_t w)
{
    uint32_t m0 = 0x64006400u, m1 = 0x54005400u;
    asm("" : "+v"(m0), "+v"(m1));
    const h2_t b0 = {(_Float16)1032.0f, (_Float16)1032.0f}, b1 = {(_Float16)72.0f, (_Float16)72.0f};
    const uint32_t v = w >> 8;
    u4_t r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2_t, (w & 0x000F000Fu) | m0) - b0);
    r[1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2_t, (w & 0x00F000F0u) | m1) - b1);
    r[2] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2_t, (v & 0x000F000Fu) | m0) - b0);
    r[3] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2_t, (v & 0x00F000F0u) | m1) - b1);
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2_t{a, b}, b2_t));
}

// bf16: v_cvt_off_f32_i4 turns a two's-complement nibble into code / 16, exact in bf16 as well; the
// factor 16 is put back at the end.
__device__ __forceinline__ u4_t widen_bf16(uint32_t w)
{
    const uint32_t a = w ^ 0x88888888u, b = a >> 4;
    // byte extracts fold into the conversions' operand selection
    auto c = [](uint32_t v, int byte) {
        return __builtin_amdgcn_cvt_off_f32_i4((int)(byte == 0 ? v : (v >> (8 * byte)) & 0xFFu));
    };
    u4_t r;
    r[0] = pack_bf16(c(a, 0), c(a, 2));
    r[1] = pack_bf16(c(b, 0), c(b, 2));
    r[2] = pack_bf16(c(a, 1), c(a, 3));
    r[3] = pack_bf16(c(b, 1), c(b, 3));
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

// Rows start anywhere an element may: the hardware's vector loads take any address.
template <int DT>
__device__ __forceinline__ ActRun<DT> load_run(const typename ActOf<DT>::raw *__restrict__ p)
{
    typedef uint32_t run_t __attribute__((ext_vector_type(4), aligned(2)));
    const run_t *q = reinterpret_cast<const run_t *>(p);
    ActRun<DT> r;
    r.v[0] = q[0];
    if constexpr (DT == W4A4_F32) r.v[1] = q[1];
    return r;
}

template <int DT> __device__ __forceinline__ void act_parts(const ActRun<DT> &x, u4_t (&p)[ActOf<DT>::PARTS])
{
    if constexpr (DT != W4A4_F32) {
        p[0] = x.v[0];
    } else {
        auto cut = [](float f) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, f) & 0xFFFF0000u); };
        auto high = [](float a, float b) {  // the upper halves of two floats, the first one's low
            return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[2], r[2], t[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f[e] = __builtin_bit_cast(float, (uint32_t)x.v[i / 2][2 * (i % 2) + e]);
                // an infinity is whole in the first part; a NaN stays one in the second
                r[e] = fabsf(f[e]) == INFINITY ? 0.0f : f[e] - cut(f[e]);
                t[e] = r[e] - cut(r[e]);
            }
            p[0][i] = high(f[0], f[1]);
            p[1][i] = high(r[0], r[1]);
            p[2][i] = high(t[0], t[1]);
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
    int row_blocks;  // set per launch
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

// One workgroup: TN tiles of C = 16 / F output channels for 16 rows, its waves splitting K. A wave turns
// the activations of U steps into matrix operands once and keeps them in registers over its TN tiles. All
// loads of the next steps are in flight while it works on these. GS groups per 128-k stage (1 for group >=
// 128). More than 16 rows are blocks of 16 in workgroups of their own: two or four blocks in one workgroup
// read the weights less often but leave too few waves (64 tokens, 16384x2048: 12.9 us with one block, 15.0
// with two, 25.6 with four).
//
// F (1, 2, 4): few activation rows leave most of the 16 x 16 results of a product unused, and few
// output channels leave CUs without work. With F > 1 a product takes F stages at once: row and column
// f C + i of the operands hold row i of the activations and channel i of stage f, so that its F diagonal
// blocks are partial sums of the same C x C results. One step is then F stages, a workgroup has C channels
// and the grid F times as many workgroups. Needs M <= C.
//
// The matrix operand wants neighbouring lanes in neighbouring rows; loading the activations that way
// touches 64 cache lines per instruction. A wave therefore loads each row's 256 bytes of a stage with
// 16 neighbouring lanes and turns the 16 x 128 tile in its own corner of LDS (no barrier), where run c
// of row r sits in slot c ^ r so that both sides are free of bank conflicts.
// Q: quads of operand rows that hold activations at most (1 for M <= 4 with F = 1, else 4).
template <int DT, int Q, int GS, int U, int TN> struct GemvStep {
    u4_t w[U][TN];
    uint16_t sc[U][TN][GS];
    ActRun<DT> x[U][Q];
};

template <int DT, int F, int Q, int GS, int U, int TN, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void k_gemv_w4g(const W4gArgs a)
{
    typedef typename ActOf<DT>::raw raw;
    constexpr int P = ActOf<DT>::PARTS, C = 16 / F;
    constexpr int TILE = P * 4 * Q * 16;  // 16-byte slots of a tile in turn
    // per wave: one tile in turn [P][4 Q][16]; afterwards [waves][TN][4][64] floats
    extern __shared__ u4_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    // consecutive workgroups go to different XCDs: the row blocks of one tile follow each other on one
    // XCD, so that its L2 holds the tile's weights for all of them
    const int block = blockIdx.x / 8;
    const int c0 = (block / a.row_blocks * 8 + blockIdx.x % 8) * (TN * C), m0 = block % a.row_blocks * 16;
    if (c0 >= a.N) return;
    const int stages = (a.K + 127) >> 7, steps = (stages + F - 1) / F, ngroups = a.K >> (5 + a.gshift);
    u4_t *turn = lds + wave * TILE;

    // as holder of the weight operand: channel c0 + t C + r % C of stage F step + r / C. With F = 1 the
    // addresses are a uniform base and a lane's fixed offset.
    const int wfold = r / C, last_tile = (a.N - 1) >> 4;
    auto weights = [&](int t, int s) {  // a tile past N reads the last one; nothing of it is stored
        const int col = c0 + t * C;
        if constexpr (F == 1) {
            const uint8_t *p = a.wt + ((int64_t)min(col >> 4, last_tile) * stages + s) * 1024;
            return reinterpret_cast<const u4_t *>(p + lane * 16u);
        } else {
            const int row = col % 16 + r % C;
            return reinterpret_cast<const u4_t *>(
                a.wt + (((int64_t)min(col >> 4, last_tile) * stages + s) * 64 + g * 16 + row) * 16);
        }
    };
    uint32_t soff[TN];
#pragma unroll
    for (int t = 0; t < TN; ++t) soff[t] = (uint32_t)min(c0 + t * C + r % C, a.N - 1);
    auto scale = [&](int t, int grp) { return (a.w_scale + (int64_t)grp * a.N)[soff[t]]; };
    // as loader: lane (g, r) holds run r of operand rows 4 q + g, row (4 q + g) % C of stage (4 q + g) / C.
    // Rows past M repeat the last one; their results are not stored. 16 rows stay inside 32-bit offsets.
    uint32_t xoff[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        xoff[q] = (uint32_t)min((4 * q) % C + g, a.M - m0 - 1) * (uint32_t)a.ldx;
    const raw *xbase = reinterpret_cast<const raw *>(a.X) + (int64_t)m0 * a.ldx;
    // start of the stage that operand row 4 q is from
    auto stage_k = [&](int step, int q) { return (step * F + 4 * q / C) * 128; };

    f4_t acc[TN];
#pragma unroll
    for (int t = 0; t < TN; ++t) acc[t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};

    typedef GemvStep<DT, Q, GS, U, TN> Step;
    // activations first: they are needed first, and the weights can then be used as they arrive
    auto load = [&](int s0, Step &d) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int step = s0 + u * waves;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k0 = stage_k(step, q), k = k0 < a.K ? k0 : 0;
                // runs past K read the last one; turn_rows makes them zeros
                d.x[u][q] = load_run<DT>(xbase + k + (xoff[q] + (uint32_t)min(8 * r, a.K - 8 - k)));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int step = s0 + u * waves;
            if (u > 0 && step >= steps) break;
            const int s = F == 1 ? step : min(step * F + wfold, stages - 1);
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int q = 0; q < GS; ++q) {
                    const int grp = GS == 1 ? (s * 4) >> a.gshift : min(s * GS + q, ngroups - 1);
                    d.sc[u][t][q] = scale(t, grp);
                }
#pragma unroll
            for (int t = 0; t < TN; ++t) d.w[u][t] = *weights(t, s);
        }
    };
    u4_t x[U][P][4];
    auto turn_rows = [&](int s0, Step &d, auto last) {  // only a wave's last steps can reach past K
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (last.value && stage_k(s0 + u * waves, q) + 8 * r >= a.K) d.x[u][q] = ActRun<DT>{};
                u4_t p[P];
                act_parts<DT>(d.x[u][q], p);
#pragma unroll
                for (int i = 0; i < P; ++i) turn[(i * 4 * Q + 4 * q + g) * 16 + (r ^ (4 * q + g))] = p[i];
            }
            turn_fence();
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)  // with one quad of rows the operand's other rows repeat them
                    x[u][i][j] = turn[(i * 4 * Q + r % (4 * Q)) * 16 + ((4 * j + g) ^ (r % (4 * Q)))];
            turn_fence();
        }
    };
    auto multiply = [&](int s0, const Step &d) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u > 0 && s0 + u * waves >= steps) break;
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                f4_t part;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u4_t b = DT == W4A4_F16 ? widen_f16(d.w[u][t][j]) : widen_bf16(d.w[u][t][j]);
                    if (j % (4 / GS) == 0) part = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = P - 1; i >= 0; --i) part = mma<DT>(x[u][i][j], b, part);
                    if ((j + 1) % (4 / GS) == 0)
                        acc[t] += part * __half2float(__ushort_as_half(d.sc[u][t][j * GS / 4]));
                }
            }
        }
    };

    Step cur;
    load(wave, cur);  // there are no more waves than steps
    int s0 = wave;
    for (; s0 + waves * U < steps; s0 += waves * U) {
        turn_rows(s0, cur, std::false_type());
        Step next;
        load(s0 + waves * U, next);
        multiply(s0, cur);
        cur = next;
    }
    turn_rows(s0, cur, std::true_type());
    multiply(s0, cur);

    float *red = reinterpret_cast<float *>(lds);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[((wave * TN + t) * 4 + i) * 64 + lane] = acc[t][i];
    __syncthreads();
    // result (m, c) of a tile: operand row f C + m (lanes of group row / 4, register row % 4), column f C + c
    const int live = min(a.M - m0, C);
    for (int e = tid; e < TN * C * live; e += blockDim.x) {
        const int c = e % C, t = e / C % TN, m = e / (C * TN);
        const int col = c0 + t * C + c;
        if (col >= a.N) continue;
        float y = 0.0f;
        for (int v = 0; v < waves; ++v)
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int row = f * C + m;
                y += red[((v * TN + t) * 4 + row % 4) * 64 + row / 4 * 16 + f * C + c];
            }
        if (DT != W4A4_F16) y *= 16.0f;  // the codes were sixteenths
        if (a.epilogue == W4A4_EPI_GELU) y = gelu_f32(y);
        else if (a.epilogue == W4A4_EPI_RESIDUAL) y += load_y<DT>(a.residual[(int64_t)(m0 + m) * a.ldr + col]);
        a.Y[(int64_t)(m0 + m) * a.ldy + col] = store_y<DT>(y);
    }
}

// Waves: enough of them to keep the memory busy, at most one per step. They double until the grid has 3000 in all
// (16384x2048, fp16, eight tokens: 19.2 us with 512, 11.6 with 1024, 8.3 with 2048, 7.7 with 4096; four tokens: 18.9,
// 11.4, 8.1 and 6.8).
template <int DT, int F, int Q, int GS, int TN>
static int run_gemv(W4gArgs a, hipStream_t s)
{
    constexpr int P = ActOf<DT>::PARTS, U = P == 1 && Q == 1 && TN <= 2 && TN * GS <= 4 ? 2 : 1;
    constexpr int MAXW = P == 1 ? 16 : 8, C = 16 / F;
    const int tiles = (a.N + TN * C - 1) / (TN * C), steps = ((a.K + 127) / 128 + F - 1) / F;
    a.row_blocks = (a.M + 15) / 16;
    int waves = 1;
    while (waves < MAXW && waves * 2 <= steps && (waves < 4 || (int64_t)tiles * a.row_blocks * waves < 3000))
        waves *= 2;
    const size_t lds = (size_t)waves * 1024 * std::max(P * Q, TN);
    const auto kernel = k_gemv_w4g<DT, F, Q, GS, U, TN, MAXW>;
    if (lds > 65536)  // more than every kernel gets unasked
        if (int rc = ensure_dynamic_lds(reinterpret_cast<const void *>(kernel), lds, "gemv_w4g")) return rc;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((int64_t)(tiles + 7) / 8 * 8 * a.row_blocks)), dim3(64 * waves),
                       lds, s, a);
    return check_launch("gemv_w4g");
}

template <int DT, int F, int Q, int TN> static int pick_group(const W4gArgs &a, hipStream_t s)
{
    // four scales a stage leave registers for two tiles of 16 rows
    if (a.gshift == 0) return run_gemv<DT, F, Q, 4, (Q == 4 && TN == 4) ? 2 : TN>(a, s);
    if (a.gshift == 1) return run_gemv<DT, F, Q, 2, TN>(a, s);
    return run_gemv<DT, F, Q, 1, TN>(a, s);
}

// Two or four tiles per workgroup share its turned activations where there are tiles enough for all CUs.
template <int DT, int Q> static int pick_tiles(const W4gArgs &a, hipStream_t s)
{
    const int64_t wgs = (int64_t)((a.N + 15) / 16) * ((a.M + 15) / 16);
    if (wgs >= 1024) return pick_group<DT, 1, Q, 4>(a, s);
    if (wgs >= 512) return pick_group<DT, 1, Q, 2>(a, s);
    return pick_group<DT, 1, Q, 1>(a, s);
}

// F stages per product while that gives the CUs workgroups they lack.
template <int DT> static int pick_rows(const W4gArgs &a, hipStream_t s)
{
    const int tiles = (a.N + 15) / 16;
    if (a.M <= 4 && a.K > 256 && tiles <= 64) return pick_group<DT, 4, 4, 1>(a, s);
    if (a.M <= 8 && a.K > 128 && tiles <= 128) return pick_group<DT, 2, 4, 1>(a, s);
    return a.M <= 4 ? pick_tiles<DT, 1>(a, s) : pick_tiles<DT, 4>(a, s);
}

int launch_gemv_w4g(const void *X, int x_dtype, int M, int K, int64_t ldx, const uint8_t *wt,
                    const uint16_t *w_scale, int gshift, int N, uint16_t *Y, int64_t ldy, int epilogue,
                    const uint16_t *residual, int64_t ldr, hipStream_t s)
{
    // a launch holds less than 2^32 threads: at most 2^22 workgroups of 1024
    const int rows = 16 * std::max(1, (1 << 22) / ((N + 15) / 16 + 8));
    for (int64_t m = 0; m < M; m += rows) {
        const char *x = reinterpret_cast<const char *>(X) + m * ldx * (x_dtype == W4A4_F32 ? 4 : 2);
        const W4gArgs a{x,         ldx, wt,       w_scale,  (int)std::min<int64_t>(rows, M - m), K, N, gshift,
                        Y + m * ldy, ldy, epilogue, residual ? residual + m * ldr : nullptr, ldr, 0};
        const int rc = x_dtype == W4A4_F16    ? pick_rows<W4A4_F16>(a, s)
                       : x_dtype == W4A4_BF16 ? pick_rows<W4A4_BF16>(a, s)
                                              : pick_rows<W4A4_F32>(a, s);
        if (rc) return rc;
    }
    return W4A4_OK;
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
