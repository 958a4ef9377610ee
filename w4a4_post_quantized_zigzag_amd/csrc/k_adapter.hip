// Low-rank adapters of many requests beside a shared projection:
//   out[m] = epilogue(Y[m] + s_a (X[m] A_a^T) B_a^T),  a = ids[m];  rows whose id names no adapter get no product.
//
// Two launches. The inner product t = X A^T (R numbers a row) and the outer one t B^T both go to the matrix cores, 16
// rows at a time. Rows of one tile may have different adapters: the tile is multiplied once with each adapter that
// occurs among its rows, and of every such pass only the rows that asked for it are kept. So each adapter is read once
// per tile that needs it, nothing has to be sorted, no row ever meets another's weights, and a batch with one adapter
// for all rows pays for one pass.
//  - inner: [ranks x rows] = A (A operand) . X^T, K cut over workgroups (parts of t are fp32 and are added in a fixed
//    order by the readers) and over the waves of each.
//  - outer: [channels x rows] = B (A operand) . t^T. t stays fp32 in effect: it enters the product as two 16-bit parts,
//    in fp16 scaled by a power of two per 32 ranks, so that neither part leaves fp16's range.
#include <algorithm>

#include "decode_core.h"

namespace w4a4 {

constexpr int AD_WAVES = 4;

// The distinct adapters among a tile's rows, in the order of their first rows: calls f(id, rows) for the `lead`-th,
// `lead + leads`-th, ... of them. Rows without an adapter have id -1 and come as one of them.
template <typename F> __device__ __forceinline__ void for_adapters(const AdapterArgs &a, int64_t m0, int lead, F f)
{
    const int r = threadIdx.x & 15;
    int id = -1;
    if (m0 + r < a.M) {
        id = a.ids[m0 + r];
        if ((unsigned)id >= (unsigned)a.n) id = -1;
    }
    uint32_t left = (uint32_t)__ballot(m0 + r < a.M) & 0xFFFFu;
    for (int i = 0; left; ++i) {
        const int who = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
        const uint32_t rows = (uint32_t)__ballot(id == who) & left;
        left &= ~rows;
        if (i % a.leads == lead) f(who, rows);
    }
}

template <int DT, int RT> __global__ __launch_bounds__(64 * AD_WAVES) void k_adapter_in(const AdapterArgs a)
{
    __shared__ float red[AD_WAVES][RT][64][4];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = blockIdx.x % a.parts, lead = blockIdx.x / a.parts % a.leads, r0 = blockIdx.z * 16 * RT;
    const int64_t m0 = (int64_t)(blockIdx.y + a.tile0) * 16;
    const uint16_t *x = a.X + min(m0 + r, a.M - 1) * a.ldx;
    const int steps = (a.K + 31) / 32, per = (steps + a.parts * AD_WAVES - 1) / (a.parts * AD_WAVES);
    const int s0 = (part * AD_WAVES + wave) * per, s1 = min(steps, s0 + per);
    for_adapters(a, m0, lead, [&](int id, uint32_t rows) {
        if (id < 0) return;
        const uint16_t *w[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
            w[t] = a.A + (int64_t)id * a.stride_a + (int64_t)min(r0 + 16 * t + r, a.R - 1) * a.K;
        f4_t acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int s = s0; s < s1; ++s) {
            const int k = 32 * s + 8 * g, kc = min(k, a.K - 8);
            const u4_t zero = {0, 0, 0, 0};
            u4_t xv = load8_any(x + kc), wv[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) wv[t] = load8_any(w[t] + kc);
            if (32 * s + 32 > a.K) {  // runs past K are zeros on both sides
                xv = k < a.K ? xv : zero;
#pragma unroll
                for (int t = 0; t < RT; ++t) wv[t] = k < a.K ? wv[t] : zero;
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[t] = mma32<DT>(wv[t], xv, acc[t]);
        }
        __syncthreads();  // of the pass before this
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][t][lane][i] = acc[t][i];
        __syncthreads();
        // entry (t, l, i): rank r0 + 16 t + 4 (l / 16) + i of row l % 16
        for (int e = threadIdx.x; e < RT * 256; e += 64 * AD_WAVES) {
            const int i = e % 4, l = e / 4 % 64, t = e / 256, rank = r0 + 16 * t + l / 16 * 4 + i;
            float v = 0.0f;
#pragma unroll
            for (int u = 0; u < AD_WAVES; ++u) v += red[u][t][l][i];
            if (rank < a.R && (rows >> (l % 16) & 1))
                a.T[((int64_t)part * a.M + m0 + l % 16) * a.R + rank] = v;
        }
    });
}

__device__ __forceinline__ float gelu_erf(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

// A wave has 16 NT channels: operand row r of product t is channel 4 NT (r / 4) + 4 t + r % 4 of them, so that a lane's
// results are 4 NT neighbouring channels of its row.
template <int DT, int NT> __global__ __launch_bounds__(64 * AD_WAVES) void k_adapter_out(const AdapterArgs a)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m0 = (int64_t)(blockIdx.y + a.tile0) * 16, m = m0 + r, mc = min(m, a.M - 1);
    const int lead = blockIdx.x % a.leads, n0 = (blockIdx.x / a.leads * AD_WAVES + wave) * 16 * NT;
    if (n0 >= a.N) return;
    const int c0 = n0 + 4 * NT * g, live = a.N - c0;  // the lane's first channel, and how many there are
    for_adapters(a, m0, lead, [&](int id, uint32_t rows) {
        const bool mine = rows >> r & 1;
        if (id < 0 && a.Y == a.out && a.ldy == a.ldo && a.epilogue == W4A4_EPI_NONE) return;  // nothing to do
        float sum[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[t][i] = 0.0f;
        if (id >= 0) {
            const uint16_t *w[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                w[t] = a.B + (int64_t)id * a.stride_b +
                       (int64_t)min(n0 + 4 * NT * (r / 4) + 4 * t + r % 4, a.N - 1) * a.R;
            for (int j = 0; j < a.R; j += 32) {
                const int k = j + 8 * g, kc = min(k, a.R - 8);
                u4_t wv[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    wv[t] = load8_any(w[t] + kc);
                    if (j + 32 > a.R) wv[t] = k < a.R ? wv[t] : u4_t{0, 0, 0, 0};
                }
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.0f;
                if (mine && k < a.R) {  // rows of other adapters have no t of this one
                    const float *tp = a.T + mc * a.R + k;
                    for (int p = 0; p < a.parts; ++p, tp += a.M * a.R)
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] += tp[i];
                }
                float f = 1.0f;
                if constexpr (DT == W4A4_F16) {
                    float top = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
                    top = across_groups(top, [](float x, float y) { return fmaxf(x, y); });
                    // the largest becomes 2^14 to 2^15; nothing below 2^-100 counts
                    const uint32_t e = min(max(__builtin_bit_cast(uint32_t, top) >> 23, 27u), 240u);
                    f = __builtin_bit_cast(float, (e - 14u) << 23);
                    const float inv = __builtin_bit_cast(float, (254u - (e - 14u)) << 23);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= inv;
                }
                u4_t hi, lo;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hi[i] = pack16<DT>(v[2 * i], v[2 * i + 1]);
                    const f2_t h = unpack16<DT>(hi[i]);
                    // an infinity is whole in the first part
                    lo[i] = pack16<DT>(fabsf(h.x) == INFINITY ? 0.0f : v[2 * i] - h.x,
                                       fabsf(h.y) == INFINITY ? 0.0f : v[2 * i + 1] - h.y);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f4_t p = mma32<DT>(wv[t], lo, f4_t{0.0f, 0.0f, 0.0f, 0.0f});
                    p = mma32<DT>(wv[t], hi, p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[t][i] = fmaf(p[i], f, sum[t][i]);
                }
            }
        }
        if (!mine || live <= 0) return;
        const float s = id < 0 ? 0.0f : a.scale ? a.scale[id] : 1.0f;
        const uint16_t *y = a.Y + m * a.ldy + c0, *res = a.residual ? a.residual + m * a.ldr + c0 : nullptr;
        uint16_t *out = a.out + m * a.ldo + c0;
        auto finish = [&](float base, float v, float add) {
            v = id < 0 ? base : fmaf(v, s, base);
            return a.epilogue == W4A4_EPI_GELU ? gelu_erf(v) : v + add;
        };
        if (live >= 4 * NT) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const any2_t b = *reinterpret_cast<const any2_t *>(y + 4 * t);
                any2_t q = {0, 0};
                if (res) q = *reinterpret_cast<const any2_t *>(res + 4 * t);
                const f2_t b0 = unpack16<DT>(b[0]), b1 = unpack16<DT>(b[1]), q0 = unpack16<DT>(q[0]), q1 = unpack16<DT>(q[1]);
                *reinterpret_cast<any2_t *>(out + 4 * t) =
                    any2_t{pack16<DT>(finish(b0.x, sum[t][0], q0.x), finish(b0.y, sum[t][1], q0.y)),
                           pack16<DT>(finish(b1.x, sum[t][2], q1.x), finish(b1.y, sum[t][3], q1.y))};
            }
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * t + i < live)
                        out[4 * t + i] = (uint16_t)pack16<DT>(finish(unpack16<DT>(y[4 * t + i]).x, sum[t][i],
                                                                     res ? unpack16<DT>(res[4 * t + i]).x : 0.0f), 0.0f);
        }
    });
}

// Parts of K: enough workgroups for the chip when there are few tiles, but no fewer than 256 k each.
int adapter_parts(int64_t M, int K)
{
    const int64_t tiles = (M + 15) / 16;
    return (int)std::max<int64_t>(1, std::min<int64_t>({16, (K + 255) / 256, 256 / std::max<int64_t>(tiles, 1)}));
}

template <int DT> static int run_adapter(AdapterArgs a, hipStream_t s)
{
    const int64_t tiles = (a.M + 15) / 16;
    a.leads = tiles <= 16 ? 16 : tiles <= 128 ? 4 : 1;
    const int rt = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;
    constexpr int NT = 4;
    const int blocks = (a.N + 16 * NT * AD_WAVES - 1) / (16 * NT * AD_WAVES);
    for (a.tile0 = 0; a.tile0 < tiles; a.tile0 += 32768) {
        const unsigned y = (unsigned)std::min<int64_t>(32768, tiles - a.tile0);
        const dim3 in(a.parts * a.leads, y, (a.R + 16 * rt - 1) / (16 * rt)), out(blocks * a.leads, y);
        const dim3 block(64 * AD_WAVES);
        if (rt == 1) hipLaunchKernelGGL((k_adapter_in<DT, 1>), in, block, 0, s, a);
        else if (rt == 2) hipLaunchKernelGGL((k_adapter_in<DT, 2>), in, block, 0, s, a);
        else hipLaunchKernelGGL((k_adapter_in<DT, 4>), in, block, 0, s, a);
        if (int rc = check_launch("adapter_add inner")) return rc;
        hipLaunchKernelGGL((k_adapter_out<DT, NT>), out, block, 0, s, a);
        if (int rc = check_launch("adapter_add")) return rc;
    }
    return W4A4_OK;
}

int launch_adapter(const AdapterArgs &a, int dtype, hipStream_t s)
{
    return dtype == W4A4_BF16 ? run_adapter<W4A4_BF16>(a, s) : run_adapter<W4A4_F16>(a, s);
}

}  // namespace w4a4
