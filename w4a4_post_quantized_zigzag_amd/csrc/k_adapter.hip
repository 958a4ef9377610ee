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
#include <type_traits>

#include "decode_core.h"

namespace w4a4 {

constexpr int AD_WAVES = 4;

// The adapters of a tile's rows, one after another in the order of their first rows; this workgroup takes the `lead`-th,
// `lead + leads`-th, ... of them. Rows without an adapter count as one more, with id -1.
struct AdapterWalk {
    int id;         // of the lane's row m0 + lane % 16
    uint32_t left;  // rows not yet met
    int count;
    int who;        // the adapter met last, and its rows
    uint32_t rows;

    __device__ __forceinline__ void start(const AdapterArgs &a, int64_t m0)
    {
        const int64_t m = m0 + (threadIdx.x & 15);
        id = -1;
        if (m < a.M) {
            id = a.ids[m];
            if ((unsigned)id >= (unsigned)a.n) id = -1;
        }
        left = (uint32_t)__ballot(m < a.M) & 0xFFFFu;
        count = 0;
    }
    __device__ __forceinline__ bool next(const AdapterArgs &a, int lead)
    {
        while (left) {
            who = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
            rows = (uint32_t)__ballot(id == who) & left;
            left &= ~rows;
            if (count++ % a.leads == lead) return true;
        }
        return false;
    }
};

template <int DT, int RT> __global__ __launch_bounds__(64 * AD_WAVES) void k_adapter_in(const AdapterArgs a)
{
    constexpr int U = RT == 1 ? 8 : 4;  // steps of 32 k in flight
    __shared__ float red[AD_WAVES][RT][64][4];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = blockIdx.x % a.parts, lead = blockIdx.x / a.parts % a.leads, r0 = blockIdx.z * 16 * RT;
    const int64_t m0 = (int64_t)(blockIdx.y + a.tile0) * 16;
    const uint16_t *x = a.X + min(m0 + r, a.M - 1) * a.ldx + 8 * g;
    const int steps = (a.K + 31) / 32, per = (steps + a.parts * AD_WAVES - 1) / (a.parts * AD_WAVES);
    const int s0 = (part * AD_WAVES + wave) * per, s1 = min(steps, s0 + per);
    const int most = a.K - 8 - 8 * g;  // the last run's k
    AdapterWalk walk;
    walk.start(a, m0);
    while (walk.next(a, lead)) {
        if (walk.who < 0) continue;
        const uint16_t *w[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
            w[t] = a.A + (int64_t)walk.who * a.stride_a + (int64_t)min(r0 + 16 * t + r, a.R - 1) * a.K + 8 * g;
        f4_t acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
        auto block = [&](int s, auto last) {  // steps s .. s + U - 1; the last ones may reach past K or s1
            u4_t xv[U], wv[U][RT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = last.value ? min(32 * (s + u), most) : 32 * (s + u);
                xv[u] = load8_any(x + k);
#pragma unroll
                for (int t = 0; t < RT; ++t) wv[u][t] = load8_any(w[t] + k);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (last.value) {  // what is past the end is zeros on both sides
                    const bool on = s + u < s1 && 32 * (s + u) <= most;
                    const u4_t zero = {0, 0, 0, 0};
                    xv[u] = on ? xv[u] : zero;
#pragma unroll
                    for (int t = 0; t < RT; ++t) wv[u][t] = on ? wv[u][t] : zero;
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) acc[t] = mma32<DT>(wv[u][t], xv[u], acc[t]);
            }
        };
        int s = s0;
        for (; s + U < s1; s += U) block(s, std::false_type());
        if (s < s1) block(s, std::true_type());
        __syncthreads();  // of the pass before this
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][t][lane][i] = acc[t][i];
        __syncthreads();
        // entry (t, l, i): rank r0 + 16 t + 4 (l / 16) + i of row l % 16; R is a multiple of 8
        for (int e = threadIdx.x; e < RT * 64; e += 64 * AD_WAVES) {
            const int l = e % 64, t = e / 64, rank = r0 + 16 * t + l / 16 * 4;
            f4_t v = *reinterpret_cast<const f4_t *>(red[0][t][l]);
#pragma unroll
            for (int u = 1; u < AD_WAVES; ++u) v += *reinterpret_cast<const f4_t *>(red[u][t][l]);
            if (rank < a.R && (walk.rows >> (l % 16) & 1))
                *reinterpret_cast<f4_t *>(a.T + ((int64_t)part * a.M + m0 + l % 16) * a.R + rank) = v;
        }
    }
}

__device__ __forceinline__ float gelu_erf(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

// A wave has 16 rows and 16 NT channels: operand row r of product t is channel 4 NT (r / 4) + 4 t + r % 4 of them, so
// that a lane's results are 4 NT neighbouring channels of its row. Every row's inner products are its own adapter's,
// whichever adapter the pass is for: they are made into operands once, and each pass keeps its own rows' columns.
// J: blocks of 32 ranks.
template <int DT, int J, int NT> __global__ __launch_bounds__(64 * AD_WAVES) void k_adapter_out(const AdapterArgs a)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the waves of a workgroup are row_waves tiles of rows by AD_WAVES / row_waves blocks of channels
    const int64_t tile = (int64_t)(blockIdx.y * a.row_waves + wave % a.row_waves) + a.tile0;
    const int64_t m0 = tile * 16, m = m0 + r, mc = min(m, a.M - 1);
    const int lead = blockIdx.x % a.leads;
    const int n0 = (blockIdx.x / a.leads * (AD_WAVES / a.row_waves) + wave / a.row_waves) * 16 * NT;
    if (n0 >= a.N || m0 >= a.M) return;
    const int c0 = n0 + 4 * NT * g, live = a.N - c0;  // the lane's first channel, and how many there are
    AdapterWalk walk;
    walk.start(a, m0);

    // all that does not depend on the adapter is asked for first
    float v[J][8];
    {
        const float *tp = a.T + mc * a.R + 8 * g;
        const int64_t next = a.M * a.R;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const f4_t *q = reinterpret_cast<const f4_t *>(tp + min(32 * j, a.R - 8 - 8 * g));
            const f4_t x = q[0], y = q[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = x[i], v[j][4 + i] = y[i];
        }
        for (int p = 1; p < a.parts; ++p) {
            tp += next;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const f4_t *q = reinterpret_cast<const f4_t *>(tp + min(32 * j, a.R - 8 - 8 * g));
                const f4_t x = q[0], y = q[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j][i] += x[i], v[j][4 + i] += y[i];
            }
        }
    }
    const bool whole = live >= 4 * NT;
    any2_t base[NT], add[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) base[t] = add[t] = any2_t{0, 0};
    const uint16_t *yp = a.Y + mc * a.ldy + c0, *rp = a.residual ? a.residual + mc * a.ldr + c0 : nullptr;
    auto load4 = [&](const uint16_t *p, int t) {  // channels 4 t .. 4 t + 3
        any2_t x = {0, 0};
        if (whole) return *reinterpret_cast<const any2_t *>(p + 4 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * t + i < live) x[i / 2] |= (uint32_t)p[4 * t + i] << (16 * (i % 2));
        return x;
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) base[t] = load4(yp, t);
    if (rp)
#pragma unroll
        for (int t = 0; t < NT; ++t) add[t] = load4(rp, t);

    u4_t hi[J], lo[J];
    float f[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (32 * j + 8 * g >= a.R)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
        f[j] = 1.0f;
        if constexpr (DT == W4A4_F16) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[j][i]));
            top = across_groups(top, [](float x, float y) { return fmaxf(x, y); });
            // the largest becomes 2^14 to 2^15; what is below 2^-100 is left as small as it is
            const uint32_t e = min(max(__builtin_bit_cast(uint32_t, top) >> 23, 27u), 240u);
            f[j] = __builtin_bit_cast(float, (e - 14u) << 23);
            const float inv = __builtin_bit_cast(float, (254u - (e - 14u)) << 23);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] *= inv;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[j][i] = pack16<DT>(v[j][2 * i], v[j][2 * i + 1]);
            const uint32_t w = hi[j][i];
            const f2_t h = unpack16<DT>(w);
            // an infinity is whole in the first part
            lo[j][i] = pack16<DT>(fabsf(h.x) == INFINITY ? 0.0f : v[j][2 * i] - h.x,
                                  fabsf(h.y) == INFINITY ? 0.0f : v[j][2 * i + 1] - h.y);
        }
    }

    float sum[NT][4], s = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[t][i] = 0.0f;
    uint32_t kept = 0;  // rows that are this workgroup's to write
    bool has = false;   // the lane's row has an adapter
    int64_t wrow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        wrow[t] = (int64_t)min(n0 + 4 * NT * (r / 4) + 4 * t + r % 4, a.N - 1) * a.R + 8 * g;
    while (walk.next(a, lead)) {
        if (walk.who < 0) {
            // rows without an adapter that are already what they shall be
            if (!(a.Y == a.out && a.ldy == a.ldo && a.epilogue == W4A4_EPI_NONE)) kept |= walk.rows;
            continue;
        }
        kept |= walk.rows;
        const bool mine = walk.rows >> r & 1;
        const uint16_t *w = a.B + (int64_t)walk.who * a.stride_b;
        u4_t wv[J][NT];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int t = 0; t < NT; ++t) wv[j][t] = load8_any(w + wrow[t] + min(32 * j, a.R - 8 - 8 * g));
        const float sc = a.scale ? a.scale[walk.who] : 1.0f;
        if (mine) {
            s = sc;
            has = true;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (32 * j + 32 > a.R && 32 * j + 8 * g >= a.R) wv[j][t] = u4_t{0, 0, 0, 0};
                f4_t p = mma32<DT>(wv[j][t], lo[j], f4_t{0.0f, 0.0f, 0.0f, 0.0f});
                p = mma32<DT>(wv[j][t], hi[j], p);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[t][i] = mine ? fmaf(p[i], f[j], sum[t][i]) : sum[t][i];
            }
    }
    if (!(kept >> r & 1) || live <= 0) return;
    uint16_t *out = a.out + m * a.ldo + c0;
    auto finish = [&](float y, float x, float z) {
        y = has ? fmaf(x, s, y) : y;
        return a.epilogue == W4A4_EPI_GELU ? gelu_erf(y) : y + z;
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const f2_t y0 = unpack16<DT>(base[t][0]), y1 = unpack16<DT>(base[t][1]);
        const f2_t z0 = unpack16<DT>(add[t][0]), z1 = unpack16<DT>(add[t][1]);
        const any2_t o = {pack16<DT>(finish(y0.x, sum[t][0], z0.x), finish(y0.y, sum[t][1], z0.y)),
                          pack16<DT>(finish(y1.x, sum[t][2], z1.x), finish(y1.y, sum[t][3], z1.y))};
        if (whole) {
            *reinterpret_cast<any2_t *>(out + 4 * t) = o;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * t + i < live) out[4 * t + i] = (uint16_t)(o[i / 2] >> (16 * (i % 2)));
        }
    }
}

// Parts of K: 1024 k for the four waves of a workgroup, all loads of a wave in flight at once, while that leaves few
// enough workgroups; every part is read again by each workgroup of the second launch.
int adapter_parts(int64_t M, int K)
{
    const int64_t tiles = (M + 15) / 16;
    return (int)std::max<int64_t>(1, std::min<int64_t>({16, (K + 1023) / 1024, 64 / std::max<int64_t>(tiles, 1)}));
}

template <int DT, int J, int NT> static void run_out(AdapterArgs a, int64_t tiles, hipStream_t s)
{
    const int across = AD_WAVES / a.row_waves, blocks = (a.N + 16 * NT * across - 1) / (16 * NT * across);
    hipLaunchKernelGGL((k_adapter_out<DT, J, NT>), dim3(blocks * a.leads, (tiles + a.row_waves - 1) / a.row_waves),
                       dim3(64 * AD_WAVES), 0, s, a);
}

template <int DT, int J> static void pick_out(const AdapterArgs &a, int64_t tiles, hipStream_t s)
{
    run_out<DT, J, J >= 4 ? 2 : 4>(a, tiles, s);
}

template <int DT> static int run_adapter(AdapterArgs a, hipStream_t s)
{
    const int64_t tiles = (a.M + 15) / 16;
    const int leads = tiles <= 16 ? 16 : tiles <= 128 ? 4 : 1;
    const int rt = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;
    for (a.tile0 = 0; a.tile0 < tiles; a.tile0 += 32768) {
        const unsigned y = (unsigned)std::min<int64_t>(32768, tiles - a.tile0);
        a.leads = leads;
        a.row_waves = 1;
        const dim3 in(a.parts * a.leads, y, (a.R + 16 * rt - 1) / (16 * rt)), block(64 * AD_WAVES);
        if (rt == 1) hipLaunchKernelGGL((k_adapter_in<DT, 1>), in, block, 0, s, a);
        else if (rt == 2) hipLaunchKernelGGL((k_adapter_in<DT, 2>), in, block, 0, s, a);
        else hipLaunchKernelGGL((k_adapter_in<DT, 4>), in, block, 0, s, a);
        if (int rc = check_launch("adapter_add inner")) return rc;
        a.leads = tiles <= 16 ? 4 : 1;
        a.row_waves = tiles > 16 ? 4 : 1;
        if (a.R <= 32) pick_out<DT, 1>(a, y, s);
        else if (a.R <= 64) pick_out<DT, 2>(a, y, s);
        else if (a.R <= 128) pick_out<DT, 4>(a, y, s);
        else pick_out<DT, 8>(a, y, s);
        if (int rc = check_launch("adapter_add")) return rc;
    }
    return W4A4_OK;
}

int launch_adapter(const AdapterArgs &a, int dtype, hipStream_t s)
{
    return dtype == W4A4_BF16 ? run_adapter<W4A4_BF16>(a, s) : run_adapter<W4A4_F16>(a, s);
}

}  // namespace w4a4
