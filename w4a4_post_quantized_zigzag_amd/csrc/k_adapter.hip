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
//  - outer: [channels x rows] = B (A operand) . t^T. t enters the product as two 16-bit parts, which in bf16 drop 2^-17 of
//    it. In fp16 they are scaled by a power of two per 32 ranks that takes the largest of them to 2^14 or above, so that
//    neither part leaves fp16's range; they drop 2^-22 of t, and where the second is subnormal half its step, 2^-39 of that
//    largest.
// For up to four rows of up to 16 ranks and 2048 k one launch does both: each workgroup of the second makes the inner
// products it needs itself, in the same order.
// Measured (MI355X): 32 rows of 24 adapters, 16 ranks, 2048 -> 16384 channels: 5.0 us inner, 9.0 outer, bound by the launches
// and by one adapter's weights after another (12.6 MB at 1.4 TB/s); 1600 rows of 64 ranks, 1024 -> 4099, one adapter for 50
// rows: 8.9 inner (a tile's rows and one or two adapters, one after the other, read by few waves), 19.9 outer (37 MB in and
// out at 1.9 TB/s, vector units 26 % busy); one row, 1024 -> 1024, in one launch: 5.6.
#include <algorithm>
#include <type_traits>

#include "decode_core.h"

namespace w4a4 {

constexpr int IN_WAVES = 4, OUT_WAVES = 4;

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

// One wave's steps s0 .. s1 of 32 k each: [ranks x rows] into acc. x and w point at the lane's row and 8 k of each; U
// steps are in flight; most: the lane's last run of 8 k.
template <int DT, int RT, int U>
__device__ __forceinline__ void inner_steps(const uint16_t *x, const uint16_t *const (&w)[RT], int s0, int s1, int most,
                                            f4_t (&acc)[RT])
{
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
}

template <int DT, int RT, int U> __global__ __launch_bounds__(64 * IN_WAVES) void k_adapter_in(const AdapterArgs a)
{
    __shared__ float red[IN_WAVES][RT][64][4];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = blockIdx.x % a.parts, lead = blockIdx.x / a.parts % a.leads, r0 = blockIdx.z * 16 * RT;
    const int64_t m0 = (int64_t)(blockIdx.y + a.tile0) * 16;
    const uint16_t *x = a.X + min(m0 + r, a.M - 1) * a.ldx + 8 * g;
    const int steps = (a.K + 31) / 32, per = (steps + a.parts * IN_WAVES - 1) / (a.parts * IN_WAVES);
    const int s0 = (part * IN_WAVES + wave) * per, s1 = min(steps, s0 + per);
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
        inner_steps<DT, RT, U>(x, w, s0, s1, most, acc);
        __syncthreads();  // of the pass before this
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][t][lane][i] = acc[t][i];
        __syncthreads();
        // entry (t, l, i): rank r0 + 16 t + 4 (l / 16) + i of row l % 16; R is a multiple of 8
        for (int e = threadIdx.x; e < RT * 64; e += 64 * IN_WAVES) {
            const int l = e % 64, t = e / 64, rank = r0 + 16 * t + l / 16 * 4;
            f4_t v = *reinterpret_cast<const f4_t *>(red[0][t][l]);
#pragma unroll
            for (int u = 1; u < IN_WAVES; ++u) v += *reinterpret_cast<const f4_t *>(red[u][t][l]);
            if (rank < a.R && (walk.rows >> (l % 16) & 1))
                *reinterpret_cast<f4_t *>(a.T + ((int64_t)part * a.M + m0 + l % 16) * a.R + rank) = v;
        }
    }
}

__device__ __forceinline__ float gelu_erf(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

// A wave has 16 rows and a block of 16 NT channels at a time. What limits it is not the bytes but the lines that its
// loads touch: the matrix operands want neighbouring lanes in neighbouring rows, which is a line per lane (20 million
// line accesses for 1600 rows of 64 ranks through 4099 channels, 35 us). So the block's weights, which are one run of
// memory, are loaded as they lie there, LP lanes to a row of ranks, and pass through a corner of LDS of the wave's own
// (rows padded to an odd number of 16-byte slots, free of bank conflicts on both sides); the results go back through
// it, so that Y, the residual and the output are touched row by row as well.
// Every row's inner products are its own adapter's, whichever adapter a pass is for: they are made into operands once,
// and each pass keeps its own rows' columns.
//  - WALK: the wave walks run_blocks blocks of channels, with the next block's Y and first adapter's weights on their
//    way: few adapters per tile of rows, many tiles.
//  - else it has one block, and the next adapter's weights are on their way: many adapters, few tiles.
// What is on its way is asked for without branches (the last one once more at the end), for a wait behind a branch is
// a wait for everything. LP: lanes to a row of weights, 8 LP >= R. SMALL: N below 8. ONE: there was no first launch.
template <int DT, int LP, bool WALK, bool SMALL, bool ONE = false>
__global__ __launch_bounds__(64 * OUT_WAVES) __attribute__((amdgpu_waves_per_eu(LP < 8 ? 4 : LP == 8 ? 3 : 2)))
void k_adapter_out(const AdapterArgs a)
{
    constexpr int NT = LP <= 8 ? 4 : LP == 16 ? 2 : 1, C = 16 * NT, J = LP < 4 ? 1 : LP / 4;
    constexpr int SLOTS = LP + 1, LOADS = C * LP / 64;     // of weights per block
    constexpr int CL = C / 8, IO = 16 * CL / 64 > 0 ? 16 * CL / 64 : 1;  // lanes to a row of Y, loads of 16 rows
    constexpr int RES = C + 4;                              // floats between the rows of the results
    constexpr int AREA = C * SLOTS * 16 > 16 * RES * 4 ? C * SLOTS * 16 : 16 * RES * 4;
    __shared__ __attribute__((aligned(16))) uint8_t area[OUT_WAVES][AREA];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The waves of a workgroup are row_waves tiles of rows by OUT_WAVES / row_waves runs of blocks. Consecutive
    // workgroups go to different XCDs: a run of channels stays on one, whose L2 then reads its part of each B once.
    const int unit = blockIdx.x / 8, lead = unit % a.leads, runs8 = (a.out_runs + 7) / 8;
    const int run = unit / a.leads % runs8 * 8 + blockIdx.x % 8;
    const int64_t tile = (int64_t)(unit / a.leads / runs8) * a.row_waves + wave % a.row_waves + a.tile0;
    const int64_t m0 = tile * 16, mc = min(m0 + r, a.M - 1);
    const int first = (run * (OUT_WAVES / a.row_waves) + wave / a.row_waves) * a.run_blocks * C;
    const int end = min(a.N, first + a.run_blocks * C);
    if (run >= a.out_runs || (!ONE && (first >= end || m0 >= a.M))) return;
    u4_t *slots = reinterpret_cast<u4_t *>(area[wave]);
    float *results = reinterpret_cast<float *>(area[wave]);

    // all that does not depend on the adapter is asked for first: the rows' inner products, their part of Y, their ids
    float v[J][8];
    const float *tp = a.T + mc * a.R + 8 * g;
    auto inner = [&](int j, const float *t) {
        const f4_t *q = reinterpret_cast<const f4_t *>(t + min(32 * j, a.R - 8 - 8 * g));
        const f4_t x = q[0], y = q[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] += x[i], v[j][4 + i] += y[i];
    };
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
        if (!ONE) inner(j, tp);
    }
    // as holder of Y: row lane / CL of each 64 / CL, eight channels from 8 (lane % CL)
    const int ch = lane % CL * 8;
    int64_t row[IO];
    int rid[IO];
#pragma unroll
    for (int i = 0; i < IO; ++i) {
        row[i] = min(m0 + min(i * (64 / CL) + lane / CL, 15), a.M - 1);
        rid[i] = a.ids[row[i]];
    }
    struct Rows {
        u4_t y[IO];
    };
    const bool residual = a.residual != nullptr;
    const uint16_t *zbase = residual ? a.residual : a.Y;
    const int64_t ldz = residual ? a.ldr : a.ldy;
    auto load_rows = [&](int n0, Rows &d) {
        if constexpr (!SMALL) {
            const int c = min(n0 + ch, a.N - 8);  // what reaches past N is read again, element by element
#pragma unroll
            for (int i = 0; i < IO; ++i) d.y[i] = load8_any(a.Y + row[i] * a.ldy + c);
        }
    };
    Rows rows;
    load_rows(first, rows);
    AdapterWalk walk;
    walk.start(a, m0);
    float rscale[IO];
    bool rhas[IO];
#pragma unroll
    for (int i = 0; i < IO; ++i) {
        rhas[i] = (unsigned)rid[i] < (unsigned)a.n;
        rscale[i] = rhas[i] && a.scale ? a.scale[rid[i]] : 1.0f;
    }
    // rows without an adapter that are already what they shall be need no pass
    const bool idle = a.Y == a.out && a.ldy == a.ldo && a.epilogue == W4A4_EPI_NONE;
    auto next_adapter = [&]() {
        while (walk.next(a, lead))
            if (walk.who >= 0 || !idle) return true;
        return false;
    };
    if (!next_adapter()) return;
    // as loader of weights: row lane / LP of each 64 / LP, eight ranks from 8 (lane % LP)
    struct Weights {
        u4_t w[LOADS];
    };
    const int wrank = min(lane % LP * 8, a.R - 8);
    auto load_weights = [&](int n0, int who, Weights &d) {  // without an adapter the first one's, unused
        const uint16_t *w = a.B + (int64_t)max(who, 0) * a.stride_b + wrank;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            d.w[i] = load8_any(w + (int64_t)min(n0 + i * (64 / LP) + lane / LP, a.N - 1) * a.R);
    };
    Weights w;
    load_weights(first, walk.who, w);

    if constexpr (ONE) {  // the sums of k_adapter_in, in its order, by all waves of the workgroup
        constexpr int RT = LP < 4 ? 1 : 2;
        __shared__ __attribute__((aligned(16))) float products[16][8 * LP + 4];
        static_assert(AREA >= RT * 1024, "");
        const int steps = (a.K + 31) / 32, per = (steps + a.parts * OUT_WAVES - 1) / (a.parts * OUT_WAVES);
        AdapterWalk again;
        again.start(a, m0);
        while (again.next(a, lead)) {
            if (again.who < 0) continue;
            for (int r0 = 0; r0 < a.R; r0 += 16 * RT) {
                const uint16_t *wi[RT];
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    wi[t] = a.A + (int64_t)again.who * a.stride_a + (int64_t)min(r0 + 16 * t + r, a.R - 1) * a.K + 8 * g;
                for (int part = 0; part < a.parts; ++part) {
                    f4_t acc[RT];
#pragma unroll
                    for (int t = 0; t < RT; ++t) acc[t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
                    const int s0 = (part * OUT_WAVES + wave) * per;
                    inner_steps<DT, RT, 8>(a.X + mc * a.ldx + 8 * g, wi, s0, min(steps, s0 + per), a.K - 8 - 8 * g, acc);
                    __syncthreads();  // of the part before this
#pragma unroll
                    for (int t = 0; t < RT; ++t) reinterpret_cast<f4_t *>(area[wave])[64 * t + lane] = acc[t];
                    __syncthreads();
                    const int e = threadIdx.x, l = e % 64, rank = r0 + e / 64 * 16 + l / 16 * 4;
                    if (e < RT * 64 && rank < a.R && (again.rows >> (l % 16) & 1)) {
                        f4_t q = reinterpret_cast<const f4_t *>(area[0])[e];
#pragma unroll
                        for (int u = 1; u < OUT_WAVES; ++u) q += reinterpret_cast<const f4_t *>(area[u])[e];
                        f4_t *to = reinterpret_cast<f4_t *>(&products[l % 16][rank]);
                        *to = part ? *to + q : q;
                    }
                }
            }
        }
        __syncthreads();
        if (first >= end) return;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const f4_t *q = reinterpret_cast<const f4_t *>(&products[r][min(32 * j + 8 * g, a.R - 8)]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = q[0][i], v[j][4 + i] = q[1][i];
        }
    } else {
        for (int p = 1; p < a.parts; ++p) {
            tp += a.M * a.R;
#pragma unroll
            for (int j = 0; j < J; ++j) inner(j, tp);
        }
    }
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
            const uint32_t x = pack16<DT>(v[j][2 * i], v[j][2 * i + 1]);
            hi[j][i] = x;
            const f2_t h = unpack16<DT>(x);
            // an infinity is whole in the first part
            lo[j][i] = pack16<DT>(fabsf(h.x) == INFINITY ? 0.0f : v[j][2 * i] - h.x,
                                  fabsf(h.y) == INFINITY ? 0.0f : v[j][2 * i + 1] - h.y);
        }
    }

    f4_t sum[NT];
    uint32_t met = 0;  // rows of the passes so far
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](int who, uint32_t of, const Weights &d) {
        met |= of;
        const bool mine = who >= 0 && (of >> r & 1);
        lds_fence();
#pragma unroll
        for (int i = 0; i < LOADS; ++i) slots[(i * (64 / LP) + lane / LP) * SLOTS + lane % LP] = d.w[i];
        lds_fence();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                // runs past R are zeros on both sides
                u4_t x = slots[(16 * t + r) * SLOTS + (LP < 4 ? g % LP : 4 * j + g)];
                if ((LP < 4 || a.R != 8 * LP) && 32 * j + 8 * g >= a.R) x = u4_t{0, 0, 0, 0};
                f4_t q = mma32<DT>(x, lo[j], f4_t{0.0f, 0.0f, 0.0f, 0.0f});
                q = mma32<DT>(x, hi[j], q);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[t][i] = mine ? fmaf(q[i], f[j], sum[t][i]) : sum[t][i];
            }
    };
    auto finish = [&](int i, float y, float x, float z) {
        y = rhas[i] ? fmaf(x, rscale[i], y) : y;
        return a.epilogue == W4A4_EPI_GELU ? gelu_erf(y) : residual ? y + z : y;
    };
    auto store = [&](int n0, const Rows &d) {
        u4_t res[IO];
        if (!SMALL && residual)
#pragma unroll
            for (int i = 0; i < IO; ++i) res[i] = load8_any(zbase + row[i] * ldz + min(n0 + ch, a.N - 8));
        lds_fence();
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<f4_t *>(results + r * RES + 16 * t + 4 * g) = sum[t];
        lds_fence();
        const int c = n0 + ch;
#pragma unroll
        for (int i = 0; i < IO; ++i) {
            const int q = i * (64 / CL) + lane / CL;  // row of the tile
            const float *x = results + min(q, 15) * RES + ch;
            const f4_t x0 = reinterpret_cast<const f4_t *>(x)[0], x1 = reinterpret_cast<const f4_t *>(x)[1];
            if (q > 15 || !(met >> q & 1)) continue;
            uint16_t *out = a.out + row[i] * a.ldo + c;
            if (!SMALL && c + 8 <= a.N) {
                u4_t o;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t yw = d.y[i][e], zw = residual ? res[i][e] : 0u;
                    const f2_t y = unpack16<DT>(yw), z = unpack16<DT>(zw);
                    o[e] = pack16<DT>(finish(i, y.x, e < 2 ? x0[2 * e] : x1[2 * e - 4], z.x),
                                      finish(i, y.y, e < 2 ? x0[2 * e + 1] : x1[2 * e - 3], z.y));
                }
                store8_any(out, o);
            } else {
                const uint16_t *y = a.Y + row[i] * a.ldy + c, *z = zbase + row[i] * ldz + c;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < a.N)
                        out[e] = (uint16_t)pack16<DT>(finish(i, unpack16<DT>(y[e]).x, e < 4 ? x0[e] : x1[e - 4],
                                                             unpack16<DT>(z[e]).x), 0.0f);
            }
        }
    };
    if constexpr (WALK) {
        const int who = walk.who, behind_count = walk.count;
        const uint32_t of = walk.rows, behind = walk.left;
        for (int n0 = first; n0 < end; n0 += C) {
            const int n1 = n0 + C < end ? n0 + C : n0;
            Rows rn;
            Weights wn;
            load_rows(n1, rn);
            load_weights(n1, who, wn);
            multiply(who, of, w);
            walk.left = behind;
            walk.count = behind_count;
            while (next_adapter()) {  // the tile's other adapters
                Weights more;
                load_weights(n0, walk.who, more);
                multiply(walk.who, walk.rows, more);
            }
            store(n0, rows);
#pragma unroll
            for (int t = 0; t < NT; ++t) sum[t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
            rows = rn;
            w = wn;
        }
    } else {
        bool more = true;
        while (more) {
            const int who = walk.who;
            const uint32_t of = walk.rows;
            more = next_adapter();
            Weights next;
            load_weights(first, walk.who, next);
            multiply(who, of, w);
            w = next;
        }
        store(first, rows);
    }
}

// Parts of K for the first launch: up to 1024 workgroups of active tiles, each wave at least 64 k; every part is read
// again by each wave of the second launch.
int adapter_parts(int64_t M, int K)
{
    const int64_t tiles = (M + 15) / 16;
    if (tiles <= 16) return (int)std::clamp<int64_t>((K + 1023) / 1024, 1, 16);
    return (int)std::clamp<int64_t>(std::min<int64_t>(512 / tiles, K / 512), 1, 16);
}

template <int DT, int LP> static void run_out(AdapterArgs a, int64_t tiles, bool walk, bool one, hipStream_t s)
{
    constexpr int C = 16 * (LP <= 8 ? 4 : LP == 16 ? 2 : 1);
    a.row_waves = walk ? 4 : 1;
    const int across = OUT_WAVES / a.row_waves, blocks = (a.N + C - 1) / C;
    const int64_t groups = (tiles + a.row_waves - 1) / a.row_waves;
    // A walk is long enough to leave 8 waves a CU, 12 where a wave needs few registers (1600 rows of 64 ranks, 4099 channels:
    // 28.5 us with 8, 29.9 with 12, 32.0 with 16; 16 ranks, 16384 channels: 45.1, 37.8 and 41.4).
    constexpr int WAVES = 256 * (LP == 2 ? 12 : 8);
    a.run_blocks = walk ? (int)std::clamp<int64_t>((int64_t)blocks * groups * a.row_waves / WAVES, 1, 16) : 1;
    a.out_runs = (blocks + a.run_blocks * across - 1) / (a.run_blocks * across);
    // A tile's adapters are dealt to enough workgroups for one on each CU: fewer wait for one adapter after another, more
    // wait to start (32 rows of 24 adapters, 16384 channels: 14.5 us at 256 workgroups, 16.4 at 128, 16.2 at 512, 19.3 at
    // 1024; 64 rows of 32 adapters of 64 ranks, 4096: 19.7, 21.2, 20.4, 26.7).
    const int64_t alone = a.out_runs * tiles;
    a.leads = walk ? 1 : (int)std::min<int64_t>({(255 + alone) / alone, 16, a.n + 1, a.M});
    const dim3 grid((unsigned)((a.out_runs + 7) / 8 * 8 * a.leads * groups)), block(64 * OUT_WAVES);
    if constexpr (LP == 2) {
        if (one) {
            hipLaunchKernelGGL((k_adapter_out<DT, LP, false, false, true>), grid, block, 0, s, a);
            return;
        }
    }
    if (a.N < 8) hipLaunchKernelGGL((k_adapter_out<DT, LP, false, true>), grid, block, 0, s, a);
    else if (walk) hipLaunchKernelGGL((k_adapter_out<DT, LP, true, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_adapter_out<DT, LP, false, false>), grid, block, 0, s, a);
}

template <int DT, int RT> static void run_in(const AdapterArgs &a, int64_t tiles, hipStream_t s)
{
    const dim3 grid(a.parts * a.leads, (unsigned)tiles, (a.R + 16 * RT - 1) / (16 * RT)), block(64 * IN_WAVES);
    const int per = ((a.K + 31) / 32 + a.parts * IN_WAVES - 1) / (a.parts * IN_WAVES);  // a wave's steps
    if (per <= 2) hipLaunchKernelGGL((k_adapter_in<DT, RT, 2>), grid, block, 0, s, a);
    else if (per <= 4) hipLaunchKernelGGL((k_adapter_in<DT, RT, 4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_adapter_in<DT, RT, 8>), grid, block, 0, s, a);
}

template <int DT> static int run_adapter(AdapterArgs a, hipStream_t s)
{
    const int64_t tiles = (a.M + 15) / 16;
    const bool many = tiles > 16;
    // a launch holds less than 2^32 threads: at most 2^23 workgroups of 256
    const int64_t most = std::clamp<int64_t>(((int64_t)1 << 23) / ((int64_t)a.N / 16 + 64) / 4 * 4, 4, 32768);
    for (a.tile0 = 0; a.tile0 < tiles; a.tile0 += most) {
        const int64_t y = std::min<int64_t>(most, tiles - a.tile0);
        // A tile's adapters go to workgroups of their own while those are few. Where they are many, those without one cost
        // rows in runs more than the others wait (dealt out and not: 2048 rows, one adapter for 400, 4096 k 27.6 and 22.4 us;
        // 2000 rows of 17 adapters of 32 ranks, 1024 k, 21.5 and 17.9; 600 such rows 11.2 and 10.7). Mixed rows gain at any
        // count (307 of 27 adapters 18.8 and 26.9; 600 of 17 25.0 and 39.4; 2000 of 17 71.3 and 76.1), which only the ids,
        // on the device, could tell.
        const int64_t room = tiles > 32 ? 1 : many ? 1024 / (tiles * a.parts * ((a.R + 31) / 32)) : 16;
        a.leads = (int)std::min<int64_t>({std::max<int64_t>(room, 1), 16, a.n, a.M});
        // A launch less for a few short rows (a row of 16 ranks, 1024x1024: 5.5 us in a graph against 6.8; 2048x2048: 7.0
        // against 7.1, and 9.8 against 7.5 with four parts, 10.2 against 8.6 with 64 ranks; 16 rows of 16 adapters 13.3
        // against 10.4: the workgroups make one adapter's products after another's).
        const bool one = a.M <= 4 && a.R <= 16 && a.N >= 8 && a.parts <= 2;
        if (!one) {
            if (a.R <= 16) run_in<DT, 1>(a, y, s);
            else run_in<DT, 2>(a, y, s);
            if (int rc = check_launch("adapter_add inner")) return rc;
        }
        const bool walk = many && a.N >= 8;
        if (a.R <= 16) run_out<DT, 2>(a, y, walk, one, s);
        else if (a.R <= 32) run_out<DT, 4>(a, y, walk, one, s);
        else if (a.R <= 64) run_out<DT, 8>(a, y, walk, one, s);
        else if (a.R <= 128) run_out<DT, 16>(a, y, walk, one, s);
        else run_out<DT, 32>(a, y, walk, one, s);
        if (int rc = check_launch("adapter_add")) return rc;
    }
    return W4A4_OK;
}

int launch_adapter(const AdapterArgs &a, int dtype, hipStream_t s)
{
    return dtype == W4A4_BF16 ? run_adapter<W4A4_BF16>(a, s) : run_adapter<W4A4_F16>(a, s);
}

}  // namespace w4a4
