// The quantized key-value cache: rows into it and back, the attention of one new token per sequence over it, and the
// same attention behind a prefix that all sequences of a batch share (over a quantized or a 16-bit cache).
#include <algorithm>
#include <type_traits>

#include "kv_tile.h"

namespace w4a4 {

// ================================================================================================
// Rows as they are into the cache, and back. A lane takes eight channels of one head of one token, a head is LH
// lanes, so that the largest of a head (or of 32 channels) is found by a few moves between neighbouring lanes, and each
// access is 16 bytes of a row. Bound by the bytes: 8191 tokens of 8 + 8 heads of 128 are read back from 4 bits in 11.2 us
// (9 MB in, 34 MB out: 3.8 TB/s), 1600 of 16 + 16 heads of 64 from 8 bits in 3.4; small calls by their launch (1.6 us).
// The fused write is k_norm_rope's (8191 tokens of 32 + 8 heads of 128: 36.0 us, as with a 16-bit cache).
// ================================================================================================
template <int DT, int F, int LH> __global__ __launch_bounds__(256) void k_kv_append(const KvRowsArgs a)
{
    const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LH;  // key and value heads of all tokens
    const int d = threadIdx.x % LH * 8;
    const int64_t heads = 2 * a.kv_heads, m = id / heads;
    const int h = (int)(id % heads);
    const bool is_v = h >= a.kv_heads, on = m < a.M && d < a.D;
    const int64_t mc = min(m, a.M - 1);
    const uint16_t *row = is_v ? a.v + mc * a.ldv + (h - a.kv_heads) * a.D : a.k + mc * a.ldk + h * a.D;
    const QuantRun<F> q = quant_run<DT, F, LH>(load8_any(row + (d < a.D ? d : 0)));
    const KvSlot s = kv_slot(a.kv, a.slots[mc]);
    if (!on || s.page < 0) return;
    quant_store<F>(a.kv, is_v ? a.kv.v : a.kv.k, is_v ? a.kv.v_scale : a.kv.k_scale, s, is_v ? h - a.kv_heads : h, a.D, d,
                   q);
}

template <int DT, int F, int LH> __global__ __launch_bounds__(256) void k_kv_read(const KvRowsArgs a)
{
    const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LH;
    const int d = threadIdx.x % LH * 8;
    const int64_t heads = 2 * a.kv_heads, m = id / heads;
    int h = (int)(id % heads);
    const bool is_v = h >= a.kv_heads;
    if (m >= a.M || d >= a.D) return;
    if (is_v) h -= a.kv_heads;
    uint16_t *out = is_v ? a.v : a.k;
    if (!out) return;
    out += m * (is_v ? a.ldv : a.ldk) + h * a.D + d;
    const KvSlot s = kv_slot(a.kv, a.slots[m]);
    u4_t x = {0, 0, 0, 0};
    if (s.page >= 0) {
        const uint8_t *codes = (is_v ? a.kv.v : a.kv.k) + s.page * a.kv.page_stride;
        const void *scale = is_v ? a.kv.v_scale : a.kv.k_scale;
        const int64_t row = (int64_t)h * a.kv.page_size + s.at;
        if constexpr (F == W4A4_KV_INT8) {
            const u2_t c = *reinterpret_cast<const u2_t *>(codes + row * a.D + d);
            const float f = reinterpret_cast<const float *>(scale)[s.page * a.kv.scale_stride + row];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t w = c[i / 2] >> (16 * (i % 2));
                x[i] = pack16<DT>((float)(int8_t)w * f, (float)(int8_t)(w >> 8) * f);
            }
        } else {
            const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + row * (a.D / 2) + d / 2);
            const uint32_t e = reinterpret_cast<const uint8_t *>(
                scale)[s.page * a.kv.scale_stride + ((int64_t)h * (a.D / 32) + d / 32) * a.kv.page_size + s.at];
            typedef KvTile<DT, 128, F> T;
            const float f = T::byte_scale(e);
            x = u4_t{T::template widen4<0>(c, f), T::template widen4<1>(c, f), T::template widen4<2>(c, f),
                     T::template widen4<3>(c, f)};
        }
    }
    store8_any(out, x);
}

template <int DT, int F, int LH> static int run_rows(const KvRowsArgs &a, bool read, hipStream_t s)
{
    // a launch holds less than 2^32 threads
    const int64_t per_token = 2 * a.kv_heads * LH, rows = ((int64_t)1 << 31) / per_token;
    for (int64_t m = 0; m < a.M; m += rows) {
        KvRowsArgs b = a;
        b.M = std::min(rows, a.M - m);
        b.k = a.k ? a.k + m * a.ldk : nullptr;
        b.v = a.v ? a.v + m * a.ldv : nullptr;
        b.slots = a.slots + m;
        const dim3 grid((unsigned)((b.M * per_token + 255) / 256));
        if (read) hipLaunchKernelGGL((k_kv_read<DT, F, LH>), grid, dim3(256), 0, s, b);
        else hipLaunchKernelGGL((k_kv_append<DT, F, LH>), grid, dim3(256), 0, s, b);
        if (int rc = check_launch(read ? "kv_read_quant" : "kv_append_quant")) return rc;
    }
    return W4A4_OK;
}

template <int DT, int F> static int pick_rows(const KvRowsArgs &a, bool read, hipStream_t s)
{
    if (a.D <= 64) return run_rows<DT, F, 8>(a, read, s);
    if (a.D <= 128) return run_rows<DT, F, 16>(a, read, s);
    return run_rows<DT, F, 32>(a, read, s);
}

static int pick_rows(const KvRowsArgs &a, int dtype, bool read, hipStream_t s)
{
    if (dtype == W4A4_BF16)
        return a.kv.format == W4A4_KV_INT8 ? pick_rows<W4A4_BF16, W4A4_KV_INT8>(a, read, s)
                                           : pick_rows<W4A4_BF16, W4A4_KV_FP4>(a, read, s);
    return a.kv.format == W4A4_KV_INT8 ? pick_rows<W4A4_F16, W4A4_KV_INT8>(a, read, s)
                                       : pick_rows<W4A4_F16, W4A4_KV_FP4>(a, read, s);
}

int launch_kv_append(const KvRowsArgs &a, int dtype, hipStream_t s) { return pick_rows(a, dtype, false, s); }
int launch_kv_read(const KvRowsArgs &a, int dtype, hipStream_t s) { return pick_rows(a, dtype, true, s); }

// ================================================================================================
// Attention. A sequence's own tokens: tiles of one sequence go in equal runs to workgroups and there round-robin to
// the waves, as over the 16-bit cache. The shared prefix: the query rows of all sequences that share a key/value head
// are cut into row tiles of 16, and each wave takes RT of them over a run of the prefix, so that a tile of keys that
// has been loaded and widened serves 16 RT rows. Each (sequence, head) then has parts, of the prefix and of its own
// tokens, which k_join adds up in a fixed order.
//  - Own tokens are bound by memory: 32 ragged sequences up to 8191 int8 keys (32 heads over 8 of 128) 48.1 us, 4.4 TB/s;
//    two of 131071 and fewer fp4 keys 47.8 us, 5.0 TB/s, with the vector units busy 45 % of the time and the matrix cores 17 %
//    (counted; 4 heads to a key head use a quarter of a product's columns). One short sequence is bound by the chain of
//    length, page, keys, values: 7.8 us.
//  - The prefix is bound by how few waves there are to hide each other's waits: 64 sequences behind 16384 16-bit tokens
//    52.0 us, own tokens included; the matrix cores are busy a fifth of that, the vector units a third (counted), 1.2 waves
//    on a SIMD on average. Twice as many prefix workgroups write twice as many parts, and lose more (68 us).
// ================================================================================================

// The parts that a run of T tiles is cut into: `per` tiles each, used of them
__device__ __forceinline__ int tiles_per_part(int T, int splits, int least) { return max((T + splits - 1) / splits, least); }

// A workgroup's part of one sequence's own tokens for up to 16 of the heads that share a key/value head.
template <int DT, int D, int F>
__device__ __forceinline__ void own_tokens(const AttnArgs &a, const int id, float *sm)
{
    typedef KvShape<D, F> S;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    // all heads of one (sequence, split) run on one XCD, and the sequences move on by one XCD from split to split
    const int hts = a.kv_heads * a.head_tiles;
    const int unit = id / (8 * hts) * 8 + id % 8, head = id / 8 % hts;
    const int split = unit / a.B, b = (unit + split) % a.B;
    const int kvh = head / a.head_tiles, ht = head % a.head_tiles;
    if (split >= a.splits) return;
    const int group = a.heads / a.kv_heads, G = min(16, group - ht * 16), h0 = kvh * group + ht * 16;
    const int n = a.lens[b];
    const int32_t *table = a.table + (int64_t)b * a.ldt;
    const AttnTiles tl = attn_tiles(n, a);
    const int per = tiles_per_part(tl.T, a.splits, a.tiles_per_split);
    const int t0 = split * per, t1 = min(tl.T, t0 + per);
    uint16_t *out = a.out + (int64_t)b * a.ldo + (int64_t)h0 * D;
    if (tl.T == 0) {  // nothing visible: zeros, where no other part follows
        if (split == 0 && !a.prefix_splits)
            for (int e = threadIdx.x; e < G * D; e += blockDim.x) out[e] = 0;
        return;
    }
    if (t0 >= t1) return;

    AttnRows<DT, D, F, 1> rows;
    rows.clear();
    // operand rows past the group repeat its last head; their results are not used
    const bool flip = a.scale_log2 < 0.0f;
    rows.load_q(0, a.q + (int64_t)b * a.ldq + (int64_t)(h0 + min(r, G - 1)) * D, g, flip);
    const float scale = AttnRows<DT, D, F, 1>::scale_of(a);
    bool bad = tl.over;
    const int from = a.window > 0 ? n - a.window : 0;
    auto key_of = [&](int t) { return (t < tl.ns ? t : tl.w0 + t - tl.ns) * 32; };
    auto is_whole = [&](int key0) { return key0 <= n - 32 && (key0 >= from || key0 + 32 <= a.sinks); };

    typedef KvStage<D, F, 64> Stage;
    uint8_t *stage = reinterpret_cast<uint8_t *>(sm) + wave * Stage::BYTES;
    const int count = tl.over ? 0 : (t1 - t0 - wave + waves - 1) / waves;  // this wave's tiles
    for (int base = 0; base < count; base += 64) {
        const int some = min(64, count - base);
        KvPlaces places;
        places.look_up<D, F>(a.kv, table, key_of(t0 + wave + (base + min(lane, some - 1)) * waves), n, from, a.sinks, kvh, bad);
        KvTile<DT, D, F> tile;
        Stage keys;
        KvPlace at = places.get<F>(0);
        keys.load(a.kv.k, at, lane);
        tile.template load<false>(a.kv, at, lane);
        for (int i = 0; i < some; ++i) {
            const int key0 = at.key0;
            lds_fence();
            keys.commit(stage, lane);
            lds_fence();
            KvTile<DT, D, F> cur = tile;
            cur.keys_from(stage, lane);
            // the next tile is asked for (the last one again), without a branch: behind one the wait for this tile would
            // be a wait for that, too
            at = places.get<F>(min(i + 1, some - 1));
            keys.load(a.kv.k, at, lane);
            tile.template load<false>(a.kv, at, lane);
            rows.template add<true>(cur, is_whole(key0), [&](int e) {
                const int key = key0 + 16 * (e / 4) + 4 * g + e % 4;
                return key < n && (key >= from || key < a.sinks);
            }, scale);
        }
    }
    float sum = rows.total(0);
    if (__any(bad)) sum = NAN;

    // ---- join the waves: maximum [W][16], sum [W][16], channels [W][G][D + pad] ----
    __syncthreads();  // the keys' rows make room
    float *wm = sm, *ws = sm + waves * 16, *wa = sm + waves * 32;
    constexpr int LD = D + ATTN_PAD;
    if (g == 0) {
        wm[wave * 16 + r] = rows.mx[0];
        ws[wave * 16 + r] = sum;
    }
    if (r < G) {
        float *dst = wa + (wave * G + r) * LD;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (S::VE * 16 == D || S::VE * (4 * g + x) < D)
#pragma unroll
                for (int i = 0; i < S::VE; ++i) dst[S::VE * (4 * g + x) + i] = rows.acc[0][i][x];
    }
    __syncthreads();
    const bool alone = !a.prefix_splits && tl.T <= per;
    for (int e = threadIdx.x; e < G * (D / 4); e += blockDim.x) {
        const int h = e / (D / 4), d = e % (D / 4) * 4;
        float top = wm[h];
        for (int w = 1; w < waves; ++w) top = fmaxf(top, wm[w * 16 + h]);
        const float base = top == -INFINITY ? 0.0f : top;
        f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
        float l = 0.0f;
        for (int w = 0; w < waves; ++w) {
            const float f = __builtin_amdgcn_exp2f(wm[w * 16 + h] - base);
            o += f * *reinterpret_cast<const f4_t *>(wa + (w * G + h) * LD + d);
            l += f * ws[w * 16 + h];
        }
        if (alone) {
            const u2_t y = {pack16<DT>(o[0] / l, o[1] / l), pack16<DT>(o[2] / l, o[3] / l)};
            *reinterpret_cast<any2_t *>(out + h * D + d) = y;
        } else {
            const int64_t part = ((int64_t)b * a.heads + h0 + h) * (a.prefix_splits + a.splits) + a.prefix_splits + split;
            *reinterpret_cast<f4_t *>(a.part + part * D + d) = o;
            if (d == 0) a.stat[part] = make_float2(top, l);
        }
    }
}

template <int DT, int D, int F> __global__ __launch_bounds__(64 * ATTN_WAVES) void k_attn_own(const AttnArgs a)
{
    extern __shared__ float sm[];
    own_tokens<DT, D, F>(a, blockIdx.x, sm);
}

// Tiles of the prefix: none, or one logical tile that poisons where the table cannot hold it.
__device__ __forceinline__ int prefix_tiles(const AttnArgs &a, bool &over)
{
    const int n = a.prefix_splits ? a.prefix_len[0] : 0;
    over = (int64_t)n > (int64_t)a.prefix_width * a.kv.page_size;
    return over ? 1 : n <= 0 ? 0 : (int)(((int64_t)n + 31) >> 5);
}

// The prefix for many rows: the four waves of a workgroup have RT row tiles each and share the tile of keys, which
// passes through LDS, two tiles in turn. The scales of quantized rows come along: fp32 [2][32] of keys and values, or
// bytes [2][D / 32][32].
template <int D, int F> constexpr int prefix_buffer()
{
    return 2 * KvStage<D, F, 64 * ATTN_WAVES>::BYTES +
           (F == W4A4_KV_16BIT ? 0 : 2 * 32 * (F == W4A4_KV_INT8 ? 4 : D / 32));
}

template <int DT, int D, int F, int RT>
__device__ __forceinline__ void prefix_many(const AttnArgs &a, const int id, uint8_t *lds)
{
    typedef KvShape<D, F> S;
    typedef KvStage<D, F, 64 * ATTN_WAVES> Stage;
    constexpr int BUF = prefix_buffer<D, F>();
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // all row blocks of one (head, part, run of blocks) run on one XCD
    const int unit = id / (8 * a.prefix_row_blocks) * 8 + id % 8, keys = unit / a.prefix_row_runs;
    const int block = unit % a.prefix_row_runs * a.prefix_row_blocks + id / 8 % a.prefix_row_blocks;
    const int kvh = keys / a.prefix_splits, split = keys % a.prefix_splits;
    const int group = a.heads / a.kv_heads;
    const int64_t total = (int64_t)a.B * group, row0 = ((int64_t)block * ATTN_WAVES + wave) * 16 * RT;
    if (kvh >= a.kv_heads || (int64_t)block * ATTN_WAVES * 16 * RT >= total) return;
    bool bad;
    const int T = prefix_tiles(a, bad), n = bad ? 0 : a.prefix_len[0];
    const int per = tiles_per_part(T, a.prefix_splits, 1);
    const int t0 = split * per, t1 = min(T, t0 + per);
    if (t0 >= t1) return;

    AttnRows<DT, D, F, RT> rows;
    rows.clear();
    auto place = [&](int t, int64_t &b, int &h) {  // row r of row tile t
        const int64_t row = min(row0 + 16 * t + r, total - 1);
        b = row / group;
        h = kvh * group + (int)(row - b * group);
    };
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        int64_t b;
        int h;
        place(t, b, h);
        rows.load_q(t, a.q + b * a.ldq + (int64_t)h * D, g, a.scale_log2 < 0.0f);
    }
    const float scale = AttnRows<DT, D, F, 1>::scale_of(a);
    if (!bad) {
        Stage k, v;
        uint32_t sc = 0;
        // the thread's dword of the scales: key's or value's, group, first key (fp4: of four)
        constexpr int PER = F == W4A4_KV_INT8 ? 32 : 8, GROUPS = F == W4A4_KV_INT8 ? 1 : D / 32;
        const int sv = tid / (PER * GROUPS), sg = tid / PER % GROUPS, sk = tid % PER * (32 / PER);
        auto load = [&](const KvPlace &at) {
            k.load(a.kv.k, at, tid);
            v.load(a.kv.v, at, tid);
            if (F != W4A4_KV_16BIT && sv < 2) {
                const void *p = sv ? a.kv.v_scale : a.kv.k_scale;
                const int64_t i = (sk < 16 ? at.scales[0] : at.scales[1]) + sg * a.kv.page_size + sk % 16;
                sc = F == W4A4_KV_INT8 ? reinterpret_cast<const uint32_t *>(p)[i]
                                       : *reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(p) + i);
            }
        };
        // what is past the end becomes zeros; its scales finite, and a key's not 0, which would turn its -inf into a NaN
        auto commit = [&](int t, uint8_t *to) {
            const int live = n - t * 32;
            if (live >= 32) {
                k.commit(to, tid);
                v.commit(to + Stage::BYTES, tid);
            } else {
                k.commit(to, tid, live);
                v.commit(to + Stage::BYTES, tid, live);
            }
            if (F != W4A4_KV_16BIT && sv < 2) {
                uint32_t x = sc;
                if constexpr (F == W4A4_KV_INT8) {
                    if (sk >= live) x = sv ? 0u : 0x3F800000u;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (sk + i >= live) x = (x & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
                }
                reinterpret_cast<uint32_t *>(to + 2 * Stage::BYTES)[tid] = x;
            }
        };
        for (int base = t0; base < t1; base += 64) {
            const int some = min(64, t1 - base);
            KvPlaces places;
            places.look_up<D, F>(a.kv, a.prefix_table, (base + min(lane, some - 1)) * 32, n, 0, 0, kvh, bad);
            load(places.get<F>(0));
            commit(base, lds);
            __syncthreads();
            for (int i = 0; i < some; ++i) {
                const int t = base + i;
                const uint8_t *now = lds + (i & 1) * BUF;
                load(places.get<F>(min(i + 1, some - 1)));
                if (row0 < total) {
                    KvTile<DT, D, F> tile;
                    tile.keys_from(now, lane);
                    const uint8_t *scales = now + 2 * Stage::BYTES;
                    if constexpr (F == W4A4_KV_INT8) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            tile.ks[hf] = reinterpret_cast<const float4 *>(scales)[4 * hf + g];
                            tile.vs[hf] = reinterpret_cast<const float4 *>(scales)[8 + 4 * hf + g];
                        }
                    } else if constexpr (F == W4A4_KV_FP4) {
                        const int vg = (S::VE * r < D ? S::VE * r : 0) / 32;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                            for (int l = 0; l < S::NL; ++l)
                                tile.kb[hf][l] = scales[S::channel(l * S::NR, g) / 32 * 32 + 16 * hf + r];
                            tile.vb[hf] = reinterpret_cast<const uint32_t *>(scales + D + vg * 32 + 16 * hf)[g];
                        }
                    }
                    tile.values_from(now + Stage::BYTES, lane);
                    rows.template add<false>(tile, t * 32 <= n - 32,
                                        [&](int e) { return t * 32 + 16 * (e / 4) + 4 * g + e % 4 < n; }, scale);
                }
                if (i + 1 < some) commit(t + 1, lds + ((i + 1) & 1) * BUF);
                __syncthreads();
            }
        }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        float sum = rows.total(t);
        if (__any(bad)) sum = NAN;
        if (row0 + 16 * t + r >= total) continue;
        int64_t b;
        int h;
        place(t, b, h);
        const int64_t part = (b * a.heads + h) * (a.prefix_splits + a.splits) + split;
        if (g == 0) a.stat[part] = make_float2(rows.mx[t], sum);
        float *dst = a.part + part * D;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (S::VE * 16 == D || S::VE * (4 * g + x) < D)
#pragma unroll
                for (int i = 0; i < S::VE; ++i) dst[S::VE * (4 * g + x) + i] = rows.acc[t][i][x];
    }
}

// The prefix for few rows, fewer than four row tiles: each wave loads its own tiles of keys.
template <int DT, int D, int F> __device__ __forceinline__ void prefix_few(const AttnArgs &a, const int id)
{
    constexpr int RT = 1;
    typedef KvShape<D, F> S;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // wr waves on row tiles, the others on other keys; all row blocks of one (head, part) run on one XCD
    const int wr = a.prefix_row_waves, wk = ATTN_WAVES / wr;
    const int unit = id / (8 * a.prefix_row_blocks) * 8 + id % 8;
    const int block = id / 8 % a.prefix_row_blocks;
    const int parts = a.prefix_splits / wk;
    const int kvh = unit / parts, split = unit % parts * wk + wave / wr;
    if (kvh >= a.kv_heads) return;
    const int group = a.heads / a.kv_heads;
    const int64_t total = (int64_t)a.B * group, row0 = ((int64_t)block * wr + wave % wr) * 16 * RT;
    if (row0 >= total) return;
    bool bad;
    const int T = prefix_tiles(a, bad), n = bad ? 0 : a.prefix_len[0];
    const int per = tiles_per_part(T, a.prefix_splits, 1);
    const int t0 = split * per, t1 = min(T, t0 + per);
    if (t0 >= t1) return;

    AttnRows<DT, D, F, RT> rows;
    rows.clear();
    auto place = [&](int t, int64_t &b, int &h) {  // row r of row tile t
        const int64_t row = min(row0 + 16 * t + r, total - 1);
        b = row / group;
        h = kvh * group + (int)(row - b * group);
    };
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        int64_t b;
        int h;
        place(t, b, h);
        rows.load_q(t, a.q + b * a.ldq + (int64_t)h * D, g, a.scale_log2 < 0.0f);
    }
    const float scale = AttnRows<DT, D, F, 1>::scale_of(a);
    if (!bad) {
        for (int base = t0; base < t1; base += 64) {
            const int some = min(64, t1 - base);
            KvPlaces places;
            places.look_up<D, F>(a.kv, a.prefix_table, (base + min(lane, some - 1)) * 32, n, 0, 0, kvh, bad);
            KvTile<DT, D, F> tile;
            tile.template load<true>(a.kv, places.get<F>(0), lane);
            for (int i = 0; i < some; ++i) {
                const int key0 = (base + i) * 32;
                KvTile<DT, D, F> cur = tile;
                tile.template load<true>(a.kv, places.get<F>(min(i + 1, some - 1)), lane);
                rows.template add<true>(cur, key0 <= n - 32,
                                        [&](int e) { return key0 + 16 * (e / 4) + 4 * g + e % 4 < n; }, scale);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        float sum = rows.total(t);
        if (__any(bad)) sum = NAN;
        if (row0 + 16 * t + r >= total) continue;
        int64_t b;
        int h;
        place(t, b, h);
        const int64_t part = (b * a.heads + h) * (a.prefix_splits + a.splits) + split;
        if (g == 0) a.stat[part] = make_float2(rows.mx[t], sum);
        float *dst = a.part + part * D;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (S::VE * 16 == D || S::VE * (4 * g + x) < D)
#pragma unroll
                for (int i = 0; i < S::VE; ++i) dst[S::VE * (4 * g + x) + i] = rows.acc[t][i][x];
    }
}

// The prefix and the sequences' own tokens in one launch: the one is bound by the matrix cores, the other by memory. The
// prefix's workgroups come first, at most one for each CU where the row blocks allow it (prefix_plan), and
// the own tokens' fill in beside and behind them. RT 0: few rows.
template <int DT, int D, int F, int RT> __global__ __launch_bounds__(64 * ATTN_WAVES) void k_attn_shared(const AttnArgs a)
{
    extern __shared__ float sm[];
    const int own = blockIdx.x - 8 * a.prefix_turns;
    if (own >= 0) own_tokens<DT, D, F>(a, own, sm);
    else if constexpr (RT == 0) prefix_few<DT, D, F>(a, blockIdx.x);
    else prefix_many<DT, D, F, RT>(a, blockIdx.x, reinterpret_cast<uint8_t *>(sm));
}

// out = sum_s exp2(m_s - M) o_s / sum_s exp2(m_s - M) l_s over the parts that had tiles, one workgroup per
// (sequence, head): the prefix's parts come first, the sequence's own behind them. Bound by its launch and the parts' bytes
// (64 sequences of 32 heads, 16 parts of 128 channels of the prefix: 6.7 us; one of 8 heads, 32 parts of 256: 3.5).
constexpr int JOIN_MAX = 256;
template <int DT, int D> __global__ __launch_bounds__(256) void k_join(const AttnArgs a)
{
    constexpr int TC = D / 4, ROWS = 256 / TC;  // threads over the channels, parts at a time
    __shared__ float4 red[ROWS][TC];
    __shared__ float weight[JOIN_MAX], wave_top[4], wave_sum[4];
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, wave = tid >> 6;
    const int c = tid % TC, row = tid / TC;
    const int64_t at = ((int64_t)b * a.heads + h) * (a.prefix_splits + a.splits);
    const float4 *p = reinterpret_cast<const float4 *>(a.part + at * D) + c;
    bool over;
    int used_p = 0, used_s = 0;
    if (a.prefix_splits) {
        const int T = prefix_tiles(a, over);
        const int per = tiles_per_part(T, a.prefix_splits, 1);
        used_p = (T + per - 1) / per;
    }
    const AttnTiles tl = attn_tiles(a.lens[b], a);
    const int per = tiles_per_part(tl.T, a.splits, a.tiles_per_split);
    used_s = (tl.T + per - 1) / per;
    if (!a.prefix_splits && used_s <= 1) return;  // written by its only workgroup
    const int used = used_p + used_s;
    auto place = [&](int i) { return i < used_p ? i : a.prefix_splits + i - used_p; };
    uint16_t *out = a.out + (int64_t)b * a.ldo + (int64_t)h * D;
    if (used == 0) {
        for (int e = tid; e < D; e += 256) out[e] = 0;
        return;
    }
    const float2 st = tid < used ? a.stat[at + place(tid)] : make_float2(-INFINITY, 0.0f);
    float top = st.x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    if ((tid & 63) == 0) wave_top[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
    const float f = __builtin_amdgcn_exp2f(st.x - (top == -INFINITY ? 0.0f : top));
    weight[tid] = f;
    float l = f * st.y;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) l += __shfl_xor(l, off, 64);
    if ((tid & 63) == 0) wave_sum[wave] = l;
    __syncthreads();
    l = wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3];
    float4 o = make_float4(0, 0, 0, 0);
    if (row < ROWS) {
#pragma unroll 4
        for (int s = row; s < used; s += ROWS) {
            const float4 x = p[(int64_t)place(s) * TC];
            const float w = weight[s];
            o.x = fmaf(w, x.x, o.x);
            o.y = fmaf(w, x.y, o.y);
            o.z = fmaf(w, x.z, o.z);
            o.w = fmaf(w, x.w, o.w);
        }
        red[row][c] = o;
    }
    __syncthreads();
    if (row == 0) {
        for (int s = 1; s < ROWS; ++s) {
            const float4 v = red[s][c];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
        }
        const u2_t y = {pack16<DT>(o.x / l, o.y / l), pack16<DT>(o.z / l, o.w / l)};
        *reinterpret_cast<any2_t *>(out + 4 * c) = y;
    }
}

// How the own tokens are split, by sizes known on the host alone. A sequence short enough for one workgroup, or one of
// so many that each CU has several, is not split: its result needs no join. The smallest parts are two tiles a wave: with
// one, partials and their join cost more than the keys (64 sequences of 4000 int8 keys, one key head: 20.3 us against
// 15.3; one of 8192: 13.2 against 12.4). Few short rows take a wave each, which waits for no other. Between them: about
// two workgroups a CU for one or two sequences and eight for many, whose lengths differ and fill each other's gaps (the
// ragged int8 batch: 54.5 us at 2048 workgroups, 69.5 at 512; two of 65536 keys in 4 bits: 53.2 at 512, 61.2 at 2048);
// four behind a window, where lengths differ less (30.4 us at 1024, 35.9 at 2048); two behind a prefix, whose products
// fill the rest.
AttnPlan kv_plan(int B, int heads, int kv_heads, int max_len, int window, int sinks, bool shared)
{
    const int64_t head_tiles = ((int64_t)heads / kv_heads + 15) / 16;
    int64_t tiles = ((int64_t)max_len + 31) / 32;
    if ((int64_t)window + sinks >= max_len) window = 0;  // it hides nothing
    if (window > 0)  // a run of w keys touches at most w / 32 + 2 tiles
        tiles = std::min<int64_t>(tiles, (int64_t)window / 32 + 2 + ((int64_t)sinks + 31) / 32);
    tiles = std::max<int64_t>(tiles, 1);
    const int64_t rows = (int64_t)std::max(B, 1) * kv_heads * head_tiles;
    if (tiles <= std::clamp<int64_t>(rows / 4, 8, 32)) return {1, (int)tiles, ATTN_WAVES};
    AttnPlan p;
    p.waves = !shared && rows * tiles <= 512 && tiles <= 96 ? 1 : ATTN_WAVES;
    int64_t want = tiles, least = 1;
    if (p.waves > 1) {
        const int workgroups = shared || (B <= 2 && window <= 0) ? 512 : window > 0 ? 1024 : 2048;
        want = std::min<int64_t>(std::max<int64_t>(workgroups / rows, 1), 256);
        least = 2 * p.waves;
    }
    p.tiles_per_split = (int)std::max<int64_t>((tiles + want - 1) / want, least);
    p.splits = (int)((tiles + p.tiles_per_split - 1) / p.tiles_per_split);
    return p;
}

// How the prefix is split: at most one workgroup for each CU as long as the heads' row blocks alone are no more than the
// CUs, those counted that only fill a turn of eight, since a CU with two takes twice as long while others wait (2 key heads
// of 384 rows, 30011 int8 keys: 51.3 us with 240 workgroups, 66.2 with 264). More than 4 row tiles go two to a wave: each
// key read from LDS serves both (64 sequences of 8 heads a key head, 16384 keys: 56.2 us against 70.4 with one). More row
// blocks than an XCD has CUs are cut into runs, each on one XCD (8 heads over 1 of 128, 16384 keys: 512 sequences, 32
// blocks, 88 us; 513, 33 blocks, 152 in two runs of 17 and 755 in one run, which leaves seven XCDs idle).
PrefixPlan prefix_plan(int B, int heads, int kv_heads, int max_prefix)
{
    PrefixPlan p;
    const int64_t rows = (int64_t)std::max(B, 1) * (heads / kv_heads), row_tiles = (rows + 15) / 16;
    const int64_t tiles = std::max<int64_t>(((int64_t)max_prefix + 31) / 32, 1);
    p.rt = row_tiles > 4 ? 2 : 1;
    const int64_t wave_rows = (row_tiles + p.rt - 1) / p.rt;
    p.row_waves = p.rt == 2 || wave_rows >= 4 ? 4 : wave_rows >= 2 ? 2 : 1;  // fewer than 4: a tile's rows in each wave
    const int64_t blocks = (wave_rows + p.row_waves - 1) / p.row_waves;
    p.row_runs = (int)((blocks + 31) / 32);
    p.row_blocks = (int)((blocks + p.row_runs - 1) / p.row_runs);
    const int wk = ATTN_WAVES / p.row_waves;
    const int64_t want = std::max<int64_t>(8 * (32 / p.row_blocks) / ((int64_t)kv_heads * p.row_runs), 1);  // on a run's keys
    p.splits = (int)std::min<int64_t>({want, (tiles + wk - 1) / wk, 128 / wk}) * wk;
    return p;
}

template <int DT, int D, int F, int RT> static int run_shared(const AttnArgs &a, size_t lds, hipStream_t s)
{
    if constexpr (RT > 0) lds = std::max<size_t>(lds, 2 * prefix_buffer<D, F>());
    if (lds > 65536)  // more than every kernel gets unasked
        if (int rc = ensure_dynamic_lds(reinterpret_cast<const void *>(&k_attn_shared<DT, D, F, RT>), lds, "paged_attn_shared"))
            return rc;
    hipLaunchKernelGGL((k_attn_shared<DT, D, F, RT>), dim3(8 * (unsigned)(a.prefix_turns + a.own_turns)),
                       dim3(64 * ATTN_WAVES), lds, s, a);
    return check_launch("paged_attn_shared");
}

template <int DT, int D, int F> static int run_kv_attn(AttnArgs a, int rt, hipStream_t s)
{
    int rc;
    const int G = std::min(16, a.heads / a.kv_heads);
    const size_t lds = a.waves * std::max<size_t>((32 + G * (D + ATTN_PAD)) * sizeof(float), KvStage<D, F, 64>::BYTES);
    a.own_turns = (int)(((int64_t)a.B * a.splits + 7) / 8 * a.kv_heads * a.head_tiles);
    if (a.prefix_splits) {
        const int wk = ATTN_WAVES / a.prefix_row_waves;
        a.prefix_turns = (int)(((int64_t)a.kv_heads * (a.prefix_splits / wk) * a.prefix_row_runs + 7) / 8 * a.prefix_row_blocks);
        rc = wk > 1    ? run_shared<DT, D, F, 0>(a, lds, s)
             : rt == 2 ? run_shared<DT, D, F, 2>(a, lds, s)
                       : run_shared<DT, D, F, 1>(a, lds, s);
        if (rc) return rc;
    } else {
        if (lds > 65536 && (rc = ensure_dynamic_lds(reinterpret_cast<const void *>(&k_attn_own<DT, D, F>), lds, "paged_attn")))
            return rc;
        hipLaunchKernelGGL((k_attn_own<DT, D, F>), dim3(8 * (unsigned)a.own_turns), dim3(64 * a.waves), lds, s, a);
        if ((rc = check_launch("paged_attn")) || a.splits == 1) return rc;
    }
    hipLaunchKernelGGL((k_join<DT, D>), dim3(a.heads, a.B), dim3(256), 0, s, a);
    return check_launch("paged_attn join");
}

template <int DT, int D> static int pick_format(const AttnArgs &a, int rt, hipStream_t s)
{
    if (a.kv.format == W4A4_KV_INT8) return run_kv_attn<DT, D, W4A4_KV_INT8>(a, rt, s);
    if (a.kv.format == W4A4_KV_FP4) return run_kv_attn<DT, D, W4A4_KV_FP4>(a, rt, s);
    return run_kv_attn<DT, D, W4A4_KV_16BIT>(a, rt, s);  // behind a prefix only
}

template <int DT> static int pick_dim(const AttnArgs &a, int D, int rt, hipStream_t s)
{
    switch (D) {
    case 64: return pick_format<DT, 64>(a, rt, s);
    case 96: return pick_format<DT, 96>(a, rt, s);
    case 128: return pick_format<DT, 128>(a, rt, s);
    case 192: return pick_format<DT, 192>(a, rt, s);
    default: return pick_format<DT, 256>(a, rt, s);
    }
}

int launch_kv_attn(AttnArgs a, int dtype, int D, int rt, hipStream_t s)
{
    a.head_tiles = (a.heads / a.kv_heads + 15) / 16;
    return dtype == W4A4_BF16 ? pick_dim<W4A4_BF16>(a, D, rt, s) : pick_dim<W4A4_F16>(a, D, rt, s);
}

}  // namespace w4a4
