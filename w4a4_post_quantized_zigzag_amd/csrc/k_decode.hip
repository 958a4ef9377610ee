// The single-token path between two linears: per-head RMS norm and position rotation of queries and
// keys with the append to the paged key-value cache, and the attention of one new token per sequence
// over that cache.
#include <algorithm>

#include "kv_quant.h"

namespace w4a4 {

// ================================================================================================
// Norm, rotation, append. Per head x of D channels: y = x / sqrt(mean(x^2) + eps) * w, then the first
// rot channels in pairs (a, b) -> (a cos t - b sin t, b cos t + a sin t), t = position * inv_freq.
//
// Bound by the bytes: every element is read once and written once, in one launch for queries, keys
// and values. A head is LH lanes of eight channels (one 16-byte load each), a wave works on 64 / LH
// heads at a time and walks its token's heads with HEADS_AHEAD loads in flight. The rotation's sines and
// cosines are computed once per token (one lane per frequency, shared through LDS) and kept in registers
// over its heads, multiplied with the norm's weights: y = (x (w cos) -+ x' (w' sin)) / sqrt(..), with the
// partner channel x' taken from the neighbouring lanes' raw elements. The angle is reduced to a fraction
// of a turn in fp64, so far positions lose nothing.
// Measured: 8191 tokens of 32 + 8 heads of 128 41 us (4.9 TB/s, what a large copy reaches); 1600 tokens of 16
// + 16 heads of 64 6.7 us; one token 4.0 us per launch in a graph, most of it latency.
// ================================================================================================
constexpr int HEADS_AHEAD = 4;

// PART: with PAIRS, some channels are not rotated. KV: what the cache holds; rows for a quantized one are rounded to
// 16 bits as any other, and then quantized, so that it holds what a 16-bit cache's rows would be quantized to.
template <int DT, int LH, bool PAIRS, bool PART, int KV>
__global__ __launch_bounds__(512) void k_norm_rope(const NormRopeArgs a)
{
    extern __shared__ float2 turns[];  // [tokens of the workgroup][rot / 2] (cos, sin)
    constexpr int HP = 64 / LH;        // heads at a time
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wpt = a.waves_per_token, tpw = (blockDim.x >> 6) / wpt;  // waves on a token, tokens at a time
    const int half = a.rot >> 1, slot_t = wave / wpt, sub = wave % wpt;
    const int64_t m = (int64_t)blockIdx.x * tpw + slot_t, mc = min(m, a.M - 1);
    const int c = lane % LH, d = c * 8;
    const bool on = d < a.D;
    const int dl = on ? d : 0;

    // the first heads' loads go out before anything else
    const bool cached = KV != W4A4_KV_16BIT || a.k_cache;
    const int nq = a.heads, nk = a.kv_heads, total = nq + nk + (cached ? nk : 0);
    const uint16_t *qs = a.q + mc * a.ldq + dl, *ks = a.k + mc * a.ldk + dl;
    const uint16_t *vs = cached ? a.v + mc * a.ldv + dl : ks;
    const int D = a.D;
    auto load = [=](int h) {  // past the end: the last head
        h = min(h, total - 1);
        const uint16_t *pq = qs + h * D, *pk = ks + (h - nq) * D, *pv = vs + (h - nq - nk) * D;
        return load8_any(h < nq ? pq : h < nq + nk ? pk : pv);
    };
    const int step = wpt * HP;
    u4_t raw[HEADS_AHEAD];
#pragma unroll
    for (int u = 0; u < HEADS_AHEAD; ++u)
        if (u == 0 || sub * HP + u * step < total) raw[u] = load(sub * HP + u * step + lane / LH);
    int64_t row = -1;  // cache row offset of this token (elements), -1: not kept
    KvSlot slot{-1, 0};
    if constexpr (KV != W4A4_KV_16BIT) {
        slot = kv_slot(a.kv, a.slots[mc]);
    } else if (a.k_cache) {
        const int64_t s = a.slots[mc];
        if (s >= 0 && s < (int64_t)a.num_pages * a.page_size)
            row = (s >> a.page_shift) * a.page_stride + (s & (a.page_size - 1)) * a.D;
    }
    float2 *cs = turns + slot_t * half;
    if (half > 0) {
        const double pos = (double)a.positions[mc] * 0.15915494309189533577;  // 1 / (2 pi)
        for (int f = sub * 64 + lane; f < half; f += wpt * 64) {
            double t = pos * a.inv_freq[f];
            t -= rint(t);
            float s, co;
            sincospif(2.0f * (float)t, &s, &co);
            cs[f] = make_float2(co, s);
        }
    }
    // the partner channel: the same pair's other one, in this lane or in another
    const bool rotated = d < a.rot, first = d < half;
    const int partner = (PAIRS || !rotated) ? lane : first ? lane + half / 8 : lane - half / 8;
    const int dp = on ? (partner % LH) * 8 : 0;
    float cq[8], sq[8], ck[8], sk[8];  // of queries and of keys: w cos, w' sin
    auto weights = [=](const float *w, float (&own)[8], float (&other)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) own[i] = other[i] = 1.0f;
        if (!w) return;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const anyf4_t x = *reinterpret_cast<const anyf4_t *>(w + dl + i);
            const anyf4_t y = *reinterpret_cast<const anyf4_t *>(w + dp + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                own[i + e] = x[e];
                other[i + (PAIRS ? e ^ 1 : e)] = y[e];
            }
        }
    };
    weights(a.q_weight, cq, sq);
    weights(a.k_weight, ck, sk);
    __syncthreads();
    if (m >= a.M) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int f = PAIRS ? d / 2 + i / 2 : (first ? d : d - half) + i;
        const float2 t = rotated ? cs[f] : make_float2(1.0f, 0.0f);
        const float sn = (PAIRS ? i % 2 == 0 : first) ? -t.y : t.y;
        cq[i] *= t.x;
        sq[i] *= sn;
        ck[i] *= t.x;
        sk[i] *= sn;
    }
    const float inv_d = 1.0f / (float)a.D;

    auto finish = [&](int h0, u4_t x) {
        const int h = h0 + lane / LH;
        const bool is_q = h < nq, is_v = h >= nq + nk;
        u4_t out = x;
        if (h0 < nq + nk) {  // some of these heads are not values
            if (a.D != LH * 8) x = on ? x : u4_t{0, 0, 0, 0};
            float v[8], o[8], ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f2_t f = unpack16<DT>(x[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
                ss = fmaf(f.x, f.x, ss);
                ss = fmaf(f.y, f.y, ss);
            }
            if (PAIRS) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = v[i ^ 1];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f2_t f = unpack16<DT>((uint32_t)__builtin_amdgcn_ds_bpermute(partner * 4, (int)x[i]));
                    o[2 * i] = f.x;
                    o[2 * i + 1] = f.y;
                }
            }
            const float inv = rsqrtf(fmaf(sum_lanes<LH>(ss), inv_d, a.eps));
            float y[8];
            if (h0 + HP <= nq) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = fmaf(o[i], sq[i], v[i] * cq[i]) * inv;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s1 = sq[i], s2 = sk[i], c1 = cq[i], c2 = ck[i];
                    y[i] = fmaf(o[i], is_q ? s1 : s2, v[i] * (is_q ? c1 : c2)) * inv;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = is_v ? out[i] : pack16<DT>(y[2 * i], y[2 * i + 1]);
            // A channel that is not rotated has taken its neighbour times 0, which an infinity there turns into a
            // NaN. Such a head has inv = 0, so that the channel is 0, or NaN if it is infinite itself. (This keeps
            // the elements in seven more registers, 103 in all and one wave per SIMD less: 2 % at 1600 tokens of 16
            // + 16 heads of 64, 14 % at 5000, 6 % at 12000. Selects on every head's values: 20 % at 1600.)
            if (PART && __any(inv == 0.0f)) {
                constexpr uint32_t ONES = DT == W4A4_BF16 ? 0x7F80u : 0x7C00u;  // the exponent of what is not finite
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = (x[i] & ONES) == ONES ? 0x7FFFu : 0u;
                    const uint32_t hi = (x[i] >> 16 & ONES) == ONES ? 0x7FFF0000u : 0u;
                    out[i] = rotated || is_v || inv != 0.0f ? out[i] : lo | hi;
                }
            }
        }
        QuantRun<KV> coded;
        if constexpr (KV != W4A4_KV_16BIT)
            if (h0 + HP > nq) coded = quant_run<DT, KV, LH>(out);  // some of these heads go to the cache
        if (!on || h >= total) return;
        if (is_q) {
            store8_any(a.q_out + m * a.ldqo + h * a.D + d, out);
        } else {
            const int hk = is_v ? h - nq - nk : h - nq;
            if (!is_v && a.k_out) store8_any(a.k_out + m * a.ldko + hk * a.D + d, out);
            if constexpr (KV != W4A4_KV_16BIT) {
                if (slot.page >= 0) {
                    uint8_t *kc = a.kv.k, *vc = a.kv.v;
                    void *ksc = a.kv.k_scale, *vsc = a.kv.v_scale;
                    quant_store<KV>(a.kv, is_v ? vc : kc, is_v ? vsc : ksc, slot, hk, a.D, d, coded);
                }
            } else if (row >= 0) {
                uint16_t *kc = a.k_cache, *vc = a.v_cache;
                store8_any((is_v ? vc : kc) + row + hk * a.page_size * a.D + d, out);
            }
        }
    };
    for (int h0 = sub * HP; h0 < total; h0 += HEADS_AHEAD * step) {
#pragma unroll
        for (int u = 0; u < HEADS_AHEAD; ++u) {
            const int h = h0 + u * step;
            if (h >= total) return;
            const u4_t x = raw[u];
            if (h + HEADS_AHEAD * step < total) raw[u] = load(h + HEADS_AHEAD * step + lane / LH);
            finish(h, x);
        }
    }
}

template <int DT, int LH, int KV> static int run_norm_rope(const NormRopeArgs &a, bool pairs, hipStream_t s)
{
    const int waves = std::max(4, a.waves_per_token), tpw = waves / a.waves_per_token;
    const dim3 grid((unsigned)((a.M + tpw - 1) / tpw)), block(64 * waves);
    const size_t lds = (size_t)tpw * (a.rot / 2) * sizeof(float2);
    if (pairs && a.rot < a.D) hipLaunchKernelGGL((k_norm_rope<DT, LH, true, true, KV>), grid, block, lds, s, a);
    else if (pairs) hipLaunchKernelGGL((k_norm_rope<DT, LH, true, false, KV>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_norm_rope<DT, LH, false, false, KV>), grid, block, lds, s, a);
    return check_launch("qk_norm_rope");
}

template <int DT, int KV> static int pick_head(const NormRopeArgs &a, bool pairs, hipStream_t s)
{
    if constexpr (KV == W4A4_KV_16BIT) {
        if (a.D <= 32) return run_norm_rope<DT, 4, KV>(a, pairs, s);
        if (a.D > 256) return run_norm_rope<DT, 64, KV>(a, pairs, s);
    }
    if (a.D <= 64) return run_norm_rope<DT, 8, KV>(a, pairs, s);
    if (a.D <= 128) return run_norm_rope<DT, 16, KV>(a, pairs, s);
    return run_norm_rope<DT, 32, KV>(a, pairs, s);
}

template <int DT> static int pick_format(const NormRopeArgs &a, bool pairs, hipStream_t s)
{
    if (a.kv.format == W4A4_KV_INT8) return pick_head<DT, W4A4_KV_INT8>(a, pairs, s);
    if (a.kv.format == W4A4_KV_FP4) return pick_head<DT, W4A4_KV_FP4>(a, pairs, s);
    return pick_head<DT, W4A4_KV_16BIT>(a, pairs, s);
}

int launch_norm_rope(NormRopeArgs a, int dtype, bool interleaved, hipStream_t s)
{
    // Few tokens: up to eight waves on one. Many: a wave each, so that its sines serve all heads. The limits are
    // whole workgroups per CU: one of eight waves, three of four, four of four waves with two tokens. Measured
    // on both sides, us per launch:
    //   32 + 8 heads of 128    256 tokens: 4.6 with eight waves, 4.9 with four;  300: 5.7, 5.3
    //                          700: 7.0 with four, 7.6 with two;  850: 8.1, 8.4;  1032: 10.7, 9.3
    //                          2048: 12.1 with two, 12.3 with one;  2056: 14.6, 13.0
    //   8 + 1 heads of 256     256: 4.3, 4.5;  264: 4.9, 4.4;  700: 5.2, 5.5;  850: 5.9, 5.7;  1032: 7.2, 6.2
    //                          2048: 8.4, 8.8;  2056: 10.0, 9.2
    //   5 + 1 heads of 96      200: 3.8, 3.8;  300: 4.5, 4.2;  768: 4.4, 4.3;  850: 4.8, 4.4;  2056: 6.3, 5.5
    a.waves_per_token = a.M <= 256 ? 8 : a.M <= 768 ? 4 : a.M <= 2048 ? 2 : 1;
    a.page_shift = a.page_size ? __builtin_ctz((unsigned)a.page_size) : 0;
    return dtype == W4A4_BF16 ? pick_format<W4A4_BF16>(a, interleaved, s)
                              : pick_format<W4A4_F16>(a, interleaved, s);
}

// ================================================================================================
// Attention of one new token over the paged cache.
//
// Bound by the cache bytes: every visible key and value is read once for all the query heads that
// share it. A wave takes tiles of 32 keys:
//  - scores^T (16 keys x 16 heads, twice) = K (A operand, rows straight from the cache) . q^T;
//  - a lane then holds 8 keys of one head. Running maximum and sum as usual, the sum per lane;
//  - out^T (16 channels x 16 heads per product) += V^T (A operand) . p (B operand). The scores'
//    result layout already is the B operand of a 32-key product if key 4 g + e (e < 4) of the first
//    and of the second half of the tile are its k = 8 g + e and 8 g + 4 + e. For the A operand a lane
//    loads D / 16 neighbouring channels of those eight keys and pairs them up with byte permutes;
//    nothing passes through LDS and no cross-lane step is needed but the maximum's.
//  - p is split in two 16-bit parts (p = hi + lo to 2^-16 or better), two products per tile.
// Tiles of one sequence go in equal runs to `splits` workgroups and there round-robin to the waves (four,
// one where there is little to do), joined in LDS and by k_attn_join in a fixed order.
// Measured (calls one after another): 32 sequences of 0 to 8191 tokens, 32 heads over 8 of 128, 81 us (5.05 TB/s);
// two of 131071 and 87000 tokens 154 us (5.8 TB/s, part of it from the last-level cache); 64 with a window of 1000 and
// 16 heads of 64 42.5 us (5.0 TB/s); one of 1001 tokens, one key/value head of 256, 9.6 us, the chain of two
// launches.
// ================================================================================================

template <int DT, int D>
__global__ __launch_bounds__(64 * ATTN_WAVES) void k_attn_split(const AttnArgs a)
{
    constexpr int KJ = D / 32, VE = D / 16, DW = VE / 2;
    // p is held times 2^14 in fp16, so that what the two parts drop is 2^-38 of the largest
    constexpr float OFF = DT == W4A4_F16 ? 14.0f : 0.0f;
    extern __shared__ float sm[];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    // Consecutive workgroups go to different XCDs. All heads of one (sequence, split) run on the same XCD,
    // which then walks each page once, and the sequences move on by one XCD from split to split: the late
    // splits, which only the longest sequences have, are spread over all of them.
    const int hts = a.kv_heads * a.head_tiles;
    const int unit = blockIdx.x / (8 * hts) * 8 + blockIdx.x % 8, head = blockIdx.x / 8 % hts;
    const int split = unit / a.B, b = (unit + split) % a.B;
    const int kvh = head / a.head_tiles, ht = head % a.head_tiles;
    if (split >= a.splits) return;
    const int group = a.heads / a.kv_heads, G = min(16, group - ht * 16), h0 = kvh * group + ht * 16;
    const int n = a.lens[b];
    const int32_t *table = a.table + (int64_t)b * a.ldt;
    const int t0 = split * a.tiles_per_split;
    const AttnTiles tl = attn_tiles(n, a);
    const int t1 = split + 1 == a.splits ? tl.T : min(tl.T, t0 + a.tiles_per_split);
    uint16_t *out = a.out + (int64_t)b * a.ldo + (int64_t)h0 * D;
    if (tl.T == 0) {  // nothing visible: zeros
        if (split == 0)
            for (int e = threadIdx.x; e < G * D; e += blockDim.x) out[e] = 0;
        return;
    }
    if (t0 >= t1) return;

    u4_t q[KJ];
    {
        // operand rows past the group repeat its last head; their results are not used
        const uint16_t *qp = a.q + (int64_t)b * a.ldq + (int64_t)(h0 + min(r, G - 1)) * D + 8 * g;
#pragma unroll
        for (int j = 0; j < KJ; ++j) q[j] = load8_any(qp + 32 * j);
    }
    f4_t acc[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) acc[i] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float mx = -INFINITY, sum = 0.0f;
    bool bad = tl.over;
    const int first_in_window = a.window > 0 ? n - a.window : 0;
    auto seen = [&](int key) { return key < n && (key >= first_in_window || key < a.sinks); };

    // A tile's two halves of 16 keys lie in one page each. A half without a visible key may have no page
    // any more and reads the other half's; a page with one is there as a whole. A page that does not
    // exist reads page 0 and poisons the result.
    struct Pages {
        int key0, at[2];  // first key; first row of each half inside its page
        int64_t page[2];
    };
    auto look_up = [&](int t) {
        Pages p;
        p.key0 = (t < tl.ns ? t : tl.w0 + t - tl.ns) * 32;
        bool any[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int lo = p.key0 + 16 * hf;
            any[hf] = lo < n && (min(lo + 15, n - 1) >= first_in_window || lo < a.sinks);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int lo = p.key0 + 16 * (any[hf] ? hf : 1 - hf);
            int pid = __builtin_amdgcn_readfirstlane(table[lo >> a.page_shift]);
            if ((unsigned)pid >= (unsigned)a.num_pages) {
                bad = true;
                pid = 0;
            }
            p.page[hf] = (int64_t)pid * a.page_stride;
            p.at[hf] = (kvh * a.page_size + (lo & (a.page_size - 1))) * D;
        }
        return p;
    };
    const uint32_t koff = r * D + 8 * g, voff = 4 * g * D + VE * r;

    int t = tl.over ? t1 : t0 + wave;
    Pages pg;
    if (t < t1) pg = look_up(t);
    for (; t < t1; t += waves) {
        const int key0 = pg.key0;
        const bool whole = key0 <= n - 32 && (key0 >= first_in_window || key0 + 32 <= a.sinks);
        u4_t k[2][KJ];
        DwordRun<DW> v[8];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const uint16_t *kp = a.k_cache + pg.page[hf] + pg.at[hf];
#pragma unroll
            for (int j = 0; j < KJ; ++j) k[hf][j] = *reinterpret_cast<const u4_t *>(kp + 32 * j + koff);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const uint16_t *vp = a.v_cache + pg.page[hf] + pg.at[hf];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[4 * hf + e] = *reinterpret_cast<const DwordRun<DW> *>(vp + e * D + voff);
        }
        if (t + waves < t1) pg = look_up(t + waves);  // the next tile's pages, ahead of its loads
        float p[8];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            f4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < KJ; ++j) s = mma32<DT>(k[hf][j], q[j], s);
#pragma unroll
            for (int e = 0; e < 4; ++e) p[4 * hf + e] = s[e] * a.scale_log2;
        }
        if (!whole) {  // what is not visible counts as -inf, and its values as zeros
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool ok = seen(key0 + 16 * (e / 4) + 4 * g + e % 4);
                p[e] = ok ? p[e] : -INFINITY;
#pragma unroll
                for (int i = 0; i < DW; ++i) v[e].v[i] = ok ? v[e].v[i] : 0u;
            }
        }
        float top = p[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, p[e]);
        top = across_groups(top, [](float x, float y) { return fmaxf(x, y); });
        if (__any(top > mx)) {
            const float to = fmaxf(mx, top), f = to > mx ? __builtin_amdgcn_exp2f(mx - to) : 1.0f;
#pragma unroll
            for (int i = 0; i < VE; ++i) acc[i] *= f;
            sum *= f;
            mx = to;
        }
        const float from = (mx == -INFINITY ? 0.0f : mx) - OFF;
        u4_t hi, lo;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float x = __builtin_amdgcn_exp2f(p[e] - from), y = __builtin_amdgcn_exp2f(p[e + 1] - from);
            sum += x + y;
            hi[e / 2] = pack16<DT>(x, y);
            const f2_t h = unpack16<DT>(hi[e / 2]);
            lo[e / 2] = pack16<DT>(x - h.x, y - h.y);
        }
#pragma unroll
        for (int i = 0; i < DW; ++i) {
            u4_t even, odd;  // channels VE r + 2 i and + 2 i + 1 of the eight keys
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                even[e] = __builtin_amdgcn_perm(v[2 * e + 1].v[i], v[2 * e].v[i], 0x05040100u);
                odd[e] = __builtin_amdgcn_perm(v[2 * e + 1].v[i], v[2 * e].v[i], 0x07060302u);
            }
            acc[2 * i] = mma32<DT>(even, lo, acc[2 * i]);
            acc[2 * i + 1] = mma32<DT>(odd, lo, acc[2 * i + 1]);
            acc[2 * i] = mma32<DT>(even, hi, acc[2 * i]);
            acc[2 * i + 1] = mma32<DT>(odd, hi, acc[2 * i + 1]);
        }
    }
    sum = across_groups(sum, [](float x, float y) { return x + y; });
    if (__any(bad)) sum = NAN;

    // ---- join the waves: sm = maximum [W][16], sum [W][16], channels [W][G][D + pad] ----
    float *wm = sm, *ws = sm + waves * 16, *wa = sm + waves * 32;
    constexpr int LD = D + ATTN_PAD;
    if (g == 0) {
        wm[wave * 16 + r] = mx;
        ws[wave * 16 + r] = sum;
    }
    if (r < G) {
        float *dst = wa + (wave * G + r) * LD;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int i = 0; i < VE; ++i) dst[VE * (4 * g + x) + i] = acc[i][x];
    }
    __syncthreads();
    const bool alone = a.splits == 1 || tl.T <= a.tiles_per_split;
    for (int e = threadIdx.x; e < G * (D / 4); e += blockDim.x) {
        const int h = e / (D / 4), d = e % (D / 4) * 4;
        float top = wm[h];
        for (int w = 1; w < waves; ++w) top = fmaxf(top, wm[w * 16 + h]);
        const float from = top == -INFINITY ? 0.0f : top;
        f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
        float l = 0.0f;
        for (int w = 0; w < waves; ++w) {
            const float f = __builtin_amdgcn_exp2f(wm[w * 16 + h] - from);
            o += f * *reinterpret_cast<const f4_t *>(wa + (w * G + h) * LD + d);
            l += f * ws[w * 16 + h];
        }
        if (alone) {
            const u2_t y = {pack16<DT>(o[0] / l, o[1] / l), pack16<DT>(o[2] / l, o[3] / l)};
            *reinterpret_cast<any2_t *>(out + h * D + d) = y;
        } else {
            const int64_t at = ((int64_t)b * a.heads + h0 + h) * a.splits + split;
            *reinterpret_cast<f4_t *>(a.part + at * D + d) = o;
            if (d == 0) a.stat[at] = make_float2(top, l);
        }
    }
}

// out = sum_s exp2(m_s - M) o_s / sum_s exp2(m_s - M) l_s over the splits that had tiles: one workgroup
// per (sequence, head). The weights of all splits are made first, in parallel, so that the channels' sum
// is nothing but independent loads.
constexpr int ATTN_MAX_SPLITS = 256;
template <int DT, int D> __global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a)
{
    constexpr int TC = D / 4, ROWS = 256 / TC;  // threads over the channels, splits at a time
    constexpr int AHEAD = 8;
    __shared__ float4 red[ROWS][TC];
    __shared__ float weight[ATTN_MAX_SPLITS], wave_top[4], wave_sum[4];
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, wave = tid >> 6;
    const int c = tid % TC, row = tid / TC;
    const int64_t at = ((int64_t)b * a.heads + h) * a.splits;
    const float4 *p = reinterpret_cast<const float4 *>(a.part + at * D) + c;
    // everything is asked for before the length has arrived; what no split wrote is not used
    float2 st = tid < a.splits ? a.stat[at + tid] : make_float2(0.0f, 0.0f);
    float4 v[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (row < ROWS && row + i * ROWS < a.splits) v[i] = p[(int64_t)(row + i * ROWS) * TC];
    const AttnTiles tl = attn_tiles(a.lens[b], a);
    if (tl.T <= a.tiles_per_split) return;  // written by its only workgroup
    const int used = min(a.splits, (tl.T + a.tiles_per_split - 1) / a.tiles_per_split);
    if (tid >= used) st = make_float2(-INFINITY, 0.0f);
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
    auto add = [&](const float4 &x, float w) {
        o.x = fmaf(w, x.x, o.x);
        o.y = fmaf(w, x.y, o.y);
        o.z = fmaf(w, x.z, o.z);
        o.w = fmaf(w, x.w, o.w);
    };
    if (row < ROWS) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (row + i * ROWS < used) add(v[i], weight[row + i * ROWS]);
#pragma unroll 4
        for (int s = row + AHEAD * ROWS; s < used; s += ROWS) add(p[(int64_t)s * TC], weight[s]);
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
        *reinterpret_cast<any2_t *>(a.out + (int64_t)b * a.ldo + (int64_t)h * D + 4 * c) = y;
    }
}

// How many waves and workgroups share a sequence. The lengths are on the device; only max_len is known, and every
// sequence is cut by it: a max_len far above the lengths leaves their tiles to few workgroups (one sequence of 2000
// tokens, 32 heads over 8 of 128: 8.3 us, 23.5 with a max_len of 131072; 32 of 256 to 8191: 84 and 109). All
// figures are us per call in a graph.
//  - Short sequences get one workgroup of four waves each and no join, which costs 3 us: up to 8 tiles always
//    (64, 128 and 256 tokens, 8 key/value heads of 128: 4.2, 4.7 and 6.1, split 7.0, 7.1 and 7.5; 384 tokens 7.7
//    and 7.3), up to 32 where the rows alone fill the CUs (16 sequences of 1024 tokens, 8 heads: 13.7, split 16.7;
//    64 of 768: 38 and 42; 64 of 1 to 768: 16.4 and 16.0; but 4 of 1024: 13.3 and 9.7).
//  - Else, with at most 512 tiles in all and 96 of one sequence there are CUs left, and only the latency counts: one
//    wave and one tile per workgroup. With more the join of so many parts costs more than the shorter chains save.
//    One and four waves, one sequence with one key/value head of 256, eight heads: 1001 tokens 9.4 and 9.8, 3067:
//    11.2 and 10.0, 8000: 15.6 and 11.4; one head of 64: 6.8 and 7.3, 6.8 and 7.2, 7.8 and 7.3. 16 rows of one head
//    of 128, 507 tokens: 7.4 and 8.2, 1019: 7.8 and 8.4, 2043: 10.4 and 10.1; of eight heads: 8.2 and 8.5, 9.4 and
//    8.8, 12.3 and 10.4.
//  - With a window that hides something all sequences are about as long, and two sequences leave little to balance:
//    few long runs read fastest (64 sequences of 16 heads and 1004 visible tokens: 43.4 with 1024 workgroups, 47.0
//    with 2048; 131071 and 87000 tokens, 8 heads: 163 with 512, 169 with 2048).
//  - Otherwise the lengths differ, and the CUs stay evenly loaded with shorter ones (8 sequences of 1000 to 32000
//    tokens, 8 heads: 99 with 512, 84 with 1024, 70 with 2048; 32 of 0 to 8191: 113, 100 and 82).
AttnPlan attn_plan(int B, int heads, int kv_heads, int max_len, int window, int sinks)
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
    p.waves = rows * tiles <= 512 && tiles <= 96 ? 1 : ATTN_WAVES;
    int64_t want = tiles;
    if (p.waves > 1) {
        const int workgroups = window > 0 ? 1024 : B <= 2 ? 512 : 2048;
        want = std::min<int64_t>(std::max<int64_t>(workgroups / rows, 1), ATTN_MAX_SPLITS);
    }
    p.tiles_per_split = (int)std::max<int64_t>((tiles + want - 1) / want, p.waves);
    p.splits = (int)((tiles + p.tiles_per_split - 1) / p.tiles_per_split);
    return p;
}

template <int DT, int D> static int run_attn(const AttnArgs &a, hipStream_t s)
{
    const int G = std::min(16, a.heads / a.kv_heads);
    const size_t lds = (size_t)a.waves * (32 + G * (D + ATTN_PAD)) * sizeof(float);
    int rc;
    if (lds > 65536 &&  // more than every kernel gets unasked
        (rc = ensure_dynamic_lds(reinterpret_cast<const void *>(&k_attn_split<DT, D>), lds, "paged_attn")))
        return rc;
    hipLaunchKernelGGL((k_attn_split<DT, D>), dim3((unsigned)(((int64_t)a.B * a.splits + 7) / 8 * 8 * a.kv_heads * a.head_tiles)),
                       dim3(64 * a.waves), lds, s, a);
    if ((rc = check_launch("paged_attn_decode")) || a.splits == 1) return rc;
    hipLaunchKernelGGL((k_attn_join<DT, D>), dim3(a.heads, a.B), dim3(256), 0, s, a);
    return check_launch("paged_attn_decode join");
}

template <int DT> static int pick_dim(const AttnArgs &a, int D, hipStream_t s)
{
    switch (D) {
    case 64: return run_attn<DT, 64>(a, s);
    case 96: return run_attn<DT, 96>(a, s);
    case 128: return run_attn<DT, 128>(a, s);
    case 192: return run_attn<DT, 192>(a, s);
    default: return run_attn<DT, 256>(a, s);
    }
}

int launch_paged_attn(AttnArgs a, int dtype, int D, hipStream_t s)
{
    a.head_tiles = (a.heads / a.kv_heads + 15) / 16;
    return dtype == W4A4_BF16 ? pick_dim<W4A4_BF16>(a, D, s) : pick_dim<W4A4_F16>(a, D, s);
}

}  // namespace w4a4
