// decode4_sm100.cuh -- single-token decode over the 4-bit KV cache (row format in
// kv4_sm100.cuh), split-KV with a log-sum-exp merge.
//
//   logit(t) = scale q~ . k_t,  k_t = s n + z by group;  o = sum_t p_t v_t / sum_t p_t
//
// The visible keys of all (sequence, KV head) segments, laid end to end, are cut into one
// equal share per block; a block leaves one partial (max, sum, unnormalised output) per
// query head and segment piece.  Pieces are numbered block + segment: along the blocks
// each next piece raises the one, the other or both, so no two share a number, and
// blocks + segments slots hold them all whatever the lengths.
#pragma once
#include "decode_sm100.cuh"
#include "kv4_sm100.cuh"

namespace yr {

constexpr int kDec4Chunk = 128;      // least keys per block: a tile for each warp
constexpr int kDec4Lead = 256;       // what a segment costs besides its keys, in keys
constexpr int kDec4MaxBlocks = 640;  // most blocks of the split launch
constexpr int kDec4Warps = 4;
constexpr int kDec4Threads = kDec4Warps * 32;
constexpr int kDec4Tile = 32;  // keys of one bulk copy
constexpr int kDec4Stages = 3;

struct Decode4Params {
    const __nv_bfloat16 *q_new;          // [B][Hq][d]
    const __nv_bfloat16 *k_new, *v_new;  // [B][Hkv][d]
    uint8_t *kv4;                        // [B][Hkv][T_max][5d/4]
    const int *cache_len;                // [B]
    float *ws_o;                         // [slots][g][d]
    float *ws_ml;                        // [slots][g][2]
    __nv_bfloat16 *o;                    // [B][Hq][d]
    float *lse;                          // [B][Hq] or null
    __nv_bfloat16 *k_stored, *v_stored;  // [B][Hkv][d] or null
    int B, Hq, Hkv, T_max, group;
    int grid_blocks;
    int window, n_sink;
    float sl2;  // softmax scale times log2 e
    int alibi;
    uint64_t timeout_ns;
    double turns[64];
};

// Ranges [0, len1) and [lo2, lo2 + len2) of keys that the token at position L sees.
__device__ __forceinline__ DecRanges dec4_ranges(const Decode4Params &p, int L) {
    DecRanges r{0, 0, 0};
    if (L < 0 || L > p.T_max - 1) return r;
    const int s1 = min(p.n_sink, L + 1);
    const int w0 = p.window > 0 ? max(L - p.window + 1, 0) : 0;
    if (w0 <= s1) {
        r.len1 = L + 1;
        r.lo2 = L + 1;
    } else {
        r.len1 = s1;
        r.lo2 = w0;
        r.len2 = L + 1 - w0;
    }
    return r;
}

// The partition, as every block derives it from cache_len.  A segment is kDec4Lead units
// for what a block does once for it (query, partial result) and one for each key, so that
// blocks of many short segments and blocks of few long ones take equally long.
__device__ __forceinline__ long long dec4_units_per_block(const Decode4Params &p, long long total) {
    const long long even = (total + p.grid_blocks - 1) / p.grid_blocks;
    return even > kDec4Chunk + kDec4Lead ? even : kDec4Chunk + kDec4Lead;
}
// Units of a segment with `keys` visible keys: none for a length outside the cache.
__device__ __forceinline__ long long dec4_seg_units(long long keys) { return keys > 0 ? keys + kDec4Lead : 0; }
__device__ __forceinline__ long long dec4_seq_units(const Decode4Params &p, int b) {
    if (b >= p.B) return 0;
    const DecRanges r = dec4_ranges(p, p.cache_len[b]);
    return p.Hkv * dec4_seg_units(static_cast<long long>(r.len1) + r.len2);
}
__device__ __forceinline__ long long dec4_total(const Decode4Params &p, int lane) {
    long long t = 0;
    for (int b = lane; b < p.B; b += 32) t += dec4_seq_units(p, b);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t;
}

// The new row: rotated, quantised, into slot L of the cache, and its values to k_stored and
// v_stored.  Called by a full warp; the first HD/8 lanes hold the row.
template <int HD, bool kHalf>
__device__ __forceinline__ void dec4_append(const Decode4Params &p, int b, int kvh, uint8_t *slot,
                                            const double2 *cs, int lane) {
    const int c = lane % (HD / 8);
    const long long src = (static_cast<long long>(b) * p.Hkv + kvh) * HD;
    float y[8], x[8];
    kv4_rotate8<HD, kHalf>(p.k_new + src, c, cs, y);
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4 *>(p.v_new + src + 8 * c)), x);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) bad |= kv4_clamp(y[i]) | kv4_clamp(x[i]);
    __half2 ksz, vsz;
    const uint32_t kw = kv4_quantise8(y, ksz), vw = kv4_quantise8(x, vsz);
    ksz = __shfl_sync(0xffffffffu, ksz, lane & ~3);
    vsz = __shfl_sync(0xffffffffu, vsz, lane & ~3);
    if (lane < HD / 8) {
        kv4_store8<HD>(slot, c, kw, ksz, vw, vsz);
        if (p.k_stored != nullptr) {
            kv4_values8(kw, ksz, y);
            *reinterpret_cast<uint4 *>(p.k_stored + src + 8 * c) = kv4_pack16<false>(y);
        }
        if (p.v_stored != nullptr) {
            kv4_values8(vw, vsz, x);
            *reinterpret_cast<uint4 *>(p.v_stored + src + 8 * c) = kv4_pack16<false>(x);
        }
        if (bad) raise_status(kStatusKv4Range);
    }
}

// ---------------------------------------------------------------------------- fragments
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero accumulator to begin with.
__device__ __forceinline__ void mma0_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma0_f16_1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
        "{%7,%7,%7,%7};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar,
                                          uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], "
        "%2, [%3], %4;" ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ float lo_f(uint32_t sz) {
    return __low2float(*reinterpret_cast<const __half2 *>(&sz));
}
__device__ __forceinline__ float hi_f(uint32_t sz) {
    return __high2float(*reinterpret_cast<const __half2 *>(&sz));
}
// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// The exponent e with x in [2^e, 2^(e+1)), for normal x > 0.
__device__ __forceinline__ int exponent_of(float x) { return (__float_as_int(x) >> 23) - 127; }

// Key of a tile's fragment row i (0 .. 15).  Neighbouring lanes' shared-memory reads then
// fall into different banks: rows are 160 (80) bytes apart, a fragment reads 16 (8) bytes by
// four lanes of a row for the keys and 8 (4) bytes by eight lanes for the values.
template <int HD>
__device__ __forceinline__ int dec4_key(int i) {
    const int h = (i >> 2) & 1, m = (i >> 1) & 1, b = i & 1;
    if constexpr (HD == 128)
        return (i & 8) + 4 * h + m + 2 * (b ^ h);
    else
        return (i & 8) + 2 * (i & 3) + h;
}

template <int HD, int NT>
struct Decode4Smem {
    static constexpr int kStageBytes = kDec4Tile * kv4_row_bytes(HD);
    alignas(128) uint8_t ring[kDec4Warps][kDec4Stages][kStageBytes];  // also the warps' outputs
    alignas(16) uint8_t new_row[kv4_row_bytes(HD)];
    double2 cs[HD / 2];
    uint4 q_hi[8 * NT][HD / 8], q_lo[8 * NT][HD / 8];  // fragments, see the rotation below
    float q_sum[8 * NT][HD / kKv4Group];  // sums of the scaled query over the groups
    float q_scale[8 * NT];  // what takes the scaled query back
    float m[kDec4Warps][8 * NT], l[kDec4Warps][8 * NT];
    uint64_t full[kDec4Warps][kDec4Stages];
    int abort;
};
template <int HD, int NT>
constexpr size_t decode4_smem_bytes() {
    return sizeof(Decode4Smem<HD, NT>) + 128;
}

// Each warp takes every fourth 32-key tile of the block's share by itself: a ring of bulk
// copies with a barrier per stage, no block-wide wait in the loop, and a partial result
// (max, sum, outputs) of its own, joined at the share's end.
//   Scores: S^T[16 keys x 8 heads] by m16n8k16, keys as A.  A code enters as the fp16
//   number with its four bits as the lowest of the mantissa, n 2^-24 (or n 2^-20 from the
//   byte's upper half, where the query is scaled by 2^-4): a mask is the whole conversion,
//   and exact.  The query is split into two fp16 parts.  Each 32-element group has its own
//   accumulator, multiplied by the row's s in fp32; z (sum of q over the group) is one more
//   product of fp16 operands, again with the sum in two parts.
//   Outputs: O^T[16 dims x 8 heads], value codes as A in the same way, B = p s in fp16; sum
//   p z in fp32.  p = 2^(score - R) for a reference R per head that puts the largest p s of
//   a tile at 2^12 and is raised only once one passes 2^15: small scales keep their bits
//   (fp16 holds 2^-14 at full precision), and the common tile costs one vote.
template <int HD, int NT, bool kHalf>
__global__ void __launch_bounds__(kDec4Threads, NT == 2 ? 2 : HD == 128 ? 3 : 4)
    decode4_split_kernel(const __grid_constant__ Decode4Params p) {
    using Smem = Decode4Smem<HD, NT>;
    constexpr int kRow = kv4_row_bytes(HD), G = HD / kKv4Group;
    extern __shared__ uint8_t smem_raw[];
    Smem *sm = reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                        ~static_cast<uintptr_t>(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane >> 2, r = lane & 3;
    const int g = p.group;
    const long long total = dec4_total(p, lane);
    const long long U = dec4_units_per_block(p, total);
    const long long u_lo = static_cast<long long>(blockIdx.x) * U;
    const long long u_hi = min(u_lo + U, total);
    if (blockIdx.x == 0 && tid == 0)
        for (int b = 0; b < p.B; ++b)
            if (p.cache_len[b] < 0 || p.cache_len[b] > p.T_max - 1) raise_status(kStatusBadCacheLen);
    if (u_lo >= u_hi) return;
    if (tid == 0) {
        for (int w = 0; w < kDec4Warps; ++w)
            for (int s = 0; s < kDec4Stages; ++s) mbar_init(&sm->full[w][s], 1);
        sm->abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    uint32_t n_loads = 0, n_waits = 0;  // of this warp's ring, over all segments
    const uint64_t policy = l2_policy_evict_first();
    bool ok = true;

    // Sequences before the first one of this block.
    int b = 0;
    long long seg0 = 0;
    for (long long v; b < p.B && seg0 + (v = dec4_seq_units(p, b)) <= u_lo; ++b) seg0 += v;
    for (; b < p.B && seg0 < u_hi; ++b) {
        const int L = p.cache_len[b];
        const DecRanges rg = dec4_ranges(p, L);
        const long long V = dec4_seg_units(static_cast<long long>(rg.len1) + rg.len2);
        if (V == 0) continue;
        int kvh = seg0 < u_lo ? static_cast<int>((u_lo - seg0) / V) : 0;
        seg0 += kvh * V;
        for (; kvh < p.Hkv && seg0 < u_hi; ++kvh, seg0 += V) {
            // Units [u0, u1) of the segment's keys are this block's: keys of the first
            // range, then of the second.
            const long long k0 = seg0 + kDec4Lead;
            const int u0 = static_cast<int>(max(u_lo, k0) - k0);
            const int u1 = static_cast<int>(min(u_hi, seg0 + V) - k0);
            if (u1 <= 0) continue;
            const int lo1 = min(u0, rg.len1), hi1 = min(u1, rg.len1);
            const int lo2 = rg.lo2 + max(u0, rg.len1) - rg.len1;
            const int hi2 = rg.lo2 + max(u1, rg.len1) - rg.len1;
            const int n_t1 = (hi1 - lo1 + kDec4Tile - 1) / kDec4Tile;
            const int n_tiles = n_t1 + (hi2 - lo2 + kDec4Tile - 1) / kDec4Tile;
            const bool has_L = u1 == rg.len1 + rg.len2;  // the new row is the last of this block's keys
            uint8_t *plane = p.kv4 + (static_cast<long long>(b) * p.Hkv + kvh) * p.T_max * kRow;
            auto tile_lo = [&](int i) { return i < n_t1 ? lo1 + i * kDec4Tile : lo2 + (i - n_t1) * kDec4Tile; };
            auto tile_n = [&](int i) { return min(kDec4Tile, (i < n_t1 ? hi1 : hi2) - tile_lo(i)); };
            auto load = [&](int i) {  // the cached rows of tile i: all but the new one
                const int s = n_loads % kDec4Stages;
                const int n = tile_n(i) - (has_L && i == n_tiles - 1 ? 1 : 0);
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sm->full[warp][s], n * kRow);
                    if (n > 0)
                        bulk_load(smem_u32(sm->ring[warp][s]), plane + static_cast<long long>(tile_lo(i)) * kRow,
                                  n * kRow, &sm->full[warp][s], policy);
                }
                ++n_loads;
            };
#pragma unroll
            for (int s = 0; s < kDec4Stages; ++s)
                if (warp + s * kDec4Warps < n_tiles) load(warp + s * kDec4Warps);

            // ---- queries: rotated, scaled, as fragments of two fp16 parts
            for (int i = tid; i < HD / 2; i += kDec4Threads) sm->cs[i] = kv4_cos_sin(L, p.turns[i]);
            __syncthreads();
            for (int i = tid; i < 8 * NT * (HD / 8); i += kDec4Threads) {
                const int h = i / (HD / 8), ch = i % (HD / 8);
                float y[8], mx = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = 0.f;
                if (h < g)
                    kv4_rotate8<HD, kHalf>(p.q_new + (static_cast<long long>(b) * p.Hq + kvh * g + h) * HD,
                                           ch, sm->cs, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(y[e]));
#pragma unroll
                for (int off = 1; off < HD / 8; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                // Largest element to [2^7, 2^8): both parts and their group sums fit fp16,
                // and the second part keeps its bits.
                const int e2 = mx > 0.f ? max(-100, min(127, exponent_of(mx))) : 0;
                const float f = pow2i(7 - e2);
                // The fragment words of lane r = ch % 4 for group ch / 4: word 2 part + k
                // holds elements 2 part + k and, above it, 4 further on; those of k = 1 meet
                // codes of the byte's upper half and are scaled by 2^-4.
                uint32_t hi[4], lo[4];
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v0 = y[e] * f, v1 = y[e + 4] * f;
                    sum += v0 + v1;
                    const float t0 = e & 1 ? v0 * 0.0625f : v0, t1 = e & 1 ? v1 * 0.0625f : v1;
                    const __half2 hv = __floats2half2_rn(t0, t1);
                    hi[e] = *reinterpret_cast<const uint32_t *>(&hv);
                    lo[e] = pack_half2(t0 - __low2float(hv), t1 - __high2float(hv));
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sm->q_hi[h][ch] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                sm->q_lo[h][ch] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if ((ch & 3) == 0) sm->q_sum[h][ch >> 2] = sum;
                if (ch == 0) sm->q_scale[h] = pow2i(e2 - 7);
            }
            const int last_warp = (n_tiles - 1) % kDec4Warps;
            if (has_L && warp == last_warp) {
                dec4_append<HD, kHalf>(p, b, kvh, sm->new_row, sm->cs, lane);
                __syncwarp();
                if (lane < kRow / 16)
                    reinterpret_cast<uint4 *>(plane + static_cast<long long>(L) * kRow)[lane] =
                        reinterpret_cast<const uint4 *>(sm->new_row)[lane];
            }
            __syncthreads();
            uint32_t qh[2 * G][NT][2], ql[2 * G][NT][2], qz[NT];
            float x_scale[NT][2], slope[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int h = nt * 8 + c;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    const uint4 hi = sm->q_hi[h][4 * gr + r], lo = sm->q_lo[h][4 * gr + r];
                    qh[2 * gr][nt][0] = hi.x;
                    qh[2 * gr][nt][1] = hi.y;
                    qh[2 * gr + 1][nt][0] = hi.z;
                    qh[2 * gr + 1][nt][1] = hi.w;
                    ql[2 * gr][nt][0] = lo.x;
                    ql[2 * gr][nt][1] = lo.y;
                    ql[2 * gr + 1][nt][0] = lo.z;
                    ql[2 * gr + 1][nt][1] = lo.w;
                }
                // The z product: k = 2r, 2r+1 stand for the sums' first parts of the groups
                // 2r, 2r+1 (r < 2) and for their second parts (r >= 2).
                const int g0 = 2 * (r & 1);
                const float z0 = g0 < G ? sm->q_sum[h][g0] : 0.f, z1 = g0 < G ? sm->q_sum[h][g0 + 1] : 0.f;
                const __half2 hv = __floats2half2_rn(z0, z1);
                qz[nt] = r < 2 ? *reinterpret_cast<const uint32_t *>(&hv)
                               : pack_half2(z0 - __low2float(hv), z1 - __high2float(hv));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = nt * 8 + 2 * r + j;
                    x_scale[nt][j] = p.sl2 * sm->q_scale[col];
                    // The bias m (L - n) in units of x, before x_scale.
                    slope[nt][j] = p.alibi ? exp2f(-8.0f * static_cast<float>(kvh * g + col + 1) /
                                                   static_cast<float>(p.Hq)) * 1.4426950408889634f /
                                                 x_scale[nt][j]
                                           : 0.f;
                }
            }

            float o[G][2][NT][4], w[NT][2][G], l[NT][2], R[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    R[nt][j] = -INFINITY;
                    l[nt][j] = 0.f;
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        w[nt][j][gr] = 0.f;
                        o[gr][0][nt][j] = o[gr][0][nt][j + 2] = 0.f;
                        o[gr][1][nt][j] = o[gr][1][nt][j + 2] = 0.f;
                    }
                }

            for (int i = warp; i < n_tiles; i += kDec4Warps) {
                const int s = n_waits % kDec4Stages;
                ok = ok && mbar_wait_drain(&sm->full[warp][s], (n_waits / kDec4Stages) & 1, p.timeout_ns);
                ++n_waits;
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                uint8_t *ring = sm->ring[warp][s];
                const int n0 = tile_lo(i), n_keys = tile_n(i);
                if (has_L && i == n_tiles - 1) {
                    if (lane < kRow / 16)
                        reinterpret_cast<uint4 *>(ring + (n_keys - 1) * kRow)[lane] =
                            reinterpret_cast<const uint4 *>(sm->new_row)[lane];
                    __syncwarp();
                }
#pragma unroll 1
                for (int sub = 0; sub < kDec4Tile; sub += 16) {
                    if (sub >= n_keys) break;
                    const int ka = sub + dec4_key<HD>(c), kb = ka + 8;  // this lane's keys
                    const uint8_t *ra = ring + ka * kRow, *rb = ring + kb * kRow;
                    uint32_t ca[G], cb[G], pa[G], pb[G];  // codes and (s, z) of the two keys
                    if constexpr (G == 4) {
                        *reinterpret_cast<uint4 *>(ca) = *reinterpret_cast<const uint4 *>(ra + 16 * r);
                        *reinterpret_cast<uint4 *>(cb) = *reinterpret_cast<const uint4 *>(rb + 16 * r);
                        *reinterpret_cast<uint4 *>(pa) = *reinterpret_cast<const uint4 *>(ra + HD);
                        *reinterpret_cast<uint4 *>(pb) = *reinterpret_cast<const uint4 *>(rb + HD);
                    } else {
                        *reinterpret_cast<uint2 *>(ca) = *reinterpret_cast<const uint2 *>(ra + 8 * r);
                        *reinterpret_cast<uint2 *>(cb) = *reinterpret_cast<const uint2 *>(rb + 8 * r);
                        *reinterpret_cast<uint2 *>(pa) = *reinterpret_cast<const uint2 *>(ra + HD);
                        *reinterpret_cast<uint2 *>(pb) = *reinterpret_cast<const uint2 *>(rb + HD);
                    }
                    float x[NT][4], xz[NT][4];
                    {
                        const int at = HD + (G == 4 ? 8 * (r & 1) : 0);
                        const uint2 wa = *reinterpret_cast<const uint2 *>(ra + at);
                        const uint2 wb = *reinterpret_cast<const uint2 *>(rb + at);
                        const uint32_t za = __byte_perm(wa.x, wa.y, 0x7632), zb = __byte_perm(wb.x, wb.y, 0x7632);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma0_f16_1688(xz[nt], za, zb, qz[nt]);
                    }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        float acc[NT][4];
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            const uint32_t wa = ca[gr] >> (8 * part), wb = cb[gr] >> (8 * part);
                            const uint32_t a0 = wa & 0x000f000fu, a2 = wa & 0x00f000f0u;
                            const uint32_t a1 = wb & 0x000f000fu, a3 = wb & 0x00f000f0u;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (part == 0)
                                    mma0_f16_16816(acc[nt], a0, a1, a2, a3, qh[2 * gr][nt][0], qh[2 * gr][nt][1]);
                                else
                                    mma_f16_16816(acc[nt], a0, a1, a2, a3, qh[2 * gr + 1][nt][0], qh[2 * gr + 1][nt][1]);
                                mma_f16_16816(acc[nt], a0, a1, a2, a3, ql[2 * gr + part][nt][0], ql[2 * gr + part][nt][1]);
                            }
                        }
                        const float sa = lo_f(pa[gr]), sb = lo_f(pb[gr]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[nt][e] = gr == 0 ? (e < 2 ? sa : sb) * acc[nt][e]
                                                   : fmaf(e < 2 ? sa : sb, acc[nt][e], x[nt][e]);
                        }
                    }
                    // ---- scores over x_scale; then the values' (s, z) of the two keys
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[nt][e] = fmaf(x[nt][e], 16777216.f, xz[nt][e]);
                    if constexpr (G == 4) {
                        *reinterpret_cast<uint4 *>(pa) = *reinterpret_cast<const uint4 *>(ra + HD + 4 * G);
                        *reinterpret_cast<uint4 *>(pb) = *reinterpret_cast<const uint4 *>(rb + HD + 4 * G);
                    } else {
                        *reinterpret_cast<uint2 *>(pa) = *reinterpret_cast<const uint2 *>(ra + HD + 4 * G);
                        *reinterpret_cast<uint2 *>(pb) = *reinterpret_cast<const uint2 *>(rb + HD + 4 * G);
                    }
                    if (p.alibi) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[nt][e] = fmaf(-slope[nt][e & 1], static_cast<float>(L - n0 - (e < 2 ? ka : kb)), x[nt][e]);
                    }
                    if (n_keys < kDec4Tile) {  // rows behind the tile's end do not count
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((e < 2 ? ka : kb) >= n_keys) x[nt][e] = -INFINITY;
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            if (ka >= n_keys) pa[gr] = 0;
                            if (kb >= n_keys) pb[gr] = 0;
                        }
                    }
                    float pr[NT][4];
                    uint32_t bf[G][NT][2];
                    // Probabilities and B operands; true if one of the latter nears fp16's end
                    // (or would, but for a scale of 0).
                    auto products = [&] {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) pr[nt][e] = ex2f(fmaf(x[nt][e], x_scale[nt][e & 1], -R[nt][e & 1]));
                        float p_max = 0.f;
                        __half2 t = __half2half2(__ushort_as_half(0));
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            const float sa = lo_f(pa[gr]), sb = lo_f(pb[gr]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                bf[gr][nt][0] = pack_half2(pr[nt][0] * sa, pr[nt][1] * sa);
                                bf[gr][nt][1] = pack_half2(pr[nt][2] * sb, pr[nt][3] * sb);
                                t = __hmax2(t, *reinterpret_cast<const __half2 *>(&bf[gr][nt][0]));
                                t = __hmax2(t, *reinterpret_cast<const __half2 *>(&bf[gr][nt][1]));
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            p_max = fmaxf(p_max, fmaxf(fmaxf(pr[nt][0], pr[nt][1]), fmaxf(pr[nt][2], pr[nt][3])));
                        const uint32_t largest = *reinterpret_cast<const uint32_t *>(&t);
                        return ((largest + 0x08000800u) & 0x80008000u) != 0 || p_max > 1.1e12f;
                    };
                    if (__any_sync(0xffffffffu, products())) {
                        // Raise the references to these keys' largest p s, put at 2^12 (a scale
                        // below fp16's smallest counts as that).
                        float sa = 0.f, sb = 0.f;
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            sa = fmaxf(sa, lo_f(pa[gr]));
                            sb = fmaxf(sb, lo_f(pb[gr]));
                        }
                        sa = log2f(fmaxf(sa, 5.9604645e-8f)) - 12.f;
                        sb = log2f(fmaxf(sb, 5.9604645e-8f)) - 12.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float t = fmaxf(fmaf(x[nt][j], x_scale[nt][j], sa), fmaf(x[nt][j + 2], x_scale[nt][j], sb));
#pragma unroll
                                for (int off = 4; off < 32; off <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
                                t = fmaxf(t, R[nt][j]);
                                if (!(fabsf(t) < INFINITY)) t = R[nt][j] == -INFINITY ? 0.f : R[nt][j];
                                const float f = R[nt][j] == -INFINITY ? 0.f : ex2f(R[nt][j] - t);
                                R[nt][j] = t;
                                l[nt][j] *= f;
#pragma unroll
                                for (int gr = 0; gr < G; ++gr) {
                                    w[nt][j][gr] *= f;
                                    o[gr][0][nt][j] *= f;
                                    o[gr][0][nt][j + 2] *= f;
                                    o[gr][1][nt][j] *= f;
                                    o[gr][1][nt][j + 2] *= f;
                                }
                            }
                        products();
                    }
                    // ---- sums, and O^T += V^T P
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            l[nt][j] += pr[nt][j] + pr[nt][j + 2];
#pragma unroll
                            for (int gr = 0; gr < G; ++gr)
                                w[nt][j][gr] = fmaf(pr[nt][j], hi_f(pa[gr]), fmaf(pr[nt][j + 2], hi_f(pb[gr]), w[nt][j][gr]));
                        }
                    uint32_t vw[4][G / 2];  // value words of the four keys of this lane's k indices
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint8_t *row = ring + (sub + dec4_key<HD>((k >> 1) * 8 + 2 * r + (k & 1))) * kRow + HD / 2;
                        if constexpr (G == 4)
                            *reinterpret_cast<uint2 *>(vw[k]) = *reinterpret_cast<const uint2 *>(row + 8 * c);
                        else
                            vw[k][0] = *reinterpret_cast<const uint32_t *>(row + 4 * c);
                    }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        const uint32_t sel = gr & 1 ? 0x7632u : 0x5410u;
                        const uint32_t u = __byte_perm(vw[0][gr / 2], vw[1][gr / 2], sel);
                        const uint32_t t = __byte_perm(vw[2][gr / 2], vw[3][gr / 2], sel);
                        uint32_t b0[NT], b1[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            b0[nt] = transpose8(bf[gr][nt][0]);
                            b1[nt] = transpose8(bf[gr][nt][1]);
                        }
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t us = u >> (8 * m), ts = t >> (8 * m);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16_16816(o[gr][m][nt], us & 0x000f000fu, us & 0x00f000f0u,
                                              ts & 0x000f000fu, ts & 0x00f000f0u, b0[nt], b1[nt]);
                        }
                    }
                }
                __syncwarp();  // the whole warp is done with the stage
                const int nxt = i + kDec4Stages * kDec4Warps;
                if (nxt < n_tiles) load(nxt);
            }

            // ---- the warps' results: outputs of head h, dims, in place of the ring
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
#pragma unroll
                        for (int gr = 0; gr < G; ++gr)
                            w[nt][j][gr] += __shfl_xor_sync(0xffffffffu, w[nt][j][gr], off);
                    }
                    if (lane < 4) {
                        sm->m[warp][nt * 8 + 2 * r + j] = R[nt][j];
                        sm->l[warp][nt * 8 + 2 * r + j] = l[nt][j];
                    }
                }
            if (!ok) {  // a copy did not land: no partial result to trust
                raise_status(kStatusTimeoutDecode);
                sm->abort = 1;
                for (; n_waits < n_loads; ++n_waits)  // the copies still under way
                    mbar_wait_drain(&sm->full[warp][n_waits % kDec4Stages],
                                    (n_waits / kDec4Stages) & 1, p.timeout_ns);
            }
            __syncthreads();
            if (sm->abort) return;
            float *red = reinterpret_cast<float *>(&sm->ring[0][0][0]);  // [warps][8 NT][HD]
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float add = w[nt][j][gr];
                        const float4 out = make_float4(fmaf(o[gr][0][nt][j], 16777216.f, add),
                                                       fmaf(o[gr][0][nt][j + 2], 1048576.f, add),
                                                       fmaf(o[gr][1][nt][j], 16777216.f, add),
                                                       fmaf(o[gr][1][nt][j + 2], 1048576.f, add));
                        *reinterpret_cast<float4 *>(red + (warp * 8 * NT + nt * 8 + 2 * r + j) * HD + 32 * gr + 4 * c) = out;
                    }
            }
            __syncthreads();
            const long long slot = (blockIdx.x + static_cast<long long>(b) * p.Hkv + kvh) * g;
            for (int i = tid; i < g * HD; i += kDec4Threads) {
                const int h = i / HD, dim = i % HD;
                float top_m = -INFINITY, acc = 0.f, sum = 0.f;
#pragma unroll
                for (int k = 0; k < kDec4Warps; ++k) top_m = fmaxf(top_m, sm->m[k][h]);
#pragma unroll
                for (int k = 0; k < kDec4Warps; ++k) {
                    const float f = sm->m[k][h] == -INFINITY ? 0.f : ex2f(sm->m[k][h] - top_m);
                    acc += f * red[(k * 8 * NT + h) * HD + dim];
                    sum += f * sm->l[k][h];
                }
                p.ws_o[(slot + h) * HD + dim] = acc;
                if (dim == 0) {
                    p.ws_ml[(slot + h) * 2] = top_m;
                    p.ws_ml[(slot + h) * 2 + 1] = sum;
                }
            }
            fence_proxy_async_smem();  // the ring's next copies follow these writes and reads
            __syncthreads();
        }
    }
}

// One block per (query head, sequence): the pieces of its segment, by log-sum-exp weights.
template <int HD>
__global__ void __launch_bounds__(HD) decode4_merge_kernel(const __grid_constant__ Decode4Params p) {
    const int hq = blockIdx.x % p.Hq, b = blockIdx.x / p.Hq, dim = threadIdx.x;
    const int L = p.cache_len[b], g = p.group, kvh = hq / g, hh = hq % g;
    const long long oi = static_cast<long long>(b) * p.Hq + hq;
    const DecRanges rg = dec4_ranges(p, L);
    const long long V = dec4_seg_units(static_cast<long long>(rg.len1) + rg.len2);
    if (V == 0) {  // a length outside the cache
        p.o[oi * HD + dim] = __float2bfloat16(__int_as_float(0x7fc00000));
        if (p.lse != nullptr && dim == 0) p.lse[oi] = __int_as_float(0x7fc00000);
        return;
    }
    const int lane = dim & 31;
    const long long U = dec4_units_per_block(p, dec4_total(p, lane));
    long long seg0 = 0;
    for (int i = lane; i < b; i += 32) seg0 += dec4_seq_units(p, i);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) seg0 += __shfl_xor_sync(0xffffffffu, seg0, off);
    seg0 += kvh * V;
    const int first = static_cast<int>((seg0 + kDec4Lead) / U), last = static_cast<int>((seg0 + V - 1) / U);
    const long long seg = static_cast<long long>(b) * p.Hkv + kvh;
    float M = -INFINITY;
    for (int i = first; i <= last; ++i) M = fmaxf(M, p.ws_ml[((i + seg) * g + hh) * 2]);
    float acc = 0.f, sum = 0.f;
    for (int i = first; i <= last; ++i) {
        const long long s = (i + seg) * g + hh;
        const float w = M == -INFINITY ? 0.f : ex2f(p.ws_ml[s * 2] - M);
        sum += w * p.ws_ml[s * 2 + 1];
        acc += w * p.ws_o[s * HD + dim];
    }
    p.o[oi * HD + dim] = __float2bfloat16_rn(acc / sum);
    if (p.lse != nullptr && dim == 0) p.lse[oi] = (M + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace yr
