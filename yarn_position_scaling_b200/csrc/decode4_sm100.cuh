// decode4_sm100.cuh -- decode over the 4-bit KV cache (row format in kv4_sm100.cuh), one token
// or a few, split-KV with a log-sum-exp merge.
//
//   logit(t) = scale q~ . k_t,  k_t = s n + z by group;  o = sum_t p_t v_t / sum_t p_t
//
// The keys that the tokens of a (sequence, KV head) segment see, of all segments laid end to
// end, are cut into one equal share per block; a block leaves one partial (reference, sum,
// unnormalised output) per query head and token of each segment piece.  Pieces are numbered block + segment: along the blocks
// each next piece raises the one, the other or both, so no two share a number, and
// blocks + segments slots hold them all whatever the lengths.
#pragma once
#include "decode_sm100.cuh"
#include "kv4_sm100.cuh"

namespace yr {

constexpr int kDec4Chunk = 128;      // least keys per block: a tile for each warp
constexpr int kDec4Lead = 256;       // what a segment costs besides its keys, in keys (4 us)
constexpr int kDec4MaxBlocks = 640;  // most blocks of the split launch
constexpr int kDec4Warps = 4;
constexpr int kDec4Threads = kDec4Warps * 32;
constexpr int kDec4Tile = 32;  // keys of one bulk copy
constexpr int kDec4Stages = 2;
// The tensor cores' fp32 sums are cut off, not rounded, and the sum of p s n, all positive, is far
// larger than the output where values of both signs cancel: over 128K keys of like weight, 8 KV
// heads, a warp's 21K keys (48 sequences) give 1.2 - 1.3% error and its 3.5K keys (8 sequences)
// 0.24%.  So the accumulators are folded into rounded sums every 16 tiles: 0.17 - 0.18% for both,
// where rounding the output to bf16 gives 0.16 - 0.17%, for up to 2% of the time (8 sequences 287.6
// -> 289.5 us; with a fold every 32 or 64 tiles 0.18 and 0.19 - 0.20%, every 8 no less error).
constexpr int kDec4Fold = 16;
// The reference of a column that has seen no key yet: no finite score lies below it.
constexpr float kNoScore = -3.402823466e38f;
// Scores from 2^22 on have units of 0.5 or more, too coarse for a reference a few units off one.
constexpr float kCoarseScore = 4194304.f;

struct Decode4Params {
    const __nv_bfloat16 *q_new;          // [B][Hq][Tq][d]
    const __nv_bfloat16 *k_new, *v_new;  // [B][Hkv][d], Tq = 1: the row to append; or null
    uint8_t *kv4;                        // [B][Hkv][T_max][5d/4]
    const int *cache_len;                // [B], position of the first token; or null: P0
    float *ws_o;                         // [slots][seg_tokens g][d]
    float *ws_ml;                        // [slots][seg_tokens g][2]
    __nv_bfloat16 *o;                    // [B][Hq][Tq][d]
    float *lse;                          // [B][Hq][Tq] or null
    __nv_bfloat16 *k_stored, *v_stored;  // [B][Hkv][d] or null
    int B, Hq, Hkv, T_max, group;
    int P0, Tq;
    int seg_tokens, n_segs;  // tokens of a segment, segments of a sequence and KV head
    int grid_blocks;
    int window, n_sink;
    // Softmax scale times log2 e, as a number that goes into the queries and a power of two.  A
    // score's product with the latter is exact, and so its distance from another in an FMA: with the
    // whole scale there, the product's unrounded rest, 2^-25 of a score, stood in every exponent.
    float sl2_part, sl2_pow2;
    int alibi;
    uint64_t timeout_ns;
#ifdef YR_FAULT_HOOKS
    // Failure-detection test hook, in the test build only: warp 0 of one block (-1: none) issues
    // all its copies but one, counted from 0, so a wait that nothing will complete runs out of time.
    int fault_block, fault_copy;
#endif
    double turns[64];
};

// Segment st of the B n_segs (sequence, run of tokens) pairs: positions first .. last of its
// tokens, and the ranges [0, len1) and [lo2, lo2 + len2) of the keys that one of them sees.
struct Dec4Seg {
    int first, last;
    DecRanges keys;
};
// (kMulti: more than one token; a decode step's code is spared the divisions and masks.)
template <bool kMulti>
__device__ __forceinline__ int dec4_sequence(const Decode4Params &p, int st) {
    return kMulti ? st / p.n_segs : st;
}
// Token of a column within its segment.
template <bool kMulti>
__device__ __forceinline__ int dec4_token(const Decode4Params &p, int col) {
    return kMulti ? col / p.group : 0;
}
template <bool kMulti>
__device__ __forceinline__ Dec4Seg dec4_seg(const Decode4Params &p, int st) {
    Dec4Seg s{0, -1, {0, 0, 0}};
    const int b = dec4_sequence<kMulti>(p, st), t0 = kMulti ? (st - b * p.n_segs) * p.seg_tokens : 0;
    const int L = kMulti ? p.P0 : p.cache_len[b];
    if (L < 0 || L > p.T_max - (kMulti ? p.Tq : 1)) return s;
    s.first = L + t0;
    s.last = kMulti ? L + min(t0 + p.seg_tokens, p.Tq) - 1 : L;
    const int s1 = min(p.n_sink, s.last + 1);
    const int w0 = p.window > 0 ? max(s.first - p.window + 1, 0) : 0;
    if (w0 <= s1) {
        s.keys.len1 = s.last + 1;
        s.keys.lo2 = s.last + 1;
    } else {
        s.keys.len1 = s1;
        s.keys.lo2 = w0;
        s.keys.len2 = s.last + 1 - w0;
    }
    return s;
}

// The partition, as every block derives it from cache_len.  A segment is kDec4Lead units for
// what a block does once for it (query, partial result) and one for each key: blocks of many
// short segments and blocks of few long ones take equally long, and while there are blocks
// enough no two segments' keys fall to the same one.  (Without the lead 88 segments of two keys
// all went to one block and took 490 us.)
template <bool kMulti>
__device__ __forceinline__ int dec4_keys(const Decode4Params &p, int st) {
    const DecRanges r = dec4_seg<kMulti>(p, st).keys;
    return r.len1 + r.len2;
}
// Units of a segment: none for a length outside the cache.
__device__ __forceinline__ long long dec4_units(int keys) {
    return keys > 0 ? static_cast<long long>(keys) + kDec4Lead : 0;
}
// Units of a block.  Called by a full warp.
template <bool kMulti>
__device__ __forceinline__ long long dec4_share(const Decode4Params &p, int lane) {
    long long total = 0;
    for (int st = lane; st < (kMulti ? p.B * p.n_segs : p.B); st += 32) total += dec4_units(dec4_keys<kMulti>(p, st));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    const long long even = (total * p.Hkv + p.grid_blocks - 1) / p.grid_blocks;
    return even > kDec4Chunk ? even : kDec4Chunk;
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
__device__ __forceinline__ void mma_f16_1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0));
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

// (Kept small: what shared memory leaves of an SM's 256 KB is the L1 that spills live in.)
template <int HD, int NT, bool kMulti>
struct Decode4Smem {
    static constexpr int kStageBytes = kDec4Tile * kv4_row_bytes(HD);
    alignas(128) uint8_t ring[kDec4Warps][kDec4Stages][kStageBytes];  // also the warps' outputs
    alignas(16) uint8_t new_row[kMulti ? 16 : kv4_row_bytes(HD)];
    double2 cs[kMulti ? 1 : HD / 2];   // of the one token, for the new row
    float2 q_cs[kMulti ? 1 : HD / 2];  // and for the queries
    uint4 q_hi[8 * NT][HD / 8], q_lo[8 * NT][HD / 8];  // fragments, see the rotation below
    float q_sum[8 * NT][HD / kKv4Group];  // sums of the scaled query over the groups
    float q_scale[8 * NT];  // power of two that makes a score of the scaled query one in log2 units
    float slope[8 * NT];
    float m[kDec4Warps][8 * NT], l[kDec4Warps][8 * NT];
    uint64_t full[kDec4Warps][kDec4Stages];
    int abort;
};
template <int HD, int NT, bool kMulti>
constexpr size_t decode4_smem_bytes() {
    return sizeof(Decode4Smem<HD, NT, kMulti>) + 128;
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
//   Up to four heads leave columns free: with REP = 2 (or 4, up to two heads) each head has
//   REP of the eight.  Every second of them takes the query's second part, whose scores are
//   then added across lanes, and each stands for its own groups in the value product, which
//   divides the work on p s among the lanes that would else idle.
//   Outputs: O^T[16 dims x 8 heads], value codes as A in the same way, B = p s in fp16; sum
//   p z in fp32.  p = 2^(score - R) for a reference R per head that puts the largest p s of
//   a tile at 2^8 and is raised only once one passes 2^15: small scales keep their bits
//   (fp16 holds 2^-14 at full precision), and the common tile costs one vote.
//   Scores are the queries' products times a power of two, so that score - R is exact but for
//   one rounding however large the scores are.
template <int HD, int NT, int REP, bool kHalf, bool kMulti>
__global__ void __launch_bounds__(kDec4Threads, NT == 2 ? 2 : 4)
    decode4_split_kernel(const __grid_constant__ Decode4Params p) {
    using Smem = Decode4Smem<HD, NT, kMulti>;
    constexpr int kRow = kv4_row_bytes(HD), G = HD / kKv4Group;
    static_assert(REP == 1 || (NT == 1 && REP <= G), "columns to spare");
    // A step takes 16 H keys through scores and outputs.  Two halves overlap; with one query head
    // a KV head, where the work on p s is least, one at a time spills less (78 against 86 us on
    // 16 windowed sequences of 32 KV heads, but 183 against 175 on 8 long ones with REP = 2).
    constexpr int H = REP == 4 ? 1 : 2;
    constexpr int GL = G / REP;       // groups of a lane in the value product: k REP + copy
    constexpr int kCopy = 4 / REP;    // lanes r of a copy; the next copy is as far away
    extern __shared__ uint8_t smem_raw[];
    Smem *sm = reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                        ~static_cast<uintptr_t>(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane >> 2, r = lane & 3;
    const int g = p.group, copy = r / kCopy;
    // Where this lane's operands begin in a tile: row of fragment row c, and value codes of the
    // rows of k indices 2r and 2r + 1.
    const int key_at = dec4_key<HD>(c) * kRow;
    const int val_at0 = dec4_key<HD>(2 * r) * kRow + HD / 2 + (G == 4 ? 8 : 4) * c;
    const int val_at1 = dec4_key<HD>(2 * r + 1) * kRow + HD / 2 + (G == 4 ? 8 : 4) * c;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long U = dec4_share<kMulti>(p, lane);
    const long long u_lo = blockIdx.x * U, u_hi = u_lo + U;
    if (!kMulti && blockIdx.x == 0)
        for (int b = tid; b < p.B; b += kDec4Threads)
            if (p.cache_len[b] < 0 || p.cache_len[b] > p.T_max - 1) raise_status(kStatusBadCacheLen);
    // This warp's ring, over all segments: the stages of the next copy and the next wait,
    // and the parity of the latter.
    uint32_t s_load = 0, s_wait = 0, parity = 0;
    const uint64_t policy = l2_policy_evict_first();
#ifdef YR_FAULT_HOOKS
    int n_copies = 0;
#endif

    // Segments before the first one of this block.
    // 32 at a time, by a sum over the lanes.
    int st = 0;
    long long seg0 = 0;
    const int n_st = kMulti ? p.B * p.n_segs : p.B;
    for (; st < n_st; st += 32) {
        const long long v = st + lane < n_st ? p.Hkv * dec4_units(dec4_keys<kMulti>(p, st + lane)) : 0;
        long long upto = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += t;
        }
        const uint32_t beyond = __ballot_sync(0xffffffffu, seg0 + upto > u_lo);
        if (beyond != 0) {
            const int at = __ffs(beyond) - 1;
            seg0 += __shfl_sync(0xffffffffu, upto - v, at);
            st += at;
            break;
        }
        seg0 += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (st >= n_st) return;
    if (tid == 0) {
        for (int w = 0; w < kDec4Warps; ++w)
            for (int s = 0; s < kDec4Stages; ++s) mbar_init(&sm->full[w][s], 1);
        sm->abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    for (; st < n_st && seg0 < u_hi; ++st) {
        const Dec4Seg seg = dec4_seg<kMulti>(p, st);
        const DecRanges rg = seg.keys;
        const int L = seg.last, b = dec4_sequence<kMulti>(p, st);
        const int t0 = kMulti ? (st - b * p.n_segs) * p.seg_tokens : 0;
        const int cols = (kMulti ? seg.last - seg.first + 1 : 1) * g;  // column: token times heads plus head
        const long long V = dec4_units(rg.len1 + rg.len2);
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
            // A row to append is the last of the last block's keys.
            const bool has_L = !kMulti && u1 == rg.len1 + rg.len2;
            uint8_t *plane = p.kv4 + (static_cast<long long>(b) * p.Hkv + kvh) * p.T_max * kRow;
            // This warp's tiles, as copies and as steps pass through them: every fourth of the
            // first range, then of the second, the warps taking turns across the seam.
            constexpr int kStride = kDec4Warps * kDec4Tile;
            const int lo2w = lo2 + kDec4Tile * ((warp - n_t1) & (kDec4Warps - 1));
            int ld_key = lo1 + kDec4Tile * warp, ld_end = hi1;
            if (ld_key >= ld_end) {
                ld_key = lo2w;
                ld_end = hi2;
            }
            // After a copy that did not land the rest of the share is not read any more; its new rows
            // are still made.
            if (sm->abort) ld_key = ld_end;
            int key = ld_key, end = ld_end;
            auto advance = [&](int &k, int &e) {
                k += kStride;
                if (k >= e && k < kStride + hi1 && e == hi1 && hi2 > lo2) {
                    k = lo2w;
                    e = hi2;
                }
            };
            auto load = [&] {  // the cached rows of the next tile: all but the new one
                bool issue = lane == 0;
#ifdef YR_FAULT_HOOKS
                if (static_cast<int>(blockIdx.x) == p.fault_block && warp == 0 && n_copies++ == p.fault_copy) issue = false;
#endif
                if (issue) {
                    const int n = min(kDec4Tile, ld_end - ld_key);
                    const uint32_t bytes = (n - (has_L && ld_key + n > L ? 1 : 0)) * kRow;
                    uint64_t *bar = &sm->full[warp][s_load];
                    mbar_arrive_expect_tx(bar, bytes);
                    if (bytes > 0)
                        bulk_load(smem_u32(sm->ring[warp][s_load]),
                                  plane + static_cast<long long>(ld_key) * kRow, bytes, bar, policy);
                }
                s_load = s_load + 1 == kDec4Stages ? 0 : s_load + 1;
                advance(ld_key, ld_end);
            };
#pragma unroll
            for (int s = 0; s < kDec4Stages; ++s)
                if (ld_key < ld_end) load();

            // ---- queries: rotated, scaled, as fragments of two fp16 parts
            constexpr int kItems = 8 * NT * (HD / 8);  // chunks of eight elements
            constexpr int kPer = (kItems + kDec4Threads - 1) / kDec4Threads;
            uint4 raw[kPer], other[kPer];
#pragma unroll
            for (int n = 0; n < kPer; ++n) {
                const int i = tid + n * kDec4Threads, h = i / (HD / 8), ch = i % (HD / 8);
                raw[n] = other[n] = make_uint4(0, 0, 0, 0);
                if (i < kItems && h < cols) {
                    const uint4 *row = reinterpret_cast<const uint4 *>(
                        p.q_new + ((static_cast<long long>(b) * p.Hq + kvh * g + h - dec4_token<kMulti>(p, h) * g) * (kMulti ? p.Tq : 1) + t0 + dec4_token<kMulti>(p, h)) * HD);
                    raw[n] = __ldg(row + ch);
                    if (kHalf) other[n] = __ldg(row + (ch ^ (HD / 16)));
                }
            }
            // The new row wants its sines in 64 bits; the queries' 22 bits do with fp32 ones.  Of
            // one token they are shared by its heads, of several each thread computes its own.  They
            // carry the softmax scale's part that is not a power of two.
            auto cos_sin = [&](int pos, int i) {
                const double n = static_cast<double>(pos), tr = n * p.turns[i];
                float sn, co;
                sincospif(2.f * static_cast<float>(tr - rint(tr) + fma(n, p.turns[i], -tr)), &sn, &co);
                return make_float2(co * p.sl2_part, sn * p.sl2_part);
            };
            if constexpr (!kMulti) {
                for (int i = tid; i < HD / 2; i += kDec4Threads) {
                    if (has_L) {
                        const double2 t = kv4_cos_sin(L, p.turns[i]);
                        sm->cs[i] = t;
                        sm->q_cs[i] = make_float2(static_cast<float>(t.x) * p.sl2_part, static_cast<float>(t.y) * p.sl2_part);
                    } else {
                        sm->q_cs[i] = cos_sin(L, i);
                    }
                }
                __syncthreads();
            }
#pragma unroll
            for (int n = 0; n < kPer; ++n) {
                const int i = tid + n * kDec4Threads, h = i / (HD / 8), ch = i % (HD / 8);
                if (i >= kItems) break;
                float x[8], y[8], mx = 0.f;
                unpack_bf16x8(raw[n], x);
                const int pos = seg.first + dec4_token<kMulti>(p, h);
                if constexpr (kHalf) {
                    float z[8];
                    unpack_bf16x8(other[n], z);
                    const int c0 = 8 * (ch % (HD / 16));
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = kMulti ? cos_sin(pos, c0 + e) : sm->q_cs[c0 + e];
                        y[e] = ch < HD / 16 ? x[e] * t.x - z[e] * t.y : z[e] * t.y + x[e] * t.x;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 t = kMulti ? cos_sin(pos, 4 * ch + e) : sm->q_cs[4 * ch + e];
                        y[2 * e] = x[2 * e] * t.x - x[2 * e + 1] * t.y;
                        y[2 * e + 1] = x[2 * e] * t.y + x[2 * e + 1] * t.x;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(y[e]));
#pragma unroll
                for (int off = 1; off < HD / 8; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                // Largest element to [2^7, 2^8): both parts and their group sums fit fp16,
                // and the second part keeps its bits.  (Below 2^-60 a query scores 0 anyway, and
                // ALiBi's slope in these units has to stay within fp32.)
                const int e2 = mx > 0.f ? max(-60, min(127, exponent_of(mx))) : 0;
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
                if (ch == 0) {
                    const float back = pow2i(e2 - 7) * p.sl2_pow2;
                    sm->q_scale[h] = back;
                    // ALiBi's slope in units of a score before its scaling by q_scale.
                    sm->slope[h] = p.alibi ? exp2f(-8.0f * static_cast<float>(kvh * g + h - dec4_token<kMulti>(p, h) * g + 1) /
                                                   static_cast<float>(p.Hq)) * 1.4426950408889634f / back
                                           : 0.f;
                }
            }
            __syncthreads();
            // The warp whose tile ends with the new row makes it meanwhile.
            const int tile_L = hi2 > lo2 ? n_t1 + (L - lo2) / kDec4Tile : (L - lo1) / kDec4Tile;
            if (has_L && warp == (tile_L & (kDec4Warps - 1))) {
                dec4_append<HD, kHalf>(p, b, kvh, sm->new_row, sm->cs, lane);
                __syncwarp();
                if (lane < kRow / 16)
                    reinterpret_cast<uint4 *>(plane + static_cast<long long>(L) * kRow)[lane] =
                        reinterpret_cast<const uint4 *>(sm->new_row)[lane];
            }
            // Of the two parts, this column's with copies, else both (from shared memory, in
            // the loop: registers are short).
            uint4 q_reg[G];
            uint32_t qz[NT];
            float x_scale[NT][2];
            const int col_head = REP == 1 ? c : c % (8 / REP);
            const bool second = REP > 1 && (c / (8 / REP)) % 2 == 1;
            if constexpr (REP > 1) {
#pragma unroll
                for (int gr = 0; gr < G; ++gr)
                    q_reg[gr] = second ? sm->q_lo[col_head][4 * gr + r] : sm->q_hi[col_head][4 * gr + r];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int h = nt * 8 + col_head;
                // The z product: k = 2r, 2r+1 stand for the sums' first parts of the groups
                // 2r, 2r+1 (r < 2) and for their second parts (r >= 2).
                const int g0 = 2 * (r & 1);
                const float z0 = g0 < G && !second ? sm->q_sum[h][g0] : 0.f;
                const float z1 = g0 < G && !second ? sm->q_sum[h][g0 + 1] : 0.f;
                const __half2 hv = __floats2half2_rn(z0, z1);
                qz[nt] = r < 2 ? *reinterpret_cast<const uint32_t *>(&hv)
                               : pack_half2(z0 - __low2float(hv), z1 - __high2float(hv));
#pragma unroll
                for (int j = 0; j < 2; ++j) x_scale[nt][j] = sm->q_scale[nt * 8 + 2 * (r % kCopy) + j];
            }

            // With kShare the outputs of group k REP + copy are in o[k]: the copies' columns take
            // turns, each group's B operand being zero in the others'.  It saves registers (d =
            // 128: 195 -> 175 us on 8 long sequences of 8 KV heads); where there are enough, the
            // zeroing costs more (d = 64: 45.8 -> 47.3 us on 4 sequences of 60K keys and 8 heads).
            constexpr bool kShare = REP > 1 && HD == 128;
            constexpr int GO = kShare ? GL : G;
            float o[GO][2][NT][4], w[NT][2][GL], l[NT][2], R[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    R[nt][j] = kNoScore;
                    l[nt][j] = 0.f;
#pragma unroll
                    for (int k = 0; k < GL; ++k) w[nt][j][k] = 0.f;
#pragma unroll
                    for (int k = 0; k < GO; ++k) {
                        o[k][0][nt][j] = o[k][0][nt][j + 2] = 0.f;
                        o[k][1][nt][j] = o[k][1][nt][j + 2] = 0.f;
                    }
                }

            // What the accumulators are folded into, relative to references of their own.  In
            // memory, where the compiler has to be told to leave it: registers are short.
            float sums_mem[GO * 2 * NT * 4 + NT * 2], *sums = sums_mem;
            asm volatile("" : "+l"(sums)::"memory");
            bool folded = false;
            auto fold = [&](bool keep) {
                float *sums_R = sums + GO * 2 * NT * 4;
                float f[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        f[nt][j] = folded ? ex2f(sums_R[nt * 2 + j] - R[nt][j]) : 0.f;
                        if (!keep) sums_R[nt * 2 + j] = R[nt][j];
                    }
#pragma unroll
                for (int i = 0; i < GO; ++i)
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float *at = sums + ((i * 2 + a) * NT + nt) * 4 + e;
                                const float sum = folded ? fmaf(*at, f[nt][e & 1], o[i][a][nt][e]) : o[i][a][nt][e];
                                if (!keep) *at = sum;
                                o[i][a][nt][e] = keep ? sum : 0.f;
                            }
                folded = true;
            };
            while (key < end) {
            for (int left = kDec4Fold; left > 0 && key < end; --left) {
                bool landed = mbar_try_wait(&sm->full[warp][s_wait], parity);
                if (!__all_sync(0xffffffffu, landed)) {
                    landed = mbar_wait_drain(&sm->full[warp][s_wait], parity, p.timeout_ns);
                    if (!__all_sync(0xffffffffu, landed)) {
                        // Give up: after the copies that are still under way, or their limit.
                        if (lane == 0) raise_status(kStatusTimeoutDecode);
                        sm->abort = 1;
                        for (int k = 0; k < kDec4Stages && key < end; ++k) {
                            mbar_wait_drain(&sm->full[warp][s_wait], parity, p.timeout_ns);
                            if (++s_wait == kDec4Stages) {
                                s_wait = 0;
                                parity ^= 1;
                            }
                            advance(key, end);
                        }
                        key = end;
                        break;
                    }
                }
                const uint8_t *ring = sm->ring[warp][s_wait];
                if (++s_wait == kDec4Stages) {
                    s_wait = 0;
                    parity ^= 1;
                }
                const int n_keys = min(kDec4Tile, end - key);
                if (has_L && key + n_keys > L) {  // the tile of the new row
                    if (lane < kRow / 16)
                        reinterpret_cast<uint4 *>(const_cast<uint8_t *>(ring) + (n_keys - 1) * kRow)[lane] =
                            reinterpret_cast<const uint4 *>(sm->new_row)[lane];
                    __syncwarp();
                }
#pragma unroll 1
                for (int k0 = 0; k0 < n_keys; k0 += 16 * H) {
                // The lane's keys are fragment rows c and c + 8 of each of the step's 16 keys.
                const uint8_t *row0 = ring + key_at + k0 * kRow;
                // ---- scores over x_scale
                float x[H][NT][4];
                {
                    uint32_t code[H][2][G];
#pragma unroll
                    for (int t = 0; t < H; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint8_t *from = row0 + (16 * t + 8 * k) * kRow + 4 * G * r;
                            if constexpr (G == 4)
                                *reinterpret_cast<uint4 *>(code[t][k]) = *reinterpret_cast<const uint4 *>(from);
                            else
                                *reinterpret_cast<uint2 *>(code[t][k]) = *reinterpret_cast<const uint2 *>(from);
                        }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        uint4 hi[NT], lo[NT];
                        if constexpr (REP > 1) {
                            hi[0] = q_reg[gr];
                        } else {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                hi[nt] = sm->q_hi[nt * 8 + c][4 * gr + r];
                                lo[nt] = sm->q_lo[nt * 8 + c][4 * gr + r];
                            }
                        }
#pragma unroll
                        for (int t = 0; t < H; ++t) {
                            const uint32_t wa = code[t][0][gr], wb = code[t][1][gr];
                            const uint32_t va = wa >> 8, vb = wb >> 8;
                            const uint8_t *from = row0 + 16 * t * kRow + HD + 4 * gr;
                            const float sa = __half2float(*reinterpret_cast<const __half *>(from));
                            const float sb = __half2float(*reinterpret_cast<const __half *>(from + 8 * kRow));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float acc[4];
                                mma0_f16_16816(acc, wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u, wb & 0x00f000f0u, hi[nt].x, hi[nt].y);
                                mma_f16_16816(acc, va & 0x000f000fu, vb & 0x000f000fu, va & 0x00f000f0u, vb & 0x00f000f0u, hi[nt].z, hi[nt].w);
                                if constexpr (REP == 1) {
                                    mma_f16_16816(acc, wa & 0x000f000fu, wb & 0x000f000fu, wa & 0x00f000f0u, wb & 0x00f000f0u, lo[nt].x, lo[nt].y);
                                    mma_f16_16816(acc, va & 0x000f000fu, vb & 0x000f000fu, va & 0x00f000f0u, vb & 0x00f000f0u, lo[nt].z, lo[nt].w);
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    x[t][nt][e] = gr == 0 ? (e < 2 ? sa : sb) * acc[e] : fmaf(e < 2 ? sa : sb, acc[e], x[t][nt][e]);
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < H; ++t) {
                        const uint8_t *from = row0 + 16 * t * kRow + HD + (G == 4 ? 8 * (r & 1) : 0);
                        const uint2 za = *reinterpret_cast<const uint2 *>(from);
                        const uint2 zb = *reinterpret_cast<const uint2 *>(from + 8 * kRow);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[t][nt][e] *= 16777216.f;
                            mma_f16_1688(x[t][nt], __byte_perm(za.x, za.y, 0x7632), __byte_perm(zb.x, zb.y, 0x7632), qz[nt]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if constexpr (REP > 1) x[t][nt][e] += __shfl_xor_sync(0xffffffffu, x[t][nt][e], kCopy);
                        }
                    }
                }
                uint32_t par[H][2][GL];  // the values' (s, z) of this lane's groups
#pragma unroll
                for (int t = 0; t < H; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint8_t *from = row0 + (16 * t + 8 * k) * kRow + HD + 4 * G;
                        if constexpr (GL == 4) {
                            *reinterpret_cast<uint4 *>(par[t][k]) = *reinterpret_cast<const uint4 *>(from);
                        } else {
#pragma unroll
                            for (int i = 0; i < GL; ++i)
                                par[t][k][i] = reinterpret_cast<const uint32_t *>(from)[i * REP + copy];
                        }
                    }
                if (p.alibi) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int col = nt * 8 + 2 * (r % kCopy) + j, pos = seg.first + dec4_token<kMulti>(p, col);
                            const float slope = sm->slope[col];
#pragma unroll
                            for (int t = 0; t < H; ++t)
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    x[t][nt][2 * k + j] = fmaf(-slope, static_cast<float>(pos - key - (k0 + 16 * t + 8 * k + dec4_key<HD>(c))), x[t][nt][2 * k + j]);
                        }
                }
                // Rows behind the tile's end do not count, nor keys that a column does not see.
                if (n_keys < kDec4Tile || (kMulti && (key + kDec4Tile - 1 > seg.first ||
                                              (p.window > 0 && key <= seg.last - p.window && key + kDec4Tile > p.n_sink)))) {
#pragma unroll
                    for (int t = 0; t < H; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int i = k0 + 16 * t + 8 * k + dec4_key<HD>(c), n = key + i;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int pos = seg.first + dec4_token<kMulti>(p, nt * 8 + 2 * (r % kCopy) + j);
                                    if (i >= n_keys ||
                                        (kMulti && (n > pos || (p.window > 0 && n <= pos - p.window && n >= p.n_sink))))
                                        x[t][nt][2 * k + j] = -INFINITY;
                                }
                            if (i >= n_keys) {
#pragma unroll
                                for (int m = 0; m < GL; ++m) par[t][k][m] = 0;
                            }
                        }
                }
                // Probabilities and B operands; true if one of the latter nears fp16's end (or
                // would, but for a scale of 0).
                float pr[H][NT][4];
                uint32_t bf[H][GL][NT][2];
                auto products = [&] {
                    float p_max[H * NT];
                    __half2 top[H * NT * GL];
#pragma unroll
                    for (int t = 0; t < H; ++t)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                pr[t][nt][e] = ex2f(fmaf(x[t][nt][e], x_scale[nt][e & 1], -R[nt][e & 1]));
                            }
                            p_max[t * NT + nt] = fmaxf(fmaxf(pr[t][nt][0], pr[t][nt][1]), fmaxf(pr[t][nt][2], pr[t][nt][3]));
#pragma unroll
                            for (int i = 0; i < GL; ++i) {
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float s = lo_f(par[t][k][i]);
                                    bf[t][i][nt][k] = pack_half2(pr[t][nt][2 * k] * s, pr[t][nt][2 * k + 1] * s);
                                }
                                top[(t * NT + nt) * GL + i] = __hmax2(*reinterpret_cast<const __half2 *>(&bf[t][i][nt][0]),
                                                                      *reinterpret_cast<const __half2 *>(&bf[t][i][nt][1]));
                            }
                        }
#pragma unroll
                    for (int n = H * NT * GL / 2; n > 0; n >>= 1)
#pragma unroll
                        for (int i = 0; i < n; ++i) top[i] = __hmax2(top[i], top[i + n]);
#pragma unroll
                    for (int n = H * NT / 2; n > 0; n >>= 1)
#pragma unroll
                        for (int i = 0; i < n; ++i) p_max[i] = fmaxf(p_max[i], p_max[i + n]);
                    const uint32_t largest = *reinterpret_cast<const uint32_t *>(&top[0]);
                    return ((largest + 0x08000800u) & 0x80008000u) != 0 || p_max[0] > 1.1e12f;  // 2^15; 2^40
                };
                if (__any_sync(0xffffffffu, products())) {
                    // Raise the references to these keys' largest p s, put at 2^8 (a scale below
                    // fp16's smallest counts as that), or where scores are coarse their largest p
                    // at 1, which leaves p s at most at fp16's largest scale, 65504 2 / 15.
                    float ls[H][2];
#pragma unroll
                    for (int t = 0; t < H; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float s = 5.9604645e-8f;
#pragma unroll
                            for (int i = 0; i < GL; ++i) s = fmaxf(s, lo_f(par[t][k][i]));
                            ls[t][k] = log2f(s) - 8.f;
                        }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float t = R[nt][j];
#pragma unroll
                            for (int k = 0; k < 2 * H; ++k) {
                                const float score = x[k >> 1][nt][2 * (k & 1) + j] * x_scale[nt][j];
                                t = fmaxf(t, fabsf(score) < kCoarseScore ? score + ls[k >> 1][k & 1] : score);
                            }
#pragma unroll
                            for (int off = kCopy; off < 32; off <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
                            if (!(fabsf(t) < INFINITY)) t = R[nt][j];
                            const float f = R[nt][j] == kNoScore ? 0.f : ex2f(R[nt][j] - t);
                            R[nt][j] = t;
                            l[nt][j] *= f;
#pragma unroll
                            for (int i = 0; i < GL; ++i) w[nt][j][i] *= f;
#pragma unroll
                            for (int i = 0; i < GO; ++i) {
                                o[i][0][nt][j] *= f;
                                o[i][0][nt][j + 2] *= f;
                                o[i][1][nt][j] *= f;
                                o[i][1][nt][j + 2] *= f;
                            }
                        }
                    products();
                }
                // ---- sums, and O^T += V^T P
#pragma unroll
                for (int t = 0; t < H; ++t) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            l[nt][j] += pr[t][nt][j] + pr[t][nt][j + 2];
#pragma unroll
                            for (int i = 0; i < GL; ++i)
                                w[nt][j][i] = fmaf(pr[t][nt][j], hi_f(par[t][0][i]), fmaf(pr[t][nt][j + 2], hi_f(par[t][1][i]), w[nt][j][i]));
                        }
                    uint32_t vw[4][G / 2];  // value words of the four keys of this lane's k indices
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint8_t *from = ring + (k & 1 ? val_at1 : val_at0) + (k0 + 16 * t + 8 * (k >> 1)) * kRow;
                        if constexpr (G == 4)
                            *reinterpret_cast<uint2 *>(vw[k]) = *reinterpret_cast<const uint2 *>(from);
                        else
                            vw[k][0] = *reinterpret_cast<const uint32_t *>(from);
                    }
                    uint32_t b0[GL][NT], b1[GL][NT];
#pragma unroll
                    for (int i = 0; i < GL; ++i)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            b0[i][nt] = transpose8(bf[t][i][nt][0]);
                            b1[i][nt] = transpose8(bf[t][i][nt][1]);
                        }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        const uint32_t sel = gr & 1 ? 0x7632u : 0x5410u;
                        const uint32_t u = __byte_perm(vw[0][gr / 2], vw[1][gr / 2], sel);
                        const uint32_t v = __byte_perm(vw[2][gr / 2], vw[3][gr / 2], sel);
                        const uint32_t us = u >> 8, vs = v >> 8;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const bool mine = !kShare || c / (8 / REP) == gr % REP;
                            const uint32_t b0g = mine ? b0[gr / REP][nt] : 0u, b1g = mine ? b1[gr / REP][nt] : 0u;
                            mma_f16_16816(o[kShare ? gr / REP : gr][0][nt], u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u, b0g, b1g);
                            mma_f16_16816(o[kShare ? gr / REP : gr][1][nt], us & 0x000f000fu, us & 0x00f000f0u, vs & 0x000f000fu, vs & 0x00f000f0u, b0g, b1g);
                        }
                    }
                }
                }
                __syncwarp();  // the whole warp is done with the stage
                advance(key, end);
                if (ld_key < ld_end) load();
            }
            if (key < end) fold(false);
            }

            if (folded) fold(true);
            // ---- the warps' results: outputs of head h, dims, in place of the ring
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
#pragma unroll
                        for (int i = 0; i < GL; ++i)
                            w[nt][j][i] += __shfl_xor_sync(0xffffffffu, w[nt][j][i], off);
                    }
                    if (lane < kCopy) {
                        sm->m[warp][nt * 8 + 2 * r + j] = l[nt][j] == 0.f ? -INFINITY : R[nt][j];
                        sm->l[warp][nt * 8 + 2 * r + j] = l[nt][j];
                    }
                }
            __syncthreads();
            float *red = reinterpret_cast<float *>(&sm->ring[0][0][0]);  // [warps][8 NT][HD]
#pragma unroll
            for (int i = 0; i < GO; ++i) {
                if (!kShare && i % REP != copy) continue;  // another copy's group
                const int gr = kShare ? i * REP + copy : i;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float add = w[nt][j][kShare ? i : i / REP];
                        const float4 out = make_float4(fmaf(o[i][0][nt][j], 16777216.f, add),
                                                       fmaf(o[i][0][nt][j + 2], 1048576.f, add),
                                                       fmaf(o[i][1][nt][j], 16777216.f, add),
                                                       fmaf(o[i][1][nt][j + 2], 1048576.f, add));
                        *reinterpret_cast<float4 *>(red + (warp * 8 * NT + nt * 8 + 2 * (r % kCopy) + j) * HD + 32 * gr + 4 * c) = out;
                    }
            }
            __syncthreads();
            const long long slot = (blockIdx.x + static_cast<long long>(st) * p.Hkv + kvh) * (kMulti ? p.seg_tokens * g : g);
            for (int i = tid; i < cols * HD; i += kDec4Threads) {
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
                    // After a copy that did not land: no earlier call's partial result passes for this one.
                    p.ws_ml[(slot + h) * 2] = top_m;
                    p.ws_ml[(slot + h) * 2 + 1] = sm->abort ? __int_as_float(0x7fc00000) : sum;
                }
            }
            fence_proxy_async_smem();  // the ring's next copies follow these writes and reads
            __syncthreads();
        }
    }
}

// One block per (sequence, query head, token): the pieces of its segment, by log-sum-exp weights.
// Four warps share the pieces, a lane holding HD/32 dims, so that few loads follow one another
// (one warp's turn through 40 pieces took 8 us, this 3).
constexpr int kDec4MergeThreads = 128;
template <int HD, bool kMulti>
__global__ void __launch_bounds__(kDec4MergeThreads) decode4_merge_kernel(const __grid_constant__ Decode4Params p) {
    constexpr int kVec = HD / 32, kWarps = kDec4MergeThreads / 32;
    __shared__ float weight[kDec4MaxBlocks];
    __shared__ float red[kWarps], out[kWarps][HD];
    const int oi = blockIdx.x, Tq = kMulti ? p.Tq : 1, t = oi % Tq, hq = oi / Tq % p.Hq, b = oi / Tq / p.Hq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = p.group, kvh = hq / g;
    const int st = kMulti ? b * p.n_segs + t / p.seg_tokens : b;
    const int col = (kMulti ? t % p.seg_tokens * g : 0) + hq % g;
    const int keys = dec4_keys<kMulti>(p, st);
    if (keys == 0) {  // a length outside the cache
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (tid < HD) p.o[static_cast<long long>(oi) * HD + tid] = __float2bfloat16(__int_as_float(0x7fc00000));
        if (p.lse != nullptr && tid == 0) p.lse[oi] = __int_as_float(0x7fc00000);
        return;
    }
    const long long U = dec4_share<kMulti>(p, lane);
    long long seg0 = 0;
    for (int i = lane; i < st; i += 32) seg0 += p.Hkv * dec4_units(dec4_keys<kMulti>(p, i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) seg0 += __shfl_xor_sync(0xffffffffu, seg0, off);
    const long long V = dec4_units(keys);
    seg0 += kvh * V;
    const int first = static_cast<int>((seg0 + kDec4Lead) / U);
    const int n = static_cast<int>((seg0 + V - 1) / U) - first + 1;  // pieces, at most one a block
    const int rows = kMulti ? p.seg_tokens * g : g;
    const long long slot0 = (first + static_cast<long long>(st) * p.Hkv + kvh) * rows + col;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the split kernel's results
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
    float M = -INFINITY, sum = 0.f;
    for (int i = tid; i < n; i += kDec4MergeThreads) {
        weight[i] = ml[slot0 + static_cast<long long>(i) * rows].x;
        M = fmaxf(M, weight[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (lane == 0) red[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[w]);
    float acc[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += kWarps) {
        const long long s = slot0 + static_cast<long long>(i) * rows;
        const float w = M == -INFINITY ? 0.f : ex2f(weight[i] - M);
        const float *o = p.ws_o + s * HD + kVec * lane;
        sum = fmaf(w, ml[s].y, sum);
        if constexpr (kVec == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(o);
            acc[0] = fmaf(w, v.x, acc[0]);
            acc[1] = fmaf(w, v.y, acc[1]);
            acc[2] = fmaf(w, v.z, acc[2]);
            acc[3] = fmaf(w, v.w, acc[3]);
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(o);
            acc[0] = fmaf(w, v.x, acc[0]);
            acc[1] = fmaf(w, v.y, acc[1]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kVec; ++e) out[warp][kVec * lane + e] = acc[e];
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += red[w];
    if (tid < HD) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += out[w][tid];
        p.o[static_cast<long long>(oi) * HD + tid] = __float2bfloat16_rn(v / sum);
    }
    if (p.lse != nullptr && tid == 0) p.lse[oi] = (M + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace yr
