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

constexpr int kDec4Chunk = 128;      // least keys per block
constexpr int kDec4MaxBlocks = 640;  // most blocks of the split launch
constexpr int kDec4Threads = 128;
constexpr int kDec4Tile = 32;

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

// The partition, as every block derives it from cache_len: total keys, and the first
// sequence that reaches beyond unit `u` with the units before it.  Called by a full warp.
struct Dec4Plan {
    long long total, before;
    int b;
};
__device__ __forceinline__ long long dec4_units_per_block(const Decode4Params &p, long long total) {
    const long long even = (total + p.grid_blocks - 1) / p.grid_blocks;
    return even > kDec4Chunk ? even : kDec4Chunk;
}
__device__ __forceinline__ long long dec4_seq_units(const Decode4Params &p, int b) {
    if (b >= p.B) return 0;
    const DecRanges r = dec4_ranges(p, p.cache_len[b]);
    return static_cast<long long>(p.Hkv) * (r.len1 + r.len2);
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

template <int HD, bool kHalf>
__global__ void __launch_bounds__(kDec4Threads)
    decode4_split_kernel(const __grid_constant__ Decode4Params p) {
    constexpr int kRow = kv4_row_bytes(HD), G = HD / kKv4Group;
    __shared__ float q[16][HD], k[kDec4Tile][HD + 1], v[kDec4Tile][HD], sc[16][kDec4Tile];
    __shared__ float m_run[16], l_run[16], al[16];
    __shared__ double2 cs[HD / 2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = p.group;
    const long long total = dec4_total(p, lane);
    const long long U = dec4_units_per_block(p, total);
    const long long u_lo = static_cast<long long>(blockIdx.x) * U;
    const long long u_hi = min(u_lo + U, total);
    if (blockIdx.x == 0 && tid == 0)
        for (int b = 0; b < p.B; ++b)
            if (p.cache_len[b] < 0 || p.cache_len[b] > p.T_max - 1) raise_status(kStatusBadCacheLen);
    long long seg0 = 0;
    for (int b = 0; b < p.B && seg0 < u_hi; ++b) {
        const int L = p.cache_len[b];
        const DecRanges rg = dec4_ranges(p, L);
        const int V = rg.len1 + rg.len2;
        if (V == 0) continue;
        for (int kvh = 0; kvh < p.Hkv && seg0 < u_hi; ++kvh, seg0 += V) {
            if (seg0 + V <= u_lo) continue;
            const int a = static_cast<int>(max(u_lo, seg0) - seg0);
            const int e = static_cast<int>(min(u_hi, seg0 + V) - seg0);
            uint8_t *plane = p.kv4 + (static_cast<long long>(b) * p.Hkv + kvh) * p.T_max * kRow;
            __syncthreads();
            for (int i = tid; i < HD / 2; i += kDec4Threads) cs[i] = kv4_cos_sin(L, p.turns[i]);
            if (tid < 16) {
                m_run[tid] = -INFINITY;
                l_run[tid] = 0.f;
            }
            __syncthreads();
            if (e == V && warp == 0) dec4_append<HD, kHalf>(p, b, kvh, plane + static_cast<long long>(L) * kRow, cs, lane);
            for (int i = tid; i < g * (HD / 8); i += kDec4Threads) {
                const int h = i / (HD / 8), c = i % (HD / 8);
                float y[8];
                kv4_rotate8<HD, kHalf>(p.q_new + (static_cast<long long>(b) * p.Hq + kvh * g + h) * HD, c, cs, y);
#pragma unroll
                for (int x = 0; x < 8; ++x) q[h][8 * c + x] = y[x];
            }
            float acc[16];
#pragma unroll
            for (int h = 0; h < 16; ++h) acc[h] = 0.f;
            const int dim = tid % HD;
            for (int u = a; u < e; u += kDec4Tile) {
                __syncthreads();
                const int cnt = min(kDec4Tile, e - u);
                for (int i = tid; i < kDec4Tile * (HD / 8); i += kDec4Threads) {
                    const int r = i / (HD / 8), c = i % (HD / 8);
                    float x[8], y[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.f;
                    if (r < cnt) {
                        const int n = u + r < rg.len1 ? u + r : rg.lo2 + u + r - rg.len1;
                        const uint8_t *row = plane + static_cast<long long>(n) * kRow;
                        const __half2 *par = reinterpret_cast<const __half2 *>(row + HD);
                        const uint16_t *vu = reinterpret_cast<const uint16_t *>(row + HD / 2);
                        const int cg = c >> 2, cr = c & 3;
                        kv4_values8(reinterpret_cast<const uint32_t *>(row)[cr * G + cg], par[cg], x);
                        kv4_values8(vu[2 * cr * G + cg] | (static_cast<uint32_t>(vu[(2 * cr + 1) * G + cg]) << 16),
                                    par[G + cg], y);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        k[r][8 * c + j] = x[j];
                        v[r][8 * c + j] = y[j];
                    }
                }
                __syncthreads();
                for (int i = tid; i < g * kDec4Tile; i += kDec4Threads) {
                    const int h = i / kDec4Tile, r = i % kDec4Tile;
                    float x = -INFINITY;
                    if (r < cnt) {
                        const int n = u + r < rg.len1 ? u + r : rg.lo2 + u + r - rg.len1;
                        float dot = 0.f;
                        for (int j = 0; j < HD; ++j) dot = fmaf(q[h][j], k[r][j], dot);
                        x = dot * p.sl2;
                        if (p.alibi)
                            x -= exp2f(-8.f * static_cast<float>(kvh * g + h + 1) / static_cast<float>(p.Hq)) *
                                 1.4426950408889634f * static_cast<float>(L - n);
                    }
                    sc[h][r] = x;
                }
                __syncthreads();
                for (int h = warp; h < g; h += kDec4Threads / 32) {
                    const float x = sc[h][lane];
                    float mx = x;
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    const float mo = m_run[h], mn = fmaxf(mo, mx);
                    const float w = lane < cnt ? ex2f(x - mn) : 0.f;
                    float sum = w;
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    const float f = mo == -INFINITY ? 0.f : ex2f(mo - mn);
                    sc[h][lane] = w;
                    __syncwarp();
                    if (lane == 0) {
                        m_run[h] = mn;
                        l_run[h] = l_run[h] * f + sum;
                        al[h] = f;
                    }
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int h = j * (kDec4Threads / HD) + tid / HD;
                    if (h >= g) continue;
                    float s = acc[j] * al[h];
                    for (int r = 0; r < cnt; ++r) s = fmaf(sc[h][r], v[r][dim], s);
                    acc[j] = s;
                }
            }
            const long long slot = (blockIdx.x + static_cast<long long>(b) * p.Hkv + kvh) * g;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int h = j * (kDec4Threads / HD) + tid / HD;
                if (h >= g) continue;
                p.ws_o[(slot + h) * HD + dim] = acc[j];
                if (dim == 0) {
                    p.ws_ml[(slot + h) * 2] = m_run[h];
                    p.ws_ml[(slot + h) * 2 + 1] = l_run[h];
                }
            }
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
    const long long V = rg.len1 + rg.len2;
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
    const int first = static_cast<int>(seg0 / U), last = static_cast<int>((seg0 + V - 1) / U);
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
