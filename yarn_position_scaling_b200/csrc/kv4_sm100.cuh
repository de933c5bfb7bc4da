// kv4_sm100.cuh -- the 4-bit KV cache: its row format, the pass that rotates, quantises
// and writes new keys and values, and the pass that reads rows back in 16 bits.
//
// A row holds the rotated key and the value of one token and KV head in 5d/4 bytes:
//   [key codes d/2][value codes d/2][key (s, z) x d/32][value (s, z) x d/32]
// Elements come in groups of 32; element x of a group is kept as a code n in 0..15 and
// stands for s n + z with the group's fp16 scale s and minimum z:
//   z = fp16(min x),  s = fp16(max(0, (max x - z) / 15)),
//   n = clamp(rint((x - z) / s), 0, 15), or 0 where s = 0,
// in fp32 with ties to even; the key is rotated in fp64 and rounded once to fp32, so that
// a code does not depend on how a sine was approximated.  s n is exact in fp32 (an 11-bit
// times a 4-bit integer), so s n + z has one rounding.
// Code order: a key word (8 codes) at index r G + g holds elements 32g + 8r .. + 7, a value
// unit (4 codes) at index c G + g holds elements 32g + 4c .. + 3 (G = d/32, r in 0..3,
// c in 0..7, codes from the low bits up).  The lanes of one matrix fragment of the decode
// kernel then read neighbouring bytes, and one instruction's operand stays in one group.
#pragma once
#include "kvprep_sm100.cuh"

namespace yr {

constexpr int kKv4Group = 32;
__host__ __device__ constexpr int kv4_row_bytes(int d) { return d / 2 + d / 2 + d / 4; }

struct Kv4WriteParams {
    const __nv_bfloat16 *k, *v;  // [B][Hkv][T][d], strides in elements
    long long ksb, ksh, kst, vsb, vsh, vst;
    uint8_t *kv4;       // [B][Hkv][T_max][5d/4]
    const int *starts;  // [B] or null: row t of sequence b goes to slot pos0 + starts[b] + t
    const int *counts;  // [B] or null: rows t < counts[b] are written
    int B, Hkv, T, T_max, pos0;
    int heads;          // KV heads that a block takes in turn
    double turns[64];
};

struct Kv4ReadParams {
    const uint8_t *kv4;
    void *k, *v;  // 16-bit [B][Hkv][T][d], strides in elements; either may be null
    long long ksb, ksh, kst, vsb, vsh, vst;
    const int *starts, *counts;
    int B, Hkv, T, T_max, pos0;
    // Rows [0, n_head) and [skip_to, T) are read, what lies between is not; of those, rows
    // [zero_lo, zero_hi) are written as zeros instead (an attention reads them in a tile
    // but sees none of them).
    int n_head, skip_to, zero_lo, zero_hi;
    int zero_rest;  // 1: rows that are not read become zeros; 0: they keep their contents
};

// The slots of sequence b's rows: first slot and row count, or no rows (and the status
// bit) where they do not lie in the cache.
template <class P>
__device__ __forceinline__ int kv4_rows_of(const P &p, int b, int &first) {
    const long long s = static_cast<long long>(p.pos0) + (p.starts != nullptr ? p.starts[b] : 0);
    const int n = p.counts != nullptr ? p.counts[b] : p.T;
    if (s < 0 || n < 0 || n > p.T || s + n > p.T_max) {
        raise_status(kStatusBadCacheLen);
        first = 0;
        return 0;
    }
    first = static_cast<int>(s);
    return n;
}

// Round (x - z) / s to the nearest code.  The product with an approximate reciprocal is
// off by less than 1e-5, so only a quotient that near a border needs the division.
__device__ __forceinline__ uint32_t kv4_code(float x, float z, float s, float r) {
    const float t = __fsub_rn(x, z);
    const float q = t * r;
    float n = rintf(q);
    if (fabsf(q - n) > 0.4999f) n = rintf(__fdiv_rn(t, s));
    return static_cast<uint32_t>(fminf(fmaxf(n, 0.f), 15.f));
}

// The group's (s, z), from the eight elements of each of four neighbouring lanes, and this
// lane's eight codes, the first in the low bits.
__device__ __forceinline__ uint32_t kv4_quantise8(const float (&x)[8], __half2 &sz) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    const __half z16 = __float2half_rn(lo);
    const float z = __half2float(z16);
    const __half s16 = __float2half_rn(fmaxf(__fdiv_rn(__fsub_rn(hi, z), 15.f), 0.f));
    const float s = __half2float(s16);
    sz = __halves2half2(s16, z16);
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= (s > 0.f ? kv4_code(x[i], z, s, r) : 0u) << (4 * i);
    return w;
}

// Into the fp16 range; true if x was outside it (|x| >= 65520, or not a number).
__device__ __forceinline__ bool kv4_clamp(float &x) {
    const bool bad = f16_out_of_range(x);
    x = fmaxf(fminf(x, 65504.f), -65504.f);
    return bad;
}

// cos and sin of position * 2 pi turns, the angle reduced to one turn first.
__device__ __forceinline__ double2 kv4_cos_sin(int pos, double turns) {
    const double tr = __dmul_rn(static_cast<double>(pos), turns);
    double sn, cs;
    sincospi(2.0 * __dsub_rn(tr, rint(tr)), &sn, &cs);
    return make_double2(cs, sn);
}

// Elements 8c .. 8c+7 of the rotated key.  `cs` holds (cos, sin) of every pair at the key's
// position.
template <int HD, bool kHalf>
__device__ __forceinline__ void kv4_rotate8(const __nv_bfloat16 *row, int c, const double2 *cs,
                                            float (&y)[8]) {
    float x[8];
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4 *>(row + 8 * c)), x);
    if constexpr (kHalf) {
        constexpr int kHalfChunks = HD / 16;
        float w[8];
        const bool first = c < kHalfChunks;
        const int other = first ? c + kHalfChunks : c - kHalfChunks;
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4 *>(row + 8 * other)), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double2 t = cs[8 * (first ? c : other) + e];
            const double a = x[e], b = w[e];
            y[e] = static_cast<float>(first ? __dsub_rn(__dmul_rn(a, t.x), __dmul_rn(b, t.y))
                                            : __dadd_rn(__dmul_rn(b, t.y), __dmul_rn(a, t.x)));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const double2 t = cs[4 * c + e];
            const double a = x[2 * e], b = x[2 * e + 1];
            y[2 * e] = static_cast<float>(__dsub_rn(__dmul_rn(a, t.x), __dmul_rn(b, t.y)));
            y[2 * e + 1] = static_cast<float>(__dadd_rn(__dmul_rn(a, t.y), __dmul_rn(b, t.x)));
        }
    }
}

// One lane's share of a row: its eight key and eight value codes and, from the first lane
// of a group, the group's (s, z) pairs.  c is the lane's chunk of eight elements.
template <int HD>
__device__ __forceinline__ void kv4_store8(uint8_t *row, int c, uint32_t kw, __half2 ksz,
                                           uint32_t vw, __half2 vsz) {
    constexpr int G = HD / kKv4Group;
    const int g = c >> 2, r = c & 3;
    reinterpret_cast<uint32_t *>(row)[r * G + g] = kw;
    uint16_t *vu = reinterpret_cast<uint16_t *>(row + HD / 2);
    vu[(2 * r) * G + g] = static_cast<uint16_t>(vw);
    vu[(2 * r + 1) * G + g] = static_cast<uint16_t>(vw >> 16);
    if (r == 0) {
        __half2 *par = reinterpret_cast<__half2 *>(row + HD);
        par[g] = ksz;
        par[G + g] = vsz;
    }
}

constexpr int kKv4Threads = 256;

// A block takes kRows rows of one sequence and `heads` KV heads in turn, so that the fp64
// sines of a position are computed once for its heads; a lane takes eight elements.
template <int HD, bool kHalf>
__global__ void __launch_bounds__(kKv4Threads) kv4_write_kernel(const __grid_constant__ Kv4WriteParams p) {
    constexpr int kLanes = HD / 8;  // lanes of a row
    constexpr int kRows = kKv4Threads / kLanes;
    __shared__ double2 cs[kRows][HD / 2];
    const int b = blockIdx.y;
    int first;
    const int n = kv4_rows_of(p, b, first);
    const int t0 = static_cast<int>(blockIdx.x) * kRows;
    if (t0 >= n) return;
    for (int i = threadIdx.x; i < kRows * (HD / 2); i += kKv4Threads)
        cs[i / (HD / 2)][i % (HD / 2)] =
            kv4_cos_sin(first + t0 + i / (HD / 2), p.turns[i % (HD / 2)]);
    __syncthreads();
    const int r = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
    const int t = t0 + r;
    const bool live = t < n;
    const long long tl = live ? t : n - 1;  // idle lanes repeat the last row, without a store
    const int h0 = blockIdx.z * p.heads, h1 = min(h0 + p.heads, p.Hkv);
    bool bad = false;
    for (int h = h0; h < h1; ++h) {
        float y[8], x[8];
        kv4_rotate8<HD, kHalf>(p.k + b * p.ksb + h * p.ksh + tl * p.kst, c,
                               cs[live ? r : n - 1 - t0], y);
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4 *>(p.v + b * p.vsb + h * p.vsh +
                                                            tl * p.vst + 8 * c)), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) bad |= kv4_clamp(y[i]) | kv4_clamp(x[i]);
        __half2 ksz, vsz;
        const uint32_t kw = kv4_quantise8(y, ksz), vw = kv4_quantise8(x, vsz);
        if (live)
            kv4_store8<HD>(p.kv4 + ((static_cast<long long>(b) * p.Hkv + h) * p.T_max + first + t) *
                                       kv4_row_bytes(HD), c, kw, ksz, vw, vsz);
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) raise_status(kStatusKv4Range);
}

// Eight codes of a lane as values.
__device__ __forceinline__ void kv4_values8(uint32_t w, __half2 sz, float (&x)[8]) {
    const float s = __low2float(sz), z = __high2float(sz);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(static_cast<float>((w >> (4 * i)) & 15u), s, z);
}

// Into the 16-bit type; fp16 keeps the largest finite value where s n + z passes it.
template <bool kF16>
__device__ __forceinline__ uint4 kv4_pack16(float (&x)[8]) {
    if constexpr (kF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaxf(fminf(x[i], 65504.f), -65504.f);
        return pack_half8(x);
    } else {
        return pack_bf16x8(x);
    }
}

// A lane takes eight elements of a row; a grid-stride loop over the rows to read.
template <int HD, bool kF16>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
    constexpr int kLanes = HD / 8, G = HD / kKv4Group;
    const int b = blockIdx.z, h = blockIdx.y;
    int first;
    const int n = min(kv4_rows_of(p, b, first), p.T);
    const int c = threadIdx.x % kLanes, g = c >> 2, r = c & 3;
    const int rows = p.n_head + (p.T - p.skip_to);
    uint16_t *ko = static_cast<uint16_t *>(p.k), *vo = static_cast<uint16_t *>(p.v);
    const long long step = static_cast<long long>(gridDim.x) * (kKv4Threads / kLanes);
    for (long long i = blockIdx.x * static_cast<long long>(kKv4Threads / kLanes) + threadIdx.x / kLanes;
         i < rows; i += step) {
        const int t = static_cast<int>(i < p.n_head ? i : p.skip_to + (i - p.n_head));
        if (t >= n && !p.zero_rest) continue;
        // A row that becomes zeros reads the plane's first slot, whatever that holds.
        const bool zero = t >= n || (t >= p.zero_lo && t < p.zero_hi);
        const uint8_t *row = p.kv4 + ((static_cast<long long>(b) * p.Hkv + h) * p.T_max +
                                      (zero ? 0 : first + t)) * kv4_row_bytes(HD);
        const __half2 *par = reinterpret_cast<const __half2 *>(row + HD);
        float x[8];
        if (ko != nullptr) {
            kv4_values8(reinterpret_cast<const uint32_t *>(row)[r * G + g], par[g], x);
            uint4 out = kv4_pack16<kF16>(x);
            if (zero) out = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(ko + b * p.ksb + h * p.ksh + t * p.kst + 8 * c) = out;
        }
        if (vo != nullptr) {
            const uint16_t *vu = reinterpret_cast<const uint16_t *>(row + HD / 2);
            const uint32_t w = vu[(2 * r) * G + g] | (static_cast<uint32_t>(vu[(2 * r + 1) * G + g]) << 16);
            kv4_values8(w, par[G + g], x);
            uint4 out = kv4_pack16<kF16>(x);
            if (zero) out = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(vo + b * p.vsb + h * p.vsh + t * p.vst + 8 * c) = out;
        }
    }
}

}  // namespace yr
