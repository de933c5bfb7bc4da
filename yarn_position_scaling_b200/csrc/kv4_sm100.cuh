// kv4_sm100.cuh -- the 4-bit KV cache: its row format, the pass that rotates, quantises
// and writes new keys and values, and the pass that reads rows back in 16 bits.
//
// A row holds the rotated key and the value of one token and KV head in 5d/4 bytes:
//   [key codes d/2][value codes d/2][key (s, z) x d/32][value (s, z) x d/32]
// Elements come in groups of 32; element x of a group is kept as a code n in 0..15 and
// stands for s n + z with the group's fp16 scale s and minimum z:
//   z = fp16(min x),  s = fp16(max(0, (max x - z) / 15)),
//   n = clamp(rint((x - z) / s), 0, 15), or 0 where s = 0,
// in fp32 with ties to even; the key is rotated in fp64, by the position times the table's turns
// without a rounding of that product, and rounded once to fp32: the sines' own errors, 2^-49 in
// the passes here, reach a code only where an fp32 tie and a code's border meet.  s n is exact in
// fp32 (an 11-bit times a 4-bit integer), so s n + z has one rounding.
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

// cos and sin of position * 2 pi turns, the angle reduced to one turn first: exactly, with the
// product's rounding (up to 2^-26 turns at 2^30, which the reduction would leave in the angle) put back.
__device__ __forceinline__ double2 kv4_cos_sin(int pos, double turns) {
    const double n = static_cast<double>(pos), tr = __dmul_rn(n, turns);
    double sn, cs;
    sincospi(2.0 * __dadd_rn(__dsub_rn(tr, rint(tr)), fma(n, turns, -tr)), &sn, &cs);
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

// ------------------------------------------------------------------------------- write
// Four lanes hold a row: lane r the elements 32g + 8r .. + 7 of every group g.  Both elements
// of a pair are then the same lane's in either pair layout, a group's extremes are two
// shuffles away, and a lane's codes of a row are 16 neighbouring bytes of it.
constexpr int kKv4WriteRows = 32;  // rows of a block
constexpr int kKv4WriteThreads = 4 * kKv4WriteRows;

// The high word of a bf16 number (in the upper half of `bits`, zeros below) as fp64, in integer
// arithmetic (the conversion instruction runs at an eighth of the rate).  Zeros become 2^-127,
// which no later rounding sees; infinities and NaN become numbers beyond the fp32 range, which
// the range check then finds.
__device__ __forceinline__ double bf16_as_double(uint32_t bits) {
    const uint32_t hi = (static_cast<uint32_t>(static_cast<int32_t>(bits) >> 3) & 0x8fffffffu) + (896u << 20);
    return __hiloint2double(static_cast<int>(hi), 0);
}
__device__ __forceinline__ void unpack_double8(const uint4 &raw, double (&x)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_as_double(w[i] << 16);
        x[2 * i + 1] = bf16_as_double(w[i] & 0xffff0000u);
    }
}
// Pair (a, b) turned by the angle of t = (cos, sin), rounded to fp32 once.
__device__ __forceinline__ void kv4_turn(double a, double b, const double2 &t, float &ya, float &yb) {
    ya = static_cast<float>(fma(a, t.x, -__dmul_rn(b, t.y)));
    yb = static_cast<float>(fma(a, t.y, __dmul_rn(b, t.x)));
}

// Codes of one row from the elements of its four lanes: w[g] this lane's eight of group g, and
// `sz` the (s, z) of group r (lanes r < G).  The extremes are reduced so that lane r ends with
// those of group r, which then does that group's divisions for all four.  A code is
// rint(15 sat((x - z) / (15 s))) by a product with the reciprocal, off by less than 4e-6, and
// by the division where the quotient is that near a border; the codes of a word are added up
// with the bits of the rounding constant and the constants taken off at the end.
template <int G>
__device__ __forceinline__ void kv4_quantise_row(const float (&x)[G][8], int r, uint32_t (&w)[G], __half2 &sz) {
    float lo[G], hi[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        lo[g] = fminf(x[g][0], x[g][1]);
        hi[g] = fmaxf(x[g][0], x[g][1]);
#pragma unroll
        for (int i = 2; i < 8; i += 2) {
            lo[g] = fminf(lo[g], fminf(x[g][i], x[g][i + 1]));
            hi[g] = fmaxf(hi[g], fmaxf(x[g][i], x[g][i + 1]));
        }
    }
    if constexpr (G == 4) {  // lanes r and r ^ 2 take over groups r & 2 and (r & 2) + 1
        const bool up = (r & 2) != 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const float l = __shfl_xor_sync(0xffffffffu, up ? lo[g] : lo[g + 2], 2);
            const float h = __shfl_xor_sync(0xffffffffu, up ? hi[g] : hi[g + 2], 2);
            lo[g] = fminf(up ? lo[g + 2] : lo[g], l);
            hi[g] = fmaxf(up ? hi[g + 2] : hi[g], h);
        }
    } else {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            lo[g] = fminf(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], 2));
            hi[g] = fmaxf(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], 2));
        }
    }
    const bool odd = (r & 1) != 0;
    const float l = __shfl_xor_sync(0xffffffffu, odd ? lo[0] : lo[1], 1);
    const float h = __shfl_xor_sync(0xffffffffu, odd ? hi[0] : hi[1], 1);
    const __half z16 = __float2half_rn(fminf(odd ? lo[1] : lo[0], l));
    const __half s16 = __float2half_rn(
        fmaxf(__fdiv_rn(__fsub_rn(fmaxf(odd ? hi[1] : hi[0], h), __half2float(z16)), 15.f), 0.f));
    sz = __halves2half2(s16, z16);
    const float s_own = __half2float(s16);
    const float inv_own = s_own > 0.f ? __fdividef(1.f, 15.f * s_own) : 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const __half2 szg = __shfl_sync(0xffffffffu, sz, g, 4);
        const float inv = __shfl_sync(0xffffffffu, inv_own, g, 4);
        const float z = __high2float(szg);
        uint32_t word = 0u - 0x4B400000u * 0x11111111u;
        float far = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = __saturatef(__fsub_rn(x[g][i], z) * inv);
            const float t = fmaf(q, 15.f, 12582912.f);
            far = fmaxf(far, fabsf(fmaf(q, 15.f, 12582912.f - t)));
            word += __float_as_uint(t) << (4 * i);
        }
        if (far > 0.49999f) {
            const float s = __low2float(szg);
            word = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = rintf(__fdiv_rn(__fsub_rn(x[g][i], z), s));
                word |= static_cast<uint32_t>(fminf(fmaxf(n, 0.f), 15.f)) << (4 * i);
            }
        }
        w[g] = word;
    }
}

// A block takes 32 rows of one sequence and `heads` KV heads in turn, and computes the sines
// of its positions once for them: by angle addition from row to row, 16 (8) rows from a start
// that is computed (16 products cost 2^-49; the start's angle has no error that grows with its
// position, or all its rows would have it).
template <int HD, bool kHalf>
__global__ void __launch_bounds__(kKv4WriteThreads) kv4_write_kernel(const __grid_constant__ Kv4WriteParams p) {
    constexpr int G = HD / kKv4Group, kPairs = HD / 2, kRows = kKv4WriteRows;
    // Pair 4r + i (8r + i) of a group stands at 4i + r, and a row's end is 64 bytes longer than
    // a multiple of 128: the 16-byte reads of two rows' lanes then cover every bank once.
    constexpr int kLane = kHalf ? 8 : 4;
    __shared__ double2 cs[kRows][kPairs + 4];
    const int b = blockIdx.y;
    int first;
    const int n = kv4_rows_of(p, b, first);
    const int t0 = static_cast<int>(blockIdx.x) * kRows;
    if (t0 >= n) return;
    {
        constexpr int kRun = kRows * kPairs / kKv4WriteThreads;  // rows of a thread
        const int pair = threadIdx.x % kPairs, row0 = threadIdx.x / kPairs * kRun;
        const int at = pair / (4 * kLane) * (4 * kLane) + 4 * (pair % kLane) + pair / kLane % 4;
        const double2 step = kv4_cos_sin(1, p.turns[pair]);
        double2 u = kv4_cos_sin(first + t0 + row0, p.turns[pair]);
        cs[row0][at] = u;
#pragma unroll
        for (int i = 1; i < kRun; ++i) {
            u = make_double2(fma(u.x, step.x, -__dmul_rn(u.y, step.y)), fma(u.x, step.y, __dmul_rn(u.y, step.x)));
            cs[row0 + i][at] = u;
        }
    }
    __syncthreads();
    const int row = threadIdx.x / 4, r = threadIdx.x % 4;
    const bool live = t0 + row < n;
    const int at = live ? row : n - 1 - t0;  // idle lanes repeat the last row, without a store
    const long long t = t0 + at;
    const int h0 = blockIdx.z * p.heads, h1 = min(h0 + p.heads, p.Hkv);
    bool bad = false;
    for (int h = h0; h < h1; ++h) {
        uint4 kr[G], vr[G];
        const uint4 *krow = reinterpret_cast<const uint4 *>(p.k + b * p.ksb + h * p.ksh + t * p.kst) + r;
        const uint4 *vrow = reinterpret_cast<const uint4 *>(p.v + b * p.vsb + h * p.vsh + t * p.vst) + r;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            kr[g] = __ldg(krow + 4 * g);
            vr[g] = __ldg(vrow + 4 * g);
        }
        uint8_t *to = p.kv4 + ((static_cast<long long>(b) * p.Hkv + h) * p.T_max + first + t) * kv4_row_bytes(HD);
        float x[G][8];
        uint32_t w[G];
        __half2 sz;
        // Values outside the fp16 range, rare, are brought into it and reported.
        auto clamp = [&] {
            float top = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[g][i]));
            if (top >= kF16RoundsFinite) {
                bad = true;
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 8; ++i) kv4_clamp(x[g][i]);
            }
        };
        if constexpr (kHalf) {
#pragma unroll
            for (int g = 0; g < G / 2; ++g) {
                double a[8], c[8];
                unpack_double8(kr[g], a);
                unpack_double8(kr[g + G / 2], c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    kv4_turn(a[i], c[i], cs[at][32 * g + 4 * i + r], x[g][i], x[g + G / 2][i]);
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                double a[8];
                unpack_double8(kr[g], a);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    kv4_turn(a[2 * i], a[2 * i + 1], cs[at][16 * g + 4 * i + r], x[g][2 * i], x[g][2 * i + 1]);
            }
        }
        clamp();
        kv4_quantise_row<G>(x, r, w, sz);
        if (live) {
            if constexpr (G == 4)
                *reinterpret_cast<uint4 *>(to + 16 * r) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                *reinterpret_cast<uint2 *>(to + 8 * r) = make_uint2(w[0], w[1]);
            if (r < G) reinterpret_cast<__half2 *>(to + HD)[r] = sz;
        }
        uint32_t over = 0;  // top bits of halves whose magnitude is 65536 or more, or NaN
#pragma unroll
        for (int g = 0; g < G; ++g) {
            unpack_bf16x8(vr[g], x[g]);
            over |= ((vr[g].x & 0x7fff7fffu) + 0x38803880u) | ((vr[g].y & 0x7fff7fffu) + 0x38803880u) |
                    ((vr[g].z & 0x7fff7fffu) + 0x38803880u) | ((vr[g].w & 0x7fff7fffu) + 0x38803880u);
        }
        if (over & 0x80008000u) {
            bad = true;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) kv4_clamp(x[g][i]);
        }
        kv4_quantise_row<G>(x, r, w, sz);
        if (live) {
            // Value units 2r and 2r + 1 of every group: the words' halves, regrouped.
            if constexpr (G == 4)
                *reinterpret_cast<uint4 *>(to + HD / 2 + 16 * r) =
                    make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410),
                               __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
            else
                *reinterpret_cast<uint2 *>(to + HD / 2 + 8 * r) =
                    make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632));
            if (r < G) reinterpret_cast<__half2 *>(to + HD + 4 * G)[r] = sz;
        }
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) raise_status(kStatusKv4Range);
}

// -------------------------------------------------------------------------------- read
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

constexpr int kKv4ReadThreads = 256;

// Four lanes hold a row as in the write: 16 (8) neighbouring bytes of key and of value codes
// each, and 16-byte stores of which four lanes' are neighbours.  A grid-stride loop over the
// rows to read.
template <int HD, bool kF16>
__global__ void __launch_bounds__(kKv4ReadThreads) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
    constexpr int G = HD / kKv4Group;
    const int b = blockIdx.z, h = blockIdx.y;
    int first;
    const int n = kv4_rows_of(p, b, first);
    const int r = threadIdx.x % 4;
    const int rows = p.n_head + (p.T - p.skip_to);
    uint4 *ko = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.k) + b * p.ksb + h * p.ksh) + r;
    uint4 *vo = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.v) + b * p.vsb + h * p.vsh) + r;
    const uint8_t *plane = p.kv4 + (static_cast<long long>(b) * p.Hkv + h) * p.T_max * kv4_row_bytes(HD);
    const long long step = static_cast<long long>(gridDim.x) * (kKv4ReadThreads / 4);
    for (long long i = blockIdx.x * static_cast<long long>(kKv4ReadThreads / 4) + threadIdx.x / 4; i < rows; i += step) {
        const int t = static_cast<int>(i < p.n_head ? i : p.skip_to + (i - p.n_head));
        if (t >= n && !p.zero_rest) continue;
        // A row that becomes zeros reads the plane's first slot, whatever that holds.
        const bool zero = t >= n || (t >= p.zero_lo && t < p.zero_hi);
        const uint8_t *row = plane + (zero ? 0ll : static_cast<long long>(first) + t) * kv4_row_bytes(HD);
        uint32_t kw[G], vu[G], ksz[G], vsz[G];
        if constexpr (G == 4) {
            *reinterpret_cast<uint4 *>(kw) = __ldg(reinterpret_cast<const uint4 *>(row) + r);
            *reinterpret_cast<uint4 *>(vu) = __ldg(reinterpret_cast<const uint4 *>(row + HD / 2) + r);
            *reinterpret_cast<uint4 *>(ksz) = __ldg(reinterpret_cast<const uint4 *>(row + HD));
            *reinterpret_cast<uint4 *>(vsz) = __ldg(reinterpret_cast<const uint4 *>(row + HD) + 1);
        } else {
            *reinterpret_cast<uint2 *>(kw) = __ldg(reinterpret_cast<const uint2 *>(row) + r);
            *reinterpret_cast<uint2 *>(vu) = __ldg(reinterpret_cast<const uint2 *>(row + HD / 2) + r);
            *reinterpret_cast<uint2 *>(ksz) = __ldg(reinterpret_cast<const uint2 *>(row + HD));
            *reinterpret_cast<uint2 *>(vsz) = __ldg(reinterpret_cast<const uint2 *>(row + HD) + 1);
        }
        auto put = [&](uint4 *to, uint32_t w, uint32_t sz) {
            float x[8];
            kv4_values8(w, *reinterpret_cast<const __half2 *>(&sz), x);
            uint4 out = kv4_pack16<kF16>(x);
            if (zero) out = make_uint4(0, 0, 0, 0);
            *to = out;
        };
        if (p.k != nullptr) {
            uint4 *to = ko + t * (p.kst / 8);
#pragma unroll
            for (int g = 0; g < G; ++g) put(to + 4 * g, kw[g], ksz[g]);
        }
        if (p.v != nullptr) {
            uint4 *to = vo + t * (p.vst / 8);
#pragma unroll
            for (int g = 0; g < G; ++g)
                put(to + 4 * g, __byte_perm(vu[g / 2], vu[G / 2 + g / 2], g & 1 ? 0x7632 : 0x5410), vsz[g]);
        }
    }
}

}  // namespace yr
