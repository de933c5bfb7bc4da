// kv4_entry.cuh -- the C ABI of the 4-bit KV cache (yr_kv4_*, yr_attn_decode_kv4,
// yr_attn_prefill_chunk_kv4): argument checks and launches.  Part of yarnattn.cu, whose
// helpers it uses.
#pragma once

namespace yr_host {

constexpr long long kKv4MaxPos = 1ll << 30;

// What write and read have in common: sizes, the row range and the cache pointer.
int check_kv4_rows(const std::string &f, const void *kv4, int B, int Hkv, int T, int d, int T_max,
                   int pos0, const int32_t *starts, const int32_t *counts) {
    if (!kv4) return fail(YR_EINVAL, f + ": kv4 must be non-NULL");
    if (B < 1 || Hkv < 1 || T < 1 || T_max < 1)
        return fail(YR_EINVAL, f + ": B, Hkv, T and T_max must be >= 1");
    if (B > 65535 || Hkv > 65535) return fail(YR_EINVAL, f + ": B and Hkv must be <= 65535");
    if (d != 64 && d != 128) return fail(YR_EUNSUPPORTED, f + ": d must be 64 or 128");
    if (pos0 < 0 || T > kKv4MaxPos || T_max > kKv4MaxPos || pos0 > kKv4MaxPos)
        return fail(YR_EINVAL, f + ": need 0 <= pos0, and pos0, T and T_max <= 2^30");
    if (!starts && !counts && static_cast<long long>(pos0) + T > T_max)
        return fail(YR_EINVAL, f + ": need pos0 + T <= T_max");
    if (!aligned(kv4, 16)) return fail(YR_EINVAL, f + ": kv4 must be 16-byte aligned");
    if ((starts && !aligned(starts, 4)) || (counts && !aligned(counts, 4)))
        return fail(YR_EINVAL, f + ": starts and counts must be 4-byte aligned");
    return YR_OK;
}

int check_table(const std::string &f, const yr_rope_table *tab, int d) {
    if (!tab) return fail(YR_EINVAL, f + ": tab must be non-NULL");
    if (tab->head_dim != d) return fail(YR_EINVAL, f + ": table head_dim != d");
    if (tab->pairs != YR_PAIR_INTERLEAVED && tab->pairs != YR_PAIR_HALF)
        return fail(YR_EINVAL, f + ": table pairs must be YR_PAIR_INTERLEAVED or YR_PAIR_HALF");
    return YR_OK;
}

int launch_kv4_write(const void *k, const void *v, void *kv4, int B, int Hkv, int T, int d,
                     int T_max, const long long ks[3], const long long vs[3], int pos0,
                     const int32_t *starts, const int32_t *counts, const yr_rope_table *tab,
                     int sm_count, cudaStream_t st) {
    yr::Kv4WriteParams wp;
    std::memset(&wp, 0, sizeof wp);
    wp.k = static_cast<const __nv_bfloat16 *>(k);
    wp.v = static_cast<const __nv_bfloat16 *>(v);
    wp.ksb = ks[0]; wp.ksh = ks[1]; wp.kst = ks[2];
    wp.vsb = vs[0]; wp.vsh = vs[1]; wp.vst = vs[2];
    wp.kv4 = static_cast<uint8_t *>(kv4);
    wp.starts = starts;
    wp.counts = counts;
    wp.B = B; wp.Hkv = Hkv; wp.T = T; wp.T_max = T_max; wp.pos0 = pos0;
    for (int i = 0; i < d / 2; ++i) wp.turns[i] = tab->turns[i];
    const int rows = yr::kKv4WriteRows;
    const long long tiles = (static_cast<long long>(T) + rows - 1) / rows;
    // All heads of a row in one block where the rows alone fill the GPU, else spread.
    int split = 1;
    while (split < Hkv && tiles * B * split < 4ll * sm_count) split *= 2;
    wp.heads = (Hkv + split - 1) / split;
    const dim3 grid(static_cast<unsigned>(tiles), B, (Hkv + wp.heads - 1) / wp.heads);
    const bool half = tab->pairs == YR_PAIR_HALF;
    if (d == 128 && half)
        yr::kv4_write_kernel<128, true><<<grid, yr::kKv4WriteThreads, 0, st>>>(wp);
    else if (d == 128)
        yr::kv4_write_kernel<128, false><<<grid, yr::kKv4WriteThreads, 0, st>>>(wp);
    else if (half)
        yr::kv4_write_kernel<64, true><<<grid, yr::kKv4WriteThreads, 0, st>>>(wp);
    else
        yr::kv4_write_kernel<64, false><<<grid, yr::kKv4WriteThreads, 0, st>>>(wp);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail("kv4_write_kernel launch", e);
    return YR_OK;
}

int launch_kv4_read(yr::Kv4ReadParams rp, int d, bool f16, int sm_count, cudaStream_t st) {
    const long long rows = rp.n_head + (static_cast<long long>(rp.T) - rp.skip_to);
    const int per_block = yr::kKv4ReadThreads / 4;
    long long blocks = (rows + per_block - 1) / per_block;
    const long long planes = static_cast<long long>(rp.B) * rp.Hkv;
    const long long cap = (16ll * sm_count + planes - 1) / planes;
    if (blocks > cap) blocks = cap;
    const dim3 grid(static_cast<unsigned>(blocks), rp.Hkv, rp.B);
    if (d == 128 && f16)
        yr::kv4_read_kernel<128, true><<<grid, yr::kKv4ReadThreads, 0, st>>>(rp);
    else if (d == 128)
        yr::kv4_read_kernel<128, false><<<grid, yr::kKv4ReadThreads, 0, st>>>(rp);
    else if (f16)
        yr::kv4_read_kernel<64, true><<<grid, yr::kKv4ReadThreads, 0, st>>>(rp);
    else
        yr::kv4_read_kernel<64, false><<<grid, yr::kKv4ReadThreads, 0, st>>>(rp);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail("kv4_read_kernel launch", e);
    return YR_OK;
}

// Workspace of the split kernel: a slot per block and per segment of `rows` rows each.
size_t decode4_slots_bytes(long long segments, long long rows, long long d) {
    return static_cast<size_t>((yr::kDec4MaxBlocks + segments) * rows * (d + 2) * 4);
}
size_t decode4_ws_bytes(long long B, long long Hq, long long Hkv, long long d) {
    return decode4_slots_bytes(B * Hkv, Hq / Hkv, d);
}

// A chunk's tokens in runs that the split kernel takes as its columns (16, or 8 where all fit).
struct Decode4Runs {
    int tokens, n;
};
Decode4Runs decode4_runs(int g, int Tq) {
    const int cols = static_cast<long long>(Tq) * g <= 8 ? 8 : 16;
    int tokens = cols / g < Tq ? cols / g : Tq;
    if (tokens < 1) tokens = 1;
    tokens = (Tq + (Tq + tokens - 1) / tokens - 1) / ((Tq + tokens - 1) / tokens);  // evenly
    return {tokens, (Tq + tokens - 1) / tokens};
}

// Blocks of a split kernel per SM, set up at its first launch in a context: callers without a
// 4-bit cache do not wait for its 28 forms to be loaded.  (Two threads may both set it up.)
template <int HD, int NT, int REP, bool kHalf, bool kMulti>
int prepare_decode4_form(const DeviceState &dev, int *per_sm) {
    constexpr int form = (HD == 128 ? 16 : 0) + (NT == 2 ? 12 : REP == 1 ? 8 : REP == 2 ? 4 : 0) +
                         (kHalf ? 2 : 0) + (kMulti ? 1 : 0);
    static_assert(form < kDecode4Forms, "forms");
    int n = dev.decode4_per_sm[form].load(std::memory_order_acquire);
    if (n == 0) {
        const auto kernel = &yr::decode4_split_kernel<HD, NT, REP, kHalf, kMulti>;
        const size_t smem = yr::decode4_smem_bytes<HD, NT, kMulti>();
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
        if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute", e);
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, yr::kDec4Threads, smem);
        if (e != cudaSuccess) return cuda_fail("cudaOccupancyMaxActiveBlocksPerMultiprocessor", e);
        n = n > 0 ? n : 1;
        dev.decode4_per_sm[form].store(n, std::memory_order_release);
    }
    *per_sm = n;
    return YR_OK;
}

// One wave of the split kernel, and the places of its partial results.
template <int HD, int NT, int REP, bool kHalf, bool kMulti>
int launch_decode4_form(yr::Decode4Params &dp, const DeviceState &dev, cudaStream_t st) {
    int per_sm = 0;
    const int rc = prepare_decode4_form<HD, NT, REP, kHalf, kMulti>(dev, &per_sm);
    if (rc != YR_OK) return rc;
    const int blocks = per_sm * dev.sm_count;
    dp.grid_blocks = blocks < yr::kDec4MaxBlocks ? blocks : yr::kDec4MaxBlocks;
    const long long slots = dp.grid_blocks + static_cast<long long>(dp.B) * dp.n_segs * dp.Hkv;
    dp.ws_ml = dp.ws_o + slots * dp.seg_tokens * dp.group * HD;
    yr::decode4_split_kernel<HD, NT, REP, kHalf, kMulti>
        <<<dp.grid_blocks, yr::kDec4Threads, yr::decode4_smem_bytes<HD, NT, kMulti>(), st>>>(dp);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail("decode4_split_kernel launch", e);
    return YR_OK;
}

// The form of the kernel for a segment's columns (tokens times query heads per KV head).
template <int HD, bool kHalf, bool kMulti>
int launch_decode4(yr::Decode4Params &dp, const DeviceState &dev, cudaStream_t st) {
    const int cols = dp.seg_tokens * dp.group;
    if (cols > 8) return launch_decode4_form<HD, 2, 1, kHalf, kMulti>(dp, dev, st);
    if (cols > 4) return launch_decode4_form<HD, 1, 1, kHalf, kMulti>(dp, dev, st);
    if (cols > 2 || HD == 64) return launch_decode4_form<HD, 1, 2, kHalf, kMulti>(dp, dev, st);
    return launch_decode4_form<HD, 1, HD / 32, kHalf, kMulti>(dp, dev, st);
}

// The split kernel over dp's segments and the merge of its partial results.
template <bool kMulti>
int launch_decode4_call(yr::Decode4Params &dp, int d, const yr_rope_table *tab, const DeviceState &dev,
                        cudaStream_t st) {
    // The power of two of the scale, as far as its products with the queries' stay within fp32.
    const double sl2 = tab->softmax_scale * 1.4426950408889634;
    int sl2_exp = 0;
    std::frexp(sl2, &sl2_exp);
    sl2_exp = sl2_exp > 0 ? 0 : sl2_exp < -50 ? -50 : sl2_exp;
    dp.sl2_part = static_cast<float>(std::ldexp(sl2, -sl2_exp));
    dp.sl2_pow2 = static_cast<float>(std::ldexp(1.0, sl2_exp));
    dp.alibi = tab->method == YR_ALIBI ? 1 : 0;
    for (int i = 0; i < d / 2; ++i) dp.turns[i] = tab->turns[i];
    dp.timeout_ns = wait_timeout_ns();
#ifdef YR_FAULT_HOOKS
    // Test build only: the failure-path hook, read on every launch.
    const char *drop = std::getenv("YR_FAULT_DROP_KV4_COPY");  // block:copy
    if (!drop || std::sscanf(drop, "%d:%d", &dp.fault_block, &dp.fault_copy) != 2) dp.fault_block = -1;
#endif
    const bool half = tab->pairs == YR_PAIR_HALF;
    int rc = d == 128 ? half ? launch_decode4<128, true, kMulti>(dp, dev, st)
                         : launch_decode4<128, false, kMulti>(dp, dev, st)
         : half   ? launch_decode4<64, true, kMulti>(dp, dev, st)
                  : launch_decode4<64, false, kMulti>(dp, dev, st);
    if (rc != YR_OK) return rc;
    // The merge may start, and find its pieces, while the split kernel still runs; it waits
    // for that kernel's results itself.
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(dp.B) * dp.Hq * dp.Tq);
    cfg.blockDim = dim3(yr::kDec4MergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = d == 128 ? cudaLaunchKernelEx(&cfg, yr::decode4_merge_kernel<128, kMulti>, dp)
                                   : cudaLaunchKernelEx(&cfg, yr::decode4_merge_kernel<64, kMulti>, dp);
    if (e != cudaSuccess) return cuda_fail("decode4_merge_kernel launch", e);
    return YR_OK;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace yr_host

extern "C" size_t yr_kv4_row_bytes(int d) {
    return d == 64 || d == 128 ? static_cast<size_t>(yr::kv4_row_bytes(d)) : 0;
}

extern "C" int yr_kv4_write(const void *k, const void *v, void *kv4, int B, int Hkv, int T, int d,
                            int T_max, const int64_t *k_strides, const int64_t *v_strides,
                            int pos0, const int32_t *starts, const int32_t *counts,
                            const yr_rope_table *tab, void *stream) {
    set_error("");
    const std::string f("yr_kv4_write");
    if (!k || !v) return fail(YR_EINVAL, f + ": k and v must be non-NULL");
    int rc = check_kv4_rows(f, kv4, B, Hkv, T, d, T_max, pos0, starts, counts);
    if (rc != YR_OK) return rc;
    rc = check_table(f, tab, d);
    if (rc != YR_OK) return rc;
    if (!aligned(k, 16) || !aligned(v, 16))
        return fail(YR_EINVAL, f + ": pointers must be 16-byte aligned");
    long long ks[3], vs[3];
    strides_or_contiguous(k_strides, Hkv, T, d, ks);
    strides_or_contiguous(v_strides, Hkv, T, d, vs);
    if (!strides_ok(ks) || !strides_ok(vs))
        return fail(YR_EINVAL, f + ": strides must be positive multiples of 8 elements");
    int sm_count = 0;
    rc = prepare_device(&sm_count);
    if (rc != YR_OK) return rc;
    return launch_kv4_write(k, v, kv4, B, Hkv, T, d, T_max, ks, vs, pos0, starts, counts, tab,
                            sm_count, static_cast<cudaStream_t>(stream));
}

extern "C" int yr_kv4_read(const void *kv4, void *k, void *v, int out_type, int B, int Hkv, int T,
                           int d, int T_max, const int64_t *k_strides, const int64_t *v_strides,
                           int pos0, const int32_t *starts, const int32_t *counts, int zero_rest,
                           void *stream) {
    set_error("");
    const std::string f("yr_kv4_read");
    if (!k && !v) return fail(YR_EINVAL, f + ": one of k and v must be non-NULL");
    int rc = check_kv4_rows(f, kv4, B, Hkv, T, d, T_max, pos0, starts, counts);
    if (rc != YR_OK) return rc;
    if (out_type != YR_KV4_BF16 && out_type != YR_KV4_FP16)
        return fail(YR_EINVAL, f + ": out_type must be YR_KV4_BF16 or YR_KV4_FP16");
    if ((k && !aligned(k, 16)) || (v && !aligned(v, 16)))
        return fail(YR_EINVAL, f + ": pointers must be 16-byte aligned");
    long long ks[3], vs[3];
    strides_or_contiguous(k_strides, Hkv, T, d, ks);
    strides_or_contiguous(v_strides, Hkv, T, d, vs);
    if ((k && !strides_ok(ks)) || (v && !strides_ok(vs)))
        return fail(YR_EINVAL, f + ": strides must be positive multiples of 8 elements");
    int sm_count = 0;
    rc = prepare_device(&sm_count);
    if (rc != YR_OK) return rc;
    yr::Kv4ReadParams rp;
    std::memset(&rp, 0, sizeof rp);
    rp.kv4 = static_cast<const uint8_t *>(kv4);
    rp.k = k;
    rp.v = v;
    rp.ksb = ks[0]; rp.ksh = ks[1]; rp.kst = ks[2];
    rp.vsb = vs[0]; rp.vsh = vs[1]; rp.vst = vs[2];
    rp.starts = starts;
    rp.counts = counts;
    rp.B = B; rp.Hkv = Hkv; rp.T = T; rp.T_max = T_max; rp.pos0 = pos0;
    rp.zero_rest = zero_rest ? 1 : 0;
    return launch_kv4_read(rp, d, out_type == YR_KV4_FP16, sm_count,
                           static_cast<cudaStream_t>(stream));
}

extern "C" size_t yr_attn_decode_kv4_workspace_bytes(int B, int Hq, int Hkv, int d) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || (d != 64 && d != 128)) return 0;
    return decode4_ws_bytes(B, Hq, Hkv, d);
}

extern "C" int yr_attn_decode_kv4(const void *q_new, const void *k_new, const void *v_new,
                                  void *kv4, const int32_t *cache_len, void *o, float *lse,
                                  void *k_stored, void *v_stored, int B, int Hq, int Hkv, int d,
                                  int T_max, const yr_rope_table *tab, int window, int n_sink,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    set_error("");
    const std::string f("yr_attn_decode_kv4");
    if (!q_new || !k_new || !v_new || !kv4 || !cache_len || !o || !tab || !workspace)
        return fail(YR_EINVAL, f + ": NULL pointer argument");
    if (B < 1 || Hq < 1 || Hkv < 1 || T_max < 1)
        return fail(YR_EINVAL, f + ": B, Hq, Hkv and T_max must be >= 1");
    if (T_max > kKv4MaxPos) return fail(YR_EINVAL, f + ": T_max must be <= 2^30");
    if (static_cast<long long>(B) * Hq >= (1ll << 31))
        return fail(YR_EINVAL, f + ": problem too large for one launch");
    if (Hq % Hkv != 0) return fail(YR_EINVAL, f + ": Hq must be a multiple of Hkv");
    if (d != 64 && d != 128) return fail(YR_EUNSUPPORTED, f + ": d must be 64 or 128");
    if (Hq / Hkv > 16) return fail(YR_EUNSUPPORTED, f + ": at most 16 query heads per KV head");
    int rc = check_table(f, tab, d);
    if (rc != YR_OK) return rc;
    if (window < 0 || n_sink < 0) return fail(YR_EINVAL, f + ": window and n_sink must be >= 0");
    if (n_sink > 0 && window == 0) return fail(YR_EINVAL, f + ": sinks need a window");
    const size_t need = decode4_ws_bytes(B, Hq, Hkv, d);
    if (workspace_bytes < need)
        return fail(YR_EINVAL, f + ": workspace too small (need " + std::to_string(need) + " bytes)");
    if (!aligned(workspace, 256)) return fail(YR_EINVAL, f + ": workspace must be 256-byte aligned");
    for (const void *ptr : {q_new, k_new, v_new, static_cast<const void *>(kv4),
                            static_cast<const void *>(o), static_cast<const void *>(k_stored),
                            static_cast<const void *>(v_stored)})
        if (ptr && !aligned(ptr, 16))
            return fail(YR_EINVAL, f + ": tensor pointers must be 16-byte aligned");
    if (!aligned(cache_len, 4) || (lse && !aligned(lse, 4)))
        return fail(YR_EINVAL, f + ": cache_len and lse must be 4-byte aligned");
    DeviceState dev;
    rc = prepare_device(nullptr, &dev);
    if (rc != YR_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int g = Hq / Hkv;
    yr::Decode4Params dp;
    std::memset(&dp, 0, sizeof dp);
    dp.q_new = static_cast<const __nv_bfloat16 *>(q_new);
    dp.k_new = static_cast<const __nv_bfloat16 *>(k_new);
    dp.v_new = static_cast<const __nv_bfloat16 *>(v_new);
    dp.kv4 = static_cast<uint8_t *>(kv4);
    dp.cache_len = cache_len;
    dp.o = static_cast<__nv_bfloat16 *>(o);
    dp.lse = lse;
    dp.k_stored = static_cast<__nv_bfloat16 *>(k_stored);
    dp.v_stored = static_cast<__nv_bfloat16 *>(v_stored);
    dp.B = B; dp.Hq = Hq; dp.Hkv = Hkv; dp.T_max = T_max; dp.group = g;
    dp.window = window; dp.n_sink = n_sink;
    dp.Tq = 1; dp.seg_tokens = 1; dp.n_segs = 1;
    dp.ws_o = static_cast<float *>(workspace);
    return launch_decode4_call<false>(dp, d, tab, dev, st);
}

namespace yr_host {

// Is a chunk of Tq tokens taken by the decode kernel, over the 4-bit rows, instead of by the
// prefill kernel, over 16-bit copies of them?  The former reads the rows once for every 16
// columns (tokens times query heads of a KV head), 60 ps a row (d = 128); the latter makes the
// copies (110 ps a row) and then holds 256 query rows a tile, with a window 128, however few
// there are (95 ps a row and query head, with a window half).  At d = 64 the products of the
// prefill kernel are half as long but its softmax is not.  Both sides measured, decode and
// prefill kernel in us: after 120K keys of 8 KV heads with 32 query heads 4 tokens 78 and 462,
// 16 tokens 257 and 466, 28 tokens 441 and 467, 32 tokens 491 and 466; with 64 query heads 24
// tokens 732 and 811, 28 tokens 856 and 812; with 8 after 60K 48 tokens 109 and 125, 64 tokens
// 137 and 125; d = 64, 20K keys of 4 KV heads with 16 query heads 40 tokens 47 and 49, 48 tokens
// 51 and 48; 60K of 16 with 16 48 tokens 119 and 146, 64 tokens 153 and 145; window 4096, 32
// and 8 heads of d = 128 16 tokens 33 and 34, 20 tokens 36 and 34, 16 and 4 heads of d = 64 40
// tokens 25 and 28; window 2048, 8 and 8 heads 64 tokens 20 and 24.  The window's length does not
// move the border: 32 and 8 heads, 32K 16 tokens 86 and 105, 24 tokens 120 and 106, 64K 16 tokens
// 147 and 178, 20 tokens 183 and 178, 128K (all of 120K) 20 tokens 318 and 310, 24 tokens 378 and
// 313, by the prefill kernel's 128-row form, which calls without a window do not take.
bool chunk4_by_decode(int g, int Tq, int d, int window) {
    if (g > 16) return false;
    const long long tenths = 10ll * decode4_runs(g, Tq).n;
    if (d == 64) return tenths <= (window > 0 ? 30 + 20 * g : 16 + 22 * g);
    return tenths <= (window > 0 ? 12 + 8 * g : 15 + 15 * g);
}

// Bytes that the decode kernel's partial results take for a chunk.
size_t chunk4_decode_bytes(int B, int Hq, int Hkv, int Tq, int d) {
    const Decode4Runs runs = decode4_runs(Hq / Hkv, Tq);
    return decode4_slots_bytes(static_cast<long long>(B) * Hkv * runs.n,
                               static_cast<long long>(runs.tokens) * (Hq / Hkv), d);
}

}  // namespace yr_host

extern "C" size_t yr_attn_prefill_chunk_kv4_workspace_bytes(int B, int Hq, int Hkv, int Tq, int d,
                                                            int P0) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Tq < 1 || P0 < 0 || Hq % Hkv || (d != 64 && d != 128) ||
        static_cast<long long>(P0) + Tq > kKv4MaxPos)
        return 0;
    const size_t prefill = round256(prefill_ws_bytes(B, Hkv, static_cast<long long>(P0) + Tq, d)) +
                           kMaxSplit * split_share_bytes(B, Hq, Tq, d);
    const int g = Hq / Hkv;
    const bool by_decode = chunk4_by_decode(g, Tq, d, 0) || chunk4_by_decode(g, Tq, d, 1);
    const size_t decode = by_decode ? chunk4_decode_bytes(B, Hq, Hkv, Tq, d) : 0;
    return prefill > decode ? prefill : decode;
}

extern "C" int yr_attn_prefill_chunk_kv4(const void *q, const void *k_new, const void *v_new,
                                         void *kv4, void *o, float *lse, int B, int Hq, int Hkv,
                                         int Tq, int d, int P0, int T_max,
                                         const yr_rope_table *tab, int window, int n_sink,
                                         void *workspace, size_t workspace_bytes, void *stream) {
    set_error("");
    const std::string f("yr_attn_prefill_chunk_kv4");
    if (!q || !k_new || !v_new || !kv4 || !o || !tab || !workspace)
        return fail(YR_EINVAL, f + ": NULL pointer argument");
    if (Hq < 1) return fail(YR_EINVAL, f + ": B, Hq, Hkv and Tq must be >= 1");
    int rc = check_kv4_rows(f, kv4, B, Hkv, Tq, d, T_max, P0, nullptr, nullptr);
    if (rc != YR_OK) return rc;
    const int Tk = P0 + Tq;
    const size_t planes = round256(prefill_ws_bytes(B, Hkv, Tk, d));
    if (workspace_bytes < planes)
        return fail(YR_EINVAL, f + ": workspace too small (need " + std::to_string(planes) + " bytes)");
    long long qs[3], os[3];
    rc = check_attend(q, o, lse, nullptr, B, Hq, Hkv, Tq, d, nullptr, nullptr, tab, 1, window,
                      n_sink, workspace, planes, f.c_str(), qs, os);
    if (rc != YR_OK) return rc;
    for (const void *ptr : {k_new, v_new})
        if (!aligned(ptr, 16)) return fail(YR_EINVAL, f + ": pointers must be 16-byte aligned");
    DeviceState dev;
    rc = prepare_device(nullptr, &dev);
    if (rc != YR_OK) return rc;
    const int sm_count = dev.sm_count;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    long long ks[3];
    strides_or_contiguous(nullptr, Hkv, Tq, d, ks);
    rc = launch_kv4_write(k_new, v_new, kv4, B, Hkv, Tq, d, T_max, ks, ks, P0, nullptr, nullptr,
                          tab, sm_count, st);
    if (rc != YR_OK) return rc;
    if (chunk4_by_decode(Hq / Hkv, Tq, d, window) &&
        static_cast<long long>(B) * Hq * Tq < (1ll << 31) &&
        workspace_bytes >= chunk4_decode_bytes(B, Hq, Hkv, Tq, d)) {
        const Decode4Runs runs = decode4_runs(Hq / Hkv, Tq);
        yr::Decode4Params dp;
        std::memset(&dp, 0, sizeof dp);
        dp.q_new = static_cast<const __nv_bfloat16 *>(q);
        dp.kv4 = static_cast<uint8_t *>(kv4);
        dp.o = static_cast<__nv_bfloat16 *>(o);
        dp.lse = lse;
        dp.B = B; dp.Hq = Hq; dp.Hkv = Hkv; dp.T_max = T_max; dp.group = Hq / Hkv;
        dp.P0 = P0; dp.Tq = Tq; dp.seg_tokens = runs.tokens; dp.n_segs = runs.n;
        dp.window = window; dp.n_sink = n_sink;
        dp.ws_o = static_cast<float *>(workspace);
        return launch_decode4_call<true>(dp, d, tab, dev, st);
    }
    // The rows in 16 bits for the attention: with a window, the 128-key tiles that it reads
    // and no others (those of the sinks, and from the first query's window on).
    const KvPlanes kv = workspace_planes(workspace, B, Hkv, Tk, d);
    yr::Kv4ReadParams rp;
    std::memset(&rp, 0, sizeof rp);
    rp.kv4 = static_cast<const uint8_t *>(kv4);
    rp.k = const_cast<__half *>(kv.k16);
    rp.v = const_cast<__half *>(kv.v16);
    strides_or_contiguous(nullptr, Hkv, Tk, d, ks);
    rp.ksb = rp.vsb = ks[0]; rp.ksh = rp.vsh = ks[1]; rp.kst = rp.vst = ks[2];
    rp.B = B; rp.Hkv = Hkv; rp.T = Tk; rp.T_max = T_max;
    if (window > 0) {
        const int w0 = P0 - window + 1 > 0 ? P0 - window + 1 : 0;  // first key of the window
        rp.skip_to = w0 / 128 * 128;
        const long long sinks = (static_cast<long long>(n_sink) + 127) / 128 * 128;
        rp.n_head = static_cast<int>(sinks < rp.skip_to ? sinks : rp.skip_to);
        rp.zero_lo = n_sink < w0 ? n_sink : w0;
        rp.zero_hi = w0;
    }
    rc = launch_kv4_read(rp, d, true, sm_count, st);
    if (rc != YR_OK) return rc;
    uint8_t *split_ws = static_cast<uint8_t *>(workspace) + planes;
    return attend_planes(q, o, lse, B, Hq, Hkv, Tq, d, P0, qs, os, tab, window, n_sink, kv,
                         split_ws, workspace_bytes - planes, sm_count, st);
}
