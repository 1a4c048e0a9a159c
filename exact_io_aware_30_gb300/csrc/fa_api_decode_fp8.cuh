// fa_api_decode_fp8.cuh -- host side of decoding over an 8-bit paged cache
// (fa_decode_paged_fp8, fa_decode_fp8_workspace_query).  Included once, by
// fa_api.cu, after its shared helpers and fa_api_paged.cuh.
#pragma once

#include "fa_decode_fp8_kernel.cuh"

namespace fa {

namespace {

fa_status check_dec_fp8_sizes(int B, int H, int Hkv, int Sq, int d, int block_size, int max_blocks, int num_blocks,
                              int max_seq_len, int mask_kind, int dtype) {
    if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_UNSUPPORTED;
    const fa_status st = check_fp8_cache(num_blocks, Hkv, block_size, d);
    if (st != FA_OK) return st;
    if (mask_kind != FA_MASK_NONE && mask_kind != FA_MASK_CAUSAL) return FA_ERR_UNSUPPORTED;
    if (B < 1 || H < 1 || H % Hkv != 0 || Sq < 1) return FA_ERR_INVALID_ARG;
    if ((long long)(H / Hkv) * Sq > 128) return FA_ERR_UNSUPPORTED;  // rows of one K/V head
    if (max_blocks < 1 || max_seq_len < 1 || (long long)max_seq_len > (long long)max_blocks * block_size)
        return FA_ERR_INVALID_ARG;
    if (max_seq_len > 0x7fffffff - 512) return FA_ERR_INVALID_ARG;  // key numbers of a whole step stay below 2^31
    if ((long long)B * H * Sq > 0x7fffffffLL / 2 || (long long)B * max_blocks > 0x7fffffffLL)
        return FA_ERR_INVALID_ARG;
    if ((long long)Hkv * (H / Hkv * Sq) > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Rows per unit (the kernel's RC) for R rows per K/V head: one chunk of the
// smallest size that holds them, or equal chunks of at most 32 (24 at d = 256),
// the cache being read once more per chunk.  Beyond that tensor memory does not
// hold S's and O's part columns twice (fp16, d 256) or the registers O's rows
// (32 rows at d 256: 360 us in one chunk, 334 in two; at d 128 164 against 211).
constexpr int dec_fp8_max_rows(int d) { return d == 256 ? 24 : 32; }

// Tiles per unit up to which units are not cut: a CTA then takes whole ones, and
// the merge with its launch and its workspace is left out.  Whole against cut, us:
// 400 tokens, 1 request x 8 heads 8.0 / 8.0, 64 x 8 15.5 / 18.1, 16 x 4 of 40 rows
// at d 256 12.9 / 19.8; 1,000 tokens, 1 x 8 11.9 / 8.6, 64 x 8 25.9 / 27.6, but
// with lengths that differ the longest share would set the time.
constexpr int kDecFp8WholeTiles = 4;

struct DecFp8Plan {
    int rc = 0, chunks = 1, rows_per_chunk = 0, grid = 0;
    bool cuts = false;  // units may lie across CTAs
    size_t part_lse_off = 0, part_o_off = 0, bytes = 0;
};

// Tiles per step as they were measured: a change of the shared memory's small
// arrays must not change them unseen.
template <int D, int RC>
constexpr bool dec_fp8_tiles_per_step(int bf16, int fp16) {
    return DecFp8Cfg<D, false, RC>::KPT == bf16 && DecFp8Cfg<D, true, RC>::KPT == fp16;
}
static_assert(dec_fp8_tiles_per_step<64, 1>(1, 1) && dec_fp8_tiles_per_step<64, 4>(1, 1) && dec_fp8_tiles_per_step<64, 8>(2, 2) &&
              dec_fp8_tiles_per_step<64, 16>(2, 2) && dec_fp8_tiles_per_step<64, 24>(2, 2) && dec_fp8_tiles_per_step<64, 32>(2, 1));
static_assert(dec_fp8_tiles_per_step<128, 1>(1, 1) && dec_fp8_tiles_per_step<128, 4>(1, 1) && dec_fp8_tiles_per_step<128, 8>(1, 1) &&
              dec_fp8_tiles_per_step<128, 16>(2, 2) && dec_fp8_tiles_per_step<128, 24>(2, 2) && dec_fp8_tiles_per_step<128, 32>(2, 1));
static_assert(dec_fp8_tiles_per_step<256, 1>(1, 1) && dec_fp8_tiles_per_step<256, 4>(1, 1) && dec_fp8_tiles_per_step<256, 8>(1, 1) &&
              dec_fp8_tiles_per_step<256, 16>(1, 1) && dec_fp8_tiles_per_step<256, 24>(1, 1));

template <int D, bool kFP16>
int dec_fp8_ctas_per_sm(int rc) {
    return rc == 1    ? DecFp8Cfg<D, kFP16, 1>::CTAS_PER_SM
           : rc == 4  ? DecFp8Cfg<D, kFP16, 4>::CTAS_PER_SM
           : rc == 8  ? DecFp8Cfg<D, kFP16, 8>::CTAS_PER_SM
           : rc == 16 ? DecFp8Cfg<D, kFP16, 16>::CTAS_PER_SM
           : rc == 24 ? DecFp8Cfg<D, kFP16, 24>::CTAS_PER_SM
                      : DecFp8Cfg<D, kFP16, 32>::CTAS_PER_SM;
}

DecFp8Plan plan_decode_fp8(int B, int Hkv, int R, int d, bool fp16, int max_seq_len, int num_sms) {
    DecFp8Plan pl;
    const int max_rows = dec_fp8_max_rows(d);
    pl.chunks = (R + max_rows - 1) / max_rows;
    pl.rows_per_chunk = (R + pl.chunks - 1) / pl.chunks;
    pl.chunks = (R + pl.rows_per_chunk - 1) / pl.rows_per_chunk;
    for (int rc : {1, 4, 8, 16, 24, 32})
        if (pl.rc == 0 && rc >= pl.rows_per_chunk) pl.rc = rc;
    const int per_sm = d == 64    ? (fp16 ? dec_fp8_ctas_per_sm<64, true>(pl.rc) : dec_fp8_ctas_per_sm<64, false>(pl.rc))
                       : d == 128 ? (fp16 ? dec_fp8_ctas_per_sm<128, true>(pl.rc) : dec_fp8_ctas_per_sm<128, false>(pl.rc))
                                  : 1;
    const long long tiles = (max_seq_len + 127LL) / 128;
    const long long units = (long long)B * Hkv * pl.chunks;
    pl.cuts = tiles > kDecFp8WholeTiles;
    pl.grid = (int)std::min(pl.cuts ? units * tiles : units, (long long)num_sms * per_sm);
    size_t at = 0;
    if (pl.cuts) {
        at = (size_t)(4 + 5 * pl.grid) * 4;
        pl.part_lse_off = (at + 255) / 256 * 256;
        pl.part_o_off = (pl.part_lse_off + (size_t)2 * pl.grid * pl.rc * 4 + 255) / 256 * 256;
        at = pl.part_o_off + (size_t)2 * pl.grid * pl.rc * d * 4;
    }
    pl.bytes = at;
    return pl;
}

template <int D, bool kFP16, int RC>
fa_status launch_decode_fp8_rc(const DecFp8Params &p, const DecFp8Plan &pl, DeviceInfo &info, cudaStream_t stream) {
    using C = DecFp8Cfg<D, kFP16, RC>;
    constexpr int kind = RC == 1 ? 0 : RC == 4 ? 1 : RC == 8 ? 2 : RC == 16 ? 3 : RC == 24 ? 4 : 5;
    const int slot = ((D == 256 ? 2 : D == 128 ? 1 : 0) * 2 + (kFP16 ? 1 : 0)) * 6 + kind;
    if (set_smem(fa_decode_fp8_kernel<C>, C::SMEM_BYTES, info.attr_dec_fp8[slot]) != FA_OK) return FA_ERR_CUDA;
    const fa_status st = launch_overlapped(fa_decode_fp8_kernel<C>, dim3((unsigned)pl.grid), C::NUM_THREADS,
                                           C::SMEM_BYTES, 1, stream, p);
    if (st != FA_OK || !pl.cuts || pl.grid < 2) return st;
    return launch_overlapped(fa_decode_fp8_combine_kernel<D, kFP16, RC>, dim3((unsigned)(pl.grid - 1)),
                             kDecFp8MergeThreads<RC>, 0, 1, stream, p, pl.grid);
}

template <int D, bool kFP16>
fa_status launch_decode_fp8(const DecFp8Params &p, const DecFp8Plan &pl, DeviceInfo &info, cudaStream_t stream) {
    switch (pl.rc) {
        case 1: return launch_decode_fp8_rc<D, kFP16, 1>(p, pl, info, stream);
        case 4: return launch_decode_fp8_rc<D, kFP16, 4>(p, pl, info, stream);
        case 8: return launch_decode_fp8_rc<D, kFP16, 8>(p, pl, info, stream);
        case 16: return launch_decode_fp8_rc<D, kFP16, 16>(p, pl, info, stream);
        case 24: return launch_decode_fp8_rc<D, kFP16, 24>(p, pl, info, stream);
        default: break;
    }
    if constexpr (dec_fp8_max_rows(D) >= 32) return launch_decode_fp8_rc<D, kFP16, 32>(p, pl, info, stream);
    else return FA_ERR_UNSUPPORTED;  // (the plan keeps chunks within the limit)
}

fa_status decode_fp8_impl(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                          const float *v_scale, const int *block_table, const int *seq_lens, void *o, float *lse,
                          void *workspace, size_t workspace_bytes, int B, int H, int Hkv, int Sq, int d,
                          int block_size, int max_blocks, int num_blocks, int max_seq_len, float scale,
                          int mask_kind, int dtype, cudaStream_t stream) {
    fa_status st = check_dec_fp8_sizes(B, H, Hkv, Sq, d, block_size, max_blocks, num_blocks, max_seq_len, mask_kind,
                                       dtype);
    if (st != FA_OK) return st;
    if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !o || !lse)
        return FA_ERR_INVALID_ARG;
    const uintptr_t a16 = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) |
                          reinterpret_cast<uintptr_t>(v_cache) | reinterpret_cast<uintptr_t>(o);
    const uintptr_t a4 = reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(block_table) |
                         reinterpret_cast<uintptr_t>(seq_lens) | reinterpret_cast<uintptr_t>(k_scale) |
                         reinterpret_cast<uintptr_t>(v_scale);
    if ((a16 & 15u) || (a4 & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return FA_ERR_MISALIGNED;
    int dev = 0;
    DeviceInfo *info = nullptr;
    st = device_info(&dev, &info);
    if (st != FA_OK) return st;
    const bool fp16 = dtype == FA_DTYPE_FP16;
    const DecFp8Plan pl = plan_decode_fp8(B, Hkv, H / Hkv * Sq, d, fp16, max_seq_len, info->num_sms);
    const size_t need = pl.bytes;
    if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
    const size_t rows = (size_t)B * H * Sq, qo = rows * d * 2;
    const size_t cache = (size_t)num_blocks * Hkv * block_size * d, scales = (size_t)num_blocks * Hkv * 4;
    const Extent ins[7] = {{q, qo}, {k_cache, cache}, {v_cache, cache}, {k_scale, scales}, {v_scale, scales},
                           {block_table, (size_t)B * max_blocks * 4}, {seq_lens, (size_t)B * 4}};
    const Extent outs[3] = {{o, qo}, {lse, rows * 4}, {workspace, need}};
    if (!outputs_apart(outs, 3, ins, 7, nullptr)) return FA_ERR_INVALID_ARG;

    DecFp8Params p;
    std::memset(&p, 0, sizeof(p));
    const int row_bytes = std::min(d, 128);
    if (!make_map8(&p.tm_k, k_cache, d, block_size, Hkv, num_blocks, row_bytes, block_size) ||
        !make_map8(&p.tm_v, v_cache, d, block_size, Hkv, num_blocks, row_bytes, block_size))
        return FA_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.q = static_cast<const uint16_t *>(q);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.o = o;
    p.lse = lse;
    p.whole = pl.cuts ? 0 : 1;
    if (pl.cuts) {
        p.cuts = reinterpret_cast<int *>(ws);
        p.part_lse = reinterpret_cast<float *>(ws + pl.part_lse_off);
        p.part_o = reinterpret_cast<float *>(ws + pl.part_o_off);
    }
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.Sq = Sq;
    p.R = H / Hkv * Sq;
    p.chunks = pl.chunks;
    p.rows_per_chunk = pl.rows_per_chunk;
    p.bs_log2 = block_size_log2(block_size);
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.max_seq_len = max_seq_len;
    p.mask_kind = mask_kind;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.wait_limit_ns = fa::kWaitLimitNs;
    if (const uint64_t ns = debug_stall_ns()) {
        p.stall_test = 1;
        p.wait_limit_ns = ns;
    }
    if (log_enabled())
        std::fprintf(stderr, "[fa] fa_decode_paged_fp8 d=%d B=%d H=%d Hkv=%d Sq=%d bs=%d max_len=%d rows=%d x %d grid=%d\n",
                     d, B, H, Hkv, Sq, block_size, max_seq_len, pl.rows_per_chunk, pl.chunks, pl.grid);
    if (d == 64)
        return fp16 ? launch_decode_fp8<64, true>(p, pl, *info, stream) : launch_decode_fp8<64, false>(p, pl, *info, stream);
    if (d == 128)
        return fp16 ? launch_decode_fp8<128, true>(p, pl, *info, stream) : launch_decode_fp8<128, false>(p, pl, *info, stream);
    return fp16 ? launch_decode_fp8<256, true>(p, pl, *info, stream) : launch_decode_fp8<256, false>(p, pl, *info, stream);
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_decode_paged_fp8(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                              const float *v_scale, const int *block_table, const int *seq_lens, void *o, float *lse,
                              void *workspace, size_t workspace_bytes, int B, int H, int H_kv, int Sq, int d,
                              int block_size, int max_blocks, int num_blocks, int max_seq_len, float scale,
                              int mask_kind, int dtype, fa_stream_t stream) {
    return fa::decode_fp8_impl(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o, lse, workspace,
                               workspace_bytes, B, H, H_kv, Sq, d, block_size, max_blocks, num_blocks, max_seq_len,
                               scale, mask_kind, dtype, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_decode_fp8_workspace_query(int B, int H, int H_kv, int Sq, int d, int block_size, int max_blocks,
                                        int num_blocks, int max_seq_len, int mask_kind, int dtype, size_t *bytes) {
    if (!bytes) return FA_ERR_INVALID_ARG;
    *bytes = 0;
    const fa_status st = fa::check_dec_fp8_sizes(B, H, H_kv, Sq, d, block_size, max_blocks, num_blocks, max_seq_len,
                                                 mask_kind, dtype);
    if (st != FA_OK) return st;
    int dev = 0;
    fa::DeviceInfo *info = nullptr;
    const fa_status dst = fa::device_info(&dev, &info);
    if (dst != FA_OK) return dst;
    *bytes = fa::plan_decode_fp8(B, H_kv, H / H_kv * Sq, d, dtype == FA_DTYPE_FP16, max_seq_len, info->num_sms).bytes;
    return FA_OK;
}

}  // extern "C"
