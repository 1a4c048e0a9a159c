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
    if ((long long)B * H * Sq > 0x7fffffffLL / 2 || (long long)B * max_blocks > 0x7fffffffLL)
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

template <int D>
fa_status launch_decode_fp8(const DecFp8Params &p, bool fp16, cudaStream_t stream) {
    const unsigned grid = (unsigned)(p.B * p.H * p.Sq);
    if (fp16)
        fa_decode_fp8_kernel<D, true><<<grid, 128, 0, stream>>>(p);
    else
        fa_decode_fp8_kernel<D, false><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
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
    const size_t need = 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
    const size_t rows = (size_t)B * H * Sq, qo = rows * d * 2;
    const size_t cache = (size_t)num_blocks * Hkv * block_size * d, scales = (size_t)num_blocks * Hkv * 4;
    const Extent ins[7] = {{q, qo}, {k_cache, cache}, {v_cache, cache}, {k_scale, scales}, {v_scale, scales},
                           {block_table, (size_t)B * max_blocks * 4}, {seq_lens, (size_t)B * 4}};
    const Extent outs[3] = {{o, qo}, {lse, rows * 4}, {workspace, need}};
    if (!outputs_apart(outs, 3, ins, 7, nullptr)) return FA_ERR_INVALID_ARG;

    const bool fp16 = dtype == FA_DTYPE_FP16;
    DecFp8Params p;
    std::memset(&p, 0, sizeof(p));
    p.q = static_cast<const uint16_t *>(q);
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.Sq = Sq;
    p.bs_log2 = block_size_log2(block_size);
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.max_seq_len = max_seq_len;
    p.mask_kind = mask_kind;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    if (log_enabled())
        std::fprintf(stderr, "[fa] fa_decode_paged_fp8 d=%d B=%d H=%d Hkv=%d Sq=%d bs=%d max_len=%d\n", d, B, H, Hkv,
                     Sq, block_size, max_seq_len);
    return d == 64    ? launch_decode_fp8<64>(p, fp16, stream)
           : d == 128 ? launch_decode_fp8<128>(p, fp16, stream)
                      : launch_decode_fp8<256>(p, fp16, stream);
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
    return fa::device_info(&dev, &info);
}

}  // extern "C"
