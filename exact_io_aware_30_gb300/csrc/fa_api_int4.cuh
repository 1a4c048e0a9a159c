// fa_api_int4.cuh -- host side of the paged cache in 4 bits (fa_cache_append_int4,
// fa_cache_read_int4, fa_decode_paged_int4, fa_decode_int4_workspace_query).
// Included once, by fa_api.cu, after fa_api_rope.cuh (strided views),
// fa_api_paged.cuh and fa_api_decode_fp8.cuh.
#pragma once

#include "fa_decode_int4_kernel.cuh"

namespace fa {

namespace {

// Sizes of a 4-bit cache shared by its entry points.
fa_status check_int4_cache(int num_blocks, int Hkv, int block_size, int d, int group) {
    const fa_status st = check_fp8_cache(num_blocks, Hkv, block_size, d);
    if (st != FA_OK) return st;
    return group == 32 || group == 64 ? FA_OK : FA_ERR_UNSUPPORTED;
}

struct Int4Cache {
    const void *codes[2], *words[2];
    size_t code_bytes, word_bytes;
};

Int4Cache int4_cache(const void *k_cache, const void *v_cache, const void *k_scale, const void *v_scale, int num_blocks,
                     int Hkv, int block_size, int d, int group) {
    const size_t rows = (size_t)num_blocks * Hkv * block_size;
    return {{k_cache, v_cache}, {k_scale, v_scale}, rows * (d / 2), rows * (d / group) * 4};
}

bool int4_aligned(const Int4Cache &c) {
    return ((reinterpret_cast<uintptr_t>(c.codes[0]) | reinterpret_cast<uintptr_t>(c.codes[1]) |
             reinterpret_cast<uintptr_t>(c.words[0]) | reinterpret_cast<uintptr_t>(c.words[1])) & 15u) == 0;
}

// Threads along a row's items (the smallest power of two that holds them, at
// most a CTA's) and CTAs along them.
void int4_items(int per_row, int *items_log2, unsigned *grid_y) {
    *items_log2 = 3;
    while (*items_log2 < 8 && 1 << *items_log2 < per_row) ++*items_log2;
    *grid_y = (unsigned)((per_row + (1 << *items_log2) - 1) >> *items_log2);
}

fa_status cache_append_int4_impl(const void *k, const void *v, long long k_token_stride, long long k_head_stride,
                                 long long v_token_stride, long long v_head_stride, const int *slot_map, void *k_cache,
                                 void *v_cache, unsigned *k_scale, unsigned *v_scale, int T, int Hkv, int d, int group,
                                 int block_size, int num_blocks, int dtype, cudaStream_t stream) {
    if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_UNSUPPORTED;
    const fa_status sizes = check_int4_cache(num_blocks, Hkv, block_size, d, group);
    if (sizes != FA_OK) return sizes;
    if (T < 0 || T > (1 << 30) || Hkv > 65535) return FA_ERR_INVALID_ARG;
    if (T == 0) return FA_OK;
    if (!k || !v || !slot_map || !k_cache || !v_cache || !k_scale || !v_scale) return FA_ERR_INVALID_ARG;
    const long long strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    for (long long s : strides)
        if (s < 0 || s > (1LL << 40)) return FA_ERR_INVALID_ARG;
    // (every offset stays below 2^58 elements)
    for (int i = 0; i < 4; i += 2)
        if (strides[i] > (1LL << 57) / T || strides[i + 1] > (1LL << 57) / Hkv) return FA_ERR_INVALID_ARG;
    const uintptr_t kp = reinterpret_cast<uintptr_t>(k), vp = reinterpret_cast<uintptr_t>(v);
    const Int4Cache c = int4_cache(k_cache, v_cache, k_scale, v_scale, num_blocks, Hkv, block_size, d, group);
    if (((kp | vp) & 1u) || !int4_aligned(c) || (reinterpret_cast<uintptr_t>(slot_map) & 3u)) return FA_ERR_MISALIGNED;
    const size_t k_bytes = (size_t)((T - 1) * k_token_stride + (Hkv - 1) * k_head_stride + d) * 2;
    const size_t v_bytes = (size_t)((T - 1) * v_token_stride + (Hkv - 1) * v_head_stride + d) * 2;
    const Extent ins[3] = {{k, k_bytes}, {v, v_bytes}, {slot_map, (size_t)T * 4}};
    const Extent outs[4] = {{k_cache, c.code_bytes}, {v_cache, c.code_bytes}, {k_scale, c.word_bytes}, {v_scale, c.word_bytes}};
    if (!outputs_apart(outs, 4, ins, 3, nullptr)) return FA_ERR_INVALID_ARG;
    int dev = 0;
    DeviceInfo *info = nullptr;
    const fa_status st = device_info(&dev, &info);
    if (st != FA_OK) return st;

    Int4AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.x[0] = static_cast<const uint16_t *>(k);
    p.x[1] = static_cast<const uint16_t *>(v);
    p.token_stride[0] = k_token_stride;
    p.token_stride[1] = v_token_stride;
    p.head_stride[0] = k_head_stride;
    p.head_stride[1] = v_head_stride;
    p.codes[0] = static_cast<uint8_t *>(k_cache);
    p.codes[1] = static_cast<uint8_t *>(v_cache);
    p.words[0] = k_scale;
    p.words[1] = v_scale;
    p.slot_map = slot_map;
    p.slots = (long long)num_blocks * block_size;
    p.T = T;
    p.Hkv = Hkv;
    p.d_log2 = d == 64 ? 6 : d == 128 ? 7 : 8;
    p.g_log2 = group == 32 ? 5 : 6;
    p.bs_log2 = block_size_log2(block_size);
    unsigned y = 1;
    int4_items(2 * Hkv * (d / 16), &p.items_log2, &y);
    // Rows per CTA: one per thread, and up to sixteen while the grid has more than
    // eight CTAs per SM (8,203 rows x 8 heads at d 128: one 19.9 us, eight 17.5, sixteen
    // 16.3; 40,008 rows at d 256: 64 138 us, sixteen 112, eight 111).
    p.rows_per_cta = std::min(kInt4Threads >> p.items_log2, kInt4MaxRows);
    while (p.rows_per_cta < 16 * (kInt4Threads >> p.items_log2) && p.rows_per_cta < kInt4MaxRows &&
           (long long)((T + p.rows_per_cta - 1) / p.rows_per_cta) * y > 8LL * info->num_sms)
        p.rows_per_cta *= 2;
    const dim3 grid((unsigned)((T + p.rows_per_cta - 1) / p.rows_per_cta), y);
    long long bits = (long long)(kp | vp);
    if (T > 1) bits |= (k_token_stride | v_token_stride) * 2;
    if (Hkv > 1) bits |= (k_head_stride | v_head_stride) * 2;
    const bool vec = (bits & 15) == 0, fp16 = dtype == FA_DTYPE_FP16;
    if (log_enabled())
        std::fprintf(stderr, "[fa] fa_cache_append_int4 rows=%d Hkv=%d d=%d group=%d bs=%d vec=%d rows_per_cta=%d grid=%d x %d\n",
                     T, Hkv, d, group, block_size, vec ? 1 : 0, p.rows_per_cta, (int)grid.x, (int)grid.y);
    auto kern = fp16 ? (vec ? fa_cache_append_int4_kernel<true, true> : fa_cache_append_int4_kernel<true, false>)
                     : (vec ? fa_cache_append_int4_kernel<false, true> : fa_cache_append_int4_kernel<false, false>);
    return launch_overlapped(kern, grid, kInt4Threads, 0, 1, stream, p);
}

fa_status cache_read_int4_impl(const void *k_cache, const void *v_cache, const unsigned *k_scale, const unsigned *v_scale,
                               const int *block_table, const int *seq_lens, const int *starts, void *k_out,
                               const long long *k_strides, void *v_out, const long long *v_strides, int B, int Hkv,
                               int rows, int d, int group, int block_size, int max_blocks, int num_blocks, int dtype,
                               cudaStream_t stream) {
    if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_UNSUPPORTED;
    const fa_status sizes = check_int4_cache(num_blocks, Hkv, block_size, d, group);
    if (sizes != FA_OK) return sizes;
    if (B < 1 || rows < 0 || rows > (1 << 30) || Hkv > 65535 || max_blocks < 1) return FA_ERR_INVALID_ARG;
    if ((long long)max_blocks * block_size > 0x7fffffffLL || (long long)B * max_blocks > 0x7fffffffLL ||
        (long long)B * rows > 0x7fffffffLL)
        return FA_ERR_INVALID_ARG;
    if (rows == 0) return FA_OK;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !k_out || !v_out || !k_strides ||
        !v_strides)
        return FA_ERR_INVALID_ARG;
    const Int4Cache c = int4_cache(k_cache, v_cache, k_scale, v_scale, num_blocks, Hkv, block_size, d, group);
    if (!int4_aligned(c) || ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
                              reinterpret_cast<uintptr_t>(starts)) & 3u))
        return FA_ERR_MISALIGNED;
    void *outs[2] = {k_out, v_out};
    const long long *strides[2] = {k_strides, v_strides};
    StridedView view[2];
    for (int i = 0; i < 2; ++i) {
        view[i] = {reinterpret_cast<uintptr_t>(outs[i]), {B, Hkv, rows}, {strides[i][0], strides[i][1], strides[i][2]}, d, 2};
        if (view[i].base & 1u) return FA_ERR_MISALIGNED;
        long long reach = d;
        for (int n = 0; n < 3; ++n) {
            if (view[i].stride[n] < 0 || view[i].stride[n] > (1LL << 40)) return FA_ERR_INVALID_ARG;
            if (view[i].size[n] > 1) reach += (view[i].size[n] - 1) * view[i].stride[n];
            if (reach > (1LL << 58)) return FA_ERR_INVALID_ARG;
        }
        if (!view_injective(view[i])) return FA_ERR_INVALID_ARG;
    }
    if (!views_disjoint(view[0], view[1])) return FA_ERR_INVALID_ARG;
    const Extent ins[7] = {{k_cache, c.code_bytes}, {v_cache, c.code_bytes}, {k_scale, c.word_bytes}, {v_scale, c.word_bytes},
                           {block_table, (size_t)B * max_blocks * 4}, {seq_lens, (size_t)B * 4},
                           {starts, starts ? (size_t)B * 4 : 0}};
    for (int i = 0; i < 2; ++i) {
        const Extent out = {outs[i], (size_t)view_span(view[i], true, true, true) * 2};
        if (!outputs_apart(&out, 1, ins, 7, nullptr)) return FA_ERR_INVALID_ARG;
    }
    int dev = 0;
    DeviceInfo *info = nullptr;
    const fa_status st = device_info(&dev, &info);
    if (st != FA_OK) return st;

    Int4ReadParams p;
    std::memset(&p, 0, sizeof(p));
    long long bits = 0;
    for (int i = 0; i < 2; ++i) {
        p.codes[i] = static_cast<const uint8_t *>(c.codes[i]);
        p.words[i] = static_cast<const uint32_t *>(c.words[i]);
        p.out[i] = static_cast<uint16_t *>(outs[i]);
        bits |= (long long)view[i].base;
        for (int n = 0; n < 3; ++n) {
            p.stride[i][n] = strides[i][n];
            if (view[i].size[n] > 1) bits |= strides[i][n] * 2;
        }
    }
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.starts = starts;
    p.Hkv = Hkv;
    p.rows = rows;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.d_log2 = d == 64 ? 6 : d == 128 ? 7 : 8;
    p.g_log2 = group == 32 ? 5 : 6;
    p.bs_log2 = block_size_log2(block_size);
    unsigned y = 1;
    int4_items(2 * Hkv * (d / 16), &p.items_log2, &y);
    // Rows per CTA: four in flight per thread, and more until the grid is at most
    // eight waves of eight CTAs per SM.
    p.rows_per_cta = 4 * (kInt4Threads >> p.items_log2);
    while (p.rows_per_cta < 1024 && (long long)B * ((rows + p.rows_per_cta - 1) / p.rows_per_cta) * y > 64LL * info->num_sms)
        p.rows_per_cta *= 2;
    p.chunks = (rows + p.rows_per_cta - 1) / p.rows_per_cta;
    const dim3 grid((unsigned)((long long)B * p.chunks), y);
    const int bytes = (bits & 31) == 0 ? 32 : (bits & 15) == 0 ? 16 : 2;
    const bool fp16 = dtype == FA_DTYPE_FP16;
    if (log_enabled())
        std::fprintf(stderr, "[fa] fa_cache_read_int4 B=%d Hkv=%d rows=%d d=%d group=%d bs=%d bytes=%d rows_per_cta=%d grid=%d x %d\n",
                     B, Hkv, rows, d, group, block_size, bytes, p.rows_per_cta, (int)grid.x, (int)grid.y);
    auto kern = bytes == 32   ? (fp16 ? fa_cache_read_int4_kernel<true, 32> : fa_cache_read_int4_kernel<false, 32>)
                : bytes == 16 ? (fp16 ? fa_cache_read_int4_kernel<true, 16> : fa_cache_read_int4_kernel<false, 16>)
                              : (fp16 ? fa_cache_read_int4_kernel<true, 2> : fa_cache_read_int4_kernel<false, 2>);
    return launch_overlapped(kern, grid, kInt4Threads, 0, 1, stream, p);
}

// ------------------------------------------------------------------- decode

// Rows of 32, 64 or 128 bytes of codes: box {d / 2, bs, 1, 1}, the swizzle of that width.
bool make_map_int4_codes(CUtensorMap *m, const void *base, int d, int bs, int Hkv, int num_blocks) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t row = (cuuint64_t)d / 2;
    cuuint64_t dims[4] = {row, (cuuint64_t)bs, (cuuint64_t)Hkv, (cuuint64_t)num_blocks};
    cuuint64_t strides[3] = {row, row * bs, row * bs * Hkv};
    cuuint32_t box[4] = {(cuuint32_t)row, (cuuint32_t)bs, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               d == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : d == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernel of a unit's rows (4, 8, 16 or 32): eights of rows per warp (at d = 256 a
// warp's registers hold one) and groups of warps with different rows.
constexpr int int4_warp_eights(int rc, int d) { return rc <= 8 || d == 256 ? 1 : 2; }
constexpr int int4_row_groups(int rc, int d) { return rc <= 8 ? 1 : rc / (8 * int4_warp_eights(rc, d)); }

struct DecInt4Plan : DecFp8Plan {
    size_t sums_off = 0;  // 0: no unit is long enough to rest
};

// Rows of a K/V head: at most 4, 8 (a warp's columns), 16, or 32 in equal chunks of
// at most that, the cache being read once more per chunk.
DecInt4Plan plan_decode_int4(int B, int Hkv, int R, int d, int max_seq_len, int num_sms) {
    DecInt4Plan pl;
    pl.chunks = (R + 31) / 32;
    pl.rows_per_chunk = (R + pl.chunks - 1) / pl.chunks;
    if (pl.chunks > 1) pl.rows_per_chunk = (pl.rows_per_chunk + 7) / 8 * 8;  // (a warp has whole eights)
    pl.chunks = (R + pl.rows_per_chunk - 1) / pl.rows_per_chunk;
    pl.rc = pl.rows_per_chunk <= 4 ? 4 : pl.rows_per_chunk <= 8 ? 8 : pl.rows_per_chunk <= 16 ? 16 : 32;
    const int per_sm = d <= 128 && pl.rc <= 8 ? 3 : 2;
    const long long tiles = (max_seq_len + 127LL) / 128;
    const long long units = (long long)B * Hkv * pl.chunks;
    pl.cuts = tiles > kDecFp8WholeTiles;
    pl.grid = (int)std::min(pl.cuts ? units * tiles : units, (long long)num_sms * per_sm);
    if (pl.cuts) {
        pl.part_lse_off = ((size_t)(4 + 5 * pl.grid) * 4 + 255) / 256 * 256;
        pl.part_o_off = (pl.part_lse_off + (size_t)2 * pl.grid * pl.rc * 4 + 255) / 256 * 256;
        pl.bytes = pl.part_o_off + (size_t)2 * pl.grid * pl.rc * d * 4;
    }
    const int groups = int4_row_groups(pl.rc, d);
    if (tiles > dec_i4_rest(groups)) {
        pl.sums_off = pl.bytes;
        pl.bytes += (size_t)pl.grid * groups * dec_i4_part(d, int4_warp_eights(pl.rc, d), pl.rc == 4 ? 1 : 2);
    }
    return pl;
}

template <class C>
fa_status launch_decode_int4_c(const DecInt4Params &p, const DecInt4Plan &pl, DeviceInfo &info, cudaStream_t stream) {
    constexpr int kind = C::RC == 4 ? 0 : (C::RC == 8 ? 1 : C::RC == 16 ? 3 : 5) + (C::kTwice ? 1 : 0);
    const int slot = (((C::D == 256 ? 2 : C::D == 128 ? 1 : 0) * 2 + (C::G == 64 ? 1 : 0)) * 2 + (C::kRests ? 1 : 0)) * 7 + kind;
    if (set_smem(fa_decode_int4_kernel<C>, C::SMEM_BYTES, info.attr_dec_int4[slot]) != FA_OK) return FA_ERR_CUDA;
    const fa_status st = launch_overlapped(fa_decode_int4_kernel<C>, dim3((unsigned)pl.grid), C::NUM_THREADS, C::SMEM_BYTES,
                                           1, stream, p);
    if (st != FA_OK || !pl.cuts || pl.grid < 2) return st;
    const DecFp8Params &merge = p;
    return launch_overlapped(p.fp16 ? fa_decode_fp8_combine_kernel<C::D, true, C::RC> : fa_decode_fp8_combine_kernel<C::D, false, C::RC>,
                             dim3((unsigned)(pl.grid - 1)), kDecFp8MergeThreads<C::RC>, 0, 1, stream, merge, pl.grid);
}

template <int D, int G, int RC, bool kRests>
fa_status launch_decode_int4_rc(const DecInt4Params &p, const DecInt4Plan &pl, DeviceInfo &info, cudaStream_t stream) {
    constexpr int NT = int4_warp_eights(RC, D), RG = int4_row_groups(RC, D);
    if constexpr (RC == 4) return launch_decode_int4_c<DecI4Cfg<D, G, NT, RG, true, false, kRests>>(p, pl, info, stream);
    else
        return p.fp16 ? launch_decode_int4_c<DecI4Cfg<D, G, NT, RG, false, true, kRests>>(p, pl, info, stream)
                      : launch_decode_int4_c<DecI4Cfg<D, G, NT, RG, false, false, kRests>>(p, pl, info, stream);
}

template <int D, int G, bool kRests>
fa_status launch_decode_int4_g(const DecInt4Params &p, const DecInt4Plan &pl, DeviceInfo &info, cudaStream_t stream) {
    if (pl.rc == 4) return launch_decode_int4_rc<D, G, 4, kRests>(p, pl, info, stream);
    if (pl.rc == 8) return launch_decode_int4_rc<D, G, 8, kRests>(p, pl, info, stream);
    if (pl.rc == 16) return launch_decode_int4_rc<D, G, 16, kRests>(p, pl, info, stream);
    return launch_decode_int4_rc<D, G, 32, kRests>(p, pl, info, stream);
}

template <int D>
fa_status launch_decode_int4(int group, const DecInt4Params &p, const DecInt4Plan &pl, DeviceInfo &info, cudaStream_t stream) {
    if (group == 32)
        return pl.sums_off ? launch_decode_int4_g<D, 32, true>(p, pl, info, stream) : launch_decode_int4_g<D, 32, false>(p, pl, info, stream);
    return pl.sums_off ? launch_decode_int4_g<D, 64, true>(p, pl, info, stream) : launch_decode_int4_g<D, 64, false>(p, pl, info, stream);
}

fa_status check_dec_int4_sizes(int B, int H, int Hkv, int Sq, int d, int group, int block_size, int max_blocks,
                               int num_blocks, int max_seq_len, int mask_kind, int dtype) {
    const fa_status st = check_dec_fp8_sizes(B, H, Hkv, Sq, d, block_size, max_blocks, num_blocks, max_seq_len, mask_kind,
                                             dtype);
    return st != FA_OK ? st : check_int4_cache(num_blocks, Hkv, block_size, d, group);
}

fa_status decode_int4_impl(const void *q, const void *k_cache, const void *v_cache, const unsigned *k_scale,
                           const unsigned *v_scale, const int *block_table, const int *seq_lens, void *o, float *lse,
                           void *workspace, size_t workspace_bytes, int B, int H, int Hkv, int Sq, int d, int group,
                           int block_size, int max_blocks, int num_blocks, int max_seq_len, float scale, int mask_kind,
                           int dtype, cudaStream_t stream) {
    fa_status st = check_dec_int4_sizes(B, H, Hkv, Sq, d, group, block_size, max_blocks, num_blocks, max_seq_len, mask_kind,
                                        dtype);
    if (st != FA_OK) return st;
    if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !o || !lse)
        return FA_ERR_INVALID_ARG;
    const Int4Cache c = int4_cache(k_cache, v_cache, k_scale, v_scale, num_blocks, Hkv, block_size, d, group);
    const uintptr_t a16 = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o);
    const uintptr_t a4 = reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(block_table) |
                         reinterpret_cast<uintptr_t>(seq_lens);
    if ((a16 & 15u) || !int4_aligned(c) || (a4 & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return FA_ERR_MISALIGNED;
    int dev = 0;
    DeviceInfo *info = nullptr;
    st = device_info(&dev, &info);
    if (st != FA_OK) return st;
    const DecInt4Plan pl = plan_decode_int4(B, Hkv, H / Hkv * Sq, d, max_seq_len, info->num_sms);
    const size_t need = pl.bytes;
    if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
    const size_t rows = (size_t)B * H * Sq, qo = rows * d * 2;
    const Extent ins[7] = {{q, qo}, {k_cache, c.code_bytes}, {v_cache, c.code_bytes}, {k_scale, c.word_bytes},
                           {v_scale, c.word_bytes}, {block_table, (size_t)B * max_blocks * 4}, {seq_lens, (size_t)B * 4}};
    const Extent outs[3] = {{o, qo}, {lse, rows * 4}, {workspace, need}};
    if (!outputs_apart(outs, 3, ins, 7, nullptr)) return FA_ERR_INVALID_ARG;

    DecInt4Params p;
    std::memset(&p, 0, sizeof(p));
    if (!make_map_int4_codes(&p.tm_k, k_cache, d, block_size, Hkv, num_blocks) ||
        !make_map_int4_codes(&p.tm_v, v_cache, d, block_size, Hkv, num_blocks))
        return FA_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.q = static_cast<const uint16_t *>(q);
    p.k_words = k_scale;
    p.v_words = v_scale;
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
    if (pl.sums_off) p.sums = reinterpret_cast<float4 *>(ws + pl.sums_off);
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
    p.fp16 = dtype == FA_DTYPE_FP16;
    p.wait_limit_ns = fa::kWaitLimitNs;
    if (const uint64_t ns = debug_stall_ns()) {
        p.stall_test = 1;
        p.wait_limit_ns = ns;
    }
    if (log_enabled())
        std::fprintf(stderr, "[fa] fa_decode_paged_int4 d=%d group=%d B=%d H=%d Hkv=%d Sq=%d bs=%d max_len=%d rows=%d x %d grid=%d\n",
                     d, group, B, H, Hkv, Sq, block_size, max_seq_len, pl.rows_per_chunk, pl.chunks, pl.grid);
    if (d == 64) return launch_decode_int4<64>(group, p, pl, *info, stream);
    if (d == 128) return launch_decode_int4<128>(group, p, pl, *info, stream);
    return launch_decode_int4<256>(group, p, pl, *info, stream);
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_cache_append_int4(const void *k, const void *v, long long k_token_stride, long long k_head_stride,
                               long long v_token_stride, long long v_head_stride, const int *slot_map, void *k_cache,
                               void *v_cache, unsigned *k_scale, unsigned *v_scale, int T, int H_kv, int d, int group,
                               int block_size, int num_blocks, int dtype, fa_stream_t stream) {
    return fa::cache_append_int4_impl(k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slot_map,
                                      k_cache, v_cache, k_scale, v_scale, T, H_kv, d, group, block_size, num_blocks,
                                      dtype, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_cache_read_int4(const void *k_cache, const void *v_cache, const unsigned *k_scale, const unsigned *v_scale,
                             const int *block_table, const int *seq_lens, const int *starts, void *k_out,
                             const long long *k_strides, void *v_out, const long long *v_strides, int B, int H_kv,
                             int rows, int d, int group, int block_size, int max_blocks, int num_blocks, int dtype,
                             fa_stream_t stream) {
    return fa::cache_read_int4_impl(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, starts, k_out, k_strides,
                                    v_out, v_strides, B, H_kv, rows, d, group, block_size, max_blocks, num_blocks, dtype,
                                    reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_decode_paged_int4(const void *q, const void *k_cache, const void *v_cache, const unsigned *k_scale,
                               const unsigned *v_scale, const int *block_table, const int *seq_lens, void *o, float *lse,
                               void *workspace, size_t workspace_bytes, int B, int H, int H_kv, int Sq, int d, int group,
                               int block_size, int max_blocks, int num_blocks, int max_seq_len, float scale,
                               int mask_kind, int dtype, fa_stream_t stream) {
    return fa::decode_int4_impl(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o, lse, workspace,
                                workspace_bytes, B, H, H_kv, Sq, d, group, block_size, max_blocks, num_blocks,
                                max_seq_len, scale, mask_kind, dtype, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_decode_int4_workspace_query(int B, int H, int H_kv, int Sq, int d, int group, int block_size, int max_blocks,
                                         int num_blocks, int max_seq_len, int mask_kind, int dtype, size_t *bytes) {
    if (!bytes) return FA_ERR_INVALID_ARG;
    *bytes = 0;
    const fa_status st = fa::check_dec_int4_sizes(B, H, H_kv, Sq, d, group, block_size, max_blocks, num_blocks,
                                                  max_seq_len, mask_kind, dtype);
    if (st != FA_OK) return st;
    int dev = 0;
    fa::DeviceInfo *info = nullptr;
    const fa_status dst = fa::device_info(&dev, &info);
    if (dst != FA_OK) return dst;
    *bytes = fa::plan_decode_int4(B, H_kv, H / H_kv * Sq, d, max_seq_len, info->num_sms).bytes;
    return FA_OK;
}

}  // extern "C"
