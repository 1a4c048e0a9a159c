// fa_api_paged.cuh -- host side of the paged cache's bookkeeping and writes
// (fa_paged_update, fa_cache_append_fp8).  Included once, by fa_api.cu, after
// its shared helpers.
#pragma once

#include "fa_paged_kernel.cuh"

namespace fa {

namespace {

// log2 of a cache block size, or -1 if it is not one the cache kernels take.
int block_size_log2(int bs) { return bs == 16 ? 4 : bs == 32 ? 5 : bs == 64 ? 6 : bs == 128 ? 7 : -1; }

struct Extent {
    const void *p;
    size_t n;
};

// No output shares a byte with an input or another output, but for the pairs
// (output a, input b) with alias[a] == b that are the same buffer.
bool outputs_apart(const Extent *outs, int n_out, const Extent *ins, int n_in, const int *alias) {
    for (int a = 0; a < n_out; ++a) {
        if (!outs[a].n) continue;
        for (int b = 0; b < n_in; ++b) {
            if (!ins[b].n || (alias && alias[a] == b && outs[a].p == ins[b].p)) continue;
            if (overlaps(outs[a].p, outs[a].n, ins[b].p, ins[b].n)) return false;
        }
        for (int b = a + 1; b < n_out; ++b)
            if (outs[b].n && overlaps(outs[a].p, outs[a].n, outs[b].p, outs[b].n)) return false;
    }
    return true;
}

// Rows of slot_map that one CTA of the update serves before a second CTA pays
// for its own scan of the requests.
constexpr int kUpdateRowsPerCta = 2048;

fa_status paged_update_impl(const int *seq_lens, const int *delta, int *block_table, int *free_ring,
                            const int *ring_state, int *seq_lens_out, int *ring_state_out, int *slot_map,
                            int *positions, int *status, int B, int max_blocks, int ring_size, int block_size,
                            int max_tokens, int per_request, cudaStream_t stream) {
    const int bs_log2 = block_size_log2(block_size);
    if (bs_log2 < 0) return FA_ERR_UNSUPPORTED;
    if (B < 1 || max_blocks < 1 || ring_size < 1 || max_tokens < 0) return FA_ERR_INVALID_ARG;
    if ((long long)max_blocks * block_size > 0x7fffffffLL || (long long)B * max_blocks > 0x7fffffffLL)
        return FA_ERR_INVALID_ARG;
    if (!seq_lens || !delta || !block_table || !free_ring || !ring_state || !seq_lens_out || !ring_state_out ||
        !status || (max_tokens > 0 && (!slot_map || !positions)))
        return FA_ERR_INVALID_ARG;
    const void *all[10] = {seq_lens, delta, block_table, free_ring, ring_state,
                           seq_lens_out, ring_state_out, slot_map, positions, status};
    for (const void *x : all)
        if (reinterpret_cast<uintptr_t>(x) & 3u) return FA_ERR_MISALIGNED;
    const size_t nb = (size_t)B * 4, rows = (size_t)max_tokens * 4;
    const Extent ins[3] = {{seq_lens, nb}, {ring_state, 8}, {delta, nb}};
    const Extent outs[7] = {{seq_lens_out, nb}, {ring_state_out, 8}, {status, nb}, {slot_map, rows},
                            {positions, rows}, {block_table, (size_t)B * max_blocks * 4},
                            {free_ring, (size_t)ring_size * 4}};
    const int alias[7] = {0, 1, -1, -1, -1, -1, -1};
    if (!outputs_apart(outs, 7, ins, 3, alias)) return FA_ERR_INVALID_ARG;
    int dev = 0;
    DeviceInfo *info = nullptr;
    const fa_status st = device_info(&dev, &info);
    if (st != FA_OK) return st;

    PagedUpdateParams p;
    std::memset(&p, 0, sizeof(p));
    p.seq_lens = seq_lens;
    p.delta = delta;
    p.ring_state = ring_state;
    p.block_table = block_table;
    p.free_ring = free_ring;
    p.seq_lens_out = seq_lens_out;
    p.ring_state_out = ring_state_out;
    p.slot_map = slot_map;
    p.positions = positions;
    p.status = status;
    p.B = B;
    p.max_blocks = max_blocks;
    p.ring_size = ring_size;
    p.bs_log2 = bs_log2;
    p.max_tokens = max_tokens;
    p.per_request = per_request;
    // In place, the CTAs have to meet: one cluster of a portable size.
    const bool in_place = seq_lens_out == seq_lens || ring_state_out == ring_state;
    const int most = in_place ? 8 : 32;
    int ranks = 1;
    while (ranks < most && max_tokens > ranks * kUpdateRowsPerCta) ranks *= 2;
    p.meet = in_place && ranks > 1;
    if (log_enabled())
        std::fprintf(stderr, "[fa] fa_paged_update B=%d max_blocks=%d bs=%d rows=%d ctas=%d\n", B, max_blocks,
                     block_size, max_tokens, ranks);
    // few requests and rows: a small CTA, whose barriers cost less
    const bool small = B <= 128 && max_tokens <= 512;
    return launch_overlapped(small ? fa_paged_update_kernel<128> : fa_paged_update_kernel<1024>, dim3((unsigned)ranks),
                             small ? 128 : 1024, 0, p.meet ? (unsigned)ranks : 1u, stream, p);
}

// Sizes of an 8-bit cache shared by the append and the decode.
fa_status check_fp8_cache(int num_blocks, int Hkv, int block_size, int d) {
    if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
    if (block_size_log2(block_size) < 0) return FA_ERR_UNSUPPORTED;
    if (num_blocks < 1 || Hkv < 1) return FA_ERR_INVALID_ARG;
    if ((long long)num_blocks * block_size > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    if ((long long)num_blocks * Hkv > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

fa_status cache_append_impl(const void *k, const void *v, long long k_token_stride, long long k_head_stride,
                            long long v_token_stride, long long v_head_stride, const int *slot_map, void *k_cache,
                            void *v_cache, float *k_scale, float *v_scale, int T, int Hkv, int d, int block_size,
                            int num_blocks, int dtype, cudaStream_t stream) {
    if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_UNSUPPORTED;
    const fa_status sizes = check_fp8_cache(num_blocks, Hkv, block_size, d);
    if (sizes != FA_OK) return sizes;
    if (T < 0 || T > (1 << 30) || Hkv > 65535) return FA_ERR_INVALID_ARG;
    if (T == 0) return FA_OK;
    if (!k || !v || !slot_map || !k_cache || !v_cache || !k_scale || !v_scale) return FA_ERR_INVALID_ARG;
    const long long strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    for (long long s : strides)
        if (s < 0 || s > (1LL << 40)) return FA_ERR_INVALID_ARG;
    const uintptr_t kp = reinterpret_cast<uintptr_t>(k), vp = reinterpret_cast<uintptr_t>(v);
    if (((kp | vp) & 1u) ||
        ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15u) ||
        ((reinterpret_cast<uintptr_t>(slot_map) | reinterpret_cast<uintptr_t>(k_scale) |
          reinterpret_cast<uintptr_t>(v_scale)) & 3u))
        return FA_ERR_MISALIGNED;
    const size_t cache = (size_t)num_blocks * Hkv * block_size * d, scales = (size_t)num_blocks * Hkv * 4;
    const size_t k_bytes = (size_t)((T - 1) * k_token_stride + (Hkv - 1) * k_head_stride + d) * 2;
    const size_t v_bytes = (size_t)((T - 1) * v_token_stride + (Hkv - 1) * v_head_stride + d) * 2;
    const Extent ins[3] = {{k, k_bytes}, {v, v_bytes}, {slot_map, (size_t)T * 4}};
    const Extent outs[4] = {{k_cache, cache}, {v_cache, cache}, {k_scale, scales}, {v_scale, scales}};
    if (!outputs_apart(outs, 4, ins, 3, nullptr)) return FA_ERR_INVALID_ARG;
    int dev = 0;
    DeviceInfo *info = nullptr;
    const fa_status st = device_info(&dev, &info);
    if (st != FA_OK) return st;

    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.x[0] = static_cast<const uint8_t *>(k);
    p.x[1] = static_cast<const uint8_t *>(v);
    p.token_stride[0] = k_token_stride;
    p.token_stride[1] = v_token_stride;
    p.head_stride[0] = k_head_stride;
    p.head_stride[1] = v_head_stride;
    p.cache[0] = static_cast<uint8_t *>(k_cache);
    p.cache[1] = static_cast<uint8_t *>(v_cache);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.slot_map = slot_map;
    p.T = T;
    p.Hkv = Hkv;
    p.d_log2 = d == 64 ? 6 : d == 128 ? 7 : 8;
    p.bs_log2 = block_size_log2(block_size);
    p.slots = (long long)num_blocks * block_size;
    // Warps per pair: a lane holds eight vectors of eight values.
    const int block_log2 = p.d_log2 + p.bs_log2;
    p.wpu_log2 = std::min(std::max(block_log2 - 11, 0), 3);
    const bool big = block_log2 > 14;  // 32,768 values: sixteen vectors a lane
    // Two pairs per group, and rows until the grid is at most two waves (of four
    // CTAs per SM) or a block's: in a decode step every row leads a block of its own;
    // in a prompt one row of a block does, and the others only read their slot.
    // (Two waves at most, not one: 128 rows x 40 heads are 640 CTAs, 32 more than fit
    // at once.  Four waves 15.0 us for 8,203 rows in blocks of 16 where two take 11.8.)
    const int groups = kAppendThreads / (32 << p.wpu_log2);
    const int y = std::max(1, (2 * Hkv + 2 * groups - 1) / (2 * groups));
    p.rows_per_cta = 1;
    while (p.rows_per_cta < block_size &&
           (long long)((T + p.rows_per_cta - 1) / p.rows_per_cta) * y > 8LL * info->num_sms)
        p.rows_per_cta *= 2;
    const dim3 grid((unsigned)((T + p.rows_per_cta - 1) / p.rows_per_cta), (unsigned)y);
    long long bits = (long long)(kp | vp);
    if (T > 1) bits |= (k_token_stride | v_token_stride) * 2;
    if (Hkv > 1) bits |= (k_head_stride | v_head_stride) * 2;
    const bool vec = (bits & 15) == 0, fp16 = dtype == FA_DTYPE_FP16;
    if (log_enabled())
        std::fprintf(stderr, "[fa] fa_cache_append_fp8 rows=%d Hkv=%d d=%d bs=%d vec=%d rows_per_cta=%d grid=%d x %d\n", T,
                     Hkv, d, block_size, vec ? 1 : 0, p.rows_per_cta, (int)grid.x, (int)grid.y);
    auto kern = big ? (fp16 ? (vec ? fa_cache_append_kernel<true, true, 16> : fa_cache_append_kernel<true, false, 16>)
                            : (vec ? fa_cache_append_kernel<false, true, 16> : fa_cache_append_kernel<false, false, 16>))
                    : (fp16 ? (vec ? fa_cache_append_kernel<true, true, 8> : fa_cache_append_kernel<true, false, 8>)
                            : (vec ? fa_cache_append_kernel<false, true, 8> : fa_cache_append_kernel<false, false, 8>));
    return launch_overlapped(kern, grid, kAppendThreads, 0, 1, stream, p);
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_paged_update(const int *seq_lens, const int *delta, int *block_table, int *free_ring,
                          const int *ring_state, int *seq_lens_out, int *ring_state_out, int *slot_map,
                          int *positions, int *status, int B, int max_blocks, int ring_size, int block_size,
                          int max_tokens, fa_stream_t stream) {
    return fa::paged_update_impl(seq_lens, delta, block_table, free_ring, ring_state, seq_lens_out, ring_state_out,
                                 slot_map, positions, status, B, max_blocks, ring_size, block_size, max_tokens, 0,
                                 reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_paged_update_by_request(const int *seq_lens, const int *delta, int *block_table, int *free_ring,
                                     const int *ring_state, int *seq_lens_out, int *ring_state_out, int *slot_map,
                                     int *positions, int *status, int B, int max_blocks, int ring_size,
                                     int block_size, int rows_per_request, fa_stream_t stream) {
    if (B < 1 || rows_per_request < 1 || (long long)B * rows_per_request > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    return fa::paged_update_impl(seq_lens, delta, block_table, free_ring, ring_state, seq_lens_out, ring_state_out,
                                 slot_map, positions, status, B, max_blocks, ring_size, block_size,
                                 B * rows_per_request, rows_per_request, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_cache_append_fp8(const void *k, const void *v, long long k_token_stride, long long k_head_stride,
                              long long v_token_stride, long long v_head_stride, const int *slot_map, void *k_cache,
                              void *v_cache, float *k_scale, float *v_scale, int T, int H_kv, int d, int block_size,
                              int num_blocks, int dtype, fa_stream_t stream) {
    return fa::cache_append_impl(k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slot_map,
                                 k_cache, v_cache, k_scale, v_scale, T, H_kv, d, block_size, num_blocks, dtype,
                                 reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
