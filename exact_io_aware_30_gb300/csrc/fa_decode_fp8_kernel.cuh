// fa_decode_fp8_kernel.cuh -- attention of a few new query rows per request
// over a paged cache held in 8 bits, for sm_103a.
//
// The cache is that of fa_cache_append_fp8: e4m3 codes with one scale per
// block of tokens and K/V head.  For row r of a K/V head, and over the keys j
// it sees,
//   x_rj = scale * ks[block(j)] * (q_r . kcode_j),   p = softmax(x),
//   o_r  = sum_j p_rj vs[block(j)] vcode_j,   lse_r = ln sum_j exp(x_rj),
// by the online softmax of the tiled forward pass.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fa_paged_kernel.cuh"

namespace fa {

struct DecFp8Params {
    const uint16_t *q;       // [B, H, Sq, d] 16-bit
    const uint8_t *k_cache, *v_cache;  // [num_blocks, Hkv, bs, d] e4m3
    const float *k_scale, *v_scale;    // [num_blocks, Hkv]
    const int *block_table, *seq_lens;
    void *o;
    float *lse;
    int B, H, Hkv, Sq, bs_log2, max_blocks, num_blocks, max_seq_len;
    int mask_kind;
    float scale_log2;
};

// One CTA per query row: 128 keys at a time, a key per thread for the scores,
// d / 128 (at least one) columns per thread for the weighted sum.
template <int D, bool kFP16>
__global__ void __launch_bounds__(128) fa_decode_fp8_kernel(const __grid_constant__ DecFp8Params p) {
    __shared__ float sq[D], sp[128], red[4];
    __shared__ int s_block[128];
    const int tid = (int)threadIdx.x;
    const long long row = blockIdx.x;  // of [B, H, Sq]
    const int i = (int)(row % p.Sq);
    const int h = (int)(row / p.Sq % p.H), b = (int)(row / p.Sq / p.H);
    const int kvh = h / (p.H / p.Hkv);
    const int L = min(max(p.seq_lens[b], 0), p.max_seq_len);
    const int n_keys = p.mask_kind == kMaskCausal ? max(min(L - p.Sq + i + 1, L), 0) : L;
    for (int c = tid; c < D; c += 128) {
        const uint32_t w = p.q[row * D + c];
        sq[c] = unpack16<kFP16>(w).x;
    }
    constexpr int PER = (D + 127) / 128;
    float acc[PER] = {}, m = -INFINITY, l = 0.f;
    const int bs = 1 << p.bs_log2;
    for (int k0 = 0; k0 < n_keys; k0 += 128) {
        const int j = k0 + tid;
        int block = -1;
        if (j < n_keys) {
            block = p.block_table[(size_t)b * p.max_blocks + (j >> p.bs_log2)];
            if (block >= p.num_blocks) block = -1;
        }
        __syncthreads();
        s_block[tid] = block;
        float x = j < n_keys ? 0.f : -INFINITY;
        float vs = 0.f;
        if (block >= 0) {
            const size_t bh = (size_t)block * p.Hkv + kvh;
            const uint8_t *kr = p.k_cache + (bh * bs + (j & (bs - 1))) * D;
            float dot = 0.f;
            for (int c = 0; c < D; c += 4) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(kr + c);
                const float2 a = unpack_e4m3x2(w & 0xffffu), e = unpack_e4m3x2(w >> 16);
                dot = fmaf(a.x, sq[c], dot);
                dot = fmaf(a.y, sq[c + 1], dot);
                dot = fmaf(e.x, sq[c + 2], dot);
                dot = fmaf(e.y, sq[c + 3], dot);
            }
            x = dot * (p.scale_log2 * p.k_scale[bh]);
            vs = p.v_scale[bh];
        }
        float mt = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        if ((tid & 31) == 0) red[tid >> 5] = mt;
        __syncthreads();
        mt = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float m_new = fmaxf(m, mt), m_use = m_new == -INFINITY ? 0.f : m_new;
        const float pj = j < n_keys ? exp2f(x - m_use) : 0.f, alpha = exp2f(m - m_use);
        l = l * alpha + pj;
        m = m_new;
        sp[tid] = pj * vs;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= alpha;
        const int n = min(128, n_keys - k0);
        for (int t = 0; t < n; ++t) {
            if (s_block[t] < 0) continue;
            const uint8_t *vr = p.v_cache + (((size_t)s_block[t] * p.Hkv + kvh) * bs + ((k0 + t) & (bs - 1))) * D;
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (tid + 128 * e < D) acc[e] = fmaf(sp[t], unpack_e4m3x2(vr[tid + 128 * e]).x, acc[e]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = l;
    __syncthreads();
    l = red[0] + red[1] + red[2] + red[3];
    const float inv = n_keys > 0 ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e)
        if (tid + 128 * e < D)
            static_cast<uint16_t *>(p.o)[row * D + tid + 128 * e] =
                (uint16_t)(kFP16 ? ptx::pack_f16x2(acc[e] * inv, 0.f) : ptx::pack_bf16x2(acc[e] * inv, 0.f));
    if (tid == 0) p.lse[row] = n_keys > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace fa
