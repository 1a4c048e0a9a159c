// fa_decode_fp8_kernel.cuh -- attention of a few new query rows per request
// over a paged cache held in 8 bits, for sm_103a.
//
// The cache is that of fa_cache_append_fp8: e4m3 codes with one scale per
// block of tokens and K/V head.  For row r of a K/V head, and over the keys j
// it sees,
//   x_rj = scale * ks[block(j)] * (q_r . kcode_j),   p = softmax(x),
//   o_r  = sum_j p_rj vs[block(j)] vcode_j,   lse_r = ln sum_j exp(x_rj),
// by the online softmax of the tiled forward pass.  Bound by reading the
// cache: 2 d bytes per token and K/V head.
//
// Both products run on the 8-bit tensor path with the cache's own codes as one
// operand, straight from TMA -- widening them first would move every byte
// through shared memory three more times.  Two things make that exact enough:
//   * keys are the M side.  S^T = K Q^T has M = 128 keys and N = the few query
//     rows, O^T = V^T P^T has M = 128 columns of d (V read M-major as it lies)
//     and N = the rows again, so no part of the tensor core's work is padding
//     for the rows that are missing, and it stays far from being the limit;
//   * a 16-bit q and the fp32 weights are split into NP e4m3 parts with
//     x = x1 + x2 / 16 (+ x3 / 256), each part the rounding of what the parts
//     before it left, and the parts are columns of N beside each other; their
//     products are summed in fp32 as they are read back.  Two parts hold the 8
//     significant bits of bf16, three the 11 of fp16, so S is exact up to
//     fp32 sums (a component below 2^-14 of its row's largest keeps 2^-22 of
//     that), and a weight is rounded by at most 2^-8 (2^-12) of itself, as a
//     16-bit P would be.  Weights are taken relative to the largest score of
//     their own 128-key tile and the tiles' outputs are rescaled in fp32, so
//     that what is below the parts' range (2^-22 of the tile's largest) is
//     never a large share of a row.
//
// Work split.  The work is a line of 128-key tiles: request by request, K/V
// head by K/V head, chunk of rows by chunk of rows (a unit), tile by tile.
// CTA c of G takes tiles [c T / G, (c + 1) T / G) of the T there are, so every
// CTA has the same work whatever the lengths, and its pipelines run on from
// unit to unit.  A unit that lies in one CTA is written out by it; one that is
// cut leaves a normalised partial row and its lse per CTA, and
// fa_decode_fp8_combine_kernel (a CTA per cut) merges them in order.
//
// One CTA:
//   warps 0-3: softmax.  Thread = key for S^T (TMEM lane), = column of d for
//              O^T; O is kept in registers, rescaled per tile;
//   warp 4:    MMA issuer: S^T of tile t + 1 before O^T of tile t;
//   warp 5:    TMA, a lane per block of the tile, K and V rings.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fa_fp8_kernel.cuh"
#include "fa_paged_kernel.cuh"

namespace fa {

struct DecFp8Params {
    CUtensorMap tm_k, tm_v;  // [num_blocks, Hkv, bs, d] bytes, box {min(d, 128), bs, 1, 1}
    const uint16_t *q;       // [B, H, Sq, d] 16-bit
    const float *k_scale, *v_scale;  // [num_blocks, Hkv]
    const int *block_table, *seq_lens;
    void *o;
    float *lse;
    float *part_o;           // [2 G, RC, d]: slot 2c: CTA c's unit begun by others; 2c + 1: one it begins and others end
    float *part_lse;         // [2 G, RC], log2 units
    int *cuts;               // [4 + 4 G]: total tiles (64-bit), then per CTA its first unit: b, head and chunk, tile, tiles
    int B, H, Hkv, Sq, R;    // R = H / Hkv * Sq rows per K/V head
    int chunks;              // of at most RC rows each
    int rows_per_chunk;
    int bs_log2, max_blocks, num_blocks, max_seq_len;
    int mask_kind;
    float scale_log2;
    uint64_t wait_limit_ns;
    int stall_test;          // test only: the softmax's first wait is on a barrier nothing completes
};

template <int D_, bool kFP16_, int RC_>
struct DecFp8Cfg {
    static constexpr int D = D_;
    static constexpr bool kFP16 = kFP16_;
    static constexpr int RC = RC_;                      // query rows per unit
    static constexpr int NP = kFP16 ? 3 : 2;            // e4m3 parts of q and of the weights
    static constexpr int N = (RC * NP + 15) / 16 * 16;  // columns: part-major, then rows
    static constexpr int BN = 128;                      // keys per tile
    static constexpr int ROWB = D < 128 ? D : 128;      // bytes of a row in one column chunk
    static constexpr int NCH = D / ROWB;                // column chunks
    static constexpr int NM = D == 256 ? 2 : 1;         // M blocks of O^T
    static constexpr int TILE = BN * D;                 // bytes of a K or V tile
    static constexpr int CHUNK_BYTES = BN * ROWB;
    static constexpr int Q_BYTES = N * D;               // one buffer of q's parts
    static constexpr int QCH = N * ROWB;
    static constexpr int P_BYTES = N * 128;
    static constexpr uint32_t S_COL = 0;                // two buffers
    static constexpr uint32_t O_COL = 2 * N;
    static constexpr int COLS = (2 + NM) * N;
    static constexpr uint32_t TMEM_COLS = COLS <= 32 ? 32 : COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static constexpr int CTAS_PER_SM = (D <= 128 && TMEM_COLS <= 256) ? 2 : 1;
    static constexpr int NUM_THREADS = 192;
    static constexpr int MMA_WARP = 4;
    static constexpr int TMA_WARP = 5;
    // small arrays, in floats
    static constexpr int F_RED = 0;                        // [2][4][RC + 1] tile maxima, largest |vs|
    static constexpr int F_M = F_RED + 2 * 4 * (RC + 1);   // [4][RC] the tile's maxima, a copy per warp
    static constexpr int F_AB = (F_M + 4 * RC + 1) / 2 * 2;  // [2][4][RC] float2: rescale of O, weight of the tile
    static constexpr int F_C = F_AB + 2 * 4 * RC * 2;      // [2][RC] score multiplier
    static constexpr int F_LAST = F_C + 2 * RC;            // [2][RC] last key the row sees (int)
    static constexpr int F_L = F_LAST + 2 * RC;            // [4][RC] warps' sums
    static constexpr int F_NUM = F_L + 4 * RC;
    static constexpr int BUDGET = CTAS_PER_SM == 2 ? 113 * 1024 : 226 * 1024;
    static constexpr int FIXED = 1024 + 2 * Q_BYTES + P_BYTES + F_NUM * 4 + 512;
    static constexpr int SLOTS = (BUDGET - FIXED) / TILE;
    static constexpr int KST = SLOTS >= 12 ? 6 : (SLOTS + 1) / 2;
    static constexpr int VST = SLOTS >= 12 ? 6 : SLOTS / 2;
    static constexpr int B_KFULL = 0;
    static constexpr int B_KEMPTY = B_KFULL + KST;
    static constexpr int B_VFULL = B_KEMPTY + KST;
    static constexpr int B_VEMPTY = B_VFULL + VST;
    static constexpr int B_QFULL = B_VEMPTY + VST;  // [2]
    static constexpr int B_SFULL = B_QFULL + 2;     // [2]
    static constexpr int B_SFREE = B_SFULL + 2;     // [2]
    static constexpr int B_PFULL = B_SFREE + 2;
    static constexpr int B_OFULL = B_PFULL + 1;
    static constexpr int B_DRAIN = B_OFULL + 1;
    static constexpr int B_NEVER = B_DRAIN + 1;     // no arrivals (the stall test's wait)
    static constexpr int NUM_BARS = B_NEVER + 1;
    static constexpr int SMEM_TILES = 2 * Q_BYTES + P_BYTES + (KST + VST) * TILE;
    static constexpr int SMEM_BYTES = 1024 + SMEM_TILES + F_NUM * 4 + NUM_BARS * 8 + 64;
    static_assert(VST >= 2, "rings of at least two tiles");
    static_assert(SMEM_BYTES <= BUDGET && SMEM_BYTES <= 232448, "shared memory overflow");
    static_assert(NUM_BARS * 8 + 64 <= 512 && COLS <= 512 && N <= 256, "layout");
    static_assert(QCH % 1024 == 0 || ROWB == 64, "swizzle atoms");

    // Operand descriptors at byte address a: rows of ROWB bytes, K-major (K
    // tiles, q parts) or M-major (V tiles: rows are K).
    static __device__ __forceinline__ uint64_t desc(uint32_t a) {
        if constexpr (ROWB == 64) return smem_desc_sw64(a);
        else return smem_desc(a, 16);
    }
    // M-major with 64-byte rows: M = 128 takes two atoms of 64 columns; the
    // leading offset 0 reads the same atom twice, and lanes 64 .. 127 of O^T
    // repeat 0 .. 63 unread.
    static __device__ __forceinline__ uint64_t desc_v(uint32_t a) {
        if constexpr (ROWB == 64)
            return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
        else return smem_desc(a, 16);
    }
};

// A CTA's place in the line of tiles, stepped tile by tile.
struct DecFp8It {
    int b, hc, tile;  // request, K/V head * chunks + chunk, tile of the unit
    int L, nt;        // the request's length and tiles
    int next_len;     // the next request's length, loaded ahead
    int left;         // tiles left, this one included
};

__device__ __forceinline__ int dec_fp8_tiles(int L) { return max((L + 127) >> 7, 1); }

__device__ __forceinline__ int dec_fp8_len(const DecFp8Params &p, int b) {
    return b < p.B ? min(max(p.seq_lens[b], 0), p.max_seq_len) : 0;
}

__device__ __forceinline__ void dec_fp8_step(const DecFp8Params &p, DecFp8It &it) {
    --it.left;
    if (++it.tile < it.nt) return;
    it.tile = 0;
    if (++it.hc < p.Hkv * p.chunks) return;
    it.hc = 0;
    ++it.b;
    it.L = it.next_len;
    it.nt = dec_fp8_tiles(it.L);
    it.next_len = dec_fp8_len(p, it.b + 1);
}

// Where this CTA's tiles begin: prefix sums over the requests' tiles, by all
// threads of the CTA.  `scratch` holds 16 long longs.
template <int THREADS>
__device__ DecFp8It dec_fp8_begin(const DecFp8Params &p, long long *scratch) {
    constexpr int W = THREADS / 32;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long hc = (long long)p.Hkv * p.chunks;
    int sum = 0;
    for (int b = tid; b < p.B; b += THREADS) sum += dec_fp8_tiles(dec_fp8_len(p, b));
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) scratch[warp] = sum;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < W; ++w) total += scratch[w];
    total *= hc;
    const long long G = min((long long)gridDim.x, total), c = blockIdx.x;
    DecFp8It it;
    it.b = it.hc = it.tile = it.L = it.nt = it.next_len = it.left = 0;
    if (c == 0 && tid == 0) *reinterpret_cast<long long *>(p.cuts) = total;
    if (c >= G) return it;
    const long long lo = c * total / G, hi = (c + 1) * total / G;
    long long before = 0;  // tiles of the requests before this group of THREADS, per K/V head and chunk
    for (int b0 = 0;; b0 += THREADS) {
        const int b = b0 + tid;
        const int n = b < p.B ? dec_fp8_tiles(dec_fp8_len(p, b)) : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (tid == 0) scratch[W] = -1;
        if (lane == 31) scratch[warp] = inc;
        __syncthreads();
        long long at = before + inc - n, all = 0;
        for (int w = 0; w < W; ++w) {
            if (w < warp) at += scratch[w];
            all += scratch[w];
        }
        if (n > 0 && at * hc <= lo && lo < (at + n) * hc) {
            scratch[W + 1] = at;
            scratch[W] = b;
        }
        __syncthreads();
        if (scratch[W] >= 0) break;  // (lo lies in some request)
        before += all;
    }
    it.b = (int)scratch[W];
    it.L = dec_fp8_len(p, it.b);
    it.nt = dec_fp8_tiles(it.L);
    it.next_len = dec_fp8_len(p, it.b + 1);
    const long long off = lo - scratch[W + 1] * hc;
    it.hc = (int)(off / it.nt);
    it.tile = (int)(off - (long long)it.hc * it.nt);
    it.left = (int)(hi - lo);
    if (tid == 0) {
        int *cut = p.cuts + 4 + 4 * c;
        cut[0] = it.b;
        cut[1] = it.hc;
        cut[2] = it.tile;
        cut[3] = it.nt;
    }
    return it;
}

// ------------------------------------------------------------------- TMA

template <class C>
__device__ void dec_fp8_tma_role(const DecFp8Params &p, DecFp8It it, uint8_t *sK, uint8_t *sV, uint32_t bars, Ctl *ctl) {
    const int lane = (int)ptx::lane_id();
    const uint64_t pol = p.chunks > 1 ? ptx::policy_evict_last() : ptx::policy_evict_first();
    const int per_tile = C::BN >> p.bs_log2;  // blocks
    const int blk = lane / C::NCH, ch = lane % C::NCH;
    const bool mine = blk < per_tile;
    const uint32_t dst = (uint32_t)(ch * C::CHUNK_BYTES + (blk << p.bs_log2) * C::ROWB);
    // the physical block of this lane's box: hidden blocks, and entries outside
    // the pool, are a coordinate outside the tensor, which reads zeros
    auto look_up = [&](const DecFp8It &i) -> int {
        const int n = ((i.tile * C::BN) >> p.bs_log2) + blk;
        if (!mine || i.left <= 0 || (n << p.bs_log2) >= i.L) return p.num_blocks;
        const int e = p.block_table[(size_t)i.b * p.max_blocks + n];
        return e >= 0 && e < p.num_blocks ? e : p.num_blocks;
    };
    int n_loaded = 0;
    bool ok = true;
    int phys = look_up(it);
    for (int t = 0; it.left > 0; ++t) {
        const int kvh = it.hc / p.chunks;
        dec_fp8_step(p, it);
        const int next = look_up(it);
        const int ks = t % C::KST, vs = t % C::VST;
        if (!wait_warp_backoff(bar_addr(bars, C::B_KEMPTY + ks), ((t / C::KST) & 1) ^ 1, ctl, 71)) {
            ok = false;
            break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar_addr(bars, C::B_KFULL + ks), C::TILE);
        __syncwarp();
        if (mine)
            ptx::tma_load_4d(ptx::smem_addr(sK + ks * C::TILE) + dst, &p.tm_k, bar_addr(bars, C::B_KFULL + ks),
                             ch * 128, 0, kvh, phys, pol);
        __syncwarp();
        const bool v_ok = wait_warp_backoff(bar_addr(bars, C::B_VEMPTY + vs), ((t / C::VST) & 1) ^ 1, ctl, 72);
        if (!v_ok) {  // this K tile is in flight, its V tile is not
            wait_bar_drain(bar_addr(bars, C::B_KFULL + ks), (t / C::KST) & 1);
            ok = false;
            break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar_addr(bars, C::B_VFULL + vs), C::TILE);
        __syncwarp();
        if (mine)
            ptx::tma_load_4d(ptx::smem_addr(sV + vs * C::TILE) + dst, &p.tm_v, bar_addr(bars, C::B_VFULL + vs),
                             ch * 128, 0, kvh, phys, pol);
        __syncwarp();
        ++n_loaded;
        phys = next;
    }
    if (!ok) {
        for (int t = n_loaded - C::KST > 0 ? n_loaded - C::KST : 0; t < n_loaded; ++t)
            wait_bar_drain(bar_addr(bars, C::B_KFULL + t % C::KST), (t / C::KST) & 1);
        for (int t = n_loaded - C::VST > 0 ? n_loaded - C::VST : 0; t < n_loaded; ++t)
            wait_bar_drain(bar_addr(bars, C::B_VFULL + t % C::VST), (t / C::VST) & 1);
    }
}

// ------------------------------------------------------------------- MMA

template <class C>
__device__ void dec_fp8_mma_role(const DecFp8Params &p, DecFp8It it, uint8_t *sQ, uint8_t *sP, uint8_t *sK, uint8_t *sV,
                                 uint32_t bars, uint32_t tmem, Ctl *ctl) {
    // e4m3 x e4m3 -> fp32 (type code 0 for both); V is M-major (bit 15)
    constexpr uint32_t kIdescS = make_idesc(128, C::N, true, false);
    constexpr uint32_t kIdescO = make_idesc(128, C::N, true, false) | (1u << 15);
    const bool leader = ptx::lane_id() == 0;
    const int n = it.left;
    int unit = 0;
    bool ok = true;
    for (int t = 0; ok && t <= n; ++t) {
        if (t < n) {
            const int ks = t % C::KST, b = t & 1;
            if (t > 0) {
                dec_fp8_step(p, it);
                if (it.tile == 0) ++unit;
            }
            if ((t == 0 || it.tile == 0) &&
                !wait_warp(bar_addr(bars, C::B_QFULL + (unit & 1)), (unit >> 1) & 1, ctl, 73)) {
                ok = false;
                break;
            }
            if (!wait_warp(bar_addr(bars, C::B_KFULL + ks), (t / C::KST) & 1, ctl, 74) ||
                // the softmax has read S of tile t-2 out of this buffer
                (t >= 2 && !wait_warp(bar_addr(bars, C::B_SFREE + b), ((t >> 1) - 1) & 1, ctl, 75))) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            if (leader) {
                const uint32_t ka = ptx::smem_addr(sK + ks * C::TILE);
                const uint32_t qa = ptx::smem_addr(sQ + (unit & 1) * C::Q_BYTES);
#pragma unroll
                for (int kk = 0; kk < C::D / 32; ++kk) {
                    const int ch = (kk * 32) / C::ROWB, in = (kk * 32) % C::ROWB;
                    ptx::mma_ss_f8(tmem + C::S_COL + b * C::N, C::desc(ka + ch * C::CHUNK_BYTES + in),
                                   C::desc(qa + ch * C::QCH + in), kIdescS, kk > 0 ? 1u : 0u);
                }
                ptx::mma_commit(bar_addr(bars, C::B_SFULL + b));
                ptx::mma_commit(bar_addr(bars, C::B_KEMPTY + ks));
            }
            __syncwarp();
        }
        if (t >= 1) {
            const int tp = t - 1, vs = tp % C::VST;
            if (!wait_warp(bar_addr(bars, C::B_VFULL + vs), (tp / C::VST) & 1, ctl, 76) ||
                !wait_warp(bar_addr(bars, C::B_PFULL), tp & 1, ctl, 77)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            if (leader) {
                const uint32_t va = ptx::smem_addr(sV + vs * C::TILE), pa = ptx::smem_addr(sP);
#pragma unroll
                for (int m = 0; m < C::NM; ++m)
#pragma unroll
                    for (int kk = 0; kk < C::BN / 32; ++kk)
                        ptx::mma_ss_f8(tmem + C::O_COL + m * C::N,
                                       C::desc_v(va + m * C::CHUNK_BYTES + kk * 32 * C::ROWB),
                                       smem_desc(pa + kk * 32, 16), kIdescO, kk > 0 ? 1u : 0u);
                ptx::mma_commit(bar_addr(bars, C::B_OFULL));
                ptx::mma_commit(bar_addr(bars, C::B_VEMPTY + vs));
            }
            __syncwarp();
        }
    }
    if (leader) ptx::mma_commit(bar_addr(bars, C::B_DRAIN));
    __syncwarp();
    wait_bar_drain(bar_addr(bars, C::B_DRAIN), 0);
}

// --------------------------------------------------------------- softmax

template <int G>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[G]) {
    if constexpr (G == 1) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(taddr));
    } else if constexpr (G == 2) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
    } else if constexpr (G == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
    } else {
        static_assert(G == 8, "1, 2, 4 or 8 columns");
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    }
}

// The sum of the NP part columns of rows [g0, g0 + G) of this lane.
template <class C, int G>
__device__ __forceinline__ void dec_fp8_read(uint32_t col, int g0, float (&x)[G]) {
    uint32_t part[C::NP][G];
#pragma unroll
    for (int j = 0; j < C::NP; ++j) tmem_ld_cols<G>(col + j * C::RC + g0, part[j]);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < C::NP; ++j) ptx::reg_fence<G>(part[j]);
#pragma unroll
    for (int i = 0; i < G; ++i) {
        float s = __uint_as_float(part[C::NP - 1][i]);
#pragma unroll
        for (int j = C::NP - 2; j >= 0; --j) s = fmaf(s, 0.0625f, __uint_as_float(part[j][i]));
        x[i] = s;
    }
}

// Two values as NP parts: codes[j] holds part j of a in byte 0, of b in byte 1.
template <int NP>
__device__ __forceinline__ void split_e4m3(float a, float b, uint32_t (&codes)[NP]) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(b), "f"(a));
        codes[j] = two;
        if (j + 1 < NP) {
            const float2 back = unpack_e4m3x2(two);
            a = (a - back.x) * 16.f;
            b = (b - back.y) * 16.f;
        }
    }
}

__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Rows of unit (b, hc): the packed rows' first index in [B, H, Sq] and count.
__device__ __forceinline__ size_t dec_fp8_row0(const DecFp8Params &p, int b, int hc, int *rows) {
    const int kvh = hc / p.chunks, chunk = hc - kvh * p.chunks;
    *rows = min(p.rows_per_chunk, p.R - chunk * p.rows_per_chunk);
    return ((size_t)b * p.Hkv + kvh) * p.R + (size_t)chunk * p.rows_per_chunk;
}

// q's parts of a unit into shared memory (K-major, swizzled), its rows' score
// multipliers and last keys.  Each of the four warps takes every fourth row.
// A row is scaled by a power of two so that its largest component is in
// [128, 256); a row with an infinity or NaN becomes NaN codes.
template <class C>
__device__ void dec_fp8_load_q(const DecFp8Params &p, int b, int hc, int L, uint8_t *sQ, float *mul, int *last) {
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    int rows;
    const size_t row0 = dec_fp8_row0(p, b, hc, &rows);
    const int r_first = (hc % p.chunks) * p.rows_per_chunk;
    constexpr int PL = C::D / 32;  // components per lane
    for (int r = warp; r < C::RC; r += 4) {
        float x[PL];
        float top = 0.f;
        bool fine = true;
#pragma unroll
        for (int e = 0; e < PL; e += 2) {
            uint32_t w = 0;
            if (r < rows) w = *reinterpret_cast<const uint32_t *>(p.q + (row0 + r) * C::D + lane * PL + e);
            const float2 f = unpack16<C::kFP16>(w);
            x[e] = f.x;
            x[e + 1] = f.y;
            fine = fine && isfinite(f.x) && isfinite(f.y);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        fine = __all_sync(0xffffffffu, fine);
        // 2^(7 - exponent of top); the exponents stay within fp32's normal range for any 16-bit top
        const int ex = max((int)(__float_as_uint(top) >> 23), 20);  // biased
        const float up = __uint_as_float((uint32_t)min(261 - ex, 254) << 23);
        if (lane == 0) {
            mul[r] = p.scale_log2 / up;
            last[r] = p.mask_kind == kMaskCausal ? L - p.Sq + (r_first + r) % p.Sq : L - 1;
        }
#pragma unroll
        for (int e = 0; e < PL; e += 2) {
            uint32_t codes[C::NP];
            split_e4m3<C::NP>(x[e] * up, x[e + 1] * up, codes);
            const int c = lane * PL + e, ch = c / C::ROWB, in = c % C::ROWB;
#pragma unroll
            for (int j = 0; j < C::NP; ++j) {
                const int n = j * C::RC + r;
                const int swz = C::ROWB == 128 ? n & 7 : (n >> 1) & 3;
                const int at = ch * C::QCH + n * C::ROWB + (((in >> 4) ^ swz) << 4) + (in & 15);
                *reinterpret_cast<uint16_t *>(sQ + at) = (uint16_t)(fine ? codes[j] : 0x7F7Fu);
            }
        }
    }
}

template <class C>
__device__ void dec_fp8_softmax_role(const DecFp8Params &p, DecFp8It it, uint8_t *sQ, uint8_t *sP, uint8_t *sV,
                                     float *sF, uint32_t bars, uint32_t tmem, Ctl *ctl) {
    constexpr int RC = C::RC, G = RC < 8 ? RC : 8;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t p_addr = ptx::smem_addr(sP);
    float *sM = sF + C::F_M + warp * RC;
    if (it.left <= 0) return;

    // what this thread's key of a tile needs of its block: entry, then scales,
    // looked up one and two tiles ahead (`ahead` runs in front of `it`)
    auto entry = [&](const DecFp8It &i) -> int {
        const int key = i.tile * C::BN + tid;
        if (i.left <= 0 || key >= i.L) return -1;
        const int e = p.block_table[(size_t)i.b * p.max_blocks + (key >> p.bs_log2)];
        return e >= 0 && e < p.num_blocks ? e : -1;
    };
    DecFp8It ahead = it;
    int phys = entry(ahead);
    float ks_next = phys >= 0 ? p.k_scale[(size_t)phys * p.Hkv + ahead.hc / p.chunks] : 0.f;
    float vs_next = phys >= 0 ? p.v_scale[(size_t)phys * p.Hkv + ahead.hc / p.chunks] : 0.f;
    if (ahead.left > 0) dec_fp8_step(p, ahead);
    phys = entry(ahead);

    // units are numbered from 0 in this CTA; unit u's q sits in buffer u & 1
    dec_fp8_load_q<C>(p, it.b, it.hc, it.L, sQ, sF + C::F_C, reinterpret_cast<int *>(sF + C::F_LAST));
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(bar_addr(bars, C::B_QFULL));
    ptx::named_bar_sync(3, 128);  // every warp's rows' multipliers and last keys are in place

    float acc[C::NM][RC], l[RC];
    float m_run = -INFINITY;  // lane r: row r's running maximum
    float v_prev = 0.f;       // the tile before: its largest scale / 256, the weight of its O
    bool begun_here = it.tile == 0;
    bool first = true, bad = false;
    int unit = 0;
    for (int t = 0;; ++t) {
        const float *mul = sF + C::F_C + (unit & 1) * RC;
        const int *last = reinterpret_cast<const int *>(sF + C::F_LAST) + (unit & 1) * RC;
        const bool ends = it.tile + 1 == it.nt || it.left == 1;  // the unit, or this CTA's part of it
        if (first) {
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                l[r] = 0.f;
#pragma unroll
                for (int m = 0; m < C::NM; ++m) acc[m][r] = 0.f;
            }
            m_run = -INFINITY;
            // the next unit's q, while this unit's first scores are on their way
            const int to_end = it.nt - it.tile;
            if (it.left > to_end) {
                DecFp8It next = it;
                next.tile = it.nt - 1;
                dec_fp8_step(p, next);
                const int nb = (unit + 1) & 1;
                dec_fp8_load_q<C>(p, next.b, next.hc, next.L, sQ + nb * C::Q_BYTES, sF + C::F_C + nb * RC,
                                  reinterpret_cast<int *>(sF + C::F_LAST) + nb * RC);
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(bar_addr(bars, C::B_QFULL + nb));
            }
        }
        const float ks = ks_next, vs = vs_next;
        ks_next = phys >= 0 ? p.k_scale[(size_t)phys * p.Hkv + ahead.hc / p.chunks] : 0.f;
        vs_next = phys >= 0 ? p.v_scale[(size_t)phys * p.Hkv + ahead.hc / p.chunks] : 0.f;
        if (ahead.left > 0) dec_fp8_step(p, ahead);
        phys = entry(ahead);

        const int b = t & 1, k0 = it.tile * C::BN, key = k0 + tid;
        bad = bad || !wait_warp(bar_addr(bars, p.stall_test && t == 0 ? C::B_NEVER : C::B_SFULL + b), (t >> 1) & 1, ctl, 78);
        float x[RC];
        float *red = sF + C::F_RED + b * 4 * (RC + 1) + warp * (RC + 1);
        if (!bad) {
            ptx::tc_fence_after();
#pragma unroll
            for (int g = 0; g < RC; g += G) {
                float s[G];
                dec_fp8_read<C, G>(lane_base + C::S_COL + b * C::N, g, s);
#pragma unroll
                for (int i = 0; i < G; ++i) x[g + i] = s[i] * (mul[g + i] * ks);
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar_addr(bars, C::B_SFREE + b));
            // hidden keys: past the row's last (a select, so nothing of theirs leaks)
            const int seen_by_all = p.mask_kind == kMaskCausal ? it.L - p.Sq : it.L - 1;
            if (k0 + C::BN - 1 > seen_by_all) {
#pragma unroll
                for (int r = 0; r < RC; ++r)
                    if (key > last[r]) x[r] = -INFINITY;
            }
            float mine = -INFINITY;
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                float top = x[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (lane == r) mine = top;
            }
            float vtop = fabsf(vs);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, o));
            if (lane < RC) red[lane] = mine;
            if (lane == 0) red[RC] = vtop;
        }
        // (a warp whose wait ran out still comes here, and all leave together)
        if (ptx::named_bar_any(1, 128, bad)) return;
        const float *all = sF + C::F_RED + b * 4 * (RC + 1);
        const float vtop = fmaxf(fmaxf(all[RC], all[2 * RC + 1]), fmaxf(all[3 * RC + 2], all[4 * RC + 3]));
        float2 *ab = reinterpret_cast<float2 *>(sF + C::F_AB) + (b * 4 + warp) * RC;
        if (lane < RC) {
            const float m_tile = fmaxf(fmaxf(all[lane], all[RC + 1 + lane]), fmaxf(all[2 * RC + 2 + lane], all[3 * RC + 3 + lane]));
            const float m_new = fmaxf(m_run, m_tile), m_use = m_new == -INFINITY ? 0.f : m_new;
            sM[lane] = m_tile == -INFINITY ? 0.f : m_tile;
            ab[lane] = make_float2(ptx::ex2_approx(m_run - m_use), m_tile == -INFINITY ? 0.f : ptx::ex2_approx(m_tile - m_use));
            m_run = m_new;
        }
        __syncwarp();
        // O of the tile before (of this unit): P and O are free again after it
        if (!first) {
            bad = !wait_warp(bar_addr(bars, C::B_OFULL), (t - 1) & 1, ctl, 79);
            if (!bad) {
                ptx::tc_fence_after();
                const float2 *abp = reinterpret_cast<const float2 *>(sF + C::F_AB) + ((b ^ 1) * 4 + warp) * RC;
#pragma unroll
                for (int m = 0; m < C::NM; ++m)
#pragma unroll
                    for (int g = 0; g < RC; g += G) {
                        float o[G];
                        dec_fp8_read<C, G>(lane_base + C::O_COL + m * C::N, g, o);
#pragma unroll
                        for (int i = 0; i < G; ++i) acc[m][g + i] = fmaf(acc[m][g + i], abp[g + i].x, o[i] * (abp[g + i].y * v_prev));
                    }
                ptx::tc_fence_before();
            }
        }
        v_prev = vtop * 0.00390625f;
        if (!bad) {
            // weights: of the sum in fp32, of V (times the block's scale over
            // the tile's largest, times 256) as parts
            const float share = vtop > 0.f ? vs / vtop * 256.f : 0.f;
#pragma unroll
            for (int r = 0; r < RC; r += 2) {
                const float p0 = ptx::ex2_approx(x[r] - sM[r]);
                const float2 w0 = ab[r];
                l[r] = fmaf(l[r], w0.x, p0 * w0.y);
                float p1 = 0.f;
                if (r + 1 < RC) {
                    p1 = ptx::ex2_approx(x[(r + 1) % RC] - sM[(r + 1) % RC]);
                    const float2 w1 = ab[(r + 1) % RC];
                    l[(r + 1) % RC] = fmaf(l[(r + 1) % RC], w1.x, p1 * w1.y);
                }
                uint32_t codes[C::NP];
                split_e4m3<C::NP>(p0 * share, p1 * share, codes);
#pragma unroll
                for (int j = 0; j < C::NP; ++j) {
                    const int n = j * RC + r;
                    st_shared_u8(p_addr + n * 128 + (((tid >> 4) ^ (n & 7)) << 4) + (tid & 15), codes[j]);
                    if (r + 1 < RC)
                        st_shared_u8(p_addr + (n + 1) * 128 + (((tid >> 4) ^ ((n + 1) & 7)) << 4) + (tid & 15), codes[j] >> 8);
                }
            }
            if (k0 + C::BN > it.L && (it.L & ((1 << p.bs_log2) - 1)) != 0 && key >= it.L) {
                // a row of V past the request's keys meets weight 0, but junk (NaN)
                // in it would not vanish: zero it
                const int slot = t % C::VST;
                bad = !wait_bar(bar_addr(bars, C::B_VFULL + slot), (t / C::VST) & 1, ctl, 80);
#pragma unroll
                for (int ch = 0; ch < C::NCH; ++ch)
#pragma unroll
                    for (int c = 0; c < C::ROWB; c += 16)
                        ptx::st_shared_v4(ptx::smem_addr(sV + slot * C::TILE + ch * C::CHUNK_BYTES + tid * C::ROWB + c), 0u,
                                          0u, 0u, 0u);
            }
            bad = __any_sync(0xffffffffu, bad);
        }
        ptx::fence_proxy_async_smem();
        if (!bad) ptx::mbar_arrive(bar_addr(bars, C::B_PFULL));
        first = false;

        if (ends) {
            // the unit's last O, its sums, and the rows out
            bad = bad || !wait_warp(bar_addr(bars, C::B_OFULL), t & 1, ctl, 81);
            if (!bad) {
                ptx::tc_fence_after();
#pragma unroll
                for (int m = 0; m < C::NM; ++m)
#pragma unroll
                    for (int g = 0; g < RC; g += G) {
                        float o[G];
                        dec_fp8_read<C, G>(lane_base + C::O_COL + m * C::N, g, o);
#pragma unroll
                        for (int i = 0; i < G; ++i) acc[m][g + i] = fmaf(acc[m][g + i], ab[g + i].x, o[i] * (ab[g + i].y * v_prev));
                    }
                ptx::tc_fence_before();
            }
            float mine = 0.f;
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                float s = l[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == r) mine = s;
            }
            float *sL = sF + C::F_L;
            if (lane < RC) sL[warp * RC + lane] = mine;
            if (ptx::named_bar_any(2, 128, bad)) return;
            int rows;
            const size_t row0 = dec_fp8_row0(p, it.b, it.hc, &rows);
            const bool whole = begun_here && it.tile + 1 == it.nt;
            const size_t slot = 2 * (size_t)blockIdx.x + (begun_here ? 1 : 0);
            if (warp == 0 && lane < RC && lane < rows) {
                const float sum = (sL[lane] + sL[RC + lane]) + (sL[2 * RC + lane] + sL[3 * RC + lane]);
                // (a NaN sum is no empty row)
                const float lse2 = sum == 0.f ? -INFINITY : m_run + __log2f(sum);
                if (whole) p.lse[row0 + lane] = lse2 * kLn2;
                else p.part_lse[slot * RC + lane] = lse2;
            }
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                if (r >= rows) break;
                const float sum = (sL[r] + sL[RC + r]) + (sL[2 * RC + r] + sL[3 * RC + r]);
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int m = 0; m < C::NM; ++m) {
                    const int c = m * 128 + tid;
                    if (c >= C::D) continue;
                    const float o = acc[m][r] * inv;
                    if (whole)
                        static_cast<uint16_t *>(p.o)[(row0 + r) * C::D + c] = (uint16_t)pack2b<C::kFP16>(o, 0.f);
                    else
                        p.part_o[(slot * RC + r) * C::D + c] = o;
                }
            }
            if (it.left == 1) return;
            first = true;
            begun_here = true;
            ++unit;
            // sL is written again only behind the next tile's barrier
        }
        dec_fp8_step(p, it);
    }
}

template <class C>
__global__ void __launch_bounds__(C::NUM_THREADS, C::CTAS_PER_SM)
    fa_decode_fp8_kernel(const __grid_constant__ DecFp8Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sK = smem;
    uint8_t *sV = sK + C::KST * C::TILE;
    uint8_t *sQ = sV + C::VST * C::TILE;
    uint8_t *sP = sQ + 2 * C::Q_BYTES;
    uint64_t *bar_mem = reinterpret_cast<uint64_t *>(sP + C::P_BYTES);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bar_mem + C::NUM_BARS);
    Ctl *ctl = reinterpret_cast<Ctl *>(tmem_holder + 2);
    float *sF = reinterpret_cast<float *>(ctl + 2);
    const uint32_t bars = ptx::smem_addr(bar_mem);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::KST; ++s) {
            ptx::mbar_init(bar_addr(bars, C::B_KFULL + s), 1);
            ptx::mbar_init(bar_addr(bars, C::B_KEMPTY + s), 1);
        }
        for (int s = 0; s < C::VST; ++s) {
            ptx::mbar_init(bar_addr(bars, C::B_VFULL + s), 1);
            ptx::mbar_init(bar_addr(bars, C::B_VEMPTY + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar_addr(bars, C::B_QFULL + b), 128);
            ptx::mbar_init(bar_addr(bars, C::B_SFULL + b), 1);
            ptx::mbar_init(bar_addr(bars, C::B_SFREE + b), 128);
        }
        ptx::mbar_init(bar_addr(bars, C::B_PFULL), 128);
        ptx::mbar_init(bar_addr(bars, C::B_OFULL), 1);
        ptx::mbar_init(bar_addr(bars, C::B_DRAIN), 1);
        ptx::mbar_init(bar_addr(bars, C::B_NEVER), 1);
        ctl->abort = 0;
        ctl->limit_ns = p.wait_limit_ns;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == C::MMA_WARP) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_holder), C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    if (warp == C::TMA_WARP && ptx::lane_id() == 0) {
        ptx::prefetch_tensormap(&p.tm_k);
        ptx::prefetch_tensormap(&p.tm_v);
    }
    // (the small arrays are not yet in use: the prefix sums borrow their first bytes)
    const DecFp8It it = dec_fp8_begin<C::NUM_THREADS>(p, reinterpret_cast<long long *>(sF));
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp < 4) {
        dec_fp8_softmax_role<C>(p, it, sQ, sP, sV, sF, bars, tmem, ctl);
    } else if (warp == C::MMA_WARP) {
        dec_fp8_mma_role<C>(p, it, sQ, sP, sK, sV, bars, tmem, ctl);
    } else {
        dec_fp8_tma_role<C>(p, it, sK, sV, bars, ctl);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Merges the units that a boundary between two CTAs cuts.  CTA x stands for
// the boundary in front of CTA c = x + 1 of the attention; the first boundary
// inside a unit merges it: the partial of CTA c - 1 (slot 2c - 1), then those of
// c, c + 1, ... (slots 2c, 2c + 2, ...) up to the unit's end.  A warp per row.
template <int D, bool kFP16, int RC>
__global__ void __launch_bounds__(128) fa_decode_fp8_combine_kernel(const __grid_constant__ DecFp8Params p, int grid) {
    const int c = (int)blockIdx.x + 1, lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const long long total = *reinterpret_cast<const long long *>(p.cuts);
    const long long G = min((long long)grid, total);
    if (c >= G) return;
    const int *cut = p.cuts + 4 + 4 * c;
    if (cut[2] == 0) return;  // between two units
    const long long begin = c * total / G - cut[2], end = begin + cut[3];
    if ((c - 1) * total / G > begin) return;  // an earlier boundary merges this unit
    int n = 1;                                // partials behind the first
    while (c + n < G && (c + n) * total / G < end) ++n;
    int rows;
    const size_t row0 = dec_fp8_row0(p, cut[0], cut[1], &rows);
    constexpr int PER = D / 32;
    for (int r = warp; r < rows; r += 4) {
        float top = -INFINITY;
        bool nan = false;
        for (int i = lane; i <= n; i += 32) {
            const float v = p.part_lse[(size_t)(i == 0 ? 2 * c - 1 : 2 * (c + i - 1)) * RC + r];
            top = fmaxf(top, v);
            nan = nan || isnan(v);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (__any_sync(0xffffffffu, nan)) top = NAN;
        float acc[PER], sum = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = 0.f;
        if (top != -INFINITY) {
            for (int i = 0; i <= n; ++i) {
                const size_t slot = (size_t)(i == 0 ? 2 * c - 1 : 2 * (c + i - 1)) * RC + r;
                const float w = ptx::ex2_approx(p.part_lse[slot] - top);
                sum += w;
                const float *src = p.part_o + slot * D + lane * PER;
#pragma unroll
                for (int e = 0; e < PER; e += 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(src + e);
                    acc[e] = fmaf(w, v.x, acc[e]);
                    acc[e + 1] = fmaf(w, v.y, acc[e + 1]);
                }
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + (row0 + r) * D + lane * PER);
#pragma unroll
        for (int e = 0; e < PER; e += 2) dst[e / 2] = pack2b<kFP16>(acc[e] * inv, acc[e + 1] * inv);
        if (lane == 0) p.lse[row0 + r] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
    }
}

}  // namespace fa
