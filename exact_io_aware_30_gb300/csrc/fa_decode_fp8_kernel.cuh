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
//     x = x1 + x2 / 16 (+ x3 / 256 + x4 / 4096), each part the rounding of what
//     the parts before it left, and the parts are columns of N beside each
//     other; their products are summed in fp32 as they are read back.  Two
//     parts hold the 8 significant bits of bf16, three the 11 of fp16, so S is
//     exact up to fp32 sums (but for components far below their row's largest:
//     see dec_fp8_put_q), and a weight is rounded much as a 16-bit P would be: to
//     fp16, 2^-11 of itself, and with two parts by 2^-8 more.  Up to four rows a
//     fourth part fits into the 16 columns that N has at least: q keeps all
//     bits there and a weight 16 (2^-16 of itself), since a few rows'
//     weights are not rounded to 16 bits over the 16-bit cache either (4 rows, 606
//     MB: 97.8 us with two parts, 98.2 with four; with more rows the columns and stores
//     cost more: 8 rows at d 128 92 / 96 us, at d 64 64 / 74, 16 rows 115 / 133).  Weights
//     are taken relative to the largest score of their own step of 128 or 256
//     keys and the steps' outputs are rescaled in fp32, so that what is below
//     the parts' range (2^-22, 2^-26, 2^-30 of the step's largest with two, three,
//     four parts) is never a large share of a row.  What P V takes is a weight
//     times its block's V scale, relative to the step's largest scale; in steps
//     whose scales are far apart (V_RANGE) relative to the row's own largest
//     product, which costs an exchange more (8 rows at d 128 88 -> 93 us, 32 rows 168
//     -> 185 where every step is such a one).
//
// Work split.  The work is a line of 128-key tiles: request by request, K/V
// head by K/V head, chunk of rows by chunk of rows (a unit), tile by tile.
// CTA c of G takes tiles [c T / G, (c + 1) T / G) of the T there are, so every
// CTA has the same work whatever the lengths, and its pipelines run on from
// unit to unit.  A unit that lies in one CTA is written out by it; one that is
// cut leaves a normalised partial row and its lse per CTA, and
// fa_decode_fp8_combine_kernel (a CTA per cut) merges them in order.  Where units
// are short, a CTA takes whole ones instead, and there is nothing to merge.
//
// One CTA:
//   softmax warpgroups, one per eight rows of the unit.  Thread = key for S^T
//     (TMEM lane), = column of d for O^T; O is kept in registers, rescaled per
//     step of one or two tiles.  (All rows in one warpgroup, 16 or 32 to a thread, left the SM with
//     eight warps in long dependent chains: 115 and 240 us where 8 rows take 94,
//     64 requests x 8 K/V heads x 4,096 tokens at d 128.)
//   an MMA warp: S^T of step s + 1 before O^T of step s;
//   a TMA warp: a lane per block of the tile, K and V rings.
//
// Measured: 128 requests x 40 heads, up to 2,048 tokens, fp16: 247 us (6.2 TB/s,
// 91 % of a copy); 64 requests, 32 heads on 8, up to 8,192, bf16: 97 us (92 %).  64
// requests x 8 K/V heads, full lengths, bf16, with 1 / 4 / 8 rows: 52 / 63 / 61 us at d
// 64 (269 MB), 87 / 90 / 88 at d 128 and 83 / 84 / 87 at d 256 (537 MB); 16, 24, 32 rows
// at d 128 108, 130, 167.
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
    int whole;               // units are not cut: a CTA takes whole ones, and part_o, part_lse and cuts are unused
    int *cuts;               // [4 + 5 G]: total tiles (64-bit), then per CTA its first unit: b, head, chunk, tile, tiles
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
    static constexpr int RW = RC < 8 ? RC : 8;          // rows of one softmax warpgroup
    static constexpr int NWG = RC / RW;                 // softmax warpgroups, each with all keys of a tile
    static_assert(RW * NWG == RC, "whole warpgroups of rows");
    static constexpr int NP = RC <= 4 ? 4 : kFP16 ? 3 : 2;  // e4m3 parts of q and of the weights
    static constexpr int N = (RC * NP + 15) / 16 * 16;  // columns: part-major, then rows
    static constexpr int BN = 128;                      // keys per tile
    static constexpr int ROWB = D < 128 ? D : 128;      // bytes of a row in one column chunk
    static constexpr int NCH = D / ROWB;                // column chunks
    static constexpr int NM = D == 256 ? 2 : 1;         // M blocks of O^T
    static constexpr int TILE = BN * D;                 // bytes of a K or V tile
    static constexpr int CHUNK_BYTES = BN * ROWB;
    static constexpr int Q_BYTES = N * D;               // one buffer of q's parts
    static constexpr int QCH = N * ROWB;
    static constexpr int P_BYTES = N * 128;             // the weights' parts of a tile
    // Tensor memory: two S buffers of KPT tiles, two O buffers of NM M blocks.
    static constexpr int cols(int kpt) { return (2 * kpt + 2 * NM) * N; }
    static constexpr int ctas(int kpt) {
        return D == 64 && RC <= 4 ? 3 : D <= 128 && NWG == 1 ? 2 : 1;
    }
    static constexpr int budget(int kpt) { return ctas(kpt) == 3 ? 75 * 1024 : ctas(kpt) == 2 ? 113 * 1024 : 226 * 1024; }
    static constexpr int MMA_WARP = 4 * NWG;
    static constexpr int TMA_WARP = 4 * NWG + 1;
    static constexpr int NUM_THREADS = 32 * (TMA_WARP + 1);
    // How far the V scales of a step may be apart to be taken relative to the
    // largest of them (else each row has a reference of its own): what is then
    // lost is within 2^-20 of the row's largest weight times scale.
    static constexpr float V_RANGE = NP == 2 ? 4.f : NP == 3 ? 64.f : 1024.f;
    // small arrays of a warpgroup, in floats, rows padded to a multiple of four
    static constexpr int RP = (RW + 3) / 4 * 4;
    static constexpr int F_M = 0;                    // [4 warps] the tile's maxima
    static constexpr int F_B = F_M + 4 * RP;         // [4 warps] 2^(tile's maximum - running maximum)
    static constexpr int F_A = F_B + 4 * RP;         // [2][4 warps] rescale of what came before the tile
    static constexpr int F_V = F_A + 8 * RP;         // [2][4 warps] weight of the tile's O
    static constexpr int F_C = F_V + 8 * RP;         // [2] score multipliers
    static constexpr int F_LAST = F_C + 2 * RP;      // [2] last key the row sees (int)
    static constexpr int F_L = F_LAST + 2 * RP;      // [4 warps] sums
    static constexpr int F_N = F_L + 4 * RP;         // [4 warps] what a row's weights times V scales are multiplied by
    static constexpr int F_TOP = F_L;                // [4 warps] largest weight times |vs|
    static constexpr int F_RED = F_N + 4 * RP;       // [2][4 warps][RW + 2] tile maxima, largest |vs|, smallest but 0 negated
    static constexpr int F_WG = (F_RED + 2 * 4 * (RW + 2) + 3) / 4 * 4;
    static constexpr int F_NUM = NWG * F_WG;
    static constexpr int slots(int kpt) {
        return (budget(kpt) - (1024 + 2 * Q_BYTES + 2 * kpt * P_BYTES + F_NUM * 4 + 512)) / TILE;
    }
    // Tiles per step of the softmax: two where tensor memory holds them and the
    // rings keep two steps.  Most of a step's time is a chain of waits,
    // exchanges and short loads that does not grow with its keys (d 64, 8 rows:
    // 84 -> 66 us; d 128, 24 rows: 193 -> 145 us); with shorter rings the
    // second step's copies start late (d 128, 1 row: 92 -> 107 us).  That is two for
    // 8 to 24 rows at d 64, 16 and 24 at d 128, and 32 there in bf16.
    static constexpr int KPT = cols(2) <= 512 / ctas(2) && slots(2) >= 8 ? 2 : 1;
    static constexpr int COLS = cols(KPT);
    static constexpr int CTAS_PER_SM = ctas(KPT);
    static constexpr uint32_t TMEM_COLS = COLS <= 32 ? 32 : COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static constexpr uint32_t S_COL = 0;
    static constexpr uint32_t O_COL = 2 * KPT * N;
    static constexpr int SLOTS = slots(KPT) < 12 ? slots(KPT) : 12;
    static constexpr int VST = (SLOTS + 1) / 2;
    static constexpr int KST = SLOTS / 2;
    static constexpr int B_KFULL = 0;
    static constexpr int B_KEMPTY = B_KFULL + KST;
    static constexpr int B_VFULL = B_KEMPTY + KST;
    static constexpr int B_VEMPTY = B_VFULL + VST;
    static constexpr int B_QFULL = B_VEMPTY + VST;  // [2]
    static constexpr int B_SFULL = B_QFULL + 2;     // [2]
    static constexpr int B_SFREE = B_SFULL + 2;     // [2]
    static constexpr int B_PFULL = B_SFREE + 2;     // [2]
    static constexpr int B_OFULL = B_PFULL + 2;     // [2]
    static constexpr int B_DRAIN = B_OFULL + 2;
    static constexpr int B_NEVER = B_DRAIN + 1;     // no arrivals (the stall test's wait)
    static constexpr int NUM_BARS = B_NEVER + 1;
    static constexpr int SMEM_TILES = 2 * Q_BYTES + 2 * KPT * P_BYTES + (KST + VST) * TILE;
    static constexpr int SMEM_BYTES = 1024 + SMEM_TILES + F_NUM * 4 + NUM_BARS * 8 + 64;
    static_assert(KST >= 2 && VST >= 2, "rings of at least two tiles");
    static_assert(SMEM_BYTES <= budget(KPT) && SMEM_BYTES <= 232448, "shared memory overflow");
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
    int b, kvh, chunk, tile;  // request, K/V head, chunk of rows, tile of the unit
    int L, nt;                // the request's length and tiles
    int next_len;             // the next request's length, loaded ahead
    int left;                 // tiles left, this one included
};

__device__ __forceinline__ int dec_fp8_tiles(int L) { return max((L + 127) >> 7, 1); }

__device__ __forceinline__ int dec_fp8_len(const DecFp8Params &p, int b) {
    return b < p.B ? min(max(p.seq_lens[b], 0), p.max_seq_len) : 0;
}

__device__ __forceinline__ void dec_fp8_step(const DecFp8Params &p, DecFp8It &it) {
    --it.left;
    if (++it.tile < it.nt) return;
    it.tile = 0;
    if (++it.chunk < p.chunks) return;
    it.chunk = 0;
    if (++it.kvh < p.Hkv) return;
    it.kvh = 0;
    ++it.b;
    it.L = it.next_len;
    it.nt = dec_fp8_tiles(it.L);
    it.next_len = dec_fp8_len(p, it.b + 1);
}

// Tiles of one step of the softmax: KPT, or what is left of the unit or the CTA's share.
template <class C>
__device__ __forceinline__ int dec_fp8_span(const DecFp8It &it) {
    return C::KPT == 1 ? 1 : min(C::KPT, min(it.nt - it.tile, it.left));
}

template <class C>
__device__ __forceinline__ void dec_fp8_steps(const DecFp8Params &p, DecFp8It &it, int span) {
    it.tile += span - 1;
    it.left -= span - 1;
    dec_fp8_step(p, it);
}

// The first tile of the unit behind this one's.  (Its next_len is not loaded
// where the step does not need it: no use of the result waits for that.)
__device__ __forceinline__ DecFp8It dec_fp8_next_unit(const DecFp8Params &p, DecFp8It it) {
    it.left -= it.nt - 1 - it.tile;
    it.tile = it.nt - 1;
    dec_fp8_step(p, it);
    return it;
}

// Where this CTA's tiles begin: prefix sums over the requests' tiles, by all
// threads of the CTA.  `scratch` holds THREADS / 32 + 5 long longs.  Up to
// THREADS requests take one load each and two barriers.
template <int THREADS>
__device__ DecFp8It dec_fp8_begin(const DecFp8Params &p, long long *scratch) {
    constexpr int W = THREADS / 32;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long hc = (long long)p.Hkv * p.chunks, c = blockIdx.x;
    DecFp8It it;
    it.b = it.kvh = it.chunk = it.tile = it.L = it.nt = it.next_len = it.left = 0;
    if (p.whole) {  // an even share of the units (there are at least as many as CTAs)
        const long long units = p.B * hc, u0 = c * units / gridDim.x, u1 = (c + 1) * units / gridDim.x;
        const int b0 = (int)(u0 / hc), b1 = (int)((u1 - 1) / hc);
        int sum = 0;
        for (int b = b0 + lane; b <= b1; b += 32)
            sum += (int)(min(u1, (b + 1) * hc) - max(u0, b * hc)) * dec_fp8_tiles(dec_fp8_len(p, b));
        it.left = __reduce_add_sync(0xffffffffu, sum);
        it.b = b0;
        it.L = dec_fp8_len(p, b0);
        it.nt = dec_fp8_tiles(it.L);
        it.next_len = dec_fp8_len(p, b0 + 1);
        const int unit = (int)(u0 - b0 * hc);
        it.kvh = unit / p.chunks;
        it.chunk = unit - it.kvh * p.chunks;
        return it;
    }
    long long total = -1, G = 0, lo = 0, hi = 0;
    if (p.B > THREADS) {  // the sum first; then the requests are gone through again
        int sum = 0;
        for (int b = tid; b < p.B; b += THREADS) sum += dec_fp8_tiles(dec_fp8_len(p, b));
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) scratch[warp] = sum;
        __syncthreads();
        total = 0;
        for (int w = 0; w < W; ++w) total += scratch[w];
        total *= hc;
        __syncthreads();
    }
    long long before = 0;  // tiles of the requests before this group of THREADS, per K/V head and chunk
    for (int b0 = 0;; b0 += THREADS) {
        const int b = b0 + tid, L = dec_fp8_len(p, b);
        const int n = b < p.B ? dec_fp8_tiles(L) : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (tid == 0) scratch[W] = -1;
        if (lane == 31) scratch[warp] = inc;
        __syncthreads();
        long long at = before + inc - n, all = 0;
        for (int w = 0; w < W; ++w) {
            if (w < warp) at += scratch[w];
            all += scratch[w];
        }
        if (total < 0) total = all * hc;
        if (b0 == 0) {
            G = min((long long)gridDim.x, total);
            if (c == 0 && tid == 0) *reinterpret_cast<long long *>(p.cuts) = total;
            if (c >= G) return it;
            lo = c * total / G;
            hi = (c + 1) * total / G;
        }
        if (n > 0 && at * hc <= lo && lo < (at + n) * hc) {
            scratch[W] = b;
            scratch[W + 1] = at;
            scratch[W + 2] = L;
            scratch[W + 3] = dec_fp8_len(p, b + 1);
        }
        __syncthreads();
        if (scratch[W] >= 0) break;  // (lo lies in some request)
        before += all;
        __syncthreads();
    }
    it.b = (int)scratch[W];
    it.L = (int)scratch[W + 2];
    it.nt = dec_fp8_tiles(it.L);
    it.next_len = (int)scratch[W + 3];
    const long long off = lo - scratch[W + 1] * hc;
    const int unit = (int)(off / it.nt);
    it.tile = (int)(off - (long long)unit * it.nt);
    it.kvh = unit / p.chunks;
    it.chunk = unit - it.kvh * p.chunks;
    it.left = (int)(hi - lo);
    if (tid == 0) {
        int *cut = p.cuts + 4 + 5 * c;
        cut[0] = it.b;
        cut[1] = it.kvh;
        cut[2] = it.chunk;
        cut[3] = it.tile;
        cut[4] = it.nt;
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
        const int kvh = it.kvh;
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
    int unit = 0, t = 0;  // t: tiles of this CTA so far, as the rings count them
    int span_before = 0, t_before = 0;
    bool ok = true;
    for (int step = 0; ok; ++step) {
        const int b = step & 1, span = it.left > 0 ? dec_fp8_span<C>(it) : 0;
        if (span > 0) {
            if ((step == 0 || it.tile == 0) &&
                !wait_warp(bar_addr(bars, C::B_QFULL + (unit & 1)), (unit >> 1) & 1, ctl, 73)) {
                ok = false;
                break;
            }
            // the softmax has read S of step - 2 out of this buffer
            if (step >= 2 && !wait_warp(bar_addr(bars, C::B_SFREE + b), ((step >> 1) - 1) & 1, ctl, 75)) {
                ok = false;
                break;
            }
            for (int j = 0; j < span; ++j) {
                const int ks = (t + j) % C::KST;
                ok = wait_warp(bar_addr(bars, C::B_KFULL + ks), ((t + j) / C::KST) & 1, ctl, 74);
                if (!ok) break;
                ptx::tc_fence_after();
                if (leader) {
                    const uint32_t ka = ptx::smem_addr(sK + ks * C::TILE);
                    const uint32_t qa = ptx::smem_addr(sQ + (unit & 1) * C::Q_BYTES);
#pragma unroll
                    for (int kk = 0; kk < C::D / 32; ++kk) {
                        const int ch = (kk * 32) / C::ROWB, in = (kk * 32) % C::ROWB;
                        ptx::mma_ss_f8(tmem + C::S_COL + (b * C::KPT + j) * C::N, C::desc(ka + ch * C::CHUNK_BYTES + in),
                                       C::desc(qa + ch * C::QCH + in), kIdescS, kk > 0 ? 1u : 0u);
                    }
                    if (j + 1 == span) ptx::mma_commit(bar_addr(bars, C::B_SFULL + b));
                    ptx::mma_commit(bar_addr(bars, C::B_KEMPTY + ks));
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        if (step >= 1) {
            const int pb = b ^ 1;  // the step before
            if (!wait_warp(bar_addr(bars, C::B_PFULL + pb), ((step - 1) >> 1) & 1, ctl, 77)) {
                ok = false;
                break;
            }
            for (int j = 0; j < span_before; ++j) {
                const int vs = (t_before + j) % C::VST;
                ok = wait_warp(bar_addr(bars, C::B_VFULL + vs), ((t_before + j) / C::VST) & 1, ctl, 76);
                if (!ok) break;
                ptx::tc_fence_after();
                if (leader) {
                    const uint32_t va = ptx::smem_addr(sV + vs * C::TILE);
                    const uint32_t pa = ptx::smem_addr(sP + (pb * C::KPT + j) * C::P_BYTES);
                    const uint32_t o_col = tmem + C::O_COL + pb * C::NM * C::N;
#pragma unroll
                    for (int m = 0; m < C::NM; ++m)
#pragma unroll
                        for (int kk = 0; kk < C::BN / 32; ++kk)
                            ptx::mma_ss_f8(o_col + m * C::N, C::desc_v(va + m * C::CHUNK_BYTES + kk * 32 * C::ROWB),
                                           smem_desc(pa + kk * 32, 16), kIdescO, (j > 0 || kk > 0) ? 1u : 0u);
                    if (j + 1 == span_before) ptx::mma_commit(bar_addr(bars, C::B_OFULL + pb));
                    ptx::mma_commit(bar_addr(bars, C::B_VEMPTY + vs));
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        if (span == 0) break;
        t_before = t;
        span_before = span;
        t += span;
        dec_fp8_steps<C>(p, it, span);
        if (it.tile == 0) ++unit;  // (one more than there are behind the last)
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
    } else if constexpr (G == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
    } else {
        static_assert(G == 8, "1, 4 or 8 columns");
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    }
}

// The sums of the NP part columns of G rows of this lane, `col` the first part
// of the first of them.
template <class C, int G>
__device__ __forceinline__ void dec_fp8_read(uint32_t col, float (&x)[G]) {
    uint32_t part[C::NP][G];
#pragma unroll
    for (int j = 0; j < C::NP; ++j) tmem_ld_cols<G>(col + j * C::RC, part[j]);
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

// Two values (at most 256) as NP parts: codes[j] holds part j of a in byte 0,
// of b in byte 1.  They are rounded to fp16 first, whose 11 bits three parts
// hold, and every later step is exact in fp16: what a part leaves is at most
// half a step of it, 2^-4 of the value before.  A fourth part holds what those
// three and the rounding to fp16 left.
template <int NP>
__device__ __forceinline__ void split_e4m3(float a, float b, uint32_t (&codes)[NP]) {
    const __half2 k16 = __half2half2(__ushort_as_half(0x4C00));  // 16
    const uint32_t w = ptx::pack_f16x2(a, b);
    __half2 h = *reinterpret_cast<const __half2 *>(&w);
    float2 lost = make_float2(0.f, 0.f);
    if constexpr (NP == 4) {
        const float2 r = __half22float2(h);
        lost = make_float2(a - r.x, b - r.y);  // (exact)
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        uint16_t two;
        if (j == 3) {
            const float2 r = __half22float2(h);
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(two) : "f"(fmaf(lost.y, 4096.f, r.y)), "f"(fmaf(lost.x, 4096.f, r.x)));
            codes[j] = two;
            break;
        }
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(two) : "r"(*reinterpret_cast<const uint32_t *>(&h)));
        codes[j] = two;
        if (j + 1 < NP) {
            uint32_t back;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(two));
            h = __hmul2(__hsub2(h, *reinterpret_cast<const __half2 *>(&back)), k16);
        }
    }
}

// The largest of the warp's values (NaN only if all are), in every lane.
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// r consecutive floats of shared memory (16-byte aligned for r >= 4).
template <int R>
__device__ __forceinline__ void lds_row(const float *src, float (&dst)[R]) {
    if constexpr (R % 4 == 0) {
#pragma unroll
        for (int i = 0; i < R; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src + i);
            dst[i] = v.x;
            dst[i + 1] = v.y;
            dst[i + 2] = v.z;
            dst[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) dst[i] = src[i];
    }
}

__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
    // (no memory clobber: the loads of later rows may pass; the proxy fence
    // behind the last store is a volatile asm as well and stays behind it)
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v));
}

// Rows of a unit: the packed rows' first index in [B, H, Sq] and count.
__device__ __forceinline__ size_t dec_fp8_row0(const DecFp8Params &p, int b, int kvh, int chunk, int *rows) {
    *rows = min(p.rows_per_chunk, p.R - chunk * p.rows_per_chunk);
    return ((size_t)b * p.Hkv + kvh) * p.R + (size_t)chunk * p.rows_per_chunk;
}

// A warpgroup's q rows of a unit, 16-bit, each of its four warps every fourth
// row, a lane D / 32 adjacent components.
template <class C>
struct DecFp8Q {
    static constexpr int PL = C::D / 32;        // components per lane
    static constexpr int NR = (C::RW + 3) / 4;  // rows per warp
    uint32_t raw[NR][PL / 2];
};

template <class C>
__device__ __forceinline__ void dec_fp8_load_q(const DecFp8Params &p, const DecFp8It &u, DecFp8Q<C> &q) {
    constexpr int PL = DecFp8Q<C>::PL;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5 & 3, wg = (int)threadIdx.x >> 7;
    int rows;
    const size_t row0 = dec_fp8_row0(p, u.b, u.kvh, u.chunk, &rows);
#pragma unroll
    for (int i = 0; i < DecFp8Q<C>::NR; ++i) {
        const int r = wg * C::RW + warp + 4 * i;
        const uint16_t *src = p.q + (row0 + (r < rows ? r : 0)) * C::D + lane * PL;
        if constexpr (PL == 8) {
            const uint4 w = *reinterpret_cast<const uint4 *>(src);
            q.raw[i][0] = w.x, q.raw[i][1] = w.y, q.raw[i][2] = w.z, q.raw[i][3] = w.w;
        } else if constexpr (PL == 4) {
            const uint2 w = *reinterpret_cast<const uint2 *>(src);
            q.raw[i][0] = w.x, q.raw[i][1] = w.y;
        } else {
            q.raw[i][0] = *reinterpret_cast<const uint32_t *>(src);
        }
    }
}

// q's parts into shared memory (K-major, swizzled), its rows' score multipliers
// and last keys.  A row is scaled by a power of two so that its largest
// component is in [128, 256).  Components of at least 2^-13 (two parts, bf16) or
// 2^-14 (three, fp16) of the largest are exact; smaller ones are off by half the last
// part's smallest step, at most 2^-21 (two parts), 2^-25 (three) or 2^-29 (four)
// of the largest.  A row with an infinity or NaN becomes NaN codes.
template <class C>
__device__ __forceinline__ void dec_fp8_put_q(const DecFp8Params &p, const DecFp8It &u, const DecFp8Q<C> &q, uint8_t *sQ,
                                              float *mul, int *last) {
    constexpr int PL = DecFp8Q<C>::PL;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5 & 3, wg = (int)threadIdx.x >> 7;
    const int r_first = u.chunk * p.rows_per_chunk, rows = min(p.rows_per_chunk, p.R - r_first);
#pragma unroll
    for (int i = 0; i < DecFp8Q<C>::NR; ++i) {
        const int in_wg = warp + 4 * i, r = wg * C::RW + in_wg;
        if (in_wg >= C::RW) break;
        float x[PL];
        float top = 0.f;
        bool fine = true;
#pragma unroll
        for (int e = 0; e < PL; e += 2) {
            const float2 f = unpack16<C::kFP16>(r < rows ? q.raw[i][e / 2] : 0u);
            x[e] = f.x;
            x[e + 1] = f.y;
            fine = fine && isfinite(f.x) && isfinite(f.y);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        top = warp_max(top);
        fine = __all_sync(0xffffffffu, fine);
        // 2^(7 - exponent of top) and its inverse: with the exponent at least
        // 2^-107 both are normal for any 16-bit top
        const uint32_t ex = max(__float_as_uint(top) >> 23, 20u);  // biased
        const float up = __uint_as_float((261u - min(ex, 254u)) << 23), down = __uint_as_float((min(ex, 254u) - 7u) << 23);
        if (lane == 0) {
            // positive, so that a hidden key's -inf stays -inf: a zero scale runs as 2^-126
            mul[in_wg] = fmaxf(p.scale_log2 * down, 1.17549435e-38f);
            last[in_wg] = p.mask_kind != kMaskCausal ? u.L - 1 : p.Sq == 1 ? u.L - 1 : u.L - p.Sq + (r_first + r) % p.Sq;
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

// acc = acc * alpha + O * weight over a warpgroup's rows, O read from its buffer.
template <class C>
__device__ __forceinline__ void dec_fp8_accumulate(uint32_t o_col, const float *alpha, const float *weight,
                                                   float (&acc)[C::NM][C::RW]) {
    float a[C::RW], w[C::RW];
    lds_row<C::RW>(alpha, a);
    lds_row<C::RW>(weight, w);
#pragma unroll
    for (int m = 0; m < C::NM; ++m) {
        float o[C::RW];
        dec_fp8_read<C, C::RW>(o_col + m * C::N, o);
#pragma unroll
        for (int i = 0; i < C::RW; ++i) acc[m][i] = fmaf(acc[m][i], a[i], o[i] * w[i]);
    }
}

template <class C>
__device__ void dec_fp8_softmax_role(const DecFp8Params &p, DecFp8It it, uint8_t *sQ, uint8_t *sP, uint8_t *sV,
                                     float *sF, uint32_t bars, uint32_t tmem, Ctl *ctl) {
    constexpr int RW = C::RW, RP = C::RP;
    const int wg = (int)threadIdx.x >> 7, tid = (int)threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
    sF += wg * C::F_WG;
    // this warp's TMEM lanes, from the warpgroup's first column of a part
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16) + wg * RW;
    // this thread's byte of the warpgroup's row n of the weights: 16-byte chunk (tid >> 4) ^ (n & 7)
    const uint32_t p_addr = ptx::smem_addr(sP) + (uint32_t)(wg * RW * 128 + tid);
    if (it.left <= 0) return;

    // What this thread's key of a tile needs of its block: the table's entry,
    // then the scales, loaded three and two tiles ahead (`ahead` runs in front
    // of `it`): with the memory busy a load takes more than a tile's time.  The
    // loads are unconditional, at places clamped into the arrays, and judged
    // only when they are used, so that none is waited for early.
    DecFp8It ahead = it;
    constexpr int KPT = C::KPT;   // keys of this thread in a step
    int entry[KPT];               // of `ahead`'s step, as loaded
    bool entry_seen[KPT];         // its key exists
    float ks_next[KPT], vs_next[KPT], ks_far[KPT], vs_far[KPT];  // of the next step and the one behind it, as loaded
    bool next_seen[KPT], far_seen[KPT];
    auto load_entry = [&] {
        const int span = dec_fp8_span<C>(ahead);
        const int *row = p.block_table + (size_t)min(ahead.b, p.B - 1) * p.max_blocks;
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
            const int key = (ahead.tile + j) * C::BN + tid;
            entry_seen[j] = ahead.left > 0 && j < span && key < ahead.L;
            entry[j] = row[min(key >> p.bs_log2, p.max_blocks - 1)];
        }
    };
    auto load_scales = [&] {
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
            far_seen[j] = entry_seen[j] && entry[j] >= 0 && entry[j] < p.num_blocks;
            const int bh = (far_seen[j] ? entry[j] : 0) * p.Hkv + ahead.kvh;  // (below 2^31: the host checks)
            ks_far[j] = p.k_scale[bh];
            vs_far[j] = p.v_scale[bh];
        }
        if (ahead.left > 0) dec_fp8_steps<C>(p, ahead, dec_fp8_span<C>(ahead));
    };
    auto shift_scales = [&] {
#pragma unroll
        for (int j = 0; j < KPT; ++j) ks_next[j] = ks_far[j], vs_next[j] = vs_far[j], next_seen[j] = far_seen[j];
    };

    // Units are numbered from 0 in this CTA; unit u's q sits in buffer u & 1.
    // Its rows are loaded one unit before they are split into parts, and split
    // one unit before they are used.
    // (With four warpgroups and two keys a thread registers run out before the
    // memory's rate does: the scales are then loaded one step ahead, and q when it
    // is split; 32 rows at d 128 187 -> 164 us.)
    constexpr bool kDeep = C::NWG < 4 || C::KPT == 1;
    DecFp8Q<C> q;
    dec_fp8_load_q<C>(p, it, q);
    load_entry();
    load_scales();
    load_entry();
    dec_fp8_put_q<C>(p, it, q, sQ, sF + C::F_C, reinterpret_cast<int *>(sF + C::F_LAST));
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(bar_addr(bars, C::B_QFULL));
    shift_scales();
    if constexpr (kDeep) {
        load_scales();
        load_entry();
        if (it.left > it.nt - it.tile) dec_fp8_load_q<C>(p, dec_fp8_next_unit(p, it), q);
    }
    ptx::named_bar_sync(9 + wg, 128);  // every warp's rows' multipliers and last keys are in place

    float acc[C::NM][RW], l[RW];
    float m_run = -INFINITY;  // lane r: row r's running maximum
    bool begun_here = it.tile == 0;
    bool first = true, bad = false;
    int unit = 0, t = 0;  // t: tiles of this CTA so far
    for (int step = 0;; ++step) {
        const int span = dec_fp8_span<C>(it);
        const float *mul = sF + C::F_C + (unit & 1) * RP;
        const int *last = reinterpret_cast<const int *>(sF + C::F_LAST) + (unit & 1) * RP;
        const bool ends = it.tile + span == it.nt || it.left == span;  // the unit, or this CTA's part of it
        if (first) {
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                l[r] = 0.f;
#pragma unroll
                for (int m = 0; m < C::NM; ++m) acc[m][r] = 0.f;
            }
            m_run = -INFINITY;
            // the next unit's q, while this unit's first scores are on their way
            if (it.left > it.nt - it.tile) {
                const int nb = (unit + 1) & 1;
                DecFp8It coming = dec_fp8_next_unit(p, it);
                if constexpr (!kDeep) dec_fp8_load_q<C>(p, coming, q);
                dec_fp8_put_q<C>(p, coming, q, sQ + nb * C::Q_BYTES, sF + C::F_C + nb * RP,
                                 reinterpret_cast<int *>(sF + C::F_LAST) + nb * RP);
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(bar_addr(bars, C::B_QFULL + nb));
                if (kDeep && coming.left > coming.nt) dec_fp8_load_q<C>(p, dec_fp8_next_unit(p, coming), q);
            }
        }
        float ks[KPT], vs[KPT];
#pragma unroll
        for (int j = 0; j < KPT; ++j) ks[j] = next_seen[j] ? ks_next[j] : 0.f, vs[j] = next_seen[j] ? vs_next[j] : 0.f;
        if constexpr (kDeep) shift_scales();
        load_scales();
        if constexpr (!kDeep) shift_scales();
        load_entry();

        const int b = step & 1, k0 = it.tile * C::BN;
        bad = bad || !wait_warp(bar_addr(bars, p.stall_test && step == 0 ? C::B_NEVER : C::B_SFULL + b), (step >> 1) & 1, ctl, 78);
        float x[KPT][RW];  // scores without their row's multiplier
        float *red = sF + C::F_RED + (b * 4 + warp) * (RW + 2);
        if (!bad) {
            ptx::tc_fence_after();
#pragma unroll
            for (int j = 0; j < KPT; ++j) {
                dec_fp8_read<C, RW>(lane_base + C::S_COL + (b * KPT + j) * C::N, x[j]);
#pragma unroll
                for (int r = 0; r < RW; ++r) x[j][r] *= ks[j];
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar_addr(bars, C::B_SFREE + b));
            // hidden keys: past the row's last (a select, so nothing of theirs leaks)
            const int seen_by_all = p.mask_kind == kMaskCausal ? it.L - p.Sq : it.L - 1;
            if (k0 + KPT * C::BN - 1 > seen_by_all) {
#pragma unroll
                for (int j = 0; j < KPT; ++j) {
                    const int key = k0 + j * C::BN + tid;
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (key > last[r] || j >= span) x[j][r] = -INFINITY;
                }
            } else if (KPT > 1 && span < KPT) {
                // (the rest of the unit is another CTA's: S holds nothing of this step there)
#pragma unroll
                for (int r = 0; r < RW; ++r) x[KPT - 1][r] = -INFINITY;
            }
            float mine = -INFINITY;
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                float both = x[0][r];
                if constexpr (KPT == 2) both = fmaxf(both, x[KPT - 1][r]);
                const float top = warp_max(both);
                if (lane == r) mine = top;
            }
            float high = 0.f, low = -INFINITY;  // (a scale of zero is near any other)
#pragma unroll
            for (int j = 0; j < KPT; ++j) {
                high = fmaxf(high, fabsf(vs[j]));
                low = fmaxf(low, vs[j] != 0.f ? -fabsf(vs[j]) : -INFINITY);
            }
            const float vtop = warp_max(high), vlow = warp_max(low);
            if (lane < RW) red[lane] = mine;
            if (lane == 0) red[RW] = vtop, red[RW + 1] = vlow;
        }
        // (a warp whose wait ran out still comes here, and the warpgroup leaves together)
        if (ptx::named_bar_any(1 + wg, 128, bad)) return;
        const float *all = sF + C::F_RED + b * 4 * (RW + 2), *all1 = all + (RW + 2), *all2 = all1 + (RW + 2), *all3 = all2 + (RW + 2);
        const float vtop = fmaxf(fmaxf(all[RW], all1[RW]), fmaxf(all2[RW], all3[RW]));
        const float vlow = -fmaxf(fmaxf(all[RW + 1], all1[RW + 1]), fmaxf(all2[RW + 1], all3[RW + 1]));
        const bool apart = vtop > C::V_RANGE * vlow;  // (the same in the whole warpgroup)
        float *sM = sF + C::F_M + warp * RP, *sB = sF + C::F_B + warp * RP;
        float *sA = sF + C::F_A + (b * 4 + warp) * RP, *sW = sF + C::F_V + (b * 4 + warp) * RP;
        float *sN = sF + C::F_N + warp * RP;
        if (lane < RW) {
            const float top = fmaxf(fmaxf(all[lane], all1[lane]), fmaxf(all2[lane], all3[lane]));
            const float m_tile = top * mul[lane];
            const bool none = m_tile == -INFINITY;  // the row sees no key of the tile
            const float m_new = fmaxf(m_run, m_tile), m_use = m_new == -INFINITY ? 0.f : m_new;
            const float beta = none ? 0.f : ptx::ex2_approx(m_tile - m_use);
            sM[lane] = none ? 0.f : m_tile;
            sB[lane] = beta;
            sA[lane] = ptx::ex2_approx(m_run - m_use);
            sN[lane] = 1.f;
            sW[lane] = beta * (vtop * 0.00390625f);  // O holds 256 times its weights over vtop
            m_run = m_new;
        }
        __syncwarp();
        if (apart) {
            // A block of a much larger scale, in keys that carry little of the row
            // (or none, where the row does not see them), must not push the others
            // below the parts' range: the reference is the row's own largest weight
            // times scale, brought into [128, 256) by a power of two.  One exchange
            // more, in the steps that need it.  (The sums' array is free here: it is read
            // out before the next step's barrier, and written behind the wait for this
            // step's O, which every warp's weights come before.)
            float *sT = sF + C::F_TOP;
            float mine = 0.f;
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                float most = 0.f;
#pragma unroll
                for (int j = 0; j < KPT; ++j) most = fmaxf(most, ptx::ex2_approx(fmaf(x[j][r], mul[r], -sM[r])) * fabsf(vs[j]));
                most = warp_max(most);
                if (lane == r) mine = most;
            }
            if (lane < RW) sT[warp * RP + lane] = mine;
            ptx::named_bar_sync(1 + wg, 128);
            if (lane < RW) {
                const float most = fmaxf(fmaxf(sT[lane], sT[RP + lane]), fmaxf(sT[2 * RP + lane], sT[3 * RP + lane]));
                // biased exponent, kept where the factor and its inverse are normal numbers
                const uint32_t ex = min(max(__float_as_uint(most) >> 23, 8u), 253u);
                sN[lane] = __uint_as_float((261u - ex) << 23);
                sW[lane] = sB[lane] * __uint_as_float((ex - 7u) << 23);
            }
            __syncwarp();
        }
        // weights: of the sum in fp32, of V (times the block's scale, relative to
        // the step's largest times 1 / 256 or to the row's own reference) as
        // parts.  P V of two steps before is done (its O has been read), so its
        // buffer is free.
        {
            float share[KPT];
#pragma unroll
            for (int j = 0; j < KPT; ++j) share[j] = apart ? vs[j] : vtop > 0.f ? vs[j] / vtop * 256.f : 0.f;
            const uint32_t buf = p_addr + b * KPT * C::P_BYTES;
            constexpr int S = RW < 4 ? 1 : 4;  // rows at a time
            static_assert(RW == 1 || RW % 4 == 0, "one row, or whole fours");
#pragma unroll
            for (int g = 0; g < RW; g += S) {
                float m[S], c[S], a[S], e[S], n[S], v[KPT][(S + 1) / 2 * 2];
                lds_row<S>(sM + g, m);
                lds_row<S>(mul + g, c);
                lds_row<S>(sA + g, a);
                lds_row<S>(sB + g, e);
                lds_row<S>(sN + g, n);
#pragma unroll
                for (int r = 0; r < S; ++r) {
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < KPT; ++j) {
                        const float w = ptx::ex2_approx(fmaf(x[j][g + r], c[r], -m[r]));
                        sum += w;
                        v[j][r] = w * share[j] * n[r];
                    }
                    l[g + r] = fmaf(l[g + r], a[r], sum * e[r]);
                }
#pragma unroll
                for (int j = 0; j < KPT; ++j) {
                    if constexpr (S == 1) v[j][1] = 0.f;
#pragma unroll
                    for (int r = 0; r < S; r += 2) {
                        uint32_t codes[C::NP];
                        split_e4m3<C::NP>(v[j][r], v[j][r + 1], codes);
#pragma unroll
                        for (int i = 0; i < C::NP; ++i) {
                            const int at = i * C::RC + g + r;  // (the warpgroup's first row is 0 modulo 8)
                            st_shared_u8((buf ^ (uint32_t)((at & 7) << 4)) + j * C::P_BYTES + at * 128, codes[i]);
                            if (r + 1 < S)
                                st_shared_u8((buf ^ (uint32_t)(((at + 1) & 7) << 4)) + j * C::P_BYTES + (at + 1) * 128,
                                             codes[i] >> 8);
                        }
                    }
                }
            }
            // a row of V past the request's keys (they end in the step's last
            // tile) meets weight 0, but junk (NaN) in it would not vanish: zero it
            const int last_tile = it.tile + span - 1;
            if (wg == 0 && (last_tile + 1) * C::BN > it.L && (it.L & ((1 << p.bs_log2) - 1)) != 0 &&
                last_tile * C::BN + tid >= it.L) {
                const int slot = (t + span - 1) % C::VST;
                bad = !wait_bar(bar_addr(bars, C::B_VFULL + slot), ((t + span - 1) / C::VST) & 1, ctl, 80);
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
        ptx::tc_fence_before();
        if (!bad) ptx::mbar_arrive(bar_addr(bars, C::B_PFULL + b));
        // O of the tile before (of this unit), while P V of this one runs
        if (!first) {
            bad = bad || !wait_warp(bar_addr(bars, C::B_OFULL + (b ^ 1)), ((step - 1) >> 1) & 1, ctl, 79);
            if (!bad) {
                ptx::tc_fence_after();
                dec_fp8_accumulate<C>(lane_base + C::O_COL + (b ^ 1) * C::NM * C::N, sF + C::F_A + ((b ^ 1) * 4 + warp) * RP,
                                      sF + C::F_V + ((b ^ 1) * 4 + warp) * RP, acc);
                ptx::tc_fence_before();
            }
        }
        first = false;

        if (ends) {
            // the unit's last O, its sums, and the rows out
            bad = bad || !wait_warp(bar_addr(bars, C::B_OFULL + b), (step >> 1) & 1, ctl, 81);
            if (!bad) {
                ptx::tc_fence_after();
                dec_fp8_accumulate<C>(lane_base + C::O_COL + b * C::NM * C::N, sA, sW, acc);
                ptx::tc_fence_before();
            }
            float mine = 0.f;
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                float s = l[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == r) mine = s;
            }
            float *sL = sF + C::F_L;
            if (lane < RW) sL[warp * RP + lane] = mine;
            if (ptx::named_bar_any(5 + wg, 128, bad)) return;
            int rows;
            const size_t row0 = dec_fp8_row0(p, it.b, it.kvh, it.chunk, &rows);
            const bool whole = begun_here && it.tile + span == it.nt;
            const size_t slot = 2 * (size_t)blockIdx.x + (begun_here ? 1 : 0);
            rows -= wg * RW;  // (0 or less: the warpgroup has none of them)
            if (warp == 0 && lane < RW && lane < rows) {
                const float sum = (sL[lane] + sL[RP + lane]) + (sL[2 * RP + lane] + sL[3 * RP + lane]);
                // (a NaN sum is no empty row)
                const float lse2 = sum == 0.f ? -INFINITY : m_run + __log2f(sum);
                if (whole) p.lse[row0 + wg * RW + lane] = lse2 * kLn2;
                else p.part_lse[slot * C::RC + wg * RW + lane] = lse2;
            }
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                if (r >= rows) break;
                const float sum = (sL[r] + sL[RP + r]) + (sL[2 * RP + r] + sL[3 * RP + r]);
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int m = 0; m < C::NM; ++m) {
                    const int c = m * 128 + tid;
                    if (c >= C::D) continue;
                    const float o = acc[m][r] * inv;
                    if (whole)
                        static_cast<uint16_t *>(p.o)[(row0 + wg * RW + r) * C::D + c] = (uint16_t)pack2b<C::kFP16>(o, 0.f);
                    else
                        p.part_o[(slot * C::RC + wg * RW + r) * C::D + c] = o;
                }
            }
            if (it.left == span) return;
            first = true;
            begun_here = true;
            ++unit;
            // sL is written again only behind the next tile's barrier
        }
        t += span;
        dec_fp8_steps<C>(p, it, span);
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
    uint64_t *bar_mem = reinterpret_cast<uint64_t *>(sP + 2 * C::KPT * C::P_BYTES);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bar_mem + C::NUM_BARS);
    Ctl *ctl = reinterpret_cast<Ctl *>(tmem_holder + 2);
    float *sF = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(ctl + 1) + 15) & ~static_cast<uintptr_t>(15));
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
            ptx::mbar_init(bar_addr(bars, C::B_QFULL + b), 128 * C::NWG);
            ptx::mbar_init(bar_addr(bars, C::B_SFULL + b), 1);
            ptx::mbar_init(bar_addr(bars, C::B_SFREE + b), 128 * C::NWG);
            ptx::mbar_init(bar_addr(bars, C::B_PFULL + b), 128 * C::NWG);
            ptx::mbar_init(bar_addr(bars, C::B_OFULL + b), 1);
        }
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
    ptx::wait_for_previous_kernel();
    // (the small arrays are not yet in use: the prefix sums borrow their first bytes)
    const DecFp8It it = dec_fp8_begin<C::NUM_THREADS>(p, reinterpret_cast<long long *>(sF));
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // the merge may be set up now; it waits for this grid's end before it reads
    ptx::let_next_kernel_begin();

    if (warp < 4 * C::NWG) {
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
// c, c + 1, ... (slots 2c, 2c + 2, ...) up to the unit's end, in that order.  A
// warp per row, all at once; lane i holds the weight of partial i of 32 at a
// time.
template <int RC>
constexpr int kDecFp8MergeThreads = 32 * (RC < 4 ? 4 : RC);

template <int D, bool kFP16, int RC>
__global__ void __launch_bounds__(kDecFp8MergeThreads<RC>)
    fa_decode_fp8_combine_kernel(const __grid_constant__ DecFp8Params p, int grid) {
    const int c = (int)blockIdx.x + 1, lane = (int)threadIdx.x & 31, r = (int)threadIdx.x >> 5;
    ptx::wait_for_previous_kernel();  // (launched while the attention still runs)
    // One round of loads: the cut, the first 32 partials' lse and the first two
    // partial rows, which every unit that is merged has.
    const long long total = *reinterpret_cast<const long long *>(p.cuts);
    const int *cut = p.cuts + 4 + 5 * c;
    const int cb = cut[0], ckvh = cut[1], cchunk = cut[2], ctile = cut[3], cnt = cut[4];
    auto slot_row = [&](int i) { return (size_t)(i == 0 ? 2 * c - 1 : 2 * (c + i - 1)) * RC + r; };
    constexpr int PER = D / 32;
    const bool held = r < RC;
    float lse0 = held && c + lane - 1 < grid ? p.part_lse[slot_row(lane)] : -INFINITY;
    float row0_v[PER], row1_v[PER];
#pragma unroll
    for (int e = 0; e < PER; e += 2) {
        float2 v0 = make_float2(0.f, 0.f), v1 = v0;
        if (held) {
            v0 = *reinterpret_cast<const float2 *>(p.part_o + slot_row(0) * D + lane * PER + e);
            v1 = *reinterpret_cast<const float2 *>(p.part_o + slot_row(1) * D + lane * PER + e);
        }
        row0_v[e] = v0.x, row0_v[e + 1] = v0.y;
        row1_v[e] = v1.x, row1_v[e + 1] = v1.y;
    }
    const long long G = min((long long)grid, total);
    if (c >= G) return;
    if (ctile == 0) return;  // between two units
    const long long begin = c * total / G - ctile, end = begin + cnt;
    if ((c - 1) * total / G > begin) return;  // an earlier boundary merges this unit
    // Partials of the unit: CTA c - 1's and one for each CTA from c on that
    // begins before its end.  CTA k begins at k T / G, which is below `end` for
    // k < end G / T: the largest such k gives the last.
    const long long last = min((end * G - 1) / total, G - 1);
    const int n = (int)(last - c) + 2;
    int rows;
    const size_t row0 = dec_fp8_row0(p, cb, ckvh, cchunk, &rows);
    if (r >= rows) return;
    float acc[PER], sum = 0.f, top = -INFINITY;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const float mine = i0 + lane >= n ? -INFINITY : i0 == 0 ? lse0 : p.part_lse[slot_row(i0 + lane)];
        const bool nan = __any_sync(0xffffffffu, isnan(mine));
        const float high = nan ? NAN : fmaxf(top, warp_max(mine));
        const float use = high == -INFINITY ? 0.f : high;
        const float rescale = ptx::ex2_approx(top - use), weight = ptx::ex2_approx(mine - use);
        top = nan || isnan(top) ? NAN : high;
        sum *= rescale;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] *= rescale;
        int i = 0;
        if (i0 == 0) {
            const float w0 = __shfl_sync(0xffffffffu, weight, 0), w1 = __shfl_sync(0xffffffffu, weight, 1);
            sum = w0 + w1;
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(w1, row1_v[e], w0 * row0_v[e]);
            i = 2;
        }
#pragma unroll 4
        for (; i < min(32, n - i0); ++i) {
            const float w = __shfl_sync(0xffffffffu, weight, i);
            const float *src = p.part_o + slot_row(i0 + i) * D + lane * PER;
            sum += w;
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

}  // namespace fa
