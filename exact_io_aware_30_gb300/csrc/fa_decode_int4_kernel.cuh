// fa_decode_int4_kernel.cuh -- attention of a few new query rows per request
// over a paged cache held in 4 bits (the format of fa_int4_kernel.cuh), for
// sm_103a.
//
// For row r of a K/V head, over the keys j it sees and the groups g of d,
//   x_rj = scale sum_g s_jg (q_rg . c_jg - z_jg sum q_rg),  p = softmax(x),
//   o_rg = sum_j (p_rj s_jg) c_jg - sum_j p_rj s_jg z_jg,   lse_r = ln sum_j exp(x_rj):
// the codes go into the products as whole numbers, and scales and zeros meet
// fp32 sums (K) or the weights (V).  Bound by reading the cache: d + 8 d / G
// bytes per token and K/V head.
//
// Codes in the tensor cores.  A 32-bit word holds 8 codes; masked with 0x000F000F
// it is two fp16 numbers c 2^-24, exact, below the normal numbers, and masked with
// 0x00F000F0 two more, c 2^-20: a code costs 5/8 of an instruction.  The factor 16
// between the two is taken out of q (whose odd components are 16 times smaller)
// and of O's rows at the end.  Which components share a product's step is free,
// so every product takes one chunk of 32 adjacent components of a group: four words
// of 8, lane t of four word t.  These are products by warps (mma.sync m16n8k16, one
// in 8 cycles of an SM's quarter): the codes pass through registers anyway, and what
// they make needs no shared memory on its way in, and for up to 8 query rows a key's
// products take a third of the time that its bytes take from memory.
//   S^T = K Q^T: 16 keys x 8 rows per product, K words straight from shared memory.
//   O^T = V^T P^T: ldmatrix transposes V by units of 16 bits, four codes of one
//   key; the weights' fragment is S's, rounded to fp16 and turned by movmatrix.
// Half of the keys' codes enter O as 15 - c, with the weight negated (a complement
// is part of the same masking instruction), so that O's sums, which the tensor core
// cuts off rather than rounds, do not grow with the 7.5 that codes are on average;
// what that leaves out goes with the zeros, whose products are begun anew each step
// and summed in fp32.
//
// Weights.  What P V takes is p s / ref_g in fp16: 2^-11 of itself (with up to four
// rows, or fp16 q, 2^-22, in two numbers), and no finer than 2^-25 where 2^12 stands for the row's
// reference: rows are taken relative to a running maximum M of x + log2 max_g (s /
// ref_g), 6 above it when it moves, and each group's scales relative to a power of two
// that the step's largest is kept within 2^8 of.  So the smallest half step is 2^-31 of
// the row's largest product where a group's scales are alike, and at most 2^-23.  Both
// move rarely, by a branch of the whole warp that rescales what it has summed.
//
// Sums.  The tensor core cuts a sum off, towards 0, at each product into it; after 256
// products (4,096 keys of a warp; 512 with those of weights' rests) the sums are laid down and begun anew (REST).
//
// Work split: the line of 128-key tiles of fa_decode_fp8_kernel.cuh, an even
// share of it per CTA, cut units merged by its second kernel.  One CTA: a ring of
// tiles, K and V codes and words, that its four warps take turns at filling; a warp
// takes 32 keys of a tile, as two sixteens side by side (16 at a time where registers
// do not hold their words; with more rows fewer warps more keys, the others other
// rows), and has a running maximum and sums of its own, so that nothing is exchanged
// before the unit's end, where half of the warps hand their sums to the other half at
// a time.
//
// What bounds it (kv8: 64 requests, 32 heads on 8 K/V heads, up to 8,192 tokens, d 128,
// bf16, groups of 32, 379 MB): the copies alone run at 57 us, the floor is 56 and the
// kernel takes 87.5.  16 keys are 358 instructions of a warp, a quarter of them masks and
// shifts at half rate; the ALU is busy half of the time and the issue slots too, with
// three warps to a scheduler, whose waits for one another's pipes and for their own
// results fill the rest.  Before weights kept their rests it took 84 us, 16 warps of one
// sixteen each (128 registers) 103, 8 warps of four sixteens 85 to 93; copies by a ninth
// warp left two CTAs' warps 96 registers and spilled (216).  Short units pay for their
// ends: 128 requests x 40 heads, nine tiles to a unit, 268 us for a floor of 140.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fa_decode_fp8_kernel.cuh"
#include "fa_int4_kernel.cuh"

namespace fa {

struct DecInt4Params : DecFp8Params {  // (k_scale and v_scale are not used)
    const uint32_t *k_words, *v_words;  // [num_blocks, Hkv, bs, d / G]
    float4 *sums;                       // [G, RG, PART / 16]: what a CTA's unit has summed in front of its last rest
    int fp16;
};

// Tiles of a unit after which a warp's sums are laid down and begun anew: 4,096 keys
// of a warp, 256 products into each sum of O (512 with kTwice).  The tensor core cuts a sum off at each
// of them, always towards 0, and the weights' sum is rounded 512 times; over a million
// keys of about even weight lse was off by 2e-4 and O by 2^-10 and more.
constexpr int dec_i4_rest(int row_groups) { return 32 * (4 / row_groups); }

// Bytes of a warp's sums: nt eights of rows, of each of which a lane has e.
constexpr int dec_i4_part(int d, int nt, int e) { return (e * nt * d / 32 + nt) * 512; }

template <int D_, int G_, int NT_, int RG_, bool kFew_, bool kTwice_, bool kRests_>
struct DecI4Cfg {
    static constexpr int D = D_;
    static constexpr int G = G_;                  // components per group
    static constexpr int NT = NT_;                // eights of rows per warp
    static constexpr int RG = RG_;                // groups of warps with different rows
    // Up to four rows stand in every other column of a product, so that a lane has
    // one of them and the work on the weights halves.
    static constexpr bool kFew = kFew_;
    // The columns between them hold what rounding a weight to fp16 lost, so that it has
    // 22 bits, not 11.  fp16, 128 requests x 40 heads: the error of O 1.33 -> 1.00 times
    // its own rounding, 266 -> 273 us when it came.  bf16: two keys that nearly cancel
    // leave less than 2^-17 of their values in place of 2^-12, kv8 83 -> 87.6 us, with
    // groups of 64 72 -> 74.
    // With more rows, and where O is fp16, whose own rounding is no coarser than a
    // weight's, that rest takes the products a second time, over the same codes: the
    // error of O 1.15 to 1.8 -> 1.00 times its own rounding, 64 requests x 8 heads of 8 rows
    // 93 -> 111 us, of 8 at d 64 58 -> 65, of 32 245 -> 328.
    static constexpr bool kTwice = kTwice_;
    static_assert(!(kFew && kTwice), "one place for the rest");
    static constexpr int E = kFew ? 1 : 2;        // rows of each eight columns that are a lane's
    static constexpr int RC = 4 * E * NT * RG;    // rows per unit
    static constexpr bool kWide = D <= 128 && NT == 1;
    static constexpr int WARPS = 4;
    static constexpr int KW = WARPS / RG;         // warps along a tile's keys
    // Sixteens of keys of a step, side by side, where registers hold their words
    // (kv8, one 103 us, two 84; 16 rows at d 64 106 and 97).
    static constexpr int H = D / G * NT <= 4 ? 2 : 1;
    static constexpr int KEYS = 16 * H;
    static constexpr int BN = 128;
    static constexpr int SPT = BN / KEYS / KW;    // steps of a warp per tile
    // A kernel of its own: with rests in all of them 128 requests x 40 heads took
    // 269 us for 264, drafts at d 256 109 for 104.
    static constexpr bool kRests = kRests_;
    static constexpr int REST = dec_i4_rest(RG);
    // Which key of a step stands in row i + 8k of the products of sixteen h: SI i +
    // SK k + sixteen(h).  With two words to a key, 16 bytes hold those of two, and
    // the order is such that the transposed words have the zeros where their
    // products want them (see dec_i4_keys).
    static constexpr bool kPairs = D / G == 2;
    static constexpr int SI = kPairs ? 2 : 1;
    static constexpr int SK = !kPairs ? 8 : H > 1 ? 16 : 1;
    static __device__ __forceinline__ constexpr int sixteen(int h) { return kPairs && H > 1 ? (h & 1) + 32 * (h >> 1) : 16 * h; }
    static constexpr bool ZMMA = D / G >= 2;      // the zeros go through products
    static constexpr int ZE = D / G == 2 ? 2 * E : E;  // sums of them a lane holds per group and eight rows
    static constexpr int NG = D / G;
    static constexpr int NC = D / 32;             // chunks of 32 components, 16 bytes
    static constexpr int ROW = D / 2;             // bytes of a row of codes
    static constexpr int TILE = BN * ROW;
    static constexpr int WORDS = BN * NG * 4;     // bytes of a tile's words
    static constexpr int O_V = TILE, O_KW = 2 * TILE, O_VW = O_KW + WORDS;  // places in a stage
    static constexpr int STAGE = (O_VW + WORDS + 1023) / 1024 * 1024;
    static constexpr int PART = dec_i4_part(D, NT, E);  // a warp's sums, on their way to another's
    static constexpr int PARTS = WARPS / 2;
    static constexpr int CTAS_PER_SM = kWide ? 3 : 2;
    static constexpr int BUDGET = (227 / CTAS_PER_SM - 1) * 1024;
    static constexpr int FIXED = 1024 + PARTS * PART + 512;
    static constexpr int FIT = (BUDGET - FIXED) / STAGE;
    static constexpr int ST = FIT < 6 ? FIT : 6;
    static_assert(ST >= 2, "a ring of at least two tiles");
    static constexpr int SMEM_BYTES = FIXED + ST * STAGE;
    static constexpr int NUM_THREADS = 32 * WARPS;
    static constexpr int B_FULL = 0;
    static constexpr int B_EMPTY = ST;
    static constexpr int B_NEVER = 2 * ST;        // no arrivals (the stall test's wait)
    static constexpr int NUM_BARS = 2 * ST + 1;
    static_assert(NUM_BARS * 8 + 32 * WARPS + 16 + 4 * ST <= 512, "layout");
};

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// n consecutive words of shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = lds32(addr);
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]) : "r"(addr + 4 * i));
    }
}

__device__ __forceinline__ float4 lds_float4(uint32_t addr) {
    uint32_t w[4];
    lds_words<4>(addr, w);
    return make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
}

__device__ __forceinline__ void sts_float4(uint32_t addr, float a, float b, float c, float d) {
    ptx::st_shared_v4(addr, __float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// ------------------------------------------------------------------- copies

// A warp's next tile to copy lies in shared memory between its turns, so that the
// products have its registers.
constexpr int kI4Kept = 32;  // bytes

__device__ __forceinline__ void dec_i4_keep(const DecFp8It &it, int lane, uint32_t kept) {
    __syncwarp();
    if (lane == 0) {
        ptx::st_shared_v4(kept, it.b, it.kvh, it.chunk, it.tile);
        ptx::st_shared_v4(kept + 16, it.L, it.nt, it.next_len, it.left);
    }
    __syncwarp();
}

__device__ __forceinline__ DecFp8It dec_i4_take(uint32_t kept) {
    uint32_t x[8];
    lds_words<8>(kept, x);
    DecFp8It it;
    it.b = (int)x[0], it.kvh = (int)x[1], it.chunk = (int)x[2], it.tile = (int)x[3];
    it.L = (int)x[4], it.nt = (int)x[5], it.next_len = (int)x[6], it.left = (int)x[7];
    return it;
}

// n tiles on.
__device__ __forceinline__ void dec_i4_advance(const DecInt4Params &p, DecFp8It &it, int n) {
    while (n > 0 && it.left > 0) {
        const int in_unit = min(n, it.nt - it.tile);  // up to the first tile of the next unit
        it.left -= in_unit - 1;
        it.tile += in_unit - 1;
        dec_fp8_step(p, it);
        n -= in_unit;
    }
}

// Lanes 4k .. 4k + 3 stand for block k of a tile: whether there is such a block,
// and its table entry as loaded.  (Judged when the copy begins, so that the load is
// not waited for here.)
template <class C>
__device__ __forceinline__ bool dec_i4_entry(const DecInt4Params &p, const DecFp8It &it, int lane, int &entry) {
    const int n = ((it.tile * C::BN) >> p.bs_log2) + (lane >> 2);
    const bool some = lane >> 2 < C::BN >> p.bs_log2 && it.left > 0 && (n << p.bs_log2) < it.L;
    entry = some ? p.block_table[(size_t)it.b * p.max_blocks + n] : 0;
    return some;
}

// BYTES (4, 8 or 16) from global to shared memory, completed on a barrier by copy_arrive.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A warp issues its TMA copies lane after lane.  With blocks of 16 a tile's words
// are therefore copied by all lanes at once, those of every 32nd key each (128
// requests x 40 heads 272 -> 263 us); with larger ones, of which a tile has few, by
// TMA too (kv8, blocks of 64: by lanes 84.6 -> 87.2).
__device__ __forceinline__ bool dec_i4_words_by_lanes(const DecInt4Params &p) { return p.bs_log2 == 4; }

// Copies a tile into a stage that is free.  The whole warp: lane 4k + j has part j
// (K codes, V codes, K words, V words) of block k.  Slots behind the request's
// blocks are not read later; a block outside the pool gets zero words, whatever its
// codes.
template <class C>
__device__ __forceinline__ void dec_i4_copy(const DecInt4Params &p, int kvh, bool some, int entry, int lane, uint32_t stage, uint32_t bar) {
    const bool in = some && entry >= 0 && entry < p.num_blocks;
    const uint32_t blocks = (uint32_t)__popc(__ballot_sync(0xffffffffu, in)) / 4;
    const int part = lane & 3, row = (lane >> 2) << p.bs_log2;
    constexpr int ROW_W = C::NG * 4, PIECE = ROW_W < 16 ? ROW_W : 16;
    uint32_t bytes = blocks * ((uint32_t)(2 * C::ROW) << p.bs_log2);
    const uint32_t word_bytes = (uint32_t)ROW_W << p.bs_log2, words_at = stage + (part & 1 ? C::O_VW : C::O_KW) + row * ROW_W;
    if (some && !in && part >= 2)
        for (uint32_t i = 0; i < word_bytes; i += 16) ptx::st_shared_v4(words_at + i, 0u, 0u, 0u, 0u);
    if (dec_i4_words_by_lanes(p)) {
        const int judged = in ? entry : -1;
#pragma unroll
        for (int i = 0; i < C::BN / 32; ++i) {
            const int key = 32 * i + lane, e = __shfl_sync(0xffffffffu, judged, key >> 4 << 2);
            if (e < 0) continue;
            const uint32_t dst = stage + C::O_KW + key * ROW_W;
            const size_t at = (((size_t)e * p.Hkv + kvh) * 16 + (key & 15)) * C::NG;
#pragma unroll
            for (int x = 0; x < ROW_W; x += PIECE) {
                copy_async<PIECE>(dst + x, p.k_words + at + x / 4);
                copy_async<PIECE>(dst + C::WORDS + x, p.v_words + at + x / 4);
            }
        }
        copy_arrive(bar);
    } else {
        if (some && !in) ptx::fence_proxy_async_smem();  // (later copies of words to this stage come behind the zeros)
        bytes += 2 * blocks * word_bytes;
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
    __syncwarp();
    if (in) {
        if (part < 2) {
            const uint64_t pol = p.chunks > 1 ? ptx::policy_evict_last() : ptx::policy_evict_first();
            ptx::tma_load_4d(stage + (part ? C::O_V : 0) + row * C::ROW, part ? &p.tm_v : &p.tm_k, bar, 0, 0, kvh, entry, pol);
        } else if (!dec_i4_words_by_lanes(p)) {
            const size_t at = (((size_t)entry * p.Hkv + kvh) << p.bs_log2) * C::NG;
            ptx::bulk_load(words_at, (part & 1 ? p.v_words : p.k_words) + at, word_bytes, bar);
        }
    }
    __syncwarp();
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with sums that begin at 0.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ void ldmatrix_x2_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}

__device__ __forceinline__ void ldmatrix_x1_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x1.trans.shared.b16 {%0}, [%1];" : "=r"(r[0]) : "r"(addr));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float i4_scale(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float i4_zero(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
}

// What a warp holds of its unit.  Lane 4i + t: keys i and i + 8 of a step, rows
// 2t and 2t + 1 of each eight; of O, components 4i .. 4i + 3 of each chunk.
template <class C>
struct DecI4Warp {
    uint32_t q[C::NT][C::NC][4];     // fragments of q
    float q_sum[C::NT][C::NG][C::E]; // -2^-20 times the groups' sums of q
    float mul[C::NT][C::E];          // from a sum of products to log2 units
    float m[C::NT][C::E];            // reference of the exponents
    float l[C::NT][C::E];            // this lane's sums of weights
    float inv[C::NG];                // kI4Room / ref of the groups' V scales, a power of two; 0 before the first
    float o[C::NT][C::NC][2][4];     // sums of weights times codes
    float zo[C::NT][C::NG][C::ZE];   // sums of weights times zeros: this lane's share, or as the products leave them
};

constexpr float kI4None = -3.402823466e38f;  // the reference before the first key
// What P V takes is at most 2^12: 2^6 when a row's reference has just moved,
// which is 2^6 above its largest product then.
constexpr float kI4Room = 4096.f;
constexpr float kI4RoomLog2 = 12.f, kI4Ahead = 6.f;

// q's rows of a unit, 16-bit: lane 4i + t has components 8t .. 8t + 7 of each chunk of rows i.
template <class C>
__device__ __forceinline__ void dec_i4_load_q(const DecInt4Params &p, const DecFp8It &u, int rg, int lane, uint4 (&raw)[C::NT][C::NC]) {
    const int i = lane >> 2, t = lane & 3;
    int rows;
    const size_t row0 = dec_fp8_row0(p, u.b, u.kvh, u.chunk, &rows);
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        const int r = C::kFew ? i >> 1 : (rg * C::NT + n) * 8 + i;
#pragma unroll
        for (int c = 0; c < C::NC; ++c) {
            raw[n][c] = make_uint4(0, 0, 0, 0);
            if (r < rows && !(C::kFew && (i & 1))) raw[n][c] = *reinterpret_cast<const uint4 *>(p.q + (row0 + r) * C::D + 32 * c + 8 * t);
        }
    }
}

// q's rows into fragments, and empty sums.  A row is scaled by a power of two so
// that its largest component is in [2^10, 2^11); 16-bit components are then
// exact in fp16 down to 2^-24 of it (and 2^-25 of the row's scale is the most a
// smaller one is off).  A row with an infinity, a NaN or a component of 2^112 or
// more is NaN.
template <class C, bool kFP16>
__device__ __forceinline__ void dec_i4_q_unit(const DecInt4Params &p, const uint4 (&raw)[C::NT][C::NC], int lane,
                                                  DecI4Warp<C> &w) {
    const int t = lane & 3;
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        uint32_t mag = 0;
#pragma unroll
        for (int c = 0; c < C::NC; ++c)
            mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(raw[n][c].x & 0x7fff7fffu, raw[n][c].y & 0x7fff7fffu),
                                         __vmaxu2(raw[n][c].z & 0x7fff7fffu, raw[n][c].w & 0x7fff7fffu)));
        mag = max(mag & 0xffffu, mag >> 16);
        mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
        mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
        const float top = unpack16<kFP16>(mag).x;
        const uint32_t ex = max(__float_as_uint(top) >> 23, 20u);  // biased exponent
        const bool fine = ex < 127u + 112u;
        const float up = __uint_as_float((264u - min(ex, 238u)) << 23);
        // positive, so that a hidden key's -inf stays -inf: a zero scale runs as 2^-126
        const float mul = fmaxf(p.scale_log2 * __uint_as_float((min(ex, 238u) + 10u) << 23), 1.17549435e-38f);
        float sum[C::NG];
#pragma unroll
        for (int g = 0; g < C::NG; ++g) sum[g] = 0.f;
#pragma unroll
        for (int c = 0; c < C::NC; ++c) {
            const uint32_t ws[4] = {raw[n][c].x, raw[n][c].y, raw[n][c].z, raw[n][c].w};
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack16<kFP16>(ws[e]);
                x[2 * e] = f.x * up;
                x[2 * e + 1] = f.y * up;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[c * 32 / C::G] += x[e];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w.q[n][c][2 * h] = fine ? ptx::pack_f16x2(16.f * x[2 * h], 16.f * x[2 * h + 4]) : 0x7fff7fffu;
                w.q[n][c][2 * h + 1] = fine ? ptx::pack_f16x2(x[2 * h + 1], x[2 * h + 5]) : 0x7fff7fffu;
            }
        }
#pragma unroll
        for (int g = 0; g < C::NG; ++g) {
            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
            sum[g] = fine ? sum[g] * -9.5367431640625e-7f : 0.f;
        }
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            const int from = (2 * t + e) * 4;
#pragma unroll
            for (int g = 0; g < C::NG; ++g) w.q_sum[n][g][e] = __shfl_sync(0xffffffffu, sum[g], from);
            w.mul[n][e] = __shfl_sync(0xffffffffu, mul, from);
            w.m[n][e] = kI4None;
            w.l[n][e] = 0.f;
#pragma unroll
            for (int g = 0; g < C::NG; ++g)
#pragma unroll
                for (int z = e; z < C::ZE; z += C::E) w.zo[n][g][z] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < C::NC; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) w.o[n][c][h][e] = 0.f;
    }
#pragma unroll
    for (int g = 0; g < C::NG; ++g) w.inv[g] = 0.f;
}

template <class C>
__device__ __forceinline__ void dec_i4_begin_unit(const DecInt4Params &p, const uint4 (&raw)[C::NT][C::NC], int lane,
                                                  DecI4Warp<C> &w) {
    if (C::kTwice || (C::kFew && p.fp16)) dec_i4_q_unit<C, true>(p, raw, lane, w);
    else dec_i4_q_unit<C, false>(p, raw, lane, w);
}

// log2 of the largest of a key's V scales relative to their references (a:
// times kI4Room).
template <class C>
__device__ __forceinline__ float dec_i4_top(const float (&a)[C::NG]) {
    float top = 3.7252903e-9f;  // 2^-40 of kI4Room: a key without a scale does not move the reference far
#pragma unroll
    for (int g = 0; g < C::NG; ++g) top = fmaxf(top, a[g]);
    return lg2_approx(top) - kI4RoomLog2;
}

// Moves the references of the groups' scales (where the step's largest is more
// than 2^8 away) and of the exponents (where a row's largest product is above
// it) and rescales the sums.  vw: the V words of the lane's keys; s: their
// scores' sums of products.  The whole warp.
//   Where every group's reference rose, the exponents' may come down by as much, so
// that products with later, lighter keys keep their bits.  A row's sum of weights
// grows by that, and is kept below 2^kI4MostLog2: scales may be 2^240 apart, fp32's
// sums not.  A row's sums take both steps at once, by the product of the factors, as one
// of them alone could leave fp32's range.
constexpr float kI4MostLog2 = 112.f;

template <class C>
__device__ __forceinline__ void dec_i4_move(DecI4Warp<C> &w, const uint32_t (&vw)[C::H][2][C::NG], const float (&s)[C::H][C::NT][2][C::E]) {
    int rise = -1000;     // log2 of the factor of the group whose sums shrink least
    int shift[C::NG];     // log2 of the groups' factors
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
        float top = 0.f;
#pragma unroll
        for (int h = 0; h < C::H; ++h) top = fmaxf(top, fmaxf(i4_scale(vw[h][0][g]), i4_scale(vw[h][1][g])));
        top = warp_max(top);  // (a NaN scale is passed over)
        const int ex = (int)min(max(__float_as_uint(top) >> 23, 13u), 253u);
        const float old = w.inv[g] * (1.f / kI4Room), rel = top * old;
        const int from = (int)(__float_as_uint(old) >> 23);  // (a power of two)
        int to = from;
        if (old == 0.f) {
            if (top > 0.f) w.inv[g] = __uint_as_float((uint32_t)(254 - ex) << 23) * kI4Room;
        } else if (rel > 256.f) {
            to = 254 - ex;
        } else if (rel < 0.00390625f && top > 0.f) {
            // downwards as far as the sums have room in fp32
            float most = 1.f;
#pragma unroll
            for (int n = 0; n < C::NT; ++n) {
#pragma unroll
                for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        most = fmaxf(most, 16777216.f * fmaxf(fabsf(w.o[n][c][0][e]), fabsf(w.o[n][c][1][e])));
#pragma unroll
                for (int z = 0; z < C::ZE; ++z) most = fmaxf(most, fabsf(w.zo[n][g][z]));
            }
            most = warp_max(most);
            const int room = 200 - (int)min(__float_as_uint(most) >> 23, 200u);  // up to 2^73
            to = min(254 - ex, from + room);
        }
        if (to != from) w.inv[g] = __uint_as_float((uint32_t)to << 23) * kI4Room;
        shift[g] = to - from;
        rise = max(rise, shift[g]);
    }
    float la[C::H][2];
#pragma unroll
    for (int h = 0; h < C::H; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float a[C::NG];
#pragma unroll
            for (int g = 0; g < C::NG; ++g) a[g] = i4_scale(vw[h][k][g]) * w.inv[g];
            la[h][k] = dec_i4_top<C>(a);
        }
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            float top = kI4None;
#pragma unroll
            for (int h = 0; h < C::H; ++h)
                top = fmaxf(top, fmaxf(fmaf(s[h][n][0][e], w.mul[n][e], la[h][0]), fmaf(s[h][n][1][e], w.mul[n][e], la[h][1])));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            float old = w.m[n][e];
            if (rise < 0) {  // (in the whole warp)
                float l = w.l[n][e];
                l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, 4));
                l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, 8));
                l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, 16));
                old -= fminf((float)-rise, fmaxf(kI4MostLog2 - lg2_approx(fmaxf(l, 1.f)), 0.f));
            }
            const float now = top > old ? top + kI4Ahead : old;
            const float f = ptx::ex2_approx(w.m[n][e] - now);
            w.m[n][e] = now;
            w.l[n][e] *= f;
#pragma unroll
            for (int g = 0; g < C::NG; ++g) {
                const int half = shift[g] >> 1;  // (in halves, which are normal numbers)
                const float both = __uint_as_float((uint32_t)(127 + half) << 23) * f * __uint_as_float((uint32_t)(127 + shift[g] - half) << 23);
#pragma unroll
                for (int z = e; z < C::ZE; z += C::E) w.zo[n][g][z] *= both;
#pragma unroll
                for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        w.o[n][c][h][e] *= both;
                        w.o[n][c][h][2 + e] *= both;
                        if constexpr (C::kFew) {
                            w.o[n][c][h][1] *= both;
                            w.o[n][c][h][3] *= both;
                        }
                    }
            }
        }
}

// What a lane reads of a stage at its warp's first step: K words, V matrices,
// words of its keys, words as matrices.
struct DecI4Lane {
    uint32_t k, v, w, z;
};

template <class C>
__device__ __forceinline__ DecI4Lane dec_i4_lane(uint32_t ring, int lane, int first) {
    // 16-byte chunk c of row r of a box is chunk c ^ swizzle(r)
    auto swizzle = [](int r) { return C::ROW == 128 ? r & 7 : C::ROW == 64 ? (r >> 1) & 3 : (r >> 2) & 1; };
    const int k_row = C::SI * (lane >> 2), v_row = C::SI * (lane & 7) + C::SK * (lane >> 3 & 1);
    const int z_row = C::NG == 2 ? 2 * lane : lane;  // (lanes whose matrix is not loaded are not asked)
    DecI4Lane x;
    x.k = ring + (first + k_row) * C::ROW + (swizzle(k_row) << 4) + 4 * (lane & 3);
    x.v = ring + C::O_V + (first + v_row) * C::ROW + ((swizzle(v_row) ^ (lane >> 4)) << 4);
    x.w = ring + C::O_KW + (first + k_row) * C::NG * 4;
    x.z = ring + C::O_VW + (first + z_row) * C::NG * 4;
    return x;
}

// A step's keys, the first of them `key`, `at` bytes behind the lane's places.
// Row r of the K/V head, the warp's first being row0, sees keys up to L - 1 -
// back + r % (back + 1).
template <class C>
__device__ __forceinline__ void dec_i4_keys(DecI4Warp<C> &w, int key, int L, int back, int row0, int lane, const DecI4Lane &from,
                                            uint32_t at, uint32_t at_words) {
    constexpr int H = C::H, ROW_W = C::NG * 4;
    constexpr int OTHER = C::SK * C::ROW;  // to row i + 8
    const uint32_t words = from.w + at_words;
    if (key + C::KEYS > L) {  // slots past the request's tokens may hold anything: their words become 0
#pragma unroll
        for (int mine = lane; mine < C::KEYS; mine += 32)
            if (key + mine >= L) {
                const uint32_t row = words + (mine - C::SI * (lane >> 2)) * ROW_W;
#pragma unroll
                for (int g = 0; g < C::NG; ++g) {
                    sts32(row + 4 * g, 0u);
                    sts32(row + C::WORDS + 4 * g, 0u);
                }
            }
        ptx::fence_proxy_async_smem();  // (the next copy to this stage comes behind)
        __syncwarp();
    }
    uint32_t kw[H][2][C::NG], vw[H][2][C::NG];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) lds_words<C::NG>(words + (C::sixteen(h) + C::SK * k) * ROW_W, kw[h][k]);
    float s[H][C::NT][2][C::E];  // of keys i and i + 8 of a half, the lane's rows
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
        float acc[H][C::NT][4];
#pragma unroll
        for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c) {
            const uint32_t place = (from.k + at) ^ (uint32_t)(c << 4);
            uint32_t a[H], b[H];
#pragma unroll
            for (int h = 0; h < H; ++h) a[h] = lds32(place + C::sixteen(h) * C::ROW), b[h] = lds32(place + C::sixteen(h) * C::ROW + OTHER);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const uint32_t f[4] = {a[h] & 0x000f000fu, b[h] & 0x000f000fu, a[h] & 0x00f000f0u, b[h] & 0x00f000f0u};
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) {
                        if (x == 0 && c == g * C::G / 32) mma_16816_first(acc[h][n], f, w.q[n][c][0], w.q[n][c][1]);
                        else mma_16816(acc[h][n], f, w.q[n][c][2 * x], w.q[n][c][2 * x + 1]);
                    }
                    a[h] >>= 8;
                    b[h] >>= 8;
                }
        }
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float scale = i4_scale(kw[h][k][g]), zero = i4_zero(kw[h][k][g]);
#pragma unroll
                    for (int e = 0; e < C::E; ++e) {
                        const float sum = fmaf(zero, w.q_sum[n][g][e], acc[h][n][2 * k + e]);
                        s[h][n][k][e] = g == 0 ? scale * sum : fmaf(scale, sum, s[h][n][k][e]);
                    }
                }
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) lds_words<C::NG>(words + C::WORDS + (C::sixteen(h) + C::SK * k) * ROW_W, vw[h][k]);
    // hidden keys: past the row's last (a select, so nothing of theirs leaks)
    if (key + C::KEYS > L - back) {
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < C::E; ++e) {
                const int row_last = back == 0 ? L - 1 : L - 1 - back + (row0 + 8 * n + C::E * (lane & 3) + e) % (back + 1);
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (key + C::SI * (lane >> 2) + C::sixteen(h) + C::SK * k > row_last) s[h][n][k][e] = -INFINITY;
            }
    }
    float a[H][2][C::NG];  // the keys' V scales over their references
    {
        bool move = false;
        float low = INFINITY, high = 0.f;  // of the groups' largest scales of the lane's keys
        float most[C::NG];
#pragma unroll
        for (int g = 0; g < C::NG; ++g) most[g] = 0.f;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int g = 0; g < C::NG; ++g) {
                    a[h][k][g] = i4_scale(vw[h][k][g]) * w.inv[g];
                    most[g] = fmaxf(most[g], a[h][k][g]);
                }
                const float la = dec_i4_top<C>(a[h][k]);
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int e = 0; e < C::E; ++e) move |= fmaf(s[h][n][k][e], w.mul[n][e], la) > w.m[n][e];
            }
#pragma unroll
        for (int g = 0; g < C::NG; ++g) low = fminf(low, most[g]), high = fmaxf(high, most[g]);
        move |= ((low < kI4Room / 256.f) & (key + C::KEYS <= L)) | (high > kI4Room * 256.f);
        if (__any_sync(0xffffffffu, move)) {
            dec_i4_move<C>(w, vw, s);
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int g = 0; g < C::NG; ++g) a[h][k][g] = i4_scale(vw[h][k][g]) * w.inv[g];
        }
    }
    // weights, in place of the scores
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < C::E; ++e) {
                    s[h][n][k][e] = ptx::ex2_approx(fmaf(s[h][n][k][e], w.mul[n][e], -w.m[n][e]));
                    w.l[n][e] += s[h][n][k][e];
                }
    // The zeros: sum B z over keys 0 .. 7 of a half, and sum B (15 - z) over keys 8
    // .. 15, whose weights B are negated.  The words, transposed, are a first
    // factor's registers as they are: row 2g has the zeros of group g (modulo
    // four), row 2g + 1 bits of scales, which nobody reads.  15 comes from a register
    // of rows that are else empty.  With two words to a key the 16 bytes of a row
    // are two keys', so rows 0 and 2 are even keys' and 4 and 6 odd keys'.
    constexpr uint32_t kMinus = 0x80008000u, kFifteen = 0x4b804b80u;
    constexpr int ZQ = C::NG > 4 ? 2 * H : H > 1 && !C::kPairs ? H / 2 : 1;
    uint32_t zr[ZQ][4];
    if constexpr (C::ZMMA) {
        if constexpr (C::NG > 4) {
#pragma unroll
            for (int x = 0; x < ZQ; ++x) ldmatrix_x2_trans(from.z + at_words + C::sixteen(x >> 1) * ROW_W + 16 * (x & 1), zr[x]);
        } else if constexpr (H == 1 && C::kPairs) {
            ldmatrix_x1_trans(from.z + at_words, zr[0]);
        } else if constexpr (H == 1 || C::kPairs) {
            ldmatrix_x2_trans(from.z + at_words, zr[0]);
        } else {
#pragma unroll
            for (int x = 0; x < ZQ; ++x) ldmatrix_x4_trans(from.z + at_words + x * 32 * ROW_W, zr[x]);
        }
    }
    uint32_t raw[H][4];
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
        constexpr int PF = C::kTwice ? 2 : 1;
        uint32_t pf[PF][H][C::NT][2];
        float zs[C::NT][4];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            // keys 8 .. 15 of a half: code 15 - c, weight negated
            const float a0 = a[h][0][g], a1 = -a[h][1][g];
#pragma unroll
            for (int n = 0; n < C::NT; ++n) {
                float p0[2], p1[2];
#pragma unroll
                for (int e = 0; e < C::E; ++e) p0[e] = s[h][n][0][e] * a0, p1[e] = s[h][n][1][e] * a1;
                if constexpr (C::kFew) {  // the other column holds what the rounding lost
                    p0[1] = p0[0] - unpack16<true>(ptx::pack_f16x2(p0[0], p0[0])).x;
                    p1[1] = p1[0] - unpack16<true>(ptx::pack_f16x2(p1[0], p1[0])).x;
                }
#pragma unroll
                for (int x = 0; x < PF; ++x) {
                    const uint32_t h0 = ptx::pack_f16x2(p0[0], p0[1]), h1 = ptx::pack_f16x2(p1[0], p1[1]);
                    pf[x][h][n][0] = movmatrix_trans(h0);
                    pf[x][h][n][1] = movmatrix_trans(h1);
                    // (the zeros meet the rounded weights, so that a weight's rounding is of its value's share only)
                    if constexpr (!C::ZMMA) {
                        const float z0 = i4_zero(vw[h][0][g]), z1 = 15.f - i4_zero(vw[h][1][g]);
                        const float2 f0 = unpack16<true>(h0), f1 = unpack16<true>(h1);
                        w.zo[n][g][0] = fmaf(f0.x, z0, fmaf(f1.x, z1, w.zo[n][g][0]));
                        w.zo[n][g][C::E - 1] = fmaf(f0.y, z0, fmaf(f1.y, z1, w.zo[n][g][C::E - 1]));
                    } else {
                        uint32_t f[4];
                        if constexpr (C::kPairs && H == 1) {
                            f[0] = zr[0][0], f[1] = 0u, f[2] = kFifteen, f[3] = zr[0][0] ^ kMinus;
                        } else if constexpr (C::kPairs) {
                            const uint32_t z0 = zr[0][2 * (h >> 1)], z1 = zr[0][2 * (h >> 1) + 1] ^ kMinus;
                            f[0] = h & 1 ? 0u : z0, f[1] = h & 1 ? z0 : 0u, f[2] = h & 1 ? kFifteen : z1, f[3] = h & 1 ? z1 : kFifteen;
                        } else {
                            const int q = C::NG > 4 ? 2 * h + g / 4 : h / 2, y = C::NG > 4 ? 0 : 2 * (h & 1);
                            f[0] = zr[q][y], f[1] = 0u, f[2] = zr[q][y + 1] ^ kMinus, f[3] = kFifteen;
                        }
                        if (h == 0 && x == 0) mma_16816_first(zs[n], f, pf[x][h][n][0], pf[x][h][n][1]);
                        else mma_16816(zs[n], f, pf[x][h][n][0], pf[x][h][n][1]);
                    }
                    if constexpr (C::kTwice) {
                        const float2 f0 = unpack16<true>(h0), f1 = unpack16<true>(h1);
                        p0[0] -= f0.x, p0[1] -= f0.y, p1[0] -= f1.x, p1[1] -= f1.y;
                    }
                }
            }
        }
        if constexpr (C::ZMMA) {
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        w.zo[n][g][(k * C::E + (C::kFew ? 0 : e)) % C::ZE] += zs[n][2 * k + e];
        }
#pragma unroll
        for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c) {
            uint32_t lo[H], hi[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                if (c % 2 == 0) ldmatrix_x4_trans(((from.v + at) ^ (uint32_t)(c << 4)) + C::sixteen(h) * C::ROW, raw[h]);
                lo[h] = raw[h][c % 2 * 2], hi[h] = raw[h][c % 2 * 2 + 1];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const uint32_t f[4] = {lo[h] & 0x000f000fu, lo[h] & 0x00f000f0u, ~hi[h] & 0x000f000fu, ~hi[h] & 0x00f000f0u};
#pragma unroll
                    for (int n = 0; n < C::NT; ++n)
#pragma unroll
                        for (int y = 0; y < PF; ++y) mma_16816(w.o[n][c][x], f, pf[y][h][n][0], pf[y][h][n][1]);
                    lo[h] >>= 8;
                    hi[h] >>= 8;
                }
        }
    }
}

// All warps of a row group.  (A number known at compile time: a variable one
// takes all sixteen barriers for the CTA.)
template <class C>
__device__ __forceinline__ void dec_i4_meet(int rg) {
    if (C::RG == 1 || rg == 0) ptx::named_bar_sync(1, C::KW * 32);
    else if (C::RG == 2 || rg == 1) ptx::named_bar_sync(2, C::KW * 32);
    else if (rg == 2) ptx::named_bar_sync(3, C::KW * 32);
    else ptx::named_bar_sync(4, C::KW * 32);
}

// A warp's sums as float4s of each lane: put(k, x) stores the k-th, get(k) loads it.
template <class C, class Put>
__device__ __forceinline__ void dec_i4_lay_down(const DecI4Warp<C> &w, Put put) {
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        put(C::E * C::NT * C::NC + n, make_float4(w.m[n][0], w.m[n][C::E - 1], w.l[n][0], w.l[n][C::E - 1]));
#pragma unroll
        for (int c = 0; c < C::NC; ++c)
#pragma unroll
            for (int e = 0; e < C::E; ++e)
                put((n * C::NC + c) * C::E + e,
                    make_float4(w.o[n][c][0][e], w.o[n][c][0][2 + e], w.o[n][c][1][e], w.o[n][c][1][2 + e]));
    }
}

// Adds such sums to a warp's.  (kMany: of any number of pieces, so that the sum of weights is kept below 1.)
template <class C, bool kMany, class Get>
__device__ __forceinline__ void dec_i4_join(DecI4Warp<C> &w, Get get) {
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        const float4 ml = get(C::E * C::NT * C::NC + n);
        float mine[C::E], theirs[C::E];  // what the two sides' sums are multiplied by
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            const float m = e ? ml.y : ml.x, top = fmaxf(w.m[n][e], m);
            mine[e] = ptx::ex2_approx(w.m[n][e] - top);
            theirs[e] = ptx::ex2_approx(m - top);
            w.m[n][e] = top;
            w.l[n][e] = fmaf(w.l[n][e], mine[e], (e ? ml.w : ml.z) * theirs[e]);
            if (kMany && w.l[n][e] >= 1.f) w.l[n][e] *= 0.5f, mine[e] *= 0.5f, theirs[e] *= 0.5f, w.m[n][e] += 1.f;
        }
#pragma unroll
        for (int c = 0; c < C::NC; ++c)
#pragma unroll
            for (int e = 0; e < C::E; ++e) {
                const float4 y = get((n * C::NC + c) * C::E + e);
                float(&o)[2][4] = w.o[n][c];
                o[0][e] = fmaf(o[0][e], mine[e], y.x * theirs[e]);
                o[0][2 + e] = fmaf(o[0][2 + e], mine[e], y.y * theirs[e]);
                o[1][e] = fmaf(o[1][e], mine[e], y.z * theirs[e]);
                o[1][2 + e] = fmaf(o[1][2 + e], mine[e], y.w * theirs[e]);
            }
    }
}

// The unit's end, or a rest within it.  A row group's warps hand their sums down, half
// of them to the other half at a time; the last adds what it laid down at earlier
// rests and writes the rows out, or a partial of them, or lays them down.
template <class C>
__device__ __forceinline__ void dec_i4_end_unit(const DecInt4Params &p, const DecFp8It &it, DecI4Warp<C> &w, int rg, int kwi,
                                                int lane, bool whole, bool begun_here, bool rested, bool rests, uint32_t parts) {
    const int i = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) w.l[n][e] += __shfl_xor_sync(0xffffffffu, w.l[n][e], o);
            // The reference goes to where the sum of weights is in [1/8, 1/4): sums of values near the
            // largest numbers stay finite, and those of the warps can be compared by their references.
            const int to = w.l[n][e] > 0.f ? min((int)(__float_as_uint(w.l[n][e]) >> 23) - 124, 126) : 0;
            w.m[n][e] += (float)to;
            w.l[n][e] *= __uint_as_float((uint32_t)(127 - to) << 23);
#pragma unroll
            for (int g = 0; g < C::NG; ++g) {
                float z = w.zo[n][g][e];
                if constexpr (!C::ZMMA) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                } else {  // row 2g of the products (and row 12 + 2g)
                    z = __shfl_sync(0xffffffffu, z, 8 * (g & 3) + t);
                    if constexpr (C::ZE == 2 * C::E) z += __shfl_sync(0xffffffffu, w.zo[n][g][C::ZE - C::E + e], 16 + 8 * g + t);
                }
                // (the sums are kI4Room / ref too large, too; half of the step on either side of the
                // difference, as all of it could leave fp32's range)
                const uint32_t inv = __float_as_uint(w.inv[g]);
                const int step = 127 - (int)(inv >> 23) - to, half = step >> 1;
                const float first = __uint_as_float((uint32_t)(127 + half) << 23);
                const float second = inv == 0 ? 0.f : __uint_as_float((uint32_t)(127 + step - half) << 23);
                const float lower = 16777216.f * first, upper = 1048576.f * first;
                z *= first;
#pragma unroll
                for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c) {
                    if constexpr (C::kFew)
#pragma unroll
                        for (int x = 0; x < 2; ++x) w.o[n][c][x][0] += w.o[n][c][x][1], w.o[n][c][x][2] += w.o[n][c][x][3];
                    w.o[n][c][0][e] = second * fmaf(w.o[n][c][0][e], lower, -z);
                    w.o[n][c][0][2 + e] = second * fmaf(w.o[n][c][0][2 + e], upper, -z);
                    w.o[n][c][1][e] = second * fmaf(w.o[n][c][1][e], lower, -z);
                    w.o[n][c][1][2 + e] = second * fmaf(w.o[n][c][1][2 + e], upper, -z);
                }
            }
        }
    dec_i4_meet<C>(rg);  // the unit before is read
    {
#pragma unroll
        for (int half = C::KW / 2; half > 0; half >>= 1) {
            // (the last `half` places: a warp that hands its sums down writes where it has
            // itself read the ones before, each lane its own; the others may still read)
            const uint32_t at = parts + (rg * (C::KW / 2) + C::KW / 2 - half + kwi % half) * C::PART + lane * 16;
            if (kwi >= half && kwi < 2 * half)
                dec_i4_lay_down<C>(w, [&](int k, float4 x) { sts_float4(at + k * 512, x.x, x.y, x.z, x.w); });
            dec_i4_meet<C>(rg);
            if (kwi < half) dec_i4_join<C, false>(w, [&](int k) { return lds_float4(at + k * 512); });
        }
    }
    if (kwi != 0) return;
    if constexpr (C::kRests) {
        float4 *sums = p.sums + ((size_t)blockIdx.x * C::RG + rg) * (C::PART / 16) + lane;
        if (rested) dec_i4_join<C, true>(w, [&](int k) { return sums[k * 32]; });
        if (rests) {
            dec_i4_lay_down<C>(w, [&](int k, float4 x) { sums[k * 32] = x; });
            return;
        }
    }
    int rows;
    const size_t row0 = dec_fp8_row0(p, it.b, it.kvh, it.chunk, &rows);
    const size_t slot = 2 * (size_t)blockIdx.x + (begun_here ? 1 : 0);
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            const int r = (rg * C::NT + n) * 8 + C::E * t + e;
            if (r >= rows) continue;
            const float l = w.l[n][e], inv = l == 0.f ? 0.f : 1.f / l;
            const float lse2 = l == 0.f ? -INFINITY : w.m[n][e] + __log2f(l);  // (a NaN sum is no empty row)
            if (i == 0) {
                if (whole) p.lse[row0 + r] = lse2 * kLn2;
                else p.part_lse[slot * C::RC + r] = lse2;
            }
#pragma unroll
            for (int c = 0; c < C::NC; ++c) {
                const float y0 = w.o[n][c][0][e] * inv, y1 = w.o[n][c][0][2 + e] * inv;
                const float y2 = w.o[n][c][1][e] * inv, y3 = w.o[n][c][1][2 + e] * inv;
                const int d = 32 * c + 4 * i;
                if (whole)
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + (row0 + r) * C::D + d) =
                        p.fp16 ? make_uint2(ptx::pack_f16x2(y0, y1), ptx::pack_f16x2(y2, y3))
                               : make_uint2(ptx::pack_bf16x2(y0, y1), ptx::pack_bf16x2(y2, y3));
                else
                    *reinterpret_cast<float4 *>(p.part_o + (slot * C::RC + r) * C::D + d) = make_float4(y0, y1, y2, y3);
            }
        }
}

template <class C>
__device__ void dec_i4_warp(const DecInt4Params &p, DecFp8It it, uint32_t ring, uint32_t parts, uint32_t kept, uint32_t bars,
                            int *begun, Ctl *ctl) {
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5, rg = warp / C::KW, kwi = warp % C::KW;
    if (it.left <= 0) return;
    uint4 raw[C::NT][C::NC];
    dec_i4_load_q<C>(p, it, rg, lane, raw);
    // The warps take turns at the copies.  Of the first ST - 1 tiles, tile n is warp
    // n % WARPS's; warp t % WARPS copies tile t + ST - 1, behind its own keys of tile
    // t, to where tile t - 1 was, which the others have read by then.  (In front of
    // its keys it waits for them: kv8 84 -> 94 us.)
    DecFp8It ahead = it;
    int entry = 0;
    bool some;
    {
        dec_i4_advance(p, ahead, warp);
        for (int n = warp; n < C::ST - 1; n += C::WARPS) {
            if (ahead.left > 0) {
                if (lane == 0) begun[n] = n + 1;
                some = dec_i4_entry<C>(p, ahead, lane, entry);
                dec_i4_copy<C>(p, ahead.kvh, some, entry, lane, ring + n * C::STAGE, bar_addr(bars, C::B_FULL + n));
            }
            dec_i4_advance(p, ahead, C::WARPS);
        }
        ahead = it;
        dec_i4_advance(p, ahead, warp + C::ST - 1);
    }
    dec_i4_keep(ahead, lane, kept);
    some = dec_i4_entry<C>(p, ahead, lane, entry);
    const DecI4Lane from = dec_i4_lane<C>(ring, lane, kwi * C::SPT * C::KEYS);
    const int back = p.mask_kind == kMaskCausal ? p.Sq - 1 : 0;
    DecI4Warp<C> w;
    dec_i4_begin_unit<C>(p, raw, lane, w);
    bool begun_here = it.tile == 0, bad = false;
    // (one warp's wait, so that the others wind down from wherever they are)
    if (p.stall_test && warp == (int)(blockIdx.x % C::WARPS)) bad = !wait_warp(bar_addr(bars, C::B_NEVER), 0, ctl, 92);
    int slot = 0, turn = warp;      // turn: tiles until this warp's next copy
    int tiles = 0;                  // of the unit so far
    uint32_t phase = 0;
    int t = 0;
    for (;;) {
        // (a warp whose wait ran out goes on without its tiles, so that the others meet it at the units' ends)
        if (!bad) bad = !wait_warp(bar_addr(bars, C::B_FULL + slot), phase, ctl, 92);
        // (a row group behind the chunk's last rows has nothing to do)
        const bool idle = C::RG > 1 && rg * 8 * C::NT >= min(p.rows_per_chunk, p.R - it.chunk * p.rows_per_chunk);
        int key = it.tile * C::BN + kwi * C::SPT * C::KEYS;
#pragma unroll 1
        for (int j = 0; j < C::SPT; ++j, key += C::KEYS) {
            if (bad || key >= it.L || idle) break;
            dec_i4_keys<C>(w, key, it.L, back, it.chunk * p.rows_per_chunk + rg * C::NT * 8, lane, from,
                           slot * C::STAGE + j * C::KEYS * C::ROW, slot * C::STAGE + j * C::KEYS * C::NG * 4);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_addr(bars, C::B_EMPTY + slot));
        if (turn == 0) {
            turn = C::WARPS;
            DecFp8It coming = dec_i4_take(kept);
            if (coming.left > 0 && !bad) {
                const int prev = slot == 0 ? C::ST - 1 : slot - 1;
                bad = t > 0 && !wait_warp(bar_addr(bars, C::B_EMPTY + prev), slot == 0 ? phase ^ 1 : phase, ctl, 91);
                if (!bad) {
                    if (lane == 0) begun[prev] = t + C::ST;
                    dec_i4_copy<C>(p, coming.kvh, some, entry, lane, ring + prev * C::STAGE, bar_addr(bars, C::B_FULL + prev));
                    dec_i4_advance(p, coming, C::WARPS);
                    dec_i4_keep(coming, lane, kept);
                    some = dec_i4_entry<C>(p, coming, lane, entry);
                }
            }
        }
        --turn;
        ++t;
        if (++slot == C::ST) slot = 0, phase ^= 1;
        const bool ends = it.tile + 1 == it.nt, done = it.left == 1;
        const bool rests = C::kRests && ++tiles % C::REST == 0 && !ends && !done;
        if (ends || done || rests) {
            DecFp8It next = it;
            dec_fp8_step(p, next);
            if (!done) dec_i4_load_q<C>(p, next, rg, lane, raw);
            dec_i4_end_unit<C>(p, it, w, rg, kwi, lane, begun_here && ends, begun_here, tiles > C::REST, rests, parts);
            if (done) break;
            it = next;
            dec_i4_begin_unit<C>(p, raw, lane, w);
            if (ends) begun_here = true, tiles = 0;
        } else {
            ++it.tile;
            --it.left;
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::NUM_THREADS, C::CTAS_PER_SM)
    fa_decode_int4_kernel(const __grid_constant__ DecInt4Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *parts = ring + C::ST * C::STAGE;
    uint8_t *kept = parts + C::PARTS * C::PART;
    uint64_t *bar_mem = reinterpret_cast<uint64_t *>(kept + C::WARPS * kI4Kept);
    Ctl *ctl = reinterpret_cast<Ctl *>(bar_mem + C::NUM_BARS);
    int *begun = reinterpret_cast<int *>(ctl + 1);  // [ST] 1 + the tile whose copy to a place was begun last; 0: none
    const uint32_t bars = ptx::smem_addr(bar_mem);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::ST; ++s) {
            ptx::mbar_init(bar_addr(bars, C::B_FULL + s), dec_i4_words_by_lanes(p) ? 1 + 32 : 1);  // (each lane's words, too)
            ptx::mbar_init(bar_addr(bars, C::B_EMPTY + s), C::WARPS);
            begun[s] = 0;
        }
        ptx::mbar_init(bar_addr(bars, C::B_NEVER), 1);
        ctl->abort = 0;
        ctl->limit_ns = p.wait_limit_ns;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
        ptx::prefetch_tensormap(&p.tm_k);
        ptx::prefetch_tensormap(&p.tm_v);
    }
    ptx::wait_for_previous_kernel();
    const DecFp8It it = dec_fp8_begin<C::NUM_THREADS>(p, reinterpret_cast<long long *>(parts));
    __syncthreads();
    // the merge may be set up now; it waits for this grid's end before it reads
    ptx::let_next_kernel_begin();
    dec_i4_warp<C>(p, it, ptx::smem_addr(ring), ptx::smem_addr(parts),
                   ptx::smem_addr(kept) + (threadIdx.x >> 5) * kI4Kept, bars, begun, ctl);
    __syncthreads();
    // The CTA's memory stays until its last copies have landed, also where the
    // warps gave up waiting for them.  (Where one gave up, tiles that were its turn
    // are missing in between: each place has its own last tile.)
    if (ctl->abort && threadIdx.x == 0)
        for (int s = 0; s < C::ST; ++s)
            if (const int n = begun[s]) wait_bar_drain(bar_addr(bars, C::B_FULL + s), ((n - 1) / C::ST) & 1);
}

}  // namespace fa
