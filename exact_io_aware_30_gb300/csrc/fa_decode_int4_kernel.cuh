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
// so every product takes one group: 32 adjacent components, four words of 8, lane t
// of four word t.  (Products by warps, mma.sync: the codes pass through registers
// anyway, their fragments need no shared memory, and 16 keys and 8 rows to a
// product are 0.3 of its rate at the memory's pace.)
//   S^T = K Q^T: 16 keys x 8 rows per product, K words straight from shared memory.
//   O^T = V^T P^T: ldmatrix transposes V by units of 16 bits, four codes of one
//   key; the weights' fragment is S's, rounded to fp16 and turned by movmatrix.
// Every other key's codes enter as 15 - c, with its weight negated (the
// complement is part of the same masking instruction), so that O's sums, which
// the tensor core cuts off rather than rounds, do not grow with the 7.5 that
// codes are on average; what that leaves out goes with the zeros.
//
// Weights.  What P V takes is p s / ref_g in fp16: 2^-11 of itself, and no finer
// than 2^-25 of the row's largest product so far: rows are taken relative to a
// running maximum M of x + log2 max_g (s / ref_g), which may stay up to 6 below
// the true one, and each group's scales relative to a power of two that the
// step's largest is kept within 2^8 of.  Both move rarely, by a branch of the
// whole warp that rescales what it has summed.
//
// Work split: the line of 128-key tiles of fa_decode_fp8_kernel.cuh, an even
// share of it per CTA, cut units merged by its second kernel.  One CTA: a ring of
// tiles, K and V codes and words, that its eight warps take turns at filling; a
// warp takes 16 keys of a tile (or fewer warps more keys, the others other rows)
// and has a running maximum and sums of its own, so that nothing is exchanged
// before the unit's end.  (With a ninth warp for the copies two CTAs' warps get 96
// registers instead of 128.)
#pragma once

#include <math.h>
#include <stdint.h>

#include "fa_decode_fp8_kernel.cuh"
#include "fa_int4_kernel.cuh"

namespace fa {

struct DecInt4Params : DecFp8Params {  // (k_scale and v_scale are not used)
    const uint32_t *k_words, *v_words;  // [num_blocks, Hkv, bs, d / G]
    int fp16;
};

template <int D_, int G_, int NT_, int RG_>
struct DecI4Cfg {
    static constexpr int D = D_;
    static constexpr int G = G_;                  // components per group
    static constexpr int NT = NT_;                // eights of rows per warp
    static constexpr int RG = RG_;                // groups of warps with different rows
    static constexpr int RC = 8 * NT * RG;        // rows per unit
    static constexpr int WARPS = 8;
    static constexpr int KW = WARPS / RG;         // warps along a tile's keys
    static constexpr int KPW = 8 / KW;            // 16-key steps per warp and tile
    static constexpr int BN = 128;
    static constexpr int NG = D / G;
    static constexpr int NC = D / 32;             // chunks of 32 components, 16 bytes
    static constexpr int ROW = D / 2;             // bytes of a row of codes
    static constexpr int TILE = BN * ROW;
    static constexpr int WORDS = BN * NG * 4;     // bytes of a tile's words
    static constexpr int Q_BYTES = RC * D * 2;
    static constexpr int O_V = TILE, O_KW = 2 * TILE, O_VW = O_KW + WORDS, O_Q = O_VW + WORDS;  // places in a stage
    static constexpr int STAGE = (O_Q + Q_BYTES + 1023) / 1024 * 1024;
    static constexpr int OROW = D + 4;            // floats of a partial row: no two lanes of a store on a bank
    static constexpr int SCRATCH = WARPS * 8 * NT * OROW * 4;
    static constexpr int CTAS_PER_SM = D <= 128 && NT == 1 && RG == 1 ? 2 : 1;
    static constexpr int BUDGET = CTAS_PER_SM == 2 ? 113 * 1024 : 226 * 1024;
    static constexpr int FIXED = 1024 + SCRATCH + 2 * WARPS * 8 * NT * 4 + 256;
    static constexpr int FIT = (BUDGET - FIXED) / STAGE;
    static constexpr int ST = FIT < 8 ? FIT : 8;
    static_assert(ST >= 2 && ST <= WARPS, "a ring of at least two tiles, a warp to begin each");
    static constexpr int SMEM_BYTES = FIXED + ST * STAGE;
    static constexpr int NUM_THREADS = 32 * WARPS;
    static constexpr int B_FULL = 0;
    static constexpr int B_EMPTY = ST;
    static constexpr int B_NEVER = 2 * ST;
    static constexpr int NUM_BARS = 2 * ST + 1;
    static_assert(NUM_BARS * 8 + 32 <= 256, "layout");
};

// ------------------------------------------------------------------- copies

// Lane 4k + j copies part j (K codes, V codes, K words, V words) of block k of
// a tile; its table entry, or -1 where it has none to copy, -2 where the entry is
// outside the pool.
template <class C>
__device__ __forceinline__ int dec_i4_entry(const DecInt4Params &p, const DecFp8It &it) {
    const int blk = (int)ptx::lane_id() >> 2, n = ((it.tile * C::BN) >> p.bs_log2) + blk;
    if (blk >= C::BN >> p.bs_log2 || it.left <= 0 || (n << p.bs_log2) >= it.L) return -1;
    const int e = p.block_table[(size_t)it.b * p.max_blocks + n];
    return e >= 0 && e < p.num_blocks ? e : -2;
}

// Copies a tile (and q's rows, where it begins a unit here) into a stage that is
// free.  The whole warp.  Slots behind the request's blocks are not read later;
// a block outside the pool gets zero words, whatever its codes.
template <class C>
__device__ __forceinline__ void dec_i4_copy(const DecInt4Params &p, const DecFp8It &it, int entry, bool begins, uint32_t stage,
                                            uint32_t bar, uint64_t pol) {
    const int lane = (int)ptx::lane_id(), part = lane & 3, row = (lane >> 2) << p.bs_log2;
    const uint32_t word_bytes = (uint32_t)(C::NG * 4) << p.bs_log2;
    const uint32_t words_at = stage + (part & 1 ? C::O_VW : C::O_KW) + row * C::NG * 4;
    if (entry == -2 && part >= 2) {
        for (uint32_t i = 0; i < word_bytes; i += 16) ptx::st_shared_v4(words_at + i, 0u, 0u, 0u, 0u);
        ptx::fence_proxy_async_smem();
    }
    const uint32_t blocks = (uint32_t)__popc(__ballot_sync(0xffffffffu, entry >= 0)) / 4;
    if (lane == 0) {
        uint32_t bytes = blocks * (2 * word_bytes + ((uint32_t)(2 * C::ROW) << p.bs_log2));
        int rows = 0;
        size_t row0 = 0;
        if (begins) {
            row0 = dec_fp8_row0(p, it.b, it.kvh, it.chunk, &rows);
            bytes += (uint32_t)rows * C::D * 2;
        }
        ptx::mbar_arrive_expect_tx(bar, bytes);
        if (begins) ptx::bulk_load(stage + C::O_Q, p.q + row0 * C::D, (uint32_t)rows * C::D * 2, bar);
    }
    __syncwarp();
    if (entry >= 0) {
        if (part < 2) {
            ptx::tma_load_4d(stage + (part ? C::O_V : 0) + row * C::ROW, part ? &p.tm_v : &p.tm_k, bar, 0, 0, it.kvh, entry, pol);
        } else {
            const size_t at = (((size_t)entry * p.Hkv + it.kvh) << p.bs_log2) * C::NG;
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

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// (v & mask) ^ flip in one instruction
__device__ __forceinline__ uint32_t and_xor(uint32_t v, uint32_t mask, uint32_t flip) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(v), "r"(mask), "r"(flip));
    return r;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

__device__ __forceinline__ float i4_scale(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float i4_zero(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
}

// What a warp holds of its unit.  Lane i * 4 + t: keys i and i + 8 of a step,
// rows 2t and 2t + 1 of each eight; of O, components 4i .. 4i + 3 of each chunk.
template <class C>
struct DecI4Warp {
    uint32_t q[C::NT][C::NC][4];     // fragments of q
    float q_sum[C::NT][C::NG][2];    // 2^-20 times the groups' sums of q
    float mul[C::NT][2];             // from a sum of products to log2 units
    int last[C::NT][2];              // last key the row sees
    float m[C::NT][2];               // reference of the exponents, -inf before the first key
    float l[C::NT][2];               // this lane's sums of weights
    float inv[C::NG];                // 1 / ref of the groups' V scales, a power of two; 0 before the first key
    float o[C::NT][C::NC][2][4];     // sums of weights times codes
    float zo[C::NT][C::NG][2];       // this lane's sums of weights times zeros
};

// q's rows from the ring into fragments.  A row is scaled by a power of two so
// that its largest component is in [2^10, 2^11); 16-bit components are then
// exact in fp16 down to 2^-24 of it (and 2^-25 of the row's scale is the most a
// smaller one is off).  A row with an infinity, a NaN or a component of 2^112 or
// more is NaN.
template <class C>
__device__ __forceinline__ void dec_i4_begin_unit(const DecInt4Params &p, const DecFp8It &u, const uint16_t *sq, int rg,
                                                  DecI4Warp<C> &w) {
    const int lane = (int)threadIdx.x & 31, i = lane >> 2, t = lane & 3;
    const int r_first = u.chunk * p.rows_per_chunk, rows = min(p.rows_per_chunk, p.R - r_first);
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        const int r = (rg * C::NT + n) * 8 + i;
        uint4 raw[C::NC];
        uint32_t mag = 0;
#pragma unroll
        for (int c = 0; c < C::NC; ++c) {
            raw[c] = make_uint4(0, 0, 0, 0);
            if (r < rows) raw[c] = *reinterpret_cast<const uint4 *>(sq + r * C::D + 32 * c + 8 * t);
            mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(raw[c].x & 0x7fff7fffu, raw[c].y & 0x7fff7fffu),
                                         __vmaxu2(raw[c].z & 0x7fff7fffu, raw[c].w & 0x7fff7fffu)));
        }
        mag = max(mag & 0xffffu, mag >> 16);
        mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
        mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
        const float top = p.fp16 ? unpack16<true>(mag).x : unpack16<false>(mag).x;
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
            const uint32_t ws[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = p.fp16 ? unpack16<true>(ws[e]) : unpack16<false>(ws[e]);
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
            sum[g] = fine ? sum[g] * 9.5367431640625e-7f : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int from = (2 * t + e) * 4, row = r_first + (rg * C::NT + n) * 8 + 2 * t + e;
#pragma unroll
            for (int g = 0; g < C::NG; ++g) w.q_sum[n][g][e] = __shfl_sync(0xffffffffu, sum[g], from);
            w.mul[n][e] = __shfl_sync(0xffffffffu, mul, from);
            w.last[n][e] = p.mask_kind != kMaskCausal || p.Sq == 1 ? u.L - 1 : u.L - p.Sq + row % p.Sq;
            w.m[n][e] = -INFINITY;
            w.l[n][e] = 0.f;
#pragma unroll
            for (int g = 0; g < C::NG; ++g) w.zo[n][g][e] = 0.f;
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

// log2 of the largest of a key's V scales relative to their references.
template <class C>
__device__ __forceinline__ float dec_i4_top(const float (&a)[C::NG]) {
    float top = 9.09494702e-13f;  // 2^-40: a key without a scale does not move the reference far
#pragma unroll
    for (int g = 0; g < C::NG; ++g) top = fmaxf(top, a[g]);
    return lg2_approx(top);
}

// Moves the references of the groups' scales (where the step's largest is more
// than 2^8 away) and of the exponents (up to the step's largest) and rescales
// the sums.  vs: the V scales of the lane's two keys; s: their scores' sums of
// products.  The whole warp.
template <class C>
__device__ __forceinline__ void dec_i4_move(DecI4Warp<C> &w, const float (&vs)[2][C::NG], const float (&s)[C::NT][4]) {
    float rise = -INFINITY;  // log2 of the factor of the group that grows most
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
        const float top = warp_max(fmaxf(vs[0][g], vs[1][g]));  // (a NaN scale is passed over)
        const uint32_t ex = min(max(__float_as_uint(top) >> 23, 1u), 253u);
        const float old = w.inv[g], now = __uint_as_float((254u - ex) << 23);
        float factor = 1.f;
        if (old == 0.f) {
            if (top > 0.f) w.inv[g] = now;
            else rise = fmaxf(rise, 0.f);  // (still without one)
            continue;
        }
        const float rel = top * old;
        if (rel > 256.f) {
            factor = now / old;  // < 1
            w.inv[g] = now;
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
                most = fmaxf(most, fmaxf(fabsf(w.zo[n][g][0]), fabsf(w.zo[n][g][1])));
            }
            most = warp_max(most);
            const uint32_t room = 200u - min(__float_as_uint(most) >> 23, 200u);  // up to 2^73
            const uint32_t from = __float_as_uint(old) >> 23, to = min(254u - ex, from + room);
            w.inv[g] = __uint_as_float(to << 23);
            factor = __uint_as_float((to - from + 127u) << 23);
        }
        if (factor != 1.f) {
#pragma unroll
            for (int n = 0; n < C::NT; ++n) {
#pragma unroll
                for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) w.o[n][c][h][e] *= factor;
                w.zo[n][g][0] *= factor;
                w.zo[n][g][1] *= factor;
            }
        }
        rise = fmaxf(rise, lg2_approx(factor));
    }
    float la[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float a[C::NG];
#pragma unroll
        for (int g = 0; g < C::NG; ++g) a[g] = vs[k][g] * w.inv[g];
        la[k] = dec_i4_top<C>(a);
    }
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float top = fmaxf(fmaf(s[n][e], w.mul[n][e], la[0]), fmaf(s[n][2 + e], w.mul[n][e], la[1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float old = w.m[n][e], now = fmaxf(old + fminf(rise, 0.f), top);
            const float f = old == -INFINITY ? 0.f : ptx::ex2_approx(old - now);
            w.m[n][e] = now;
            w.l[n][e] *= f;
#pragma unroll
            for (int g = 0; g < C::NG; ++g) w.zo[n][g][e] *= f;
#pragma unroll
            for (int c = 0; c < C::NC; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w.o[n][c][h][e] *= f;
                    w.o[n][c][h][2 + e] *= f;
                }
        }
}

// 16 keys, the first of them `key`, at rows of codes ks and vs and words kws and vws.
template <class C>
__device__ __forceinline__ void dec_i4_keys(const DecInt4Params &p, DecI4Warp<C> &w, int key, int L, int seen_by_all,
                                            uint32_t ks, uint32_t vs, uint32_t kws, uint32_t vws) {
    const int lane = (int)threadIdx.x & 31, i = lane >> 2, t = lane & 3;
    // 16-byte chunk c of row r of a box is chunk c ^ swizzle(r)
    auto swizzle = [](int r) { return C::ROW == 128 ? r & 7 : C::ROW == 64 ? (r >> 1) & 3 : (r >> 2) & 1; };
    uint32_t kw[2][C::NG], vw[2][C::NG];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        lds_words<C::NG>(kws + (i + 8 * k) * C::NG * 4, kw[k]);
        lds_words<C::NG>(vws + (i + 8 * k) * C::NG * 4, vw[k]);
    }
    if (key + 16 > L) {  // slots past the request's tokens may hold anything
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int g = 0; g < C::NG; ++g)
                if (key + i + 8 * k >= L) kw[k][g] = vw[k][g] = 0;
    }
    float s[C::NT][4];
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
    const uint32_t k_lane = ks + i * C::ROW + (swizzle(i) << 4) + 4 * t;
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
        const float s0 = i4_scale(kw[0][g]), s1 = i4_scale(kw[1][g]);
        const float z0 = -i4_zero(kw[0][g]), z1 = -i4_zero(kw[1][g]);
        float acc[C::NT][4];
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
            acc[n][0] = z0 * w.q_sum[n][g][0];
            acc[n][1] = z0 * w.q_sum[n][g][1];
            acc[n][2] = z1 * w.q_sum[n][g][0];
            acc[n][3] = z1 * w.q_sum[n][g][1];
        }
#pragma unroll
        for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c) {
            uint32_t a = lds32(k_lane ^ (uint32_t)(c << 4)), b = lds32((k_lane ^ (uint32_t)(c << 4)) + 8 * C::ROW);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t f[4] = {a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u};
#pragma unroll
                for (int n = 0; n < C::NT; ++n) mma_16816(acc[n], f, w.q[n][c][2 * h], w.q[n][c][2 * h + 1]);
                a >>= 8;
                b >>= 8;
            }
        }
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
            s[n][0] = fmaf(s0, acc[n][0], s[n][0]);
            s[n][1] = fmaf(s0, acc[n][1], s[n][1]);
            s[n][2] = fmaf(s1, acc[n][2], s[n][2]);
            s[n][3] = fmaf(s1, acc[n][3], s[n][3]);
        }
    }
    // hidden keys: past the row's last (a select, so nothing of theirs leaks)
    if (key + 15 > seen_by_all) {
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (key + i + 8 * (e >> 1) > w.last[n][e & 1]) s[n][e] = -INFINITY;
    }
    float a[2][C::NG];
    {
        float low = INFINITY;  // the smallest group's larger scale
#pragma unroll
        for (int g = 0; g < C::NG; ++g) {
            a[0][g] = i4_scale(vw[0][g]) * w.inv[g];
            a[1][g] = i4_scale(vw[1][g]) * w.inv[g];
            low = fminf(low, fmaxf(a[0][g], a[1][g]));
        }
        float la[2];
        la[0] = dec_i4_top<C>(a[0]);
        la[1] = dec_i4_top<C>(a[1]);
        bool move = low < 0.00390625f || fmaxf(la[0], la[1]) > 8.f;
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                move = move || fmaf(s[n][e], w.mul[n][e & 1], la[e >> 1]) > w.m[n][e & 1] + 6.f;
        if (__any_sync(0xffffffffu, move)) {
            float raw[2][C::NG];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int g = 0; g < C::NG; ++g) raw[k][g] = i4_scale(vw[k][g]);
            dec_i4_move<C>(w, raw, s);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int g = 0; g < C::NG; ++g) a[k][g] = raw[k][g] * w.inv[g];
        }
    }
    // weights, in place of the scores
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float m = w.m[n][e & 1];
            s[n][e] = ptx::ex2_approx(fmaf(s[n][e], w.mul[n][e & 1], m == -INFINITY ? 0.f : -m));
            w.l[n][e & 1] += s[n][e];
        }
    // odd keys: code 15 - c, weight negated
    const float sign = i & 1 ? -1.f : 1.f, over = i & 1 ? 15.f : 0.f;
    const int v_row = lane & 15;
    const uint32_t v_lane = vs + v_row * C::ROW + ((swizzle(v_row) ^ (lane >> 4)) << 4);
    uint32_t raw[4];
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
        uint32_t pf[C::NT][2];
        const float z0 = fmaf(sign, i4_zero(vw[0][g]), over), z1 = fmaf(sign, i4_zero(vw[1][g]), over);
        const float a0 = sign * a[0][g], a1 = sign * a[1][g];
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
            const uint32_t h0 = ptx::pack_f16x2(s[n][0] * a0, s[n][1] * a0), h1 = ptx::pack_f16x2(s[n][2] * a1, s[n][3] * a1);
            // the zeros meet the rounded weights, so that a weight's rounding is of its value's share only
            const float2 f0 = unpack16<true>(h0), f1 = unpack16<true>(h1);
            w.zo[n][g][0] = fmaf(f0.x, z0, fmaf(f1.x, z1, w.zo[n][g][0]));
            w.zo[n][g][1] = fmaf(f0.y, z0, fmaf(f1.y, z1, w.zo[n][g][1]));
            pf[n][0] = movmatrix_trans(h0);
            pf[n][1] = movmatrix_trans(h1);
        }
#pragma unroll
        for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c) {
            if (c % 2 == 0) ldmatrix_x4_trans(v_lane ^ (uint32_t)(c << 4), raw);
            uint32_t lo = raw[c % 2 * 2], hi = raw[c % 2 * 2 + 1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t f[4] = {and_xor(lo, 0x000f000fu, 0x000f0000u), and_xor(lo, 0x00f000f0u, 0x00f00000u),
                                       and_xor(hi, 0x000f000fu, 0x000f0000u), and_xor(hi, 0x00f000f0u, 0x00f00000u)};
#pragma unroll
                for (int n = 0; n < C::NT; ++n) mma_16816(w.o[n][c][h], f, pf[n][0], pf[n][1]);
                lo >>= 8;
                hi >>= 8;
            }
        }
    }
}

// The unit's end: the warps of a row group leave their sums, and together
// write the rows out, or a partial of them.
template <class C>
__device__ __forceinline__ void dec_i4_end_unit(const DecInt4Params &p, const DecFp8It &it, DecI4Warp<C> &w, int rg, int kwi,
                                                bool whole, bool begun_here, float *scratch, float *ml) {
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5, i = lane >> 2, t = lane & 3;
    constexpr int RW = 8 * C::NT;
    float *mine = scratch + warp * RW * C::OROW;
    float *ml_mine = ml + warp * RW * 2;
    int rows;
    const size_t row0 = dec_fp8_row0(p, it.b, it.kvh, it.chunk, &rows);
    rows = min(rows - rg * RW, RW);  // of this row group (0 or less: none)
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        if (8 * n >= rows) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = w.l[n][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            const int r = 8 * n + 2 * t + e;
            if (i == 0) {
                ml_mine[2 * r] = w.m[n][e];
                ml_mine[2 * r + 1] = l;
            }
#pragma unroll
            for (int g = 0; g < C::NG; ++g) {
                float z = w.zo[n][g][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                const float ref = w.inv[g] == 0.f ? 0.f : __uint_as_float((254u << 23) - __float_as_uint(w.inv[g]));
                if (r >= rows) continue;
#pragma unroll
                for (int c = g * C::G / 32; c < (g + 1) * C::G / 32; ++c) {
                    float4 y;
                    y.x = ref * fmaf(w.o[n][c][0][e], 16777216.f, -z);
                    y.y = ref * fmaf(w.o[n][c][0][2 + e], 1048576.f, -z);
                    y.z = ref * fmaf(w.o[n][c][1][e], 16777216.f, -z);
                    y.w = ref * fmaf(w.o[n][c][1][2 + e], 1048576.f, -z);
                    *reinterpret_cast<float4 *>(mine + r * C::OROW + 32 * c + 4 * i) = y;
                }
            }
        }
    }
    ptx::named_bar_sync(1 + rg, C::KW * 32);
    const float *group_o = scratch + rg * C::KW * RW * C::OROW, *group_ml = ml + rg * C::KW * RW * 2;
    const size_t slot = 2 * (size_t)blockIdx.x + (begun_here ? 1 : 0);
    // a warp per row, lanes along its components
    for (int r = kwi; r < rows; r += C::KW) {
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < C::KW; ++k) top = fmaxf(top, group_ml[(k * RW + r) * 2]);
        const float use = top == -INFINITY ? 0.f : top;
        float l = 0.f, acc[C::D / 32];
#pragma unroll
        for (int e = 0; e < C::D / 32; ++e) acc[e] = 0.f;
#pragma unroll
        for (int k = 0; k < C::KW; ++k) {
            const float f = ptx::ex2_approx(group_ml[(k * RW + r) * 2] - use);
            l = fmaf(f, group_ml[(k * RW + r) * 2 + 1], l);
#pragma unroll
            for (int e = 0; e < C::D / 32; e += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(group_o + (k * RW + r) * C::OROW + 32 * e + 2 * lane);
                acc[e] = fmaf(f, v.x, acc[e]);
                acc[e + 1] = fmaf(f, v.y, acc[e + 1]);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float lse2 = l == 0.f ? -INFINITY : use + __log2f(l);  // (a NaN sum is no empty row)
        const int row = rg * RW + r;
        if (whole) {
            if (lane == 0) p.lse[row0 + row] = lse2 * kLn2;
            uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + (row0 + row) * C::D);
#pragma unroll
            for (int e = 0; e < C::D / 32; e += 2)
                dst[16 * e + lane] = p.fp16 ? ptx::pack_f16x2(acc[e] * inv, acc[e + 1] * inv)
                                            : ptx::pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        } else {
            if (lane == 0) p.part_lse[slot * C::RC + row] = lse2;
            float *dst = p.part_o + (slot * C::RC + row) * C::D;
#pragma unroll
            for (int e = 0; e < C::D / 32; e += 2)
                *reinterpret_cast<float2 *>(dst + 32 * e + 2 * lane) = make_float2(acc[e] * inv, acc[e + 1] * inv);
        }
    }
    ptx::named_bar_sync(1 + rg, C::KW * 32);  // the scratch is free again
}

template <class C>
__device__ void dec_i4_warp(const DecInt4Params &p, DecFp8It it, uint8_t *ring, float *scratch, float *ml, uint32_t bars,
                            int *copied, Ctl *ctl) {
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5, rg = warp / C::KW, kwi = warp % C::KW;
    const uint64_t pol = p.chunks > 1 ? ptx::policy_evict_last() : ptx::policy_evict_first();
    const uint32_t ring_addr = ptx::smem_addr(ring);
    // The warps take turns at the copies: tile n is copied by warp n of the first
    // ST - 1 and by the warp whose turn tile n - ST + 1 is, behind its own keys of
    // that one; the stage's last readers were busy with the tile in front.
    DecFp8It ahead = it;
    for (int n = 0; n < C::ST - 1 && ahead.left > 0; ++n) {
        if (warp == n) {
            if (lane == 0) atomicMax(copied, n + 1);
            dec_i4_copy<C>(p, ahead, dec_i4_entry<C>(p, ahead), n == 0 || ahead.tile == 0, ring_addr + n * C::STAGE,
                           bar_addr(bars, C::B_FULL + n), pol);
        }
        dec_fp8_step(p, ahead);
    }
    DecI4Warp<C> w;
    bool begins = true, begun_here = it.tile == 0, bad = false;
    int slot = 0, prev = C::ST - 1;  // the stages of this tile and of the one in front
    uint32_t phase = 0, prev_phase = 1;
    for (int t = 0; it.left > 0; ++t) {
        const bool turn = (t & (C::WARPS - 1)) == warp && ahead.left > 0;
        int entry = -1;
        if (turn) entry = dec_i4_entry<C>(p, ahead);
        // (a warp whose wait ran out goes on without its tiles, so that the others meet it at the units' ends)
        if (!bad) bad = !wait_warp(bar_addr(bars, p.stall_test && t == 0 ? C::B_NEVER : C::B_FULL + slot), phase, ctl, 92);
        const uint8_t *stage = ring + slot * C::STAGE;
        if (begins) dec_i4_begin_unit<C>(p, it, reinterpret_cast<const uint16_t *>(stage + C::O_Q), rg, w);
        begins = false;
        const int seen_by_all = p.mask_kind == kMaskCausal ? it.L - p.Sq : it.L - 1;
#pragma unroll 1
        for (int j = 0; j < C::KPW; ++j) {
            const int at = (kwi * C::KPW + j) * 16, key = it.tile * C::BN + at;
            if (bad || key >= it.L) break;
            const uint32_t base = ring_addr + slot * C::STAGE;
            dec_i4_keys<C>(p, w, key, it.L, seen_by_all, base + at * C::ROW, base + C::O_V + at * C::ROW,
                           base + C::O_KW + at * C::NG * 4, base + C::O_VW + at * C::NG * 4);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_addr(bars, C::B_EMPTY + slot));
        if (turn && !bad) {
            // tile t + ST - 1 goes where tile t - 1 was
            bad = t > 0 && !wait_warp(bar_addr(bars, C::B_EMPTY + prev), prev_phase, ctl, 91);
            if (!bad) {
                if (lane == 0) atomicMax(copied, t + C::ST);
                dec_i4_copy<C>(p, ahead, entry, ahead.tile == 0, ring_addr + prev * C::STAGE, bar_addr(bars, C::B_FULL + prev), pol);
            }
        }
        if (ahead.left > 0) dec_fp8_step(p, ahead);
        const bool ends = it.tile + 1 == it.nt;
        if (ends || it.left == 1) {
            dec_i4_end_unit<C>(p, it, w, rg, kwi, begun_here && ends, begun_here, scratch, ml);
            begins = true;
            begun_here = true;
        }
        dec_fp8_step(p, it);
        prev = slot;
        prev_phase = phase;
        if (++slot == C::ST) slot = 0, phase ^= 1;
    }
}

template <class C>
__global__ void __launch_bounds__(C::NUM_THREADS, C::CTAS_PER_SM)
    fa_decode_int4_kernel(const __grid_constant__ DecInt4Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float *scratch = reinterpret_cast<float *>(ring + C::ST * C::STAGE);
    float *ml = scratch + C::SCRATCH / 4;
    uint64_t *bar_mem = reinterpret_cast<uint64_t *>(ml + 2 * C::WARPS * 8 * C::NT);
    Ctl *ctl = reinterpret_cast<Ctl *>(bar_mem + C::NUM_BARS);
    int *copied = reinterpret_cast<int *>(ctl + 1);  // tiles that copies were begun for
    const uint32_t bars = ptx::smem_addr(bar_mem);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::ST; ++s) {
            ptx::mbar_init(bar_addr(bars, C::B_FULL + s), 1);
            ptx::mbar_init(bar_addr(bars, C::B_EMPTY + s), C::WARPS);
        }
        ptx::mbar_init(bar_addr(bars, C::B_NEVER), 1);
        ctl->abort = 0;
        ctl->limit_ns = p.wait_limit_ns;
        *copied = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
        ptx::prefetch_tensormap(&p.tm_k);
        ptx::prefetch_tensormap(&p.tm_v);
    }
    ptx::wait_for_previous_kernel();
    const DecFp8It it = dec_fp8_begin<C::NUM_THREADS>(p, reinterpret_cast<long long *>(scratch));
    __syncthreads();
    // the merge may be set up now; it waits for this grid's end before it reads
    ptx::let_next_kernel_begin();
    dec_i4_warp<C>(p, it, ring, scratch, ml, bars, copied, ctl);
    __syncthreads();
    // the CTA's memory stays until its last copies have landed, also where the
    // warps gave up waiting for them
    if (ctl->abort && threadIdx.x == 0) {
        const int n = *copied;
        for (int t = n - C::ST > 0 ? n - C::ST : 0; t < n; ++t)
            wait_bar_drain(bar_addr(bars, C::B_FULL + t % C::ST), (t / C::ST) & 1);
    }
}

}  // namespace fa
