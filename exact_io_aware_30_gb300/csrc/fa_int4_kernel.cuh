// fa_int4_kernel.cuh -- a paged K/V cache held in 4 bits, for sm_103a: the write
// that quantises rows (fa_cache_append_int4) and reading rows back in 16 bits
// (fa_cache_read_int4).  The attention over it is in fa_decode_int4_kernel.cuh.
//
// A cached row of d components is in groups of G (32 or 64) adjacent ones.  A
// group is G codes c = 0 .. 15, two to a byte (component 2i in the low half of
// byte i), and one word: the scale s >= 0 (bf16) in its high half, the zero z (a
// whole number, |z| <= 2048, in fp16) in its low half.  The value is s (c - z).
//
// Write, per group of finite values x_i, lo and hi the smallest and largest:
//     t   = max((hi - lo) / 15, max |x| / 2048)      in fp32
//     s   = t rounded up to bf16
//     n_i = x_i / s rounded to nearest even, c_i = min(n_i - min n, 15), z = -min n
// The second term bounds z: a group whose values lie close together far from 0
// is held to 2^-12 of its largest, finer than bf16.  Rounding s up keeps the
// grid over [lo, hi], so a value is off by at most s / 2.  All zero: s = c = z =
// 0.  A group with an infinity or NaN: s is NaN, c = z = 0, and it reads as NaN.
#pragma once

#include <stdint.h>

#include "fa_paged_kernel.cuh"

namespace fa {

constexpr int kInt4Threads = 256;
constexpr int kInt4Look = 128;     // a slot's later writer is looked for among this many rows
constexpr int kInt4MaxRows = 64;   // rows of a CTA of the append

struct Int4AppendParams {
    const uint16_t *x[2];       // new K and V rows, 16-bit
    long long token_stride[2], head_stride[2];  // in elements
    uint8_t *codes[2];          // [num_blocks, Hkv, bs, d / 2]
    uint32_t *words[2];         // [num_blocks, Hkv, bs, d / G]
    const int *slot_map;        // [T]
    long long slots;            // num_blocks * bs
    int T, Hkv, d_log2, g_log2, bs_log2, rows_per_cta;
    int items_log2;             // threads along a row's (K or V, head, vector of 16) items
};

// The integer nearest to y (ties to even), |y| < 2^22: in [2^23, 2^24) the step
// of fp32 is 1.
__device__ __forceinline__ float round_even(float y) { return (y + 12582912.f) - 12582912.f; }

// x / d by a rounded inverse of d and one correction by the quotient's own
// remainder (Markstein's step): the correctly rounded quotient wherever it has
// few bits, and else within the last place.  |d| and |x| far from the ends of
// fp32's range.
__device__ __forceinline__ float quotient(float x, float d, float inv) {
    const float y = x * inv;
    return fmaf(fmaf(-y, d, x), inv, y);
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The larger (smaller) of each half; NaN if either is.
template <bool kFP16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kFP16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool kFP16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kFP16) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

struct Int4Group {
    uint32_t codes[2];  // of the thread's 16 values
    uint32_t word;
};

// Quantises the 16 values of each thread; 1 << lanes_log2 adjacent threads hold a
// group.  What bounds it is instructions, so the extremes are found two values at
// a time in 16 bits, and a division is three steps: ties are found all the same,
// as a quotient x / s that is a half has few bits, and one that is not is at
// least 2^-13 away from one (x has at most 11 bits and s 8).
template <bool kFP16>
__device__ __forceinline__ Int4Group int4_quantise(const uint32_t (&w)[8], int lanes_log2) {
    constexpr uint32_t kInf = kFP16 ? 0x7c00u : 0x7f80u;
    uint32_t top2 = w[0], bottom2 = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top2 = max2<kFP16>(top2, w[i]), bottom2 = min2<kFP16>(bottom2, w[i]);
    // low half: the largest; high half: the smallest, negated
    uint32_t ends = max2<kFP16>(__byte_perm(top2, bottom2, 0x5410) ^ 0x80000000u, __byte_perm(top2, bottom2, 0x7632) ^ 0x80000000u);
    for (int i = 0; i < lanes_log2; ++i) ends = max2<kFP16>(ends, __shfl_xor_sync(0xffffffffu, ends, 1 << i));
    Int4Group out;
    out.codes[0] = out.codes[1] = 0;
    out.word = 0x7fc00000u;
    if (max(ends & 0x7fffu, ends >> 16 & 0x7fffu) >= kInf) return out;
    const float2 hl = unpack16<kFP16>(ends);
    const float hi = hl.x, lo = -hl.y;
    // (hi - lo) / 15, from sixteenths so that the difference cannot overflow
    const float wide = hi * 0.0625f - lo * 0.0625f, most = fmaxf(fabsf(hi), fabsf(lo));
    const bool small = most < 2.58493941e-26f;  // 2^-85: below, the steps of a quotient might leave the normal numbers
    const float t = fmaxf(small ? __fdiv_rn(wide, 0.9375f) : quotient(wide, 0.9375f, 1.06666672f), most * 0.00048828125f);
    const float s = __uint_as_float((__float_as_uint(t) + 0xffffu) & 0xffff0000u);
    const float inv = rcp_approx(s);
    const float base = small ? (s > 0.f ? round_even(__fdiv_rn(lo, s)) : 0.f) : round_even(quotient(lo, s, inv));
    // four codes as the digits of one number below 2^16, read off its place in [2^23, 2^24)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t half[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float sum = 8388608.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 x = unpack16<kFP16>(w[4 * h + 2 * j + i]);
                float n0 = round_even(quotient(x.x, s, inv)), n1 = round_even(quotient(x.y, s, inv));
                if (small) {
                    n0 = s > 0.f ? round_even(__fdiv_rn(x.x, s)) : 0.f;
                    n1 = s > 0.f ? round_even(__fdiv_rn(x.y, s)) : 0.f;
                }
                sum = fmaf(fminf(n0 - base, 15.f), (float)(1 << (8 * i)), sum);
                sum = fmaf(fminf(n1 - base, 15.f), (float)(16 << (8 * i)), sum);
            }
            half[j] = __float_as_uint(sum);
        }
        out.codes[h] = __byte_perm(half[0], half[1], 0x5410);
    }
    out.word = __float_as_uint(s) | (ptx::pack_f16x2(0.f - base, 0.f) & 0xffffu);
    return out;
}

// A thread stands for 16 adjacent values of one head of K or V and goes through
// its CTA's rows, U in flight.  Bound by instructions (with 8 values a thread it ran
// 206 of them per row, the issue slots 75 % busy): 40,008 rows x 8 heads at d 256
// (430 MB) 172 us with 8 values and plain divisions, 159 with extremes in pairs and
// quotients in three steps, 112 with 16 values; four rows in flight 120, as registers
// leave fewer warps.  128 rows x 40 heads 4.7 us: slots, then the later writers, then
// the stores.
template <bool kFP16, bool kVec>
__global__ void __launch_bounds__(kInt4Threads) fa_cache_append_int4_kernel(const __grid_constant__ Int4AppendParams p) {
    __shared__ int s_slot[kInt4MaxRows + kInt4Look];
    __shared__ int s_late[kInt4MaxRows];        // the slot is written by a later row
    __shared__ long long s_row[kInt4MaxRows];   // the row's place in the cache, head 0; -1: it is not written
    constexpr int U = 2;
    const int tid = (int)threadIdx.x;
    const int per_row = 2 * p.Hkv << (p.d_log2 - 4);
    const int item = ((int)blockIdx.y << p.items_log2) + (tid & ((1 << p.items_log2) - 1));
    const int lane_row = tid >> p.items_log2, rows_at_once = kInt4Threads >> p.items_log2;
    const bool have = item < per_row;
    const int vec = item & ((1 << (p.d_log2 - 4)) - 1);
    const int unit = have ? item >> (p.d_log2 - 4) : 0, kv = unit >= p.Hkv ? 1 : 0, head = unit - (kv ? p.Hkv : 0);
    const int row0 = (int)blockIdx.x * p.rows_per_cta, rows = min(p.rows_per_cta, p.T - row0);
    const uint16_t *x = p.x[kv] + row0 * p.token_stride[kv] + head * p.head_stride[kv] + vec * 16;
    ptx::wait_for_previous_kernel();
    for (int j = tid; j < p.rows_per_cta + kInt4Look; j += kInt4Threads)
        s_slot[j] = append_slot(p.slot_map, p.slots, p.T, row0 + j);
    if (tid < kInt4MaxRows) s_late[tid] = 0;
    uint32_t held[U][8];
    auto fetch = [&](int u, int r) {
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (have && r < rows) {
            const uint16_t *src = x + r * p.token_stride[kv];
            a = load8_16<kVec>(src);
            b = load8_16<kVec>(src + 8);
        }
        held[u][0] = a.x, held[u][1] = a.y, held[u][2] = a.z, held[u][3] = a.w;
        held[u][4] = b.x, held[u][5] = b.y, held[u][6] = b.z, held[u][7] = b.w;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(u, u * rows_at_once + lane_row);
    __syncthreads();
    for (int i = tid; i < rows * kInt4Look; i += kInt4Threads) {
        const int r = i / kInt4Look, k = i % kInt4Look;
        if (k > 0 && s_slot[r] >= 0 && s_slot[r + k] == s_slot[r]) s_late[r] = 1;
    }
    __syncthreads();
    for (int r = tid; r < rows; r += kInt4Threads) {
        const int slot = s_slot[r];
        s_row[r] = slot < 0 || s_late[r] ? -1 : (((long long)(slot >> p.bs_log2) * p.Hkv) << p.bs_log2) + (slot & ((1 << p.bs_log2) - 1));
    }
    __syncthreads();
    const bool writes_word = (vec & ((1 << (p.g_log2 - 4)) - 1)) == 0;
    uint8_t *codes = p.codes[kv] + (((long long)head << p.bs_log2) << (p.d_log2 - 1)) + vec * 8;
    uint32_t *words = p.words[kv] + (((long long)head << p.bs_log2) << (p.d_log2 - p.g_log2)) + (vec >> (p.g_log2 - 4));
    for (int r0 = 0; r0 < rows; r0 += U * rows_at_once) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r0 + u * rows_at_once >= rows) break;  // (the same in the whole CTA)
            const int r = r0 + u * rows_at_once + lane_row;
            const Int4Group q = int4_quantise<kFP16>(held[u], p.g_log2 - 4);
            fetch(u, r + U * rows_at_once);
            const long long at = have && r < rows ? s_row[r] : -1;
            if (at < 0) continue;
            *reinterpret_cast<uint2 *>(codes + (at << (p.d_log2 - 1))) = make_uint2(q.codes[0], q.codes[1]);
            if (writes_word) words[at << (p.d_log2 - p.g_log2)] = q.word;
        }
    }
}

// --------------------------------------------------------------- reading back

struct Int4ReadParams {
    const uint8_t *codes[2];
    const uint32_t *words[2];
    const int *block_table, *seq_lens, *starts;
    uint16_t *out[2];
    long long stride[2][3];     // of (request, head, row), in elements
    int Hkv, rows, max_blocks, num_blocks, d_log2, g_log2, bs_log2;
    int rows_per_cta, chunks;   // CTAs of a request
    int items_log2;
};

// A thread stands for 16 adjacent values of one head of K or V; its rows' table
// entries, then codes and words, U rows in flight.
// BYTES: what the outputs' addresses are multiples of: 32, 16 or 2.  (Prefixes of up
// to 8,191 tokens x 8 heads at d 128: 32 bytes a store 58.7 us, 16 62.6.)
template <bool kFP16, int BYTES>
__global__ void __launch_bounds__(kInt4Threads) fa_cache_read_int4_kernel(const __grid_constant__ Int4ReadParams p) {
    constexpr int U = 4;
    const int tid = (int)threadIdx.x;
    const int per_row = 2 * p.Hkv << (p.d_log2 - 4);
    const int item = ((int)blockIdx.y << p.items_log2) + (tid & ((1 << p.items_log2) - 1));
    const int lane_row = tid >> p.items_log2, rows_at_once = kInt4Threads >> p.items_log2;
    const int b = (int)blockIdx.x / p.chunks, row0 = ((int)blockIdx.x - b * p.chunks) * p.rows_per_cta;
    const int vec = item & ((1 << (p.d_log2 - 4)) - 1);
    const int unit = item >> (p.d_log2 - 4), kv = unit >= p.Hkv ? 1 : 0, head = unit - (kv ? p.Hkv : 0);
    ptx::wait_for_previous_kernel();
    if (item >= per_row) return;
    const long long first = p.starts ? p.starts[b] : 0;
    const long long len = min(max(p.seq_lens[b], 0), p.max_blocks << p.bs_log2);
    // rows whose positions lie in [0, len)
    const int stop = min(row0 + p.rows_per_cta, p.rows);
    const int begin = (int)min(max((long long)row0, -first), (long long)stop);
    const int end = (int)min((long long)stop, len - first);
    const int *table = p.block_table + (size_t)b * p.max_blocks;
    uint16_t *out = p.out[kv] + b * p.stride[kv][0] + head * p.stride[kv][1] + vec * 16;
    const uint8_t *codes = p.codes[kv] + vec * 8;
    const uint32_t *words = p.words[kv] + (vec >> (p.g_log2 - 4));
    for (int r0 = begin + lane_row; r0 < end; r0 += U * rows_at_once) {
        int entry[U];
        uint2 c[U];
        uint32_t w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = min(r0 + u * rows_at_once, end - 1);
            entry[u] = table[(first + r) >> p.bs_log2];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = min(r0 + u * rows_at_once, end - 1);
            const bool in = entry[u] >= 0 && entry[u] < p.num_blocks;  // (outside the pool: zeros)
            const long long at = (((long long)(in ? entry[u] : 0) * p.Hkv + head) << p.bs_log2) +
                                 ((first + r) & ((1 << p.bs_log2) - 1));
            c[u] = *reinterpret_cast<const uint2 *>(codes + (at << (p.d_log2 - 1)));
            w[u] = words[at << (p.d_log2 - p.g_log2)];
            if (!in) w[u] = 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * rows_at_once;
            if (r >= end) break;
            const float s = __uint_as_float(w[u] & 0xffff0000u);
            // 2^23 + z: whole, as every step of s (c - z) before the product is
            const float z = 8388608.f + unpack16<true>(w[u]).x;
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t x = i < 4 ? c[u].x : c[u].y;
                const float a = __uint_as_float(0x4b000000u | ((x >> (8 * (i & 3))) & 15u)) - z;
                const float e = __uint_as_float(0x4b000000u | ((x >> (8 * (i & 3) + 4)) & 15u)) - z;
                y[i] = pack2b<kFP16>(s * a, s * e);
            }
            uint16_t *dst = out + r * p.stride[kv][2];
            if constexpr (BYTES == 32) {
                ptx::st_global_v8(dst, y);
            } else if constexpr (BYTES == 16) {
                reinterpret_cast<uint4 *>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
                reinterpret_cast<uint4 *>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dst[2 * i] = (uint16_t)y[i];
                    dst[2 * i + 1] = (uint16_t)(y[i] >> 16);
                }
            }
        }
    }
}

}  // namespace fa
