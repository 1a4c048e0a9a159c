// fa_paged_kernel.cuh -- the bookkeeping and the writes of a paged cache on the
// GPU, for sm_103a: block tables, slot maps and positions from request lengths
// (fa_paged_update), and the quantising append to an 8-bit cache
// (fa_cache_append_fp8).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "fa.h"
#include "sm103_ptx.cuh"

namespace fa {

// ------------------------------------------------------------ paged update
//
// Requests in index order; for request b with old tokens and a change delta:
//   add = max(delta, 0), first = sum of add over the requests before it,
//   have = ceil(old / bs), need = ceil((old + add) / bs) - have,
//   start = sum of need before it: its new blocks are ring entries
//   head + start .. head + start + need.
// So everything follows from two prefix sums, and a token's block from its own
// request's numbers: logical block n is table[b][n] for n < have, else ring
// entry head + start + n - have.  One launch: every CTA scans all requests
// (1,024 at a time) by itself and then takes its share of the token rows; a
// binary search over the chunk's prefix sums finds a row's request (where every
// request has per_request rows of its own, a division does; its tokens are the
// last of them, as the attention of a few new rows per request takes them).  The bytes
// are few (8 per row, 16 per request); what it costs is the launch and the
// latency of a scan, a search and a dependent load, which is why it is one
// launch and no workspace.  Where an output is its input (lengths, ring state)
// the CTAs are one cluster of at most eight, which meets after every CTA has
// read a chunk and before its one writer stores it; where none is, nothing one
// CTA reads is written by another, and there are as many as the rows keep busy.


struct PagedUpdateParams {
    const int *seq_lens, *delta, *ring_state;
    int *block_table, *free_ring;
    int *seq_lens_out, *ring_state_out, *slot_map, *positions, *status;
    int B, max_blocks, ring_size, bs_log2, max_tokens;
    int per_request;         // rows of each request, or 0: the tokens' rows follow each other
    int meet;                // the grid is one cluster, and outputs may be inputs
};

// Exclusive prefix sum over the CTA's threads (W warps); *total gets the sum.
template <int W>
__device__ __forceinline__ long long paged_scan(long long x, long long *warp_sums, long long *total) {
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();  // the previous scan's sums have been read
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    long long before = 0, all = 0;
    const long long mine = lane < W ? warp_sums[lane] : 0;
    long long w = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    before = __shfl_sync(0xffffffffu, w - mine, warp);
    all = __shfl_sync(0xffffffffu, w, 31);
    *total = all;
    return before + inc - x;
}

__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int kPagedThreads>
__global__ void __launch_bounds__(kPagedThreads) fa_paged_update_kernel(const PagedUpdateParams p) {
    constexpr int W = kPagedThreads / 32;
    __shared__ long long warp_sums[32];
    __shared__ unsigned long long s_used;  // blocks given out
    __shared__ int s_first[kPagedThreads];  // first row of the request, at most max_tokens
    __shared__ int s_old[kPagedThreads], s_start[kPagedThreads], s_gone[kPagedThreads];
    __shared__ int s_ok[kPagedThreads];
    const int tid = (int)threadIdx.x, bs = 1 << p.bs_log2;
    const int rank = (int)blockIdx.x, ranks = (int)gridDim.x;
    ptx::wait_for_previous_kernel();
    const long long head = min(max(p.ring_state[0], 0), p.ring_size - 1);
    const long long count = min(max(p.ring_state[1], 0), p.ring_size);
    const long long most = (long long)p.max_blocks << p.bs_log2;
    long long tokens = 0, needed = 0, freed = 0;  // sums over earlier chunks
    if (tid == 0) s_used = 0;

    for (int c0 = 0; c0 < p.B; c0 += kPagedThreads) {
        const int b = c0 + tid;
        const bool real = b < p.B;
        const long long old = real ? min(max((long long)p.seq_lens[b], 0LL), most) : 0;
        const long long delta = real ? p.delta[b] : 0;
        const long long add = max(delta, 0LL);
        const int n_req = min(kPagedThreads, p.B - c0);
        long long sum, first;
        bool no_rows;
        if (p.per_request > 0) {
            sum = (long long)n_req * p.per_request;
            first = (b + 1LL) * p.per_request - add;
            no_rows = add > p.per_request;
        } else {
            first = tokens + paged_scan<W>(add, warp_sums, &sum);
            no_rows = first + add > p.max_tokens;
        }
        const long long have = (old + bs - 1) >> p.bs_log2;
        const bool too_long = old + add > most;
        const long long need =
            add > 0 && !too_long && !no_rows ? ((old + add + bs - 1) >> p.bs_log2) - have : 0;
        const long long left = max(old + min(delta, 0LL), 0LL);  // a shrinking request's new length
        const long long gone = have - ((left + bs - 1) >> p.bs_log2);
        // both below 2^31 over all requests (the host checks B * max_blocks)
        long long both;
        const long long before = paged_scan<W>(need << 32 | gone, warp_sums, &both);
        const long long start = needed + (before >> 32), freed_before = freed + (before & 0xffffffffLL);
        const bool short_of = need > 0 && start + need > count;
        const int status = add == 0   ? FA_PAGED_OK
                           : too_long ? FA_PAGED_TOO_LONG
                           : no_rows  ? FA_PAGED_NO_ROWS
                           : short_of ? FA_PAGED_NO_BLOCKS
                                      : FA_PAGED_OK;
        const int given = __reduce_add_sync(0xffffffffu, (int)(short_of ? 0 : need));
        if ((tid & 31) == 0 && given) atomicAdd(&s_used, (unsigned long long)given);

        s_first[tid] = (int)min(first, (long long)p.max_tokens);
        s_old[tid] = (int)old;
        s_start[tid] = (int)min(start, 0x7fffffffLL);
        s_gone[tid] = (int)gone;
        s_ok[tid] = status == FA_PAGED_OK;
        __syncthreads();

        // rows of this chunk's tokens
        const int n_pow2 = n_req > 1 ? 1 << (31 - __clz(n_req - 1)) : 0;  // first stride of the search
        const int t0 = (int)min(tokens, (long long)p.max_tokens);
        const int t1 = (int)min(tokens + sum, (long long)p.max_tokens);
        // (four rows at a time where there are that many: the search and the load
        // behind it are all latency)
        auto rows = [&](auto count) {
            constexpr int U = decltype(count)::value;
            for (long long base = t0 + (long long)rank * kPagedThreads * U + tid; base < t1;
                 base += (long long)ranks * kPagedThreads * U) {
                int req[U];
#pragma unroll
                for (int u = 0; u < U; ++u) req[u] = 0;
                if (p.per_request > 0) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        req[u] = (int)(min(base + u * kPagedThreads, t1 - 1LL) / p.per_request) - c0;
                }
                // the last request whose first row is <= t
                for (int half = p.per_request > 0 ? 0 : n_pow2; half > 0; half >>= 1) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int mid = req[u] + half;
                        if (mid < n_req && s_first[mid] <= base + u * kPagedThreads) req[u] = mid;
                    }
                }
                int block[U], pos[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const long long t = base + u * kPagedThreads;
                    const int q = req[u], old_q = s_old[q];
                    pos[u] = t < t1 && s_ok[q] && t >= s_first[q] ? old_q + (int)(t - s_first[q]) : -1;
                    const int n = max(pos[u], 0) >> p.bs_log2, n_have = (old_q + bs - 1) >> p.bs_log2;
                    long long at = head + s_start[q] + n - n_have;  // below twice the ring's size
                    at -= at >= p.ring_size ? p.ring_size : 0;
                    const int *src = n < n_have ? p.block_table + (size_t)(c0 + q) * p.max_blocks + n : p.free_ring + at;
                    block[u] = pos[u] >= 0 ? *src : -1;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const long long t = base + u * kPagedThreads;
                    if (t >= t1) break;
                    const int q = req[u], n = max(pos[u], 0) >> p.bs_log2, in = max(pos[u], 0) & (bs - 1);
                    // a block's first token enters it in the table
                    if (pos[u] >= 0 && in == 0 && n >= (s_old[q] + bs - 1) >> p.bs_log2)
                        p.block_table[(size_t)(c0 + q) * p.max_blocks + n] = block[u];
                    const long long at = ((long long)block[u] << p.bs_log2) + in;
                    const bool good = block[u] >= 0 && at <= 0x7fffffffLL;
                    p.slot_map[t] = good ? (int)at : -1;
                    p.positions[t] = good ? pos[u] : 0;
                }
            }
        };
        if (t1 - t0 > ranks * kPagedThreads) rows(std::integral_constant<int, 4>());
        else rows(std::integral_constant<int, 1>());
        // blocks that shrinking requests give back, a warp per request
        if (both & 0xffffffffLL) {
            __shared__ long long s_freed[kPagedThreads];
            s_freed[tid] = freed_before;
            __syncthreads();
            for (int r = rank * (kPagedThreads / 32) + (tid >> 5); r < n_req; r += ranks * (kPagedThreads / 32)) {
                const int n = s_gone[r];
                if (n == 0) continue;
                const int n_have = (s_old[r] + bs - 1) >> p.bs_log2;
                const int *row = p.block_table + (size_t)(c0 + r) * p.max_blocks + (n_have - n);
                for (int j = tid & 31; j < n; j += 32) {
                    const long long at = s_freed[r] + j;
                    if (at < p.ring_size - count) {
                        long long to = head + count + at;  // below twice the ring's size
                        to -= to >= p.ring_size ? p.ring_size : 0;
                        p.free_ring[to] = row[j];
                    }
                }
            }
        }
        tokens += sum;
        needed += both >> 32;
        freed += both & 0xffffffffLL;
        if (p.meet) cluster_meet();
        if (rank == 0 && real) {
            p.seq_lens_out[b] = (int)(status == FA_PAGED_OK ? (delta < 0 ? left : old + add) : old);
            p.status[b] = status;
        }
        __syncthreads();
    }
    for (long long t = min(tokens, (long long)p.max_tokens) + (long long)rank * kPagedThreads + tid; t < p.max_tokens;
         t += (long long)ranks * kPagedThreads) {
        p.slot_map[t] = -1;
        p.positions[t] = 0;
    }
    if (rank == 0 && tid == 0) {  // (a cluster has met since the others read the state)
        const long long used = (long long)s_used;
        p.ring_state_out[0] = (int)((head + used) % p.ring_size);
        p.ring_state_out[1] = (int)(count - used + min(freed, p.ring_size - count));
    }
}

// ------------------------------------------------------- append to 8 bits
//
// A block of bs tokens of one K/V head is one scale s and bs x d e4m3 codes;
// the value of a code is code x s.  Appending to a block, K and V apart:
//   need = the smallest power of two s with max |x| <= 448 s over the finite
//          values now written (at least 2^-126),
//   s'   = need if slot 0 of the block is written (the block starts anew),
//          else max(s, need);
//   where s' > s, the codes not written now become e4m3(code * s / s');
//   the new codes are e4m3(x / s'), saturating.
// Powers of two cost at most one bit of range and none of precision, keep
// x / s' exact, and make re-encoding exact for every code that stays a normal
// number, so a block filled token by token does not lose a little more with
// every growth of its scale.
//
// The tokens of one block stand together in slot_map, so the first of them
// (the leader) stands for the block.  Of G CTAs, one takes the leaders with rows
// behind them among a few consecutive rows of slot_map, those that stand alone
// among every G-th row (a prompt's blocks lie apart; the live rows of a decode step
// in a map that is mostly padding lie together), and some of the (head, K or V)
// pairs; it works out which row writes which slot of the block, and then gives each
// pair's block to a group of WPU warps: enough that a lane holds its whole
// share, eight 16-byte vectors (sixteen for blocks of 32,768 values), between
// finding the maximum and writing the codes.  So a row is read once.  Bound by
// latency, slots then rows and scale then stores: 128 rows x 40 heads 9.1 us, 8,203
// rows x 8 heads (50 MB) 17.3 us, where the copy rate would take 0.6 and 7.4.  64
// live rows in front of 65,472 skipped ones 38 us, behind them 22 (950 and 988
// where every CTA walked back through them 32 at a time), every row skipped 8.

struct AppendParams {
    const uint8_t *x[2];        // new K and V rows, 16-bit
    long long token_stride[2], head_stride[2];  // in elements
    uint8_t *cache[2];          // e4m3 [num_blocks, Hkv, bs, d]
    float *scale[2];            // [num_blocks, Hkv]
    const int *slot_map;        // [T]
    int T, Hkv, d_log2, bs_log2, rows_per_cta;
    int wpu_log2;               // warps per (block, head, K or V)
    long long slots;            // num_blocks * bs
};

constexpr int kAppendThreads = 256;

template <bool kFP16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if constexpr (kFP16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

// Eight consecutive 16-bit values; kVec: the address is 16-byte aligned.
template <bool kVec>
__device__ __forceinline__ uint4 load8_16(const uint16_t *src) {
    if constexpr (kVec) return *reinterpret_cast<const uint4 *>(src);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)src[2 * i] | (uint32_t)src[2 * i + 1] << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The smallest power of two s >= 2^-126 with amax <= 448 s.  448 = 1.75 * 2^8:
// with amax = f 2^k, 1 <= f < 2, that is 2^(k - 8), or 2^(k - 7) for f > 1.75.
// Adding the mantissa's distance of 1.75 to 2 carries into the exponent for
// exactly those.
__device__ __forceinline__ float scale_for(float amax) {
    const int k = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;  // biased exponent of s
    return __uint_as_float((uint32_t)max(k, 1) << 23);
}

__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The slot of a row, -1 where it is skipped or there is none.  (The load is
// unconditional, so that several are on their way at once.)
__device__ __forceinline__ int append_slot(const int *slot_map, long long slots, int T, int row) {
    const int s = slot_map[min(max(row, 0), T - 1)];
    return row >= 0 && row < T && s >= 0 && s < slots ? s : -1;
}

// Long runs of skipped rows (a captured step with room for many tokens) are
// looked through by the whole CTA, 16 rows per thread at a time.  (Out of line:
// few calls need it.)
constexpr int kAppendLook = 16;

// The last live row before `hi`, or -1.  All threads of the CTA.
__device__ __noinline__ int append_last_live(const int *slot_map, long long slots, int T, int hi, int *s_row) {
    const int tid = (int)threadIdx.x;
    for (; hi > 0; hi -= kAppendLook * kAppendThreads) {
        if (tid == 0) *s_row = -1;
        __syncthreads();
        int last = -1;
#pragma unroll
        for (int i = 0; i < kAppendLook; ++i) {
            const int row = hi - 1 - i * kAppendThreads - tid;
            if (append_slot(slot_map, slots, T, row) >= 0) last = max(last, row);
        }
        if (last >= 0) atomicMax(s_row, last);
        __syncthreads();
        last = *s_row;
        __syncthreads();
        if (last >= 0) return last;
    }
    return -1;
}

// Enters the rows of `block` from r0 on, up to the first live row of another
// block, into owner.  All threads of the CTA.
__device__ __noinline__ void append_rows_after(const int *slot_map, long long slots, int T, int bs_log2, int r0, int block,
                                               int *owner, int *s_row) {
    const int tid = (int)threadIdx.x, bs = 1 << bs_log2;
    int stop = T;
    if (r0 < stop) {  // (most blocks end soon: one row per thread first)
        __syncthreads();
        if (tid == 0) *s_row = stop;
        __syncthreads();
        const int s = append_slot(slot_map, slots, T, r0 + tid);
        if (s >= 0 && s >> bs_log2 != block) atomicMin(s_row, r0 + tid);
        __syncthreads();
        stop = *s_row;
        if (s >= 0 && r0 + tid < stop) atomicMax(&owner[s & (bs - 1)], r0 + tid);
        r0 += kAppendThreads;
    }
    for (; r0 < stop; r0 += kAppendLook * kAppendThreads) {
        __syncthreads();
        if (tid == 0) *s_row = stop;
        __syncthreads();
        int s[kAppendLook], other = stop, high = -1;
#pragma unroll
        for (int i = 0; i < kAppendLook; ++i) s[i] = append_slot(slot_map, slots, T, r0 + i * kAppendThreads + tid);
#pragma unroll
        for (int i = kAppendLook - 1; i >= 0; --i) {
            if (s[i] >= 0 && s[i] >> bs_log2 != block) other = r0 + i * kAppendThreads + tid;
            high = max(high, s[i]);
        }
        if (other < stop) atomicMin(s_row, other);
        const bool any = __syncthreads_or(high >= 0);
        stop = *s_row;
        if (!any) continue;
#pragma unroll
        for (int i = 0; i < kAppendLook; ++i) {
            const int row = r0 + i * kAppendThreads + tid;
            if (s[i] >= 0 && row < stop) atomicMax(&owner[s[i] & (bs - 1)], row);
        }
    }
}

template <bool kFP16, bool kVec, int HOLD>
__global__ void __launch_bounds__(kAppendThreads, HOLD == 8 ? 4 : 2) fa_cache_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int BACK = 128;       // rows looked at before a row, and from it on
    __shared__ int win[3 * BACK];   // slots of rows row0 - BACK .., -1 where a row is skipped or there is none
    __shared__ int near[2 * BACK];  // the same round one row outside the CTA's
    __shared__ int owner[128];      // row that writes this slot of the block, or -1
    __shared__ int found[2 * 128];
    __shared__ int s_row, s_found;
    __shared__ uint32_t s_max[kAppendThreads / 32];
    static_assert(2 * BACK == kAppendThreads, "a slot of `near` per thread");
    const int tid = (int)threadIdx.x, lane = tid & 31, bs = 1 << p.bs_log2;
    const int row0 = (int)blockIdx.x * p.rows_per_cta;
    const int row1 = min(row0 + p.rows_per_cta, p.T);
    const int first = row0 - BACK;
    auto slot_of = [&](int row) { return append_slot(p.slot_map, p.slots, p.T, row); };
    auto same = [&](int s, int of) { return s >= 0 && s >> p.bs_log2 == of >> p.bs_log2; };
    ptx::wait_for_previous_kernel();
    for (int j = tid; j < BACK + p.rows_per_cta + BACK; j += kAppendThreads) win[j] = slot_of(first + j);
    int alone = -1;  // a row that leads and is not followed by another of its block
    if (tid < p.rows_per_cta) {
        const int row = (int)blockIdx.x + (int)gridDim.x * tid;
        const int s = slot_of(row);
        if (s >= 0 && !same(slot_of(row - 1), s) && !same(slot_of(row + 1), s)) alone = row;
    }
    if (tid < bs) owner[tid] = -1;
    if (tid == 0) s_found = 0;
    // this thread's group, its place in it, and the pairs it takes
    const int gsize = 32 << p.wpu_log2, group = tid / gsize, in_group = tid & (gsize - 1);
    const int groups = kAppendThreads / gsize, pairs = 2 * p.Hkv;
    const int vec_log2 = p.d_log2 - 3, units = 1 << (vec_log2 + p.bs_log2);  // 8-value vectors of a row, a block
    __syncthreads();
    if (tid < row1 - row0) {
        const int *w = win + BACK + tid;
        if (w[0] >= 0 && !same(w[-1], w[0]) && same(w[1], w[0])) found[atomicAdd(&s_found, 1)] = row0 + tid;
    }
    if (alone >= 0) found[atomicAdd(&s_found, 1)] = alone;
    __syncthreads();
    // (in any order: each has a block of its own)
    for (int f = 0; f < s_found; ++f) {
        const int row = found[f];
        if (f > 0) {
            __syncthreads();  // the block before is done with
            if (tid < bs) owner[tid] = -1;
        }
        const int *w = win + (row - row0);  // w[BACK] is the row's slot
        if (row < row0 || row >= row1) {
            near[tid] = slot_of(row - BACK + tid);
            w = near;
        }
        __syncthreads();
        const int block = w[BACK] >> p.bs_log2;

        // the block of the last live row before it (every warp for itself)
        int prev = -1, at = -1;
#pragma unroll
        for (int k = 0; k < BACK / 32; ++k) {
            const uint32_t live = __ballot_sync(0xffffffffu, w[k * 32 + lane] >= 0);
            if (live) at = k * 32 + 31 - __clz(live);
        }
        if (at >= 0) {
            prev = w[at] >> p.bs_log2;
        } else if (row > BACK) {  // (a long run of skipped rows)
            const int seen = append_last_live(p.slot_map, p.slots, p.T, row - BACK, &s_row);
            if (seen >= 0) prev = p.slot_map[seen] >> p.bs_log2;
        }
        if (prev == block) continue;

        // its rows: up to the first live row of another block
        int end = BACK;
#pragma unroll
        for (int k = BACK / 32 - 1; k >= 0; --k) {
            const int s = w[BACK + k * 32 + lane];
            const uint32_t other = __ballot_sync(0xffffffffu, s >= 0 && s >> p.bs_log2 != block);
            if (other) end = k * 32 + __ffs(other) - 1;
        }
        if (tid < end) {  // a slot named twice: the later row
            const int s = w[BACK + tid];
            if (s >= 0) atomicMax(&owner[s & (bs - 1)], row + tid);
        }
        if (end == BACK)  // (past the first look)
            append_rows_after(p.slot_map, p.slots, p.T, p.bs_log2, row + BACK, block, owner, &s_row);
        __syncthreads();

        const bool begun = owner[0] >= 0;
        for (int pair = (int)blockIdx.y * groups + group; pair < pairs; pair += (int)gridDim.y * groups) {
            const int kv = pair >= p.Hkv, head = pair - (kv ? p.Hkv : 0);
            const uint16_t *x = reinterpret_cast<const uint16_t *>(p.x[kv]) + head * p.head_stride[kv];
            const size_t bh = (size_t)block * p.Hkv + head;
            uint8_t *codes = p.cache[kv] + (bh << (p.d_log2 + p.bs_log2));
            const float old = p.scale[kv][bh];
            auto source = [&](int u, int r) {
                return x + r * p.token_stride[kv] + ((u & ((1 << vec_log2) - 1)) << 3);
            };
            // Only what every call does is unrolled (registers cannot be indexed
            // otherwise); infinities, scales that are no powers of two and growth
            // of the scale take the short loops, which read again: the whole in
            // line was several times the code, and fetching it cost a decode step
            // more than its data (128 rows x 40 heads: 19 us against 12; 8,203 rows
            // of prompts x 8 heads: 45 against 24).
            uint4 held[HOLD];
            uint32_t mine = 0;  // which of this lane's vectors are written
#pragma unroll
            for (int i = 0; i < HOLD; ++i) {
                const int u = in_group + i * gsize;
                const int r = u < units ? owner[u >> vec_log2] : -1;
                held[i] = make_uint4(0, 0, 0, 0);
                if (r >= 0) {
                    mine |= 1u << i;
                    held[i] = load8_16<kVec>(source(u, r));
                }
            }
            // 16-bit magnitudes are ordered as whole numbers
            uint32_t top2 = 0;
#pragma unroll
            for (int i = 0; i < HOLD; ++i) {
                top2 = __vmaxu2(top2, __vmaxu2(held[i].x & 0x7fff7fffu, held[i].y & 0x7fff7fffu));
                top2 = __vmaxu2(top2, __vmaxu2(held[i].z & 0x7fff7fffu, held[i].w & 0x7fff7fffu));
            }
            constexpr uint32_t kInf = kFP16 ? 0x7c00u : 0x7f80u;
            uint32_t top = max(top2 & 0xffffu, top2 >> 16);
            if (top >= kInf) {  // the largest finite one
                top = 0;
                for (int u = in_group; u < units; u += gsize) {
                    const int r = owner[u >> vec_log2];
                    for (int j = 0; r >= 0 && j < 8; ++j) {
                        const uint32_t v = source(u, r)[j] & 0x7fffu;
                        top = max(top, v < kInf ? v : 0u);
                    }
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            if (p.wpu_log2 > 0) {
                if ((tid & 31) == 0) s_max[tid >> 5] = top;
                ptx::named_bar_sync(1 + group, gsize);  // also: the group has read the old scale
                for (int w = 0; w < gsize / 32; ++w) top = max(top, s_max[group * (gsize / 32) + w]);
                ptx::named_bar_sync(1 + group, gsize);
            }
            __syncwarp();
            const float need = scale_for(unpack16<kFP16>(top).x);
            // (an old scale that is no positive finite number counts as none)
            const float now = begun || !(old > need) || isinf(old) ? need : old;
            const bool grew = !begun && old > 0.f && now > old;
            const uint32_t nb = __float_as_uint(now);
            if ((nb & 0x7fffffu) == 0 && (nb >> 23) < 254) {  // x / now by its exact inverse
                const float inv = __uint_as_float((254u - (nb >> 23)) << 23);
#pragma unroll
                for (int i = 0; i < HOLD; ++i) {
                    if (!(mine >> i & 1)) continue;
                    const uint32_t ws[4] = {held[i].x, held[i].y, held[i].z, held[i].w};
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 y = unpack16<kFP16>(ws[j]);
                        f[2 * j] = y.x * inv;
                        f[2 * j + 1] = y.y * inv;
                    }
                    *reinterpret_cast<uint2 *>(codes + (size_t)(in_group + i * gsize) * 8) =
                        make_uint2(ptx::pack_e4m3x4(f[0], f[1], f[2], f[3]), ptx::pack_e4m3x4(f[4], f[5], f[6], f[7]));
                }
            } else {
#pragma unroll 1
                for (int u = in_group; u < units; u += gsize) {
                    const int r = owner[u >> vec_log2];
#pragma unroll 1
                    for (int j = 0; r >= 0 && j < 8; ++j)
                        codes[(size_t)u * 8 + j] =
                            (uint8_t)ptx::pack_e4m3x4(__fdiv_rn(unpack16<kFP16>(source(u, r)[j]).x, now), 0.f, 0.f, 0.f);
                }
            }
            if (grew) {
#pragma unroll 1
                for (int u = in_group; u < units; u += gsize) {
                    if (owner[u >> vec_log2] >= 0) continue;
                    uint2 *dst = reinterpret_cast<uint2 *>(codes + (size_t)u * 8);
                    const uint2 w = *dst;
                    uint32_t out[2] = {0, 0};
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        const float2 y = unpack_e4m3x2((j < 2 ? w.x : w.y) >> (16 * (j & 1)));
                        const uint32_t two = ptx::pack_e4m3x4(__fdiv_rn(y.x * old, now), __fdiv_rn(y.y * old, now), 0.f, 0.f);
                        if (j < 2) out[0] |= two << (16 * j);
                        else out[1] |= two << (16 * (j - 2));
                    }
                    *dst = make_uint2(out[0], out[1]);
                }
            }
            if (in_group == 0) p.scale[kv][bh] = now;
        }
    }
}

}  // namespace fa
