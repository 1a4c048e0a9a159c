// fa_paged_kernel.cuh -- the bookkeeping and the writes of a paged cache on the
// GPU, for sm_103a: block tables, slot maps and positions from request lengths
// (fa_paged_update), and the quantising append to an 8-bit cache
// (fa_cache_append_fp8).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

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
// entry head + start + n - have.  One launch: a cluster of up to eight CTAs,
// each of which scans all requests (1,024 at a time) by itself and then takes
// every eighth 1,024 of the token rows; a binary search over the chunk's
// prefix sums finds a row's request.  The bytes are few (8 per row, 16 per
// request); what it costs is the launch and the latency of a scan, a search
// and two dependent loads, which is why it is one launch and no workspace.
// Outputs may alias inputs (lengths, ring state): the cluster meets after
// every CTA has read a chunk and before its one writer stores it.

constexpr int kPagedThreads = 1024;

struct PagedUpdateParams {
    const int *seq_lens, *delta, *ring_state;
    int *block_table, *free_ring;
    int *seq_lens_out, *ring_state_out, *slot_map, *positions, *status;
    int B, max_blocks, ring_size, bs_log2, max_tokens;
};

// Exclusive prefix sum over the block's 1,024 threads; *total gets the sum.
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
    const long long mine = warp_sums[lane];
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

__global__ void __launch_bounds__(kPagedThreads) fa_paged_update_kernel(const PagedUpdateParams p) {
    __shared__ long long warp_sums[32];
    __shared__ int s_first[kPagedThreads];  // first row of the request, at most max_tokens
    __shared__ int s_old[kPagedThreads], s_start[kPagedThreads], s_gone[kPagedThreads];
    __shared__ int s_ok[kPagedThreads];
    const int tid = (int)threadIdx.x, bs = 1 << p.bs_log2;
    const int rank = (int)blockIdx.x, ranks = (int)gridDim.x;  // the grid is one cluster
    const long long head = min(max(p.ring_state[0], 0), p.ring_size - 1);
    const long long count = min(max(p.ring_state[1], 0), p.ring_size);
    const long long most = (long long)p.max_blocks << p.bs_log2;
    long long tokens = 0, needed = 0, used = 0, freed = 0;  // sums over earlier chunks

    for (int c0 = 0; c0 < p.B; c0 += kPagedThreads) {
        const int b = c0 + tid;
        const bool real = b < p.B;
        const long long old = real ? min(max((long long)p.seq_lens[b], 0LL), most) : 0;
        const long long delta = real ? p.delta[b] : 0;
        const long long add = max(delta, 0LL);
        long long sum;
        const long long first = tokens + paged_scan(add, warp_sums, &sum);
        const long long have = (old + bs - 1) >> p.bs_log2;
        const bool too_long = old + add > most, no_rows = first + add > p.max_tokens;
        const long long need =
            add > 0 && !too_long && !no_rows ? ((old + add + bs - 1) >> p.bs_log2) - have : 0;
        const long long left = max(old + min(delta, 0LL), 0LL);  // a shrinking request's new length
        const long long gone = have - ((left + bs - 1) >> p.bs_log2);
        // both below 2^31 over all requests (the host checks B * max_blocks)
        long long both;
        const long long before = paged_scan(need << 32 | gone, warp_sums, &both);
        const long long start = needed + (before >> 32), freed_before = freed + (before & 0xffffffffLL);
        const bool short_of = need > 0 && start + need > count;
        const int status = add == 0 ? 0 : too_long ? 2 : no_rows ? 3 : short_of ? 1 : 0;
        long long used_sum;
        paged_scan(short_of ? 0 : need, warp_sums, &used_sum);

        s_first[tid] = (int)min(first, (long long)p.max_tokens);
        s_old[tid] = (int)old;
        s_start[tid] = (int)min(start, 0x7fffffffLL);
        s_gone[tid] = (int)gone;
        s_ok[tid] = status == 0;
        __syncthreads();

        // rows of this chunk's tokens
        const int n_req = min(kPagedThreads, p.B - c0);
        const int t0 = (int)min(tokens, (long long)p.max_tokens);
        const int t1 = (int)min(tokens + sum, (long long)p.max_tokens);
        for (long long t = t0 + (long long)rank * kPagedThreads + tid; t < t1; t += (long long)ranks * kPagedThreads) {
            int lo = 0, hi = n_req;  // the last request whose first row is <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_first[mid] <= t) lo = mid;
                else hi = mid;
            }
            int slot = -1, position = 0;
            if (s_ok[lo]) {
                const long long pos = (long long)s_old[lo] + t - s_first[lo];
                const int n = (int)(pos >> p.bs_log2), n_have = (s_old[lo] + bs - 1) >> p.bs_log2;
                int *row = p.block_table + (size_t)(c0 + lo) * p.max_blocks;
                int block;
                if (n < n_have) {
                    block = row[n];
                } else {
                    block = p.free_ring[(head + s_start[lo] + n - n_have) % p.ring_size];
                    if ((pos & (bs - 1)) == 0) row[n] = block;  // the block's first token enters it
                }
                const long long at = ((long long)block << p.bs_log2) + (pos & (bs - 1));
                if (block >= 0 && at <= 0x7fffffffLL) {
                    slot = (int)at;
                    position = (int)pos;
                }
            }
            p.slot_map[t] = slot;
            p.positions[t] = position;
        }
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
                    if (at < p.ring_size - count) p.free_ring[(head + count + at) % p.ring_size] = row[j];
                }
            }
        }
        tokens += sum;
        needed += both >> 32;
        freed += both & 0xffffffffLL;
        used += used_sum;
        if (ranks > 1) cluster_meet();
        if (rank == 0 && real) {
            p.seq_lens_out[b] = (int)(status == 0 ? (delta < 0 ? left : old + add) : old);
            p.status[b] = status;
        }
        __syncthreads();
    }
    for (long long t = min(tokens, (long long)p.max_tokens) + (long long)rank * kPagedThreads + tid; t < p.max_tokens;
         t += (long long)ranks * kPagedThreads) {
        p.slot_map[t] = -1;
        p.positions[t] = 0;
    }
    if (rank == 0 && tid == 0) {  // (the cluster has met since the others read the state)
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
// (the leader) stands for the block: a CTA takes a few consecutive rows of
// slot_map, one head and one of K and V, and for each leader among its rows
// does the whole block.  HBM bound for prompts (6 bytes per element), latency
// for a decode step.

struct AppendParams {
    const uint8_t *x[2];        // new K and V rows, 16-bit
    long long token_stride[2], head_stride[2];  // in elements
    uint8_t *cache[2];          // e4m3 [num_blocks, Hkv, bs, d]
    float *scale[2];            // [num_blocks, Hkv]
    const int *slot_map;        // [T]
    int T, Hkv, d, bs_log2, rows_per_cta;
    long long slots;            // num_blocks * bs
};

constexpr int kAppendThreads = 128;

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

__device__ __forceinline__ float finite_abs(float x) {
    const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
    return a < 0x7f800000u ? __uint_as_float(a) : 0.f;
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

template <bool kFP16, bool kVec>
__global__ void __launch_bounds__(kAppendThreads) fa_cache_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ int owner[128];  // row of slot_map that writes this slot of the block, or -1
    __shared__ int s_prev, s_end;
    __shared__ float s_max[kAppendThreads / 32];
    const int tid = (int)threadIdx.x, bs = 1 << p.bs_log2, kv = (int)blockIdx.z, head = (int)blockIdx.y;
    const int row0 = (int)blockIdx.x * p.rows_per_cta;
    const int row1 = min(row0 + p.rows_per_cta, p.T);
    int prev = -2;  // block of the last live row before `row`; -2: not looked up yet
    for (int row = row0; row < row1; ++row) {
        const int slot = p.slot_map[row];
        if (slot < 0 || slot >= p.slots) continue;  // a skipped row
        const int block = slot >> p.bs_log2;
        if (prev == -2) {  // the last live row before this CTA's rows
            prev = -1;
            for (int hi = row; hi > 0 && prev < 0; hi -= kAppendThreads) {
                __syncthreads();
                if (tid == 0) s_prev = -1;
                __syncthreads();
                const int r = hi - 1 - tid;
                const int s = r >= 0 ? p.slot_map[r] : -1;
                const bool live = s >= 0 && s < p.slots;
                if (live) atomicMax(&s_prev, r);
                __syncthreads();
                if (s_prev >= 0) prev = p.slot_map[s_prev] >> p.bs_log2;
            }
        }
        if (block == prev) continue;  // an earlier row leads this block
        prev = block;

        // the rows of this block: from `row` to the next live row of another block
        __syncthreads();
        for (int i = tid; i < bs; i += kAppendThreads) owner[i] = -1;
        if (tid == 0) s_end = p.T;
        __syncthreads();
        int end = p.T;
        for (int r0 = row; r0 < end; r0 += kAppendThreads) {
            const int r = r0 + tid;
            const int s = r < p.T ? p.slot_map[r] : -1;
            const bool live = s >= 0 && s < p.slots;
            if (live && s >> p.bs_log2 != block) atomicMin(&s_end, r);
            __syncthreads();
            end = s_end;
            if (live && r < end) atomicMax(&owner[s & (bs - 1)], r);  // a slot named twice: the later row
            __syncthreads();
        }

        const uint16_t *x = reinterpret_cast<const uint16_t *>(p.x[kv]) + head * p.head_stride[kv];
        const size_t bh = (size_t)block * p.Hkv + head;
        uint8_t *codes = p.cache[kv] + bh * ((size_t)p.d << p.bs_log2);
        const float old = p.scale[kv][bh];
        const int per_row = p.d / 8, units = per_row << p.bs_log2;
        float amax = 0.f;
        for (int u = tid; u < units; u += kAppendThreads) {
            const int at = u / per_row, r = owner[at];
            if (r < 0) continue;
            const uint4 w = load8_16<kVec>(x + r * p.token_stride[kv] + (u - at * per_row) * 8);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack16<kFP16>(ws[i]);
                amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if ((tid & 31) == 0) s_max[tid >> 5] = amax;
        __syncthreads();  // also: every thread has read the old scale
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
        const float need = scale_for(amax);
        const bool begun = owner[0] >= 0;
        // (an old scale that is no positive finite number counts as none)
        const float now = begun || !(old > need) || isinf(old) ? need : old;
        const bool grew = !begun && old > 0.f && now > old;
        for (int u = tid; u < units; u += kAppendThreads) {
            const int at = u / per_row, r = owner[at], c = (u - at * per_row) * 8;
            uint2 *dst = reinterpret_cast<uint2 *>(codes + (size_t)at * p.d + c);
            float f[8];
            if (r >= 0) {
                const uint4 w = load8_16<kVec>(x + r * p.token_stride[kv] + c);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = unpack16<kFP16>(ws[i]);
                    f[2 * i] = __fdiv_rn(y.x, now);
                    f[2 * i + 1] = __fdiv_rn(y.y, now);
                }
            } else if (grew) {
                const uint2 w = *dst;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = unpack_e4m3x2((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
                    f[2 * i] = __fdiv_rn(y.x * old, now);
                    f[2 * i + 1] = __fdiv_rn(y.y * old, now);
                }
            } else {
                continue;
            }
            *dst = make_uint2(ptx::pack_e4m3x4(f[0], f[1], f[2], f[3]), ptx::pack_e4m3x4(f[4], f[5], f[6], f[7]));
        }
        if (tid == 0) p.scale[kv][bh] = now;
    }
}

}  // namespace fa
