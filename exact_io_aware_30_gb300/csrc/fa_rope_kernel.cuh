// fa_rope_kernel.cuh -- rotary positions, forward and backward, for sm_103a.
//
// A rotated head keeps its first rot of d components in pairs (x1, x2); pair i
// of a row at position n turns by theta = n * f_i and is scaled by a:
//   y1 = a (x1 cos theta - x2 sin theta),  y2 = a (x1 sin theta + x2 cos theta).
// The pairs are components (i, i + rot/2) ("half") or (2i, 2i + 1)
// ("interleaved"); components rot .. d pass through.  The map is linear and,
// apart from a, orthogonal, so its gradient is the turn by -theta: the
// backward is this kernel with the sine negated.
//
// Angles: f_i arrives as turns per position in 64-bit fixed point (units of
// 2^-64 turn), so n * f_i modulo one turn is one wrapping integer product, as
// exact at position 10^9 as at 0 -- an fp32 product would lose the angle of
// far positions (2^-24 n radians) and an fp64 one would run at a few per cent
// of the fp32 rate.  Of the top 32 bits the nearest quarter turn comes off in whole
// numbers, and the rest, at most an eighth of a turn, becomes half turns in fp32 for
// sincospi: off by 2^-27 of a half turn, where the whole angle in one float was
// off by up to 2^-25.
// Products and sums are fp32, each output rounded once.
//
// What bounds it: every element is read and written once, 3 flops each, so
// HBM (268 MB in 45 us, 87 % of a copy).  A thread owns two 16-byte vectors of
// one token (in either layout, of the turning or of the other components) and
// walks eight heads with the same sines and cosines in registers.  q and k go in
// one launch.  Strides are free, so the rows can be read straight out of a
// packed projection and written as the contiguous [B, H, S, d] the attention
// takes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "sm103_ptx.cuh"

namespace fa {

struct RopeView {
    const uint8_t *in;
    uint8_t *out;
    long long is[3], os[3];  // strides in elements: batch, head, token
    int copy;                // components past rot are copied (not in place)
};

struct RopeParams {
    RopeView t[2];           // q heads [0, H), then k heads [H, H + Hkv)
    const int *positions;    // [B, S] with batch stride pos_stride, or null: 0 .. S-1
    long long pos_stride;
    const unsigned long long *freq;  // [rot / 2], turns per position * 2^64
    long long offset;        // added to every position
    float amplitude, sin_sign;
    int H, heads, heads_per_chunk;
    int S, d, rot;
    long long units;         // B * S * slots
    int slots;               // per token: rot / 2 / V turning, then half of (d - rot) / V passing through
};

template <typename T>
struct RopeType;
template <>
struct RopeType<__nv_bfloat16> {
    static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct RopeType<__half> {
    static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};
template <>
struct RopeType<float> {
    static __device__ __forceinline__ float up(float x) { return x; }
    static __device__ __forceinline__ float down(float x) { return x; }
};

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
    T e[V];
};

// V elements per vector; each thread rotates V pairs (two vectors).  U heads are
// in flight at once: four CTAs of 64 registers a thread hide the memory's
// latency; two heads fill those registers (the host's comment has the figures).
template <typename T, int V, bool kInterleaved, int U>
__global__ void __launch_bounds__(256, 4) fa_rope_kernel(const __grid_constant__ RopeParams p) {
    using Vec = RopeVec<T, V>;
    using C = RopeType<T>;
    ptx::wait_for_previous_kernel();
    const long long unit = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (unit >= p.units) return;
    const int half = p.rot >> 1, turning = half / V, passing = (p.d - p.rot) / V;
    long long token;
    int slot;
    if (passing == 0) {
        token = unit / p.slots;
        slot = (int)(unit - token * p.slots);
    } else {
        // 32 tokens at a time, their turning slots first: a warp turns or copies,
        // and no lane waits for its neighbours' sines (31 -> 29 us for half of d 128)
        const long long group = unit / (32 * p.slots);
        const int in_group = (int)min(32LL, p.units / p.slots - group * 32);
        int at = (int)(unit - group * (32 * p.slots));
        const bool copies = at >= in_group * turning;
        if (copies) at -= in_group * turning;
        const int per = copies ? p.slots - turning : turning, in = at / per;
        slot = at - in * per + (copies ? turning : 0);
        token = group * 32 + in;
    }
    const int b = (int)(token / p.S), s = (int)(token - (long long)b * p.S);
    const int h0 = (int)blockIdx.y * p.heads_per_chunk;
    const int h1 = min(h0 + p.heads_per_chunk, p.heads);

    // Two vectors per thread.  A turning slot: at components e0 and e0 + half;
    // half layout: they are the two sides of V pairs; interleaved: V / 2 whole
    // pairs each (V = 1: one pair, components 2 slot and 2 slot + 1).  A slot
    // past those: two vectors of the components that pass through.
    const bool turns = slot < turning;
    const int pass0 = slot - turning, pass_step = (passing + 1) / 2;
    const bool two = turns || pass0 + pass_step < passing;
    const int e0 = !turns ? p.rot + pass0 * V : (kInterleaved && V == 1) ? 2 * slot : slot * V;
    const int e1 = !turns ? (two ? e0 + pass_step * V : e0) : (kInterleaved && V == 1) ? e0 + 1 : e0 + half;
    Vec x0[U], x1[U];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool k = h + u >= p.H;
            const RopeView &t = p.t[k];
            if (h + u < h1 && (turns || t.copy)) {
                const T *in = reinterpret_cast<const T *>(t.in) + b * t.is[0] +
                              (h + u - (k ? p.H : 0)) * t.is[1] + s * t.is[2];
                x0[u] = *reinterpret_cast<const Vec *>(in + e0);
                x1[u] = *reinterpret_cast<const Vec *>(in + e1);
            }
        }
    };
    float cs[V], sn[V];
    if (turns) {
        const long long n = (p.positions ? (long long)p.positions[b * p.pos_stride + s] : (long long)s) + p.offset;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            int pair = slot * V + i;
            if (kInterleaved && V > 1) pair = i < V / 2 ? e0 / 2 + i : e1 / 2 + i - V / 2;
            const unsigned long long phase = (unsigned long long)n * p.freq[pair];
            const uint32_t turned = (uint32_t)(phase >> 32) + (1u << 29);  // from an eighth of a turn before
            const float x = (float)((int)(turned & 0x3fffffffu) - (1 << 29)) * 4.656612873077393e-10f;  // 2^-31
            float si, co;
            sincospif(x, &si, &co);
            if (turned & (1u << 30)) {  // a quarter turn on
                const float was = si;
                si = co;
                co = -was;
            }
            if (turned & (1u << 31)) {
                si = -si;
                co = -co;
            }
            cs[i] = co * p.amplitude;
            sn[i] = si * p.amplitude * p.sin_sign;
        }
    }

    for (int h = h0; h < h1; h += U) {
        load(h);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool k = h + u >= p.H;
            const RopeView &t = p.t[k];
            if (h + u < h1 && (turns || t.copy)) {
                Vec y0 = x0[u], y1 = x1[u];
                if (turns) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (!kInterleaved || V == 1) {
                            const float a = C::up(x0[u].e[i]), c = C::up(x1[u].e[i]);
                            y0.e[i] = C::down(a * cs[i] - c * sn[i]);
                            y1.e[i] = C::down(a * sn[i] + c * cs[i]);
                        } else if (i < V / 2) {
                            const float a = C::up(x0[u].e[(2 * i) % V]), c = C::up(x0[u].e[(2 * i + 1) % V]);
                            y0.e[(2 * i) % V] = C::down(a * cs[i] - c * sn[i]);
                            y0.e[(2 * i + 1) % V] = C::down(a * sn[i] + c * cs[i]);
                            const int j = i + V / 2;
                            const float f = C::up(x1[u].e[(2 * i) % V]), g = C::up(x1[u].e[(2 * i + 1) % V]);
                            y1.e[(2 * i) % V] = C::down(f * cs[j] - g * sn[j]);
                            y1.e[(2 * i + 1) % V] = C::down(f * sn[j] + g * cs[j]);
                        }
                    }
                }
                T *out = reinterpret_cast<T *>(t.out) + b * t.os[0] +
                         (h + u - (k ? p.H : 0)) * t.os[1] + s * t.os[2];
                *reinterpret_cast<Vec *>(out + e0) = y0;
                if (two) *reinterpret_cast<Vec *>(out + e1) = y1;
            }
        }
    }
}

}  // namespace fa
