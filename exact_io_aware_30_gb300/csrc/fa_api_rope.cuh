// fa_api_rope.cuh -- host side of rotary positions (fa_rope,
// fa_rope_frequencies).  Included once, by fa_api.cu, after its shared
// helpers.
#pragma once

#include "fa_rope_kernel.cuh"

namespace fa {

namespace {

// A strided [B, heads, S, d] view in bytes-free form: base address, sizes and
// element strides of (batch, head, token); components are adjacent.
struct StridedView {
    uintptr_t base;
    long long size[3], stride[3];
    long long d;
    int elem;
};

long long view_span(const StridedView &v, bool with0, bool with1, bool with2) {
    const bool with[3] = {with0, with1, with2};
    long long n = v.d;
    for (int i = 0; i < 3; ++i)
        if (with[i]) n += (v.size[i] - 1) * v.stride[i];
    return n;
}

// Every element of the view has an address of its own: sorted by stride, each
// dimension steps over everything inside it.
bool view_injective(const StridedView &v) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return v.stride[a] < v.stride[b]; });
    long long inner = v.d;
    for (int i : order) {
        if (v.size[i] == 1) continue;
        if (v.stride[i] < inner) return false;
        inner += (v.size[i] - 1) * v.stride[i];
    }
    return true;
}

long long gcd_ll(long long a, long long b) {
    while (b) {
        const long long t = a % b;
        a = b;
        b = t;
    }
    return a;
}

// True when the two views provably share no byte: their extents are apart, or
// they step through memory alike in some dimensions and the spans of the
// others lie beside each other within every step (heads of one packed tensor).
bool views_disjoint(const StridedView &a, const StridedView &b) {
    const long long ea = view_span(a, true, true, true) * a.elem, eb = view_span(b, true, true, true) * b.elem;
    if (a.base + (uintptr_t)ea <= b.base || b.base + (uintptr_t)eb <= a.base) return true;
    const StridedView &lo = a.base <= b.base ? a : b, &hi = a.base <= b.base ? b : a;
    const long long apart_bytes = (long long)(hi.base - lo.base);
    if (apart_bytes % lo.elem) return false;
    const long long apart = apart_bytes / lo.elem;
    for (int set = 1; set < 8; ++set) {
        long long step = 0;
        bool alike = true;
        for (int i = 0; i < 3; ++i) {
            if (!(set >> i & 1)) continue;
            const bool used = lo.size[i] > 1 || hi.size[i] > 1;
            if (!used) continue;
            if (lo.stride[i] != hi.stride[i]) alike = false;
            step = gcd_ll(step, lo.stride[i]);
        }
        if (!alike || step <= 0) continue;
        const bool w0 = !(set & 1), w1 = !(set & 2), w2 = !(set & 4);
        const long long rest = apart % step;
        if (view_span(lo, w0, w1, w2) <= rest && rest + view_span(hi, w0, w1, w2) <= step) return true;
    }
    return false;
}

bool same_view(const StridedView &a, const StridedView &b) {
    if (a.base != b.base) return false;
    for (int i = 0; i < 3; ++i)
        if (a.size[i] > 1 && a.stride[i] != b.stride[i]) return false;
    return true;
}

template <typename T, int V>
fa_status launch_rope(const RopeParams &p, int layout, dim3 grid, cudaStream_t stream) {
    // Two heads in flight; one for interleaved pairs of part of the head (bf16,
    // half of d 128, 134 MB: one 29 us, two 31, four 47; all of it, fp16, 268 MB:
    // one 55 us, two 48, four 47; half layout: one 54 us, two 48, four 49).  With two, whole
    // heads in bf16 spill 12 to 16 bytes a thread.
    auto kern = layout != FA_ROPE_INTERLEAVED ? fa_rope_kernel<T, V, false, 2>
                : p.rot < p.d                 ? fa_rope_kernel<T, V, true, 1>
                                              : fa_rope_kernel<T, V, true, 2>;
    return launch_overlapped(kern, grid, 256, 0, 1, stream, p);
}

fa_status rope_impl(const void *q, const long long *q_strides, void *q_out, const long long *q_out_strides,
                    const void *k, const long long *k_strides, void *k_out, const long long *k_out_strides,
                    const int *positions, long long pos_stride, long long offset,
                    const unsigned long long *freq, float amplitude, int B, int H, int Hkv, int S, int d,
                    int rot_dim, int layout, int direction, int dtype, cudaStream_t stream) {
    if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16 && dtype != FA_DTYPE_FP32) return FA_ERR_UNSUPPORTED;
    if (layout != FA_ROPE_HALF && layout != FA_ROPE_INTERLEAVED) return FA_ERR_UNSUPPORTED;
    if (direction != FA_ROPE_FORWARD && direction != FA_ROPE_BACKWARD) return FA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || Hkv < 0 || S < 0 || d < 2 || d > 1024) return FA_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim > d || (rot_dim & 1)) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(amplitude)) return FA_ERR_INVALID_ARG;
    if ((long long)H + Hkv > 65535 || (long long)B * S > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    if (S == 0) return FA_OK;
    if (!q || !q_strides || !q_out || !q_out_strides || !freq) return FA_ERR_INVALID_ARG;
    if (Hkv > 0 && (!k || !k_strides || !k_out || !k_out_strides)) return FA_ERR_INVALID_ARG;
    if (pos_stride < 0 || pos_stride > (1LL << 40)) return FA_ERR_INVALID_ARG;  // (as the other strides below)

    const int elem = dtype == FA_DTYPE_FP32 ? 4 : 2;
    const int n_views = Hkv > 0 ? 2 : 1;
    const void *ins[2] = {q, k};
    void *outs[2] = {q_out, k_out};
    const long long *is[2] = {q_strides, k_strides}, *os[2] = {q_out_strides, k_out_strides};
    StridedView vin[2], vout[2];
    for (int t = 0; t < n_views; ++t) {
        const int heads = t ? Hkv : H;
        vin[t] = {reinterpret_cast<uintptr_t>(ins[t]), {B, heads, S}, {is[t][0], is[t][1], is[t][2]}, d, elem};
        vout[t] = {reinterpret_cast<uintptr_t>(outs[t]), {B, heads, S}, {os[t][0], os[t][1], os[t][2]}, d, elem};
        for (const StridedView *v : {&vin[t], &vout[t]}) {
            if (v->base % elem) return FA_ERR_MISALIGNED;
            long long reach = d;
            for (int i = 0; i < 3; ++i) {
                // (the limit keeps every offset below 2^61 elements)
                if (v->stride[i] < 0 || v->stride[i] > (1LL << 40)) return FA_ERR_INVALID_ARG;
                if (v->size[i] > 1) reach += (v->size[i] - 1) * v->stride[i];
                if (reach > (1LL << 58)) return FA_ERR_INVALID_ARG;
            }
        }
        if (!view_injective(vout[t])) return FA_ERR_INVALID_ARG;
    }
    if ((reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(freq) & 7u))
        return FA_ERR_MISALIGNED;
    for (int t = 0; t < n_views; ++t) {
        for (int u = 0; u < n_views; ++u) {
            if (!(t == u && same_view(vin[u], vout[t])) && !views_disjoint(vout[t], vin[u]))
                return FA_ERR_INVALID_ARG;
            if (t < u && !views_disjoint(vout[t], vout[u])) return FA_ERR_INVALID_ARG;
        }
        const size_t bytes = (size_t)view_span(vout[t], true, true, true) * elem;
        const size_t pos_bytes = positions ? (size_t)((B - 1) * pos_stride + S) * 4 : 0;
        if ((positions && overlaps(outs[t], bytes, positions, pos_bytes)) ||
            overlaps(outs[t], bytes, freq, (size_t)rot_dim * 4))
            return FA_ERR_INVALID_ARG;
    }

    int dev = 0;
    DeviceInfo *info = nullptr;
    const fa_status st = device_info(&dev, &info);
    if (st != FA_OK) return st;

    // Vector width: 16 bytes when every row start, pair half and pass-through
    // run is a whole number of them; else 4 bytes (16-bit types); else one
    // element.
    const int half = rot_dim / 2;
    long long bits = (long long)half * elem | (long long)(d - rot_dim) * elem;
    for (int t = 0; t < n_views; ++t) {
        const int heads = t ? Hkv : H;
        const long long size[3] = {B, heads, S};
        bits |= (long long)(vin[t].base | vout[t].base);
        for (int i = 0; i < 3; ++i)
            if (size[i] > 1) bits |= (vin[t].stride[i] | vout[t].stride[i]) * elem;
    }
    const int V = (bits & 15) == 0 ? 16 / elem : (elem == 2 && (bits & 3) == 0) ? 2 : 1;

    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    for (int t = 0; t < n_views; ++t) {
        p.t[t].in = static_cast<const uint8_t *>(ins[t]);
        p.t[t].out = static_cast<uint8_t *>(outs[t]);
        const long long size[3] = {B, t ? Hkv : H, S};
        for (int i = 0; i < 3; ++i) {  // the stride of a single entry is never stepped
            p.t[t].is[i] = size[i] > 1 ? is[t][i] : 0;
            p.t[t].os[i] = size[i] > 1 ? os[t][i] : 0;
        }
        p.t[t].copy = ins[t] != outs[t];
    }
    p.positions = positions;
    p.pos_stride = pos_stride;
    p.freq = freq;
    p.offset = offset;
    p.amplitude = amplitude;
    p.sin_sign = direction == FA_ROPE_BACKWARD ? -1.f : 1.f;
    p.H = H;
    p.heads = H + Hkv;
    p.S = S;
    p.d = d;
    p.rot = rot_dim;
    p.slots = half / V + ((d - rot_dim) / V + 1) / 2;
    p.units = (long long)B * S * p.slots;
    const long long blocks = (p.units + 255) / 256;
    if (blocks > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    // Heads per thread share the sines: eight, as long as that leaves a wave of
    // CTAs (four per SM), else fewer (one in a decode step: latency).  268 MB in
    // fp16: eight heads 48 us, four 49, one 90.
    const long long wave = 4LL * info->num_sms;
    p.heads_per_chunk = 8;
    while (p.heads_per_chunk > 1 && blocks * ((p.heads + p.heads_per_chunk - 1) / p.heads_per_chunk) < wave)
        p.heads_per_chunk /= 2;
    const dim3 grid((unsigned)blocks, (unsigned)((p.heads + p.heads_per_chunk - 1) / p.heads_per_chunk));
    if (log_enabled())
        std::fprintf(stderr, "[fa] fa_rope B=%d H=%d Hkv=%d S=%d d=%d rot=%d %s vector=%d heads_per_thread=%d\n", B,
                     H, Hkv, S, d, rot_dim, direction == FA_ROPE_BACKWARD ? "backward" : "forward", V,
                     p.heads_per_chunk);
    if (dtype == FA_DTYPE_FP32)
        return V == 4 ? launch_rope<float, 4>(p, layout, grid, stream) : launch_rope<float, 1>(p, layout, grid, stream);
    if (dtype == FA_DTYPE_FP16)
        return V == 8   ? launch_rope<__half, 8>(p, layout, grid, stream)
               : V == 2 ? launch_rope<__half, 2>(p, layout, grid, stream)
                        : launch_rope<__half, 1>(p, layout, grid, stream);
    return V == 8   ? launch_rope<__nv_bfloat16, 8>(p, layout, grid, stream)
           : V == 2 ? launch_rope<__nv_bfloat16, 2>(p, layout, grid, stream)
                    : launch_rope<__nv_bfloat16, 1>(p, layout, grid, stream);
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_rope(const void *q, const long long *q_strides, void *q_out, const long long *q_out_strides,
                  const void *k, const long long *k_strides, void *k_out, const long long *k_out_strides,
                  const int *positions, long long position_stride, long long offset,
                  const unsigned long long *freq, float amplitude, int B, int H, int H_kv, int S, int d,
                  int rot_dim, int layout, int direction, int dtype, fa_stream_t stream) {
    return fa::rope_impl(q, q_strides, q_out, q_out_strides, k, k_strides, k_out, k_out_strides, positions,
                         position_stride, offset, freq, amplitude, B, H, H_kv, S, d, rot_dim, layout, direction,
                         dtype, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_length,
                              double low_turns, double high_turns, unsigned long long *freq, float *amplitude) {
    if (rot_dim < 2 || rot_dim > 1024 || (rot_dim & 1) || !freq || !amplitude) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(base) || base < 1.0) return FA_ERR_INVALID_ARG;
    if (scaling != FA_ROPE_SCALE_NONE && scaling != FA_ROPE_SCALE_LINEAR && scaling != FA_ROPE_SCALE_NTK &&
        scaling != FA_ROPE_SCALE_BY_PARTS)
        return FA_ERR_UNSUPPORTED;
    if (scaling != FA_ROPE_SCALE_NONE && (!std::isfinite(factor) || factor < 1.0)) return FA_ERR_INVALID_ARG;
    if (scaling == FA_ROPE_SCALE_BY_PARTS &&
        (!std::isfinite(original_length) || original_length <= 0.0 || !std::isfinite(low_turns) ||
         !std::isfinite(high_turns) || low_turns >= high_turns))
        return FA_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == FA_ROPE_SCALE_NTK && rot_dim > 2) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    if (!std::isfinite(base)) return FA_ERR_INVALID_ARG;
    *amplitude = 1.0f;
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);  // radians per position, at most 1
        if (scaling == FA_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == FA_ROPE_SCALE_BY_PARTS) {
            const double turns = original_length * f / two_pi;
            const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low_turns) / (high_turns - low_turns)));
            f *= keep + (1.0 - keep) / factor;
        }
        freq[i] = (unsigned long long)std::llrint(std::ldexp(f / two_pi, 64));
    }
    if (scaling == FA_ROPE_SCALE_BY_PARTS) *amplitude = (float)(0.1 * std::log(factor) + 1.0);
    return FA_OK;
}

}  // extern "C"
