// Gated linear recurrence over the tokens of a sequence, channel by channel:
//
//   a_t = sigmoid(gate_t),  h_t = a_t h_{t-1} + s_t x_t,  s_t = 1 - a_t or 1
//
// (coupled or not), its gradient
//
//   G_t = dh_t + a_{t+1} G_{t+1},  dx_t = G_t s_t,
//   dgate_t = G_t (h_{t-1} - x_t | h_{t-1}) a_t (1 - a_t),  dh0 = a_0 G_0,
//
// and the single step for decoding.  States and sums are fp32; h is rounded
// once when it is stored.  1 - a is formed as e / (1 + e), e = exp(-gate), so
// that it keeps its digits where a is near 1.
#include <math.h>

#include "common.cuh"
#include "entry.h"
#include "internal.h"
#include "ptx.cuh"

namespace ta {

namespace {

struct ScanArgs {
    const void *gate, *x, *h, *dh;     // h, dh: backward
    const float *first, *last;         // the state before the first token, the last state's gradient; or NULL
    const int32_t* lengths;            // or NULL
    void *y, *dgate, *dx;              // h (forward); gradients
    float* end;                        // the last state, or the first one's gradient; or NULL
    int64_t gs[2], xs[2], dgs[2], dxs[2];  // strides of batch and token
    int B, N, D, coupled;
};

// a = sigmoid(g) and 1 - a.  The exponent is capped so that e a is finite: a
// gate of -inf leaves a = 2^-126 of the state and 1 - a = 1.  NaN stays NaN.
__device__ __forceinline__ void gates(float g, float& a, float& keep) {
    float t = g * -1.4426950408889634f;
    asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(t));  // 126
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(1.0f + e));
    keep = e * a;
}

template <typename T>
__device__ __forceinline__ T round_to(float x);
template <>
__device__ __forceinline__ float round_to<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One thread per channel, token by token.
template <typename T>
__global__ void __launch_bounds__(128) scan_channel_kernel(const __grid_constant__ ScanArgs a) {
    const int d = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
    if (d >= a.D) return;
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
    const T* g = static_cast<const T*>(a.gate) + b * a.gs[0] + d;
    const T* x = static_cast<const T*>(a.x) + b * a.xs[0] + d;
    T* y = static_cast<T*>(a.y) + (int64_t)b * a.N * a.D + d;
    float h = a.first ? a.first[(int64_t)b * a.D + d] : 0.f;
    for (int t = 0; t < a.N; ++t) {
        float out = 0.f;
        if (t < len) {
            float al, keep;
            gates(to_float(g[t * a.gs[1]]), al, keep);
            const float v = to_float(x[t * a.xs[1]]);
            out = h = fmaf(al, h, a.coupled ? keep * v : v);
        }
        y[(int64_t)t * a.D] = round_to<T>(out);
    }
    if (a.end) a.end[(int64_t)b * a.D + d] = h;
}

template <typename T>
__global__ void __launch_bounds__(128) scan_channel_backward_kernel(const __grid_constant__ ScanArgs a) {
    const int d = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
    if (d >= a.D) return;
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
    const T* g = static_cast<const T*>(a.gate) + b * a.gs[0] + d;
    const T* x = static_cast<const T*>(a.x) + b * a.xs[0] + d;
    const T* h = static_cast<const T*>(a.h) + (int64_t)b * a.N * a.D + d;
    const T* dh = static_cast<const T*>(a.dh) + (int64_t)b * a.N * a.D + d;
    T* dg = static_cast<T*>(a.dgate) + b * a.dgs[0] + d;
    T* dx = static_cast<T*>(a.dx) + b * a.dxs[0] + d;
    float c = a.last ? a.last[(int64_t)b * a.D + d] : 0.f;
    const float h0 = a.first ? a.first[(int64_t)b * a.D + d] : 0.f;
    for (int t = a.N - 1; t >= 0; --t) {
        float og = 0.f, ox = 0.f;
        if (t < len) {
            float al, keep;
            gates(to_float(g[t * a.gs[1]]), al, keep);
            const float v = to_float(x[t * a.xs[1]]);
            const float before = t ? to_float(h[(int64_t)(t - 1) * a.D]) : h0;
            const float G = to_float(dh[(int64_t)t * a.D]) + c;
            og = G * (a.coupled ? before - v : before) * (al * keep);
            ox = a.coupled ? G * keep : G;
            c = al * G;
        }
        dg[t * a.dgs[1]] = round_to<T>(og);
        dx[t * a.dxs[1]] = round_to<T>(ox);
    }
    if (a.end) a.end[(int64_t)b * a.D + d] = c;
}

template <typename T, bool BWD>
cudaError_t launch_scan(const ScanArgs& a, cudaStream_t stream) {
    const dim3 grid((a.D + 127) / 128, a.B);
    if (BWD) {
        TA_TIMED(stream, "scan_channel_backward_kernel", scan_channel_backward_kernel<T><<<grid, 128, 0, stream>>>(a));
    } else {
        TA_TIMED(stream, "scan_channel_kernel", scan_channel_kernel<T><<<grid, 128, 0, stream>>>(a));
    }
    return cudaGetLastError();
}

// One token: VE channels a thread.
template <typename T, int VE>
__global__ void __launch_bounds__(256)
gated_step_kernel(const T* __restrict__ gate, const T* __restrict__ x, const float* in, float* out, T* __restrict__ y,
                  int64_t gs, int64_t xs, int B, int D, int coupled) {
    const int per = D / VE;
    const int64_t total = (int64_t)B * per;
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int b = (int)(i / per), d = (int)(i - (int64_t)b * per) * VE;
        T g[VE], v[VE], o[VE];
        float s[VE];
        const int64_t at = (int64_t)b * D + d;
        if constexpr (VE == 4) {
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint2*>(g) = *reinterpret_cast<const uint2*>(gate + b * gs + d);
                *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(x + b * xs + d);
            } else {
                *reinterpret_cast<uint4*>(g) = *reinterpret_cast<const uint4*>(gate + b * gs + d);
                *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(x + b * xs + d);
            }
            *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(in + at);
        } else {
            g[0] = gate[b * gs + d], v[0] = x[b * xs + d], s[0] = in[at];
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            float a, keep;
            gates(to_float(g[e]), a, keep);
            const float xv = to_float(v[e]);
            s[e] = fmaf(a, s[e], coupled ? keep * xv : xv);
            o[e] = round_to<T>(s[e]);
        }
        if constexpr (VE == 4) {
            *reinterpret_cast<float4*>(out + at) = *reinterpret_cast<float4*>(s);
            if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(y + at) = *reinterpret_cast<uint2*>(o);
            else *reinterpret_cast<uint4*>(y + at) = *reinterpret_cast<uint4*>(o);
        } else {
            out[at] = s[0], y[at] = o[0];
        }
    }
}

template <typename T>
int step_entry(const T* gate, const T* x, const float* in, float* out, T* y, int B, int D, int64_t gs, int64_t xs,
               int coupled, cudaStream_t stream) {
    if (B < 0 || D < 0 || gs < 0 || xs < 0) return TAYLOR_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return TAYLOR_OK;
    if (!gate || !x || !in || !out || !y) return TAYLOR_ERR_INVALID_ARG;
    if (!entry::aligned(gate, sizeof(T)) || !entry::aligned(x, sizeof(T)) || !entry::aligned(y, sizeof(T)) ||
        !entry::aligned(in, 4) || !entry::aligned(out, 4))
        return TAYLOR_ERR_MISALIGNED;
    const size_t four = 4 * sizeof(T);
    const bool wide = D % 4 == 0 && gs % 4 == 0 && xs % 4 == 0 && entry::aligned(gate, four) && entry::aligned(x, four) &&
                      entry::aligned(y, four) && entry::aligned(in, 16) && entry::aligned(out, 16);
    const int64_t pieces = (int64_t)B * D / (wide ? 4 : 1);
    int64_t grid = (pieces + 255) / 256;
    const int64_t most = (int64_t)entry::num_sms() * 16;
    if (grid > most) grid = most;
    if (wide) {
        TA_TIMED(stream, "gated_step_kernel", gated_step_kernel<T, 4><<<(unsigned)grid, 256, 0, stream>>>(
            gate, x, in, out, y, gs, xs, B, D, coupled));
    } else {
        TA_TIMED(stream, "gated_step_kernel", gated_step_kernel<T, 1><<<(unsigned)grid, 256, 0, stream>>>(
            gate, x, in, out, y, gs, xs, B, D, coupled));
    }
    return entry::status(cudaGetLastError());
}

// Checks of both directions; a holds what the caller passed.
template <typename T, bool BWD>
int scan_entry(ScanArgs a, const int64_t* gs, const int64_t* xs, const int64_t* dgs, const int64_t* dxs,
               cudaStream_t stream) {
    if (a.B < 0 || a.N < 0 || a.D < 0) return TAYLOR_ERR_INVALID_ARG;
    if ((int64_t)a.B * a.N >= ((int64_t)1 << 31) || (int64_t)a.B * a.D >= ((int64_t)1 << 31))
        return TAYLOR_ERR_UNSUPPORTED;
    if (a.B == 0 || a.D == 0) return TAYLOR_OK;
    if ((a.first && !entry::aligned(a.first, 4)) || (a.last && !entry::aligned(a.last, 4)) ||
        (a.end && !entry::aligned(a.end, 4)) || (a.lengths && !entry::aligned(a.lengths, 4)))
        return TAYLOR_ERR_MISALIGNED;
    const size_t state = (size_t)a.B * a.D * sizeof(float);
    if (a.N == 0) {
        // no token: the state, or its gradient, passes through
        const float* from = BWD ? a.last : a.first;
        if (!a.end || a.end == from) return TAYLOR_OK;
        if (!from) return entry::status(cudaMemsetAsync(a.end, 0, state, stream));
        return entry::status(cudaMemcpyAsync(a.end, from, state, cudaMemcpyDeviceToDevice, stream));
    }
    if (!a.gate || !a.x || !gs || !xs) return TAYLOR_ERR_INVALID_ARG;
    if (BWD ? (!a.h || !a.dh || !a.dgate || !a.dx || !dgs || !dxs) : !a.y) return TAYLOR_ERR_INVALID_ARG;
    const void* p[] = {a.gate, a.x, a.h, a.dh, a.y, a.dgate, a.dx};
    for (const void* q : p)
        if (q && !entry::aligned(q, sizeof(T))) return TAYLOR_ERR_MISALIGNED;
    const int64_t size[2] = {a.B, a.N};
    for (int i = 0; i < 2; ++i) {
        if (gs[i] < 0 || xs[i] < 0) return TAYLOR_ERR_INVALID_ARG;
        a.gs[i] = gs[i], a.xs[i] = xs[i];
        if (BWD) a.dgs[i] = dgs[i], a.dxs[i] = dxs[i];
    }
    if (BWD && (!entry::disjoint(size, a.dgs, a.D) || !entry::disjoint(size, a.dxs, a.D)))
        return TAYLOR_ERR_INVALID_ARG;
    return entry::status(launch_scan<T, BWD>(a, stream));
}

template <typename T>
int scan_forward(const void* gate, const void* x, const float* h0, const int32_t* lengths, void* h, float* h_last,
                 int B, int N, int D, const int64_t* gs, const int64_t* xs, int coupled, cudaStream_t stream) {
    ScanArgs a = {};
    a.gate = gate, a.x = x, a.first = h0, a.lengths = lengths, a.y = h, a.end = h_last;
    a.B = B, a.N = N, a.D = D, a.coupled = coupled != 0;
    return scan_entry<T, false>(a, gs, xs, nullptr, nullptr, stream);
}

template <typename T>
int scan_backward(const void* gate, const void* x, const void* h, const void* dh, const float* h0,
                  const int32_t* lengths, const float* dh_last, void* dgate, void* dx, float* dh0, int B, int N, int D,
                  const int64_t* gs, const int64_t* xs, const int64_t* dgs, const int64_t* dxs, int coupled,
                  cudaStream_t stream) {
    ScanArgs a = {};
    a.gate = gate, a.x = x, a.h = h, a.dh = dh, a.first = h0, a.last = dh_last, a.lengths = lengths;
    a.dgate = dgate, a.dx = dx, a.end = dh0;
    a.B = B, a.N = N, a.D = D, a.coupled = coupled != 0;
    return scan_entry<T, true>(a, gs, xs, dgs, dxs, stream);
}

}  // namespace

}  // namespace ta

extern "C" {

int taylor_attn_gated_scan(const void* gate, const void* x, const float* h0, const int32_t* lengths, void* h,
                           float* h_last, int B, int N, int D, const int64_t* gate_strides, const int64_t* x_strides,
                           int coupled, cudaStream_t stream) {
    return ta::scan_forward<__nv_bfloat16>(gate, x, h0, lengths, h, h_last, B, N, D, gate_strides, x_strides, coupled,
                                           stream);
}

int taylor_attn_gated_scan_f32(const float* gate, const float* x, const float* h0, const int32_t* lengths, float* h,
                               float* h_last, int B, int N, int D, const int64_t* gate_strides,
                               const int64_t* x_strides, int coupled, cudaStream_t stream) {
    return ta::scan_forward<float>(gate, x, h0, lengths, h, h_last, B, N, D, gate_strides, x_strides, coupled, stream);
}

int taylor_attn_gated_scan_backward(const void* gate, const void* x, const void* h, const void* dh, const float* h0,
                                    const int32_t* lengths, const float* dh_last, void* dgate, void* dx, float* dh0,
                                    int B, int N, int D, const int64_t* gate_strides, const int64_t* x_strides,
                                    const int64_t* dgate_strides, const int64_t* dx_strides, int coupled,
                                    cudaStream_t stream) {
    return ta::scan_backward<__nv_bfloat16>(gate, x, h, dh, h0, lengths, dh_last, dgate, dx, dh0, B, N, D,
                                            gate_strides, x_strides, dgate_strides, dx_strides, coupled, stream);
}

int taylor_attn_gated_scan_backward_f32(const float* gate, const float* x, const float* h, const float* dh,
                                        const float* h0, const int32_t* lengths, const float* dh_last, float* dgate,
                                        float* dx, float* dh0, int B, int N, int D, const int64_t* gate_strides,
                                        const int64_t* x_strides, const int64_t* dgate_strides,
                                        const int64_t* dx_strides, int coupled, cudaStream_t stream) {
    return ta::scan_backward<float>(gate, x, h, dh, h0, lengths, dh_last, dgate, dx, dh0, B, N, D, gate_strides,
                                    x_strides, dgate_strides, dx_strides, coupled, stream);
}

int taylor_attn_gated_step(const void* gate, const void* x, const float* state_in, float* state_out, void* out, int B,
                           int D, int64_t gate_stride, int64_t x_stride, int coupled, cudaStream_t stream) {
    using bf = __nv_bfloat16;
    return ta::step_entry<bf>(static_cast<const bf*>(gate), static_cast<const bf*>(x), state_in, state_out,
                              static_cast<bf*>(out), B, D, gate_stride, x_stride, coupled, stream);
}

int taylor_attn_gated_step_f32(const float* gate, const float* x, const float* state_in, float* state_out, float* out,
                               int B, int D, int64_t gate_stride, int64_t x_stride, int coupled,
                               cudaStream_t stream) {
    return ta::step_entry<float>(gate, x, state_in, state_out, out, B, D, gate_stride, x_stride, coupled, stream);
}

}  // extern "C"
