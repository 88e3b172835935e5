// Norms of queries and keys for each head with the position rotation in the
// same pass, and its gradient.
//
//   u = w (.) x / sqrt(sum x^2 + eps),   y = R(p) u
//
// per head row x of d values; w is optional (one weight per entry, shared by
// the heads).  R(p) turns the first `rot` entries of a row at position p:
// the pair (a, b) of frequency theta_j becomes (a cos - b sin, b cos + a sin)
// at the angle p theta_j; pairs are (j, j + rot/2), or (2j, 2j + 1) when
// interleaved.  Inputs are token-major with any strides (a projection's
// output, or a slice of a packed one), outputs are the dense head-major
// [B][H][N][d] that the attention calls take.  The gradient, with the same
// angles and the norm recomputed from x:
//
//   du = R(p)^T dy,  dw = sum du (.) xhat,  dx = (g - xhat (xhat . g)) inv
//
// with xhat = x inv, g = du (.) w, inv = 1 / sqrt(sum x^2 + eps).
//
// Angles: p theta_j / (2 pi) is formed in fp64 and reduced to its fraction of
// a turn there, so that far positions lose nothing; the sine and cosine of
// the fraction are fp32.  Everything else is fp32, rounded once at the end.
#include <math.h>

#include "common.cuh"
#include "entry.h"
#include "internal.h"

namespace ta {

namespace {

constexpr int kMaxHalf = kMaxDk / 2;

struct QkArgs {
    const void* x[2];        // q, k
    const void* dy[2];       // gradients of the outputs (backward)
    void* y[2];              // outputs, or gradients of q and k (backward)
    const float* w[2];       // weights or NULL
    int64_t xs[2][3];        // strides of x: batch, token, head
    int64_t ys[2][3];        // strides of the strided output (backward)
    int H[2];                // heads
    const int64_t* pos;      // [B][N] or NULL: pos0 + n
    int64_t pos0;
    float* dw;               // per-CTA partial weight gradients [grid][2][d], or NULL
    float eps;
    int B, N, d, rot, inter;
    double turn[kMaxHalf];   // turns per position
};

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__device__ __forceinline__ float2 cos_sin(const QkArgs& a, int64_t p, int j) {
    const double t = (double)p * a.turn[j];
    float s, c;
    sincospif(2.0f * (float)(t - rint(t)), &s, &c);
    return make_float2(c, s);
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// 1 / sqrt(sum x^2 + eps) over a group of G lanes.  Where the sum of squares
// leaves fp32's comfortable range, x is first divided by its largest entry m,
// and the result belongs to x / m (m is returned, else 1).  A row of zeros
// with eps 0 gives 0: its output and its gradient are zero.  All 32 lanes
// call it together.
template <int G, int E>
__device__ __forceinline__ float inv_norm(float (&x)[E], float eps, float& m) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(x[e], x[e], s);
    s = group_sum<G>(s);
    m = 1.f;
    const bool far = !(s > 1e-30f && s < 1e37f);
    if (__any_sync(0xffffffffu, far)) {
        float big = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) big = fmaxf(big, fabsf(x[e]));
        big = group_max<G>(big);
        if (far && s == s && big > 0.f && big < INFINITY) m = big;
        float s2 = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (m != 1.f) x[e] /= m;
            s2 = fmaf(x[e], x[e], s2);
        }
        s = group_sum<G>(s2) + (m != 1.f && eps > 0.f ? eps / m / m : eps);
        return s == 0.f ? 0.f : rsqrtf(s);
    }
    return rsqrtf(s + eps);
}

// Any d: one warp per token and head slice, lane l holding the entries l and
// l + 32, looping over the heads so that the angles are formed once.  Rows
// are read and written element by element; the vector kernel below takes the
// rows whose length and alignment allow wider accesses.
template <typename T, bool BWD>
__global__ void __launch_bounds__(256)
qk_any_kernel(const __grid_constant__ QkArgs a, int slices) {
    __shared__ float red[8][2][kMaxDk];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = a.rot >> 1;
    const int64_t items = (int64_t)a.B * a.N * slices;
    float acc[2][2] = {};
    for (int64_t it = (int64_t)blockIdx.x * 8 + warp; it < items; it += (int64_t)gridDim.x * 8) {
        const int slice = (int)(it % slices);
        const unsigned t = (unsigned)(it / slices);
        const int b = t / (unsigned)a.N, n = t - (unsigned)b * (unsigned)a.N;
        const int64_t p = a.pos ? a.pos[t] : a.pos0 + n;
        float c[2], s[2];
        int mate[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = lane + 32 * e;
            c[e] = 1.f, s[e] = 0.f, mate[e] = i;
            if (i < a.rot) {
                const bool first = a.inter ? (i & 1) == 0 : i < half;
                mate[e] = a.inter ? i ^ 1 : (first ? i + half : i - half);
                const float2 cs = cos_sin(a, p, a.inter ? i >> 1 : (first ? i : i - half));
                c[e] = cs.x;
                s[e] = (first != BWD) ? -cs.y : cs.y;
            }
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const float* w = a.w[z];
            const float w0 = w && lane < a.d ? w[lane] : 1.f, w1 = w && lane + 32 < a.d ? w[lane + 32] : 1.f;
            for (int h = slice; h < a.H[z]; h += slices) {
                const T* xr = static_cast<const T*>(a.x[z]) + b * a.xs[z][0] + n * a.xs[z][1] + h * a.xs[z][2];
                const int64_t dense = (((int64_t)b * a.H[z] + h) * a.N + n) * a.d;
                float x[2] = {lane < a.d ? to_float(xr[lane]) : 0.f,
                              lane + 32 < a.d ? to_float(xr[lane + 32]) : 0.f};
                float m;
                const float inv = inv_norm<32>(x, a.eps, m);
                float in[2];
                if (BWD) {
                    const T* gr = static_cast<const T*>(a.dy[z]) + dense;
                    in[0] = lane < a.d ? to_float(gr[lane]) : 0.f;
                    in[1] = lane + 32 < a.d ? to_float(gr[lane + 32]) : 0.f;
                } else {
                    in[0] = x[0] * w0;
                    in[1] = x[1] * w1;
                }
                float out[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float lo = __shfl_sync(0xffffffffu, in[0], mate[e] & 31);
                    const float hi = __shfl_sync(0xffffffffu, in[1], mate[e] & 31);
                    const float other = mate[e] & 32 ? hi : lo;
                    out[e] = lane + 32 * e < a.rot ? fmaf(other, s[e], in[e] * c[e]) : in[e];
                }
                if (BWD) {
                    const float xh0 = x[0] * inv, xh1 = x[1] * inv;
                    acc[z][0] = fmaf(out[0], xh0, acc[z][0]);
                    acc[z][1] = fmaf(out[1], xh1, acc[z][1]);
                    const float g0 = out[0] * w0, g1 = out[1] * w1;
                    const float along = group_sum<32>(g0 * xh0 + g1 * xh1);
                    T* o = static_cast<T*>(a.y[z]) + b * a.ys[z][0] + n * a.ys[z][1] + h * a.ys[z][2];
                    out[0] = (g0 - xh0 * along) * inv;
                    out[1] = (g1 - xh1 * along) * inv;
                    if (m != 1.f) out[0] /= m, out[1] /= m;
                    if (lane < a.d) o[lane] = from_float<T>(out[0]);
                    if (lane + 32 < a.d) o[lane + 32] = from_float<T>(out[1]);
                } else {
                    T* o = static_cast<T*>(a.y[z]) + dense;
                    if (lane < a.d) o[lane] = from_float<T>(out[0] * inv);
                    if (lane + 32 < a.d) o[lane + 32] = from_float<T>(out[1] * inv);
                }
            }
        }
    }
    if (BWD && a.dw) {
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int e = 0; e < 2; ++e) red[warp][z][lane + 32 * e] = acc[z][e];
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.d; i += 256) {
            const int z = i / a.d, c = i - z * a.d;
            float v = 0.f;
            for (int r = 0; r < 8; ++r) v += red[r][z][c];
            a.dw[(int64_t)blockIdx.x * 2 * a.d + i] = v;
        }
    }
}

// dw[z][c] = sum of the CTAs' partials, one warp per column, in a fixed order.
__global__ void __launch_bounds__(256)
qk_weight_grad_kernel(const float* __restrict__ part, int parts, int d, float* dqw, float* dkw) {
    const int col = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (col >= 2 * d) return;
    float v = 0.f;
    for (int i = lane; i < parts; i += 32) v += part[(int64_t)i * 2 * d + col];
    v = group_sum<32>(v);
    float* out = col < d ? dqw : dkw;
    if (lane == 0 && out) out[col < d ? col : col - d] = v;
}

template <typename T, bool BWD>
cudaError_t launch_qk(QkArgs& a, float* dqw, float* dkw, cudaStream_t stream) {
    const int sms = entry::num_sms();
    const int64_t tokens = (int64_t)a.B * a.N;
    const int heads = a.H[0] > a.H[1] ? a.H[0] : a.H[1];
    // enough warps to fill the GPU before a warp takes several heads
    int slices = 1;
    while (slices < heads && tokens * slices < (int64_t)sms * 32) slices *= 2;
    if (slices > heads) slices = heads;
    int64_t grid = (tokens * slices + 7) / 8;
    if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
    float* part = nullptr;
    if (BWD && (dqw || dkw)) {
        const cudaError_t e = workspace_alloc(reinterpret_cast<void**>(&part), (size_t)grid * 2 * a.d * 4, stream);
        if (e != cudaSuccess) return e;
    }
    a.dw = part;
    TA_TIMED(stream, "qk_any_kernel", qk_any_kernel<T, BWD><<<(unsigned)grid, 256, 0, stream>>>(a, slices));
    cudaError_t e = cudaGetLastError();
    if (part) {
        if (e == cudaSuccess) {
            TA_TIMED(stream, "qk_weight_grad_kernel",
                     qk_weight_grad_kernel<<<(2 * a.d + 7) / 8, 256, 0, stream>>>(part, (int)grid, a.d, dqw, dkw));
            e = cudaGetLastError();
        }
        const cudaError_t f = workspace_free(part, stream);
        if (e == cudaSuccess) e = f;
    }
    return e;
}

// Checks and argument packing of all four entry points.
template <typename T, bool BWD>
int qk_entry(const void* q, const void* k, const void* dqo, const void* dko, const float* qw, const float* kw,
             const int64_t* positions, int64_t pos0, const double* freqs, int rot, int interleaved, void* yq, void* yk,
             float* dqw, float* dkw, int B, int N, int Hq, int Hk, int d, const int64_t* qs, const int64_t* ks,
             const int64_t* dqs, const int64_t* dks, float eps, cudaStream_t stream) {
    if (B < 0 || N < 0 || Hq < 0 || Hk < 0 || d < 0 || rot < 0) return TAYLOR_ERR_INVALID_ARG;
    if (d < 1 || d > kMaxDk || rot > d || (rot & 1)) return TAYLOR_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !isfinite(eps)) return TAYLOR_ERR_INVALID_ARG;
    if (rot > 0 && !freqs) return TAYLOR_ERR_INVALID_ARG;
    for (int j = 0; j < rot / 2; ++j)
        if (!isfinite(freqs[j])) return TAYLOR_ERR_INVALID_ARG;
    if ((dqw && !qw) || (dkw && !kw)) return TAYLOR_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 31;
    const int64_t tokens = (int64_t)B * N;
    if (tokens >= most || tokens * Hq >= most || tokens * Hk >= most) return TAYLOR_ERR_UNSUPPORTED;
    if (tokens == 0 || (Hq == 0 && Hk == 0)) {
        cudaError_t e = cudaSuccess;
        if (BWD && dqw) e = cudaMemsetAsync(dqw, 0, (size_t)d * 4, stream);
        if (BWD && dkw && e == cudaSuccess) e = cudaMemsetAsync(dkw, 0, (size_t)d * 4, stream);
        return entry::status(e);
    }
    QkArgs a = {};
    const void* x[2] = {q, k};
    const void* dy[2] = {dqo, dko};
    void* y[2] = {yq, yk};
    const float* w[2] = {qw, kw};
    const int64_t* xs[2] = {qs, ks};
    const int64_t* ys[2] = {dqs, dks};
    const int H[2] = {Hq, Hk};
    for (int z = 0; z < 2; ++z) {
        if (H[z] == 0) continue;
        if (!x[z] || !y[z] || !xs[z] || (BWD && (!dy[z] || !ys[z]))) return TAYLOR_ERR_INVALID_ARG;
        if (!entry::aligned(x[z], sizeof(T)) || !entry::aligned(y[z], sizeof(T)) ||
            (BWD && !entry::aligned(dy[z], sizeof(T))) || (w[z] && !entry::aligned(w[z], 4)))
            return TAYLOR_ERR_MISALIGNED;
        for (int i = 0; i < 3; ++i) {
            a.xs[z][i] = xs[z][i];
            if (xs[z][i] < 0) return TAYLOR_ERR_INVALID_ARG;
            if (BWD) a.ys[z][i] = ys[z][i];
        }
        if (BWD) {
            const int64_t size[3] = {B, N, H[z]};
            if (!entry::disjoint(size, a.ys[z], d)) return TAYLOR_ERR_INVALID_ARG;
        }
        a.x[z] = x[z], a.dy[z] = dy[z], a.y[z] = y[z], a.w[z] = w[z], a.H[z] = H[z];
    }
    if (positions && !entry::aligned(positions, 8)) return TAYLOR_ERR_MISALIGNED;
    a.pos = positions, a.pos0 = pos0, a.eps = eps;
    a.B = B, a.N = N, a.d = d, a.rot = rot, a.inter = interleaved != 0;
    for (int j = 0; j < rot / 2; ++j) a.turn[j] = freqs[j] / 6.283185307179586476925286766559;
    return entry::status(launch_qk<T, BWD>(a, dqw, dkw, stream));
}

}  // namespace

}  // namespace ta

extern "C" {

int taylor_attn_qk_norm_rope(const void* q, const void* k, const float* q_weight, const float* k_weight,
                             const int64_t* positions, int64_t pos0, const double* freqs, int rot, int interleaved,
                             void* q_out, void* k_out, int B, int N, int Hq, int Hk, int d, const int64_t* q_strides,
                             const int64_t* k_strides, float eps, cudaStream_t stream) {
    return ta::qk_entry<__nv_bfloat16, false>(q, k, nullptr, nullptr, q_weight, k_weight, positions, pos0, freqs, rot,
                                              interleaved, q_out, k_out, nullptr, nullptr, B, N, Hq, Hk, d, q_strides,
                                              k_strides, nullptr, nullptr, eps, stream);
}

int taylor_attn_qk_norm_rope_f32(const float* q, const float* k, const float* q_weight, const float* k_weight,
                                 const int64_t* positions, int64_t pos0, const double* freqs, int rot,
                                 int interleaved, float* q_out, float* k_out, int B, int N, int Hq, int Hk, int d,
                                 const int64_t* q_strides, const int64_t* k_strides, float eps, cudaStream_t stream) {
    return ta::qk_entry<float, false>(q, k, nullptr, nullptr, q_weight, k_weight, positions, pos0, freqs, rot,
                                      interleaved, q_out, k_out, nullptr, nullptr, B, N, Hq, Hk, d, q_strides,
                                      k_strides, nullptr, nullptr, eps, stream);
}

int taylor_attn_qk_norm_rope_backward(const void* q, const void* k, const void* dq_out, const void* dk_out,
                                      const float* q_weight, const float* k_weight, const int64_t* positions,
                                      int64_t pos0, const double* freqs, int rot, int interleaved, void* dq, void* dk,
                                      float* dq_weight, float* dk_weight, int B, int N, int Hq, int Hk, int d,
                                      const int64_t* q_strides, const int64_t* k_strides, const int64_t* dq_strides,
                                      const int64_t* dk_strides, float eps, cudaStream_t stream) {
    return ta::qk_entry<__nv_bfloat16, true>(q, k, dq_out, dk_out, q_weight, k_weight, positions, pos0, freqs, rot,
                                             interleaved, dq, dk, dq_weight, dk_weight, B, N, Hq, Hk, d, q_strides,
                                             k_strides, dq_strides, dk_strides, eps, stream);
}

int taylor_attn_qk_norm_rope_backward_f32(const float* q, const float* k, const float* dq_out, const float* dk_out,
                                          const float* q_weight, const float* k_weight, const int64_t* positions,
                                          int64_t pos0, const double* freqs, int rot, int interleaved, float* dq,
                                          float* dk, float* dq_weight, float* dk_weight, int B, int N, int Hq, int Hk,
                                          int d, const int64_t* q_strides, const int64_t* k_strides,
                                          const int64_t* dq_strides, const int64_t* dk_strides, float eps,
                                          cudaStream_t stream) {
    return ta::qk_entry<float, true>(q, k, dq_out, dk_out, q_weight, k_weight, positions, pos0, freqs, rot,
                                     interleaved, dq, dk, dq_weight, dk_weight, B, N, Hq, Hk, d, q_strides, k_strides,
                                     dq_strides, dk_strides, eps, stream);
}

}  // extern "C"
