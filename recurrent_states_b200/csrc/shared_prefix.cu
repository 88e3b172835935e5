// One new token for every sequence of a batch that shares a long prefix.
//
// The Taylor state is additive over tokens, so with the prefix's state S (one
// for the whole batch) and a sequence's own tokens j <= L in a key and value
// cache, L the new one,
//
//   y = (c (.) phi(q))^T S + sum_{j <= L} K(tau q.k_j) [v_j | 1],
//   out = y[0:d_v] / y[d_v],
//
// K the truncated series: the own tokens are taken pairwise, exactly as their
// state would count them, and no sequence keeps, reads or writes a state of
// its own.  The new k and v are appended to the cache in the same call.
#include <math.h>

#include "common.cuh"
#include "entry.h"
#include "feature_table.cuh"
#include "internal.h"

namespace ta {

namespace {

constexpr unsigned int kErrLength = 32u;  // bit of the device error word

struct PrefixArgs {
    const void *q, *k, *v;
    const float* state;       // [H][stride]
    void *kc, *vc;            // [B][H][cap][d], [B][H][cap][dv]
    const int32_t* lengths;   // [B]
    float* out;               // [B][H][dv]
    unsigned int* err;
    int64_t F, stride;
    int B, H, cap, d, dv, n;
    float tau;
};

// One CTA per sequence and head.
template <typename T>
__global__ void __launch_bounds__(256) prefix_head_kernel(const __grid_constant__ PrefixArgs a) {
    __shared__ float qs[kMaxDk], phi[256], coef[kMaxN], num[kMaxDv + 1];
    const int tid = threadIdx.x, bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    const T* q = static_cast<const T*>(a.q) + (int64_t)bh * a.d;
    const T* k = static_cast<const T*>(a.k) + (int64_t)bh * a.d;
    const T* v = static_cast<const T*>(a.v) + (int64_t)bh * a.dv;
    T* kc = static_cast<T*>(a.kc) + (int64_t)bh * a.cap * a.d;
    T* vc = static_cast<T*>(a.vc) + (int64_t)bh * a.cap * a.dv;
    const int L = a.lengths[b];
    if (L < 0 || L >= a.cap) {
        if (tid < a.dv) a.out[(int64_t)bh * a.dv + tid] = nanf("");
        if (tid == 0) atomicOr(a.err, kErrLength);
        return;
    }
    if (tid < a.d) qs[tid] = to_float(q[tid]);
    if (tid < a.n) coef[tid] = query_coeff(tid, a.tau);
    __syncthreads();
    const PackedFeat* tab = feat_table(a.d, a.n);
    const float* S = a.state + (int64_t)h * a.stride;
    // thread c sums column c, thread 0 column d_v too
    float y = 0.f, z = 0.f;
    for (int64_t f0 = 0; f0 < a.F; f0 += 256) {
        if (f0 + tid < a.F) phi[tid] = eval_desc(get_desc(tab, a.d, a.n, f0 + tid, a.tau, coef, true), qs);
        __syncthreads();
        const int nf = (int)min64(256, a.F - f0);
        if (tid < a.dv)
            for (int f = 0; f < nf; ++f) y = fmaf(phi[f], S[(f0 + f) * a.dv + tid], y);
        if (tid == 0)
            for (int f = 0; f < nf; ++f) z = fmaf(phi[f], S[a.F * a.dv + f0 + f], z);
        __syncthreads();
    }
    for (int j0 = 0; j0 <= L; j0 += 256) {
        const int j = j0 + tid;
        if (j <= L) {
            const T* row = j < L ? kc + (int64_t)j * a.d : k;
            float x = 0.f;
            for (int i = 0; i < a.d; ++i) x = fmaf(qs[i], to_float(row[i]), x);
            phi[tid] = taylor_kernel(a.tau * x, a.n);
        }
        __syncthreads();
        const int nj = min(256, L + 1 - j0);
        for (int i = 0; i < nj; ++i) {
            const T* row = j0 + i < L ? vc + (int64_t)(j0 + i) * a.dv : v;
            if (tid < a.dv) y = fmaf(phi[i], to_float(row[tid]), y);
            if (tid == 0) z += phi[i];
        }
        __syncthreads();
    }
    if (tid < a.dv) num[tid] = y;
    if (tid == 0) num[a.dv] = z;
    __syncthreads();
    if (tid < a.dv) a.out[(int64_t)bh * a.dv + tid] = num[tid] / num[a.dv];
    if (tid < a.d) kc[(int64_t)L * a.d + tid] = k[tid];
    if (tid < a.dv) vc[(int64_t)L * a.dv + tid] = v[tid];
}

template <typename T>
cudaError_t launch_prefix(PrefixArgs& a, cudaStream_t stream) {
    TA_TIMED(stream, "prefix_head_kernel", prefix_head_kernel<T><<<(unsigned)(a.B * a.H), 256, 0, stream>>>(a));
    return cudaGetLastError();
}

template <typename T>
int prefix_entry(const T* q, const T* k, const T* v, const float* state, T* kc, T* vc, const int32_t* lengths,
                 float* out, int B, int H, int cap, int d, int dv, int n, float tau, cudaStream_t stream) {
    if (B < 0 || H < 0 || cap < 0 || d < 0 || dv < 0 || n < 0 || !isfinite(tau)) return TAYLOR_ERR_INVALID_ARG;
    if (n < 1 || n > kMaxN || d < 1 || d > kMaxDk || dv < 4 || dv > kMaxDv || dv % 4 != 0) return TAYLOR_ERR_UNSUPPORTED;
    if ((int64_t)B * H >= ((int64_t)1 << 24)) return TAYLOR_ERR_UNSUPPORTED;
    if (B == 0 || H == 0) return TAYLOR_OK;
    if (cap < 1 || !q || !k || !v || !state || !kc || !vc || !lengths || !out) return TAYLOR_ERR_INVALID_ARG;
    const void* p[] = {q, k, v, state, kc, vc, out};
    for (const void* x : p)
        if (!entry::aligned(x, 16)) return TAYLOR_ERR_MISALIGNED;
    if (!entry::aligned(lengths, 4)) return TAYLOR_ERR_MISALIGNED;
    PrefixArgs a = {};
    a.q = q, a.k = k, a.v = v, a.state = state, a.kc = kc, a.vc = vc, a.lengths = lengths, a.out = out;
    a.F = num_features(d, n);
    a.stride = (a.F * (dv + 1) + 31) / 32 * 32;
    a.B = B, a.H = H, a.cap = cap, a.d = d, a.dv = dv, a.n = n, a.tau = tau;
    a.err = device_error_word();
    if (!a.err) return TAYLOR_ERR_CUDA;
    return entry::status(launch_prefix<T>(a, stream));
}

}  // namespace

}  // namespace ta

extern "C" {

int taylor_attn_shared_prefix_decode(const void* q, const void* k, const void* v, const float* prefix_state,
                                     void* k_cache, void* v_cache, const int32_t* lengths, float* out, int B, int H,
                                     int cap, int d_k, int d_v, int n, float tau, cudaStream_t stream) {
    using bf = __nv_bfloat16;
    return ta::prefix_entry<bf>(static_cast<const bf*>(q), static_cast<const bf*>(k), static_cast<const bf*>(v),
                                prefix_state, static_cast<bf*>(k_cache), static_cast<bf*>(v_cache), lengths, out, B, H,
                                cap, d_k, d_v, n, tau, stream);
}

int taylor_attn_shared_prefix_decode_f32(const float* q, const float* k, const float* v, const float* prefix_state,
                                         float* k_cache, float* v_cache, const int32_t* lengths, float* out, int B,
                                         int H, int cap, int d_k, int d_v, int n, float tau, cudaStream_t stream) {
    return ta::prefix_entry<float>(q, k, v, prefix_state, k_cache, v_cache, lengths, out, B, H, cap, d_k, d_v, n, tau,
                                   stream);
}

}  // extern "C"
