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
#include "pairs.cuh"
#include "ptx.cuh"

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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Whether t = sum x^2 + eps is out of fp32's comfortable range, or NaN.  Above
// 1e-30 the squares that underflow in the sum are nothing beside t, be it the
// row's or eps that makes it so large.
__device__ __forceinline__ bool out_of_range(float t) { return !(t > 1e-30f && t < 1e37f); }

// 1 / sqrt(sum x^2 + eps) of rows held by groups of `lanes` neighbouring lanes,
// from a lane's entries x and the group's sum of squares s.  Where s + eps is
// out of range, x is first divided by m, the larger of its largest entry and
// sqrt(eps), so that neither x / m nor eps / m^2 is above 1, and the result
// belongs to x / m (m is returned, else 1).  A row of zeros with eps 0 gives 0:
// its output and its gradient are zero.  All 32 lanes call it together.
template <int E>
__device__ __forceinline__ float far_norm(float (&x)[E], float s, float eps, float& m, int lanes) {
    m = 1.f;
    const float t = s + eps;
    const bool far = out_of_range(t);
    if (__any_sync(0xffffffffu, far)) {
        float big = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) big = fmaxf(big, fabsf(x[e]));
        for (int o = lanes >> 1; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        const float size = fmaxf(big, sqrtf(eps));
        if (far && t == t && size > 0.f && big < INFINITY) m = size;
        float s2 = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (m != 1.f) x[e] /= m;
            s2 = fmaf(x[e], x[e], s2);
        }
        for (int o = lanes >> 1; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        s = s2 + (m != 1.f ? eps / m / m : eps);
        return s != 0.f ? rsqrtf(s) : 0.f;
    }
    return rsqrtf(t);
}

// Any d: LPR neighbouring lanes per token and head slice, lane l holding entry
// l (and l + 32 where E is 2: then one head at a time, four need too many
// registers), walking the heads four at a time so that the angles are formed
// once.  Rows are read and written element by element; the
// vector kernel below takes the rows whose length and alignment allow wider
// accesses.
template <typename T, int LPR, int E, bool BWD>
__global__ void __launch_bounds__(256)
qk_any_kernel(const __grid_constant__ QkArgs a, int slices) {
    __shared__ float red[8][2][kMaxDk];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int PER = 32 / LPR, kAnyRows = E == 2 ? 1 : 4;  // tokens of a warp; heads in flight
    const int l = lane & (LPR - 1), base = lane & ~(LPR - 1);
    const int half = a.rot >> 1;
    const int64_t tokens = (int64_t)a.B * a.N, groups = (tokens + PER - 1) / PER;
    float acc[2][E] = {};
    for (int64_t it = (int64_t)blockIdx.x * 8 + warp; it < groups * slices; it += (int64_t)gridDim.x * 8) {
        const int slice = (int)(it % slices);
        const int64_t at = it / slices * PER + base / LPR;
        const bool live = at < tokens;
        const unsigned t = live ? (unsigned)at : 0u;
        const int b = t / (unsigned)a.N, n = t - (unsigned)b * (unsigned)a.N;
        const int64_t p = a.pos ? a.pos[t] : a.pos0 + n;
        float c[E], s[E];
        int mate[E];
        bool on[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = l + 32 * e;
            on[e] = live && i < a.d;
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
            float w[E];
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = a.w[z] && l + 32 * e < a.d ? a.w[z][l + 32 * e] : 1.f;
            const T* xb = static_cast<const T*>(a.x[z]) + b * a.xs[z][0] + n * a.xs[z][1] + l;
            const int64_t dense = ((int64_t)b * a.H[z] * a.N + n) * a.d + l, dense_h = (int64_t)a.N * a.d;
            for (int h0 = slice; h0 < a.H[z]; h0 += kAnyRows * slices) {
                float x[kAnyRows][E], in[kAnyRows][E], sq[kAnyRows];
#pragma unroll
                for (int u = 0; u < kAnyRows; ++u) {
                    const int h = h0 + u * slices;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const bool use = on[e] && h < a.H[z];
                        x[u][e] = use ? to_float(xb[h * a.xs[z][2] + 32 * e]) : 0.f;
                        if (BWD) in[u][e] = use ? to_float(static_cast<const T*>(a.dy[z])[dense + h * dense_h + 32 * e]) : 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < kAnyRows; ++u) {
                    sq[u] = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) sq[u] = fmaf(x[u][e], x[u][e], sq[u]);
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int u = 0; u < kAnyRows; ++u) sq[u] += __shfl_xor_sync(0xffffffffu, sq[u], o);
#pragma unroll
                for (int u = 0; u < kAnyRows; ++u) {
                    const int h = h0 + u * slices;
                    if (h >= a.H[z]) break;  // the same in all lanes
                    float m;
                    const float inv = far_norm<E>(x[u], live ? sq[u] : 1.f, a.eps, m, LPR);
                    float out[E];
                    if (!BWD) {
#pragma unroll
                        for (int e = 0; e < E; ++e) in[u][e] = x[u][e] * w[e];
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int from = base + (mate[e] & 31);
                        float other = __shfl_sync(0xffffffffu, in[u][0], from);
                        if constexpr (E == 2) {
                            const float hi = __shfl_sync(0xffffffffu, in[u][1], from);
                            other = mate[e] & 32 ? hi : other;
                        }
                        out[e] = fmaf(other, s[e], in[u][e] * c[e]);  // s is 0 past the rotation, other its own entry
                    }
                    if (BWD) {
                        float along = 0.f;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            x[u][e] *= inv;
                            acc[z][e] = fmaf(out[e], x[u][e], acc[z][e]);
                            out[e] *= w[e];
                            along = fmaf(out[e], x[u][e], along);
                        }
#pragma unroll
                        for (int o = LPR / 2; o > 0; o >>= 1) along += __shfl_xor_sync(0xffffffffu, along, o);
                        T* o = static_cast<T*>(a.y[z]) + b * a.ys[z][0] + n * a.ys[z][1] + h * a.ys[z][2] + l;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            out[e] = (out[e] - x[u][e] * along) * inv;
                            if (m != 1.f) out[e] /= m;
                            if (on[e]) o[32 * e] = from_float<T>(out[e]);
                        }
                    } else {
                        T* o = static_cast<T*>(a.y[z]) + dense + h * dense_h;
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (on[e]) o[32 * e] = from_float<T>(out[e] * inv);
                    }
                }
            }
        }
    }
    if (BWD && a.dw) {
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // the warp's tokens first
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) acc[z][e] += __shfl_xor_sync(0xffffffffu, acc[z][e], o);
                if (base == 0) red[warp][z][l + 32 * e] = acc[z][e];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.d; i += 256) {
            const int z = i / a.d, c = i - z * a.d;
            float v = 0.f;
            for (int r = 0; r < 8; ++r) v += red[r][z][c];
            a.dw[(int64_t)blockIdx.x * 2 * a.d + i] = v;
        }
    }
}

template <typename T, bool BWD>
auto qk_any(int d) -> void (*)(QkArgs, int) {
    if (d > 32) return qk_any_kernel<T, 32, 2, BWD>;
    if (d > 16) return qk_any_kernel<T, 32, 1, BWD>;
    if (d > 8) return qk_any_kernel<T, 16, 1, BWD>;
    if (d > 4) return qk_any_kernel<T, 8, 1, BWD>;
    if (d > 2) return qk_any_kernel<T, 4, 1, BWD>;
    return qk_any_kernel<T, 2, 1, BWD>;
}

// A row's piece of VE entries as it lies in memory: 4, 8 or 16 bytes.
template <int W>
struct __align__(4 * W) Piece {
    uint32_t w[W];
};
// Asynchronous copy of one piece into shared memory.
template <int W>
__device__ __forceinline__ void fetch_piece(Piece<W>* dst, const void* src) {
    if constexpr (W == 4)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "n"(4 * W)
                     : "memory");
}
template <int W>
__device__ __forceinline__ void store_piece(void* p, const Piece<W>& r) {
    if constexpr (W == 4) *static_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else if constexpr (W == 2) *static_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    else *static_cast<unsigned int*>(p) = r.w[0];
}
__device__ __forceinline__ float total2(f32x2 v) {
    const float2 f = split2(v);
    return f.x + f.y;
}
__device__ __forceinline__ f32x2 swap2(f32x2 v) {
    const float2 f = split2(v);
    return make2(f.y, f.x);
}

template <typename T, int VE>
__device__ __forceinline__ void unpack(const Piece<VE * (int)sizeof(T) / 4>& r, f32x2 (&x)[VE / 2]) {
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) {
        if constexpr (sizeof(T) == 4) x[e] = make2(__uint_as_float(r.w[2 * e]), __uint_as_float(r.w[2 * e + 1]));
        else x[e] = make2(__uint_as_float(r.w[e] << 16), __uint_as_float(r.w[e] & 0xffff0000u));
    }
}
template <typename T, int VE>
__device__ __forceinline__ Piece<VE * (int)sizeof(T) / 4> pack(const f32x2 (&x)[VE / 2]) {
    Piece<VE * (int)sizeof(T) / 4> r;
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) {
        const float2 f = split2(x[e]);
        if constexpr (sizeof(T) == 4) {
            r.w[2 * e] = __float_as_uint(f.x);
            r.w[2 * e + 1] = __float_as_uint(f.y);
        } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
            r.w[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    return r;
}

// v summed over groups of `lanes` neighbouring lanes, which LPR states where
// it is not 0.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, int lanes) {
    if constexpr (LPR > 0) {
#pragma unroll
        for (int o = LPR >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else {
        for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// Where t = sum x^2 + eps of a row is out of range, scales the row by a power
// of two that takes the larger of its largest entry and sqrt(eps) to [1, 2)
// (exactly, but for entries that are nothing beside it), and eps by its square;
// the returned norm is that of the scaled row.  A row of zeros with eps 0 has
// the norm's inverse 0, one with infinities or NaN is left as it is.  Out of
// line: rows of ordinary size never come here.
template <int W>
struct Rescaled {
    Piece<W> row;
    float inv;
    int by;  // the row was multiplied by 2^-by
};
template <typename T, int VE>
__device__ __noinline__ Rescaled<VE * (int)sizeof(T) / 4> rescale(Piece<VE * (int)sizeof(T) / 4> r, float t, float eps,
                                                                  int lanes) {
    f32x2 x[VE / 2];
    unpack<T, VE>(r, x);
    float big = 0.f;
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) {
        const float2 f = split2(x[e]);
        big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    const float size = fmaxf(big, sqrtf(eps));
    const bool far = out_of_range(t) && t == t && size > 0.f && big < INFINITY;
    const int by = far ? ilogbf(size) : 0;
    float s2 = 0.f;
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) {
        float2 f = split2(x[e]);
        f.x = ldexpf(f.x, -by);
        f.y = ldexpf(f.y, -by);
        s2 += f.x * f.x + f.y * f.y;
        x[e] = make2(f.x, f.y);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    if (far) {
        r = pack<T, VE>(x);
        t = s2 + ldexpf(eps, -2 * by);
    }
    return {r, t == 0.f ? 0.f : rsqrtf(t), by};
}

constexpr int kDepth = 4;  // pieces a thread has in flight: four rows forward, two backward (x and dy)
constexpr int kCtas = 4;   // CTAs an SM holds, forward: 64 registers
constexpr int kBackCtas = 3;

// Rows in pieces of VE entries.  A row is held by `lpr` neighbouring lanes
// (a power of two, one piece each; lanes past the row hold nothing), a CTA
// takes `tok` tokens x `slices` head slices.  The tokens' angles are formed
// once per CTA in shared memory; a thread keeps one token's and one piece's
// cosines and sines (times the weights) in registers and walks its heads,
// q's and then k's.  Its pieces arrive by asynchronous copies into a ring of
// its own in shared memory, so that the bytes in flight cost no registers and
// the first ones travel while the angles are formed.  The other entry of a
// pair is in another lane's piece, exchanged as it was loaded.  Sums over a
// row's lanes go through shuffles, all lanes of a warp together.
//
// Bytes bound the operator (about 10 to 14 operations a value), instructions
// this kernel: at 8 bf16 a lane the 44 B a nanosecond and SM of the memory
// leave some 180 issue slots a row and lane.  Four rows held in registers at
// two CTAs an SM ran 113 us (B4 N8192, 16 + 16 heads of 64, bf16, forward,
// 268 MB); the ring at four CTAs 79 us, 79 % of the issue slots taken; pairs
// in f32x2 instructions, row pointers that step and lane counts known at
// compile time 58 us.  Backward (403 MB), in the same way, 84 us without weights
// and 101 us with; at 4 CTAs an SM it spills (152 us), at 2 it waits (109 us).
// Ring depths of 4 and 8 are within 2 %.  All these are single launches; replayed
// from a graph over two sets of buffers in turn, and with the weights' partial
// sums joined by a launch that starts early, it takes now 54 us forward (5.0
// TB/s), 84 us backward (4.8) and 94 us with weights (4.3); fp32 91, 130 and 133
// us (5.9 to 6.2 TB/s).
template <typename T, int VE, int LPR, bool BWD>
__global__ void __launch_bounds__(256, BWD ? kBackCtas : kCtas)
qk_vec_kernel(const __grid_constant__ QkArgs a, int lpr, int tok, int slices, int tiles) {
    constexpr int W = VE * (int)sizeof(T) / 4, P = VE / 2;
    constexpr int D = BWD ? kDepth / 2 : kDepth;  // rows in flight
    __shared__ Piece<W> ring[kDepth][256];
    __shared__ __align__(16) float cs[2][128 * VE];  // cos, sin: tok * rot / 2 <= 256 / lpr * VE * lpr / 2
    __shared__ __align__(16) float ws[2][kMaxDk];    // weights of q and k, 1 without
    __shared__ __align__(16) float dw[BWD ? 2 : 1][BWD ? 256 : 1][VE];  // this thread's share of the weights' gradients
    if (LPR > 0) lpr = LPR;
    const int tid = threadIdx.x, lane = tid & 31;
    const int half = a.rot >> 1;
    const int c = tid & (lpr - 1), tl = tid / lpr % tok, slice = tid / (lpr * tok);
    const int hc = half / VE;  // pieces of half a rotation
    const bool moved = !a.inter && c < 2 * hc;
    const int mate = (lane & ~(lpr - 1)) + (moved ? (c < hc ? c + hc : c - hc) : c);
    const unsigned tokens = (unsigned)a.B * (unsigned)a.N;
    // rows of a thread in q and in both
    const int rq = (a.H[0] + slices - 1) / slices, rows = rq + (a.H[1] + slices - 1) / slices;
    for (int i = tid; i < 2 * kMaxDk; i += 256) {
        const int z = i / kMaxDk, e = i % kMaxDk;
        ws[z][e] = a.w[z] && e < a.d ? a.w[z][e] : 1.f;
    }
    if (BWD) {
#pragma unroll
        for (int e = 0; e < VE; ++e) dw[0][tid][e] = dw[1][tid][e] = 0.f;
    }
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const unsigned t0 = (unsigned)tile * (unsigned)tok, t = t0 + tl;
        const bool live = t < tokens && c * VE < a.d;
        const int b = live ? t / (unsigned)a.N : 0, n = live ? t - (unsigned)b * (unsigned)a.N : 0;
        const T* xk = static_cast<const T*>(a.x[1]) + b * a.xs[1][0] + n * a.xs[1][1] + slice * a.xs[1][2] + c * VE;
        const T* xr = static_cast<const T*>(a.x[0]) + b * a.xs[0][0] + n * a.xs[0][1] + slice * a.xs[0][2] + c * VE;
        int64_t xstep = slices * a.xs[0][2];
        // rows of the dense head-major tensors: dy, or the output
        const int64_t dense = (int64_t)a.N * a.d, gstep = slices * dense;
        const int64_t at[2] = {((int64_t)b * a.H[0] + slice) * dense + (int64_t)n * a.d + c * VE,
                               ((int64_t)b * a.H[1] + slice) * dense + (int64_t)n * a.d + c * VE};
        const T* gr = BWD ? static_cast<const T*>(a.dy[0]) + at[0] : nullptr;
        int fr = 0, fh = slice, fH = a.H[0];  // the next row to fetch, its head
        if (rq == 0) xr = xk, xstep = slices * a.xs[1][2], fH = a.H[1], gr = static_cast<const T*>(a.dy[1]) + at[1];
        auto fetch = [&]() {
            if (fr < rows) {
                if (live && fh < fH) {
                    fetch_piece<W>(&ring[fr % D][tid], xr);
                    if (BWD) fetch_piece<W>(&ring[D + fr % D][tid], gr);
                }
                ++fr;
                fh += slices;
                xr += xstep;
                if (BWD) gr += gstep;
                if (fr == rq) {
                    xr = xk, xstep = slices * a.xs[1][2];
                    fh = slice, fH = a.H[1];
                    if (BWD) gr = static_cast<const T*>(a.dy[1]) + at[1];
                }
            }
            ptx::cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < D; ++i) fetch();
        if (half > 0) {
            int hp = 1;  // lanes of one token's frequencies
            while (hp < half) hp *= 2;
            const int j = tid & (hp - 1);
            const unsigned n0 = t0 % (unsigned)a.N;
            for (int ti = tid / hp; ti < tok; ti += 256 / hp) {
                const unsigned ta = t0 + ti, na = n0 + ti;
                if (j < half) {
                    // tokens past the last one: rows of zeros, whose sums an angle that is not a number would spoil
                    float2 v = make_float2(1.f, 0.f);
                    if (ta < tokens) v = cos_sin(a, a.pos ? a.pos[ta] : a.pos0 + (na < a.N ? na : na % (unsigned)a.N), j);
                    cs[0][ti * half + j] = v.x;
                    cs[1][ti * half + j] = v.y;
                }
            }
        }
        __syncthreads();
        int r = 0;
#pragma unroll 1
        for (int z = 0; z < 2; ++z) {
            f32x2 C[P], S[P], acc[P] = {};
            const f32x2* wc = reinterpret_cast<const f32x2*>(&ws[z][c * VE]);
            if (!a.inter) {
                // the pair's frequencies and the partner's weights lie as the entries do
                const int m = moved ? (c < hc ? c + hc : c - hc) : c;
                const int j = tl * half + (moved ? (c < hc ? c : c - hc) * VE : 0);
                const f32x2* wm = reinterpret_cast<const f32x2*>(&ws[z][m * VE]);
                const float sign = (c < hc) != BWD ? -1.f : 1.f;
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    C[e] = moved ? reinterpret_cast<const f32x2*>(&cs[0][j])[e] : make2(1.f, 1.f);
                    S[e] = moved ? mul2(reinterpret_cast<const f32x2*>(&cs[1][j])[e], make2(sign, sign)) : 0;
                    if (!BWD) C[e] = mul2(C[e], wc[e]), S[e] = mul2(S[e], wm[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const int i = c * VE + 2 * e;
                    const bool in = i < a.rot;
                    const float co = in ? cs[0][tl * half + i / 2] : 1.f, si = in ? cs[1][tl * half + i / 2] : 0.f;
                    C[e] = make2(co, co);
                    S[e] = BWD ? make2(si, -si) : make2(-si, si);
                    if (!BWD) C[e] = mul2(C[e], wc[e]), S[e] = mul2(S[e], swap2(wc[e]));
                }
            }
            T* y = BWD ? static_cast<T*>(a.y[z]) + b * a.ys[z][0] + n * a.ys[z][1] + slice * a.ys[z][2] + c * VE
                       : static_cast<T*>(a.y[z]) + at[z];
            const int64_t ystep = BWD ? slices * a.ys[z][2] : gstep;
            const int end = z ? rows : rq, heads = a.H[z];
#pragma unroll 1
            for (int h = slice; r < end; ++r, h += slices, y += ystep) {
                const bool on = live && h < heads;
                ptx::cp_async_wait<D - 1>();
                Piece<W> px = {}, pg = {};
                if (on) {
                    px = ring[r % D][tid];
                    if (BWD) pg = ring[D + r % D][tid];
                }
                fetch();
                f32x2 x[P];
                unpack<T, VE>(px, x);
                f32x2 sq = mul2(x[0], x[0]);
#pragma unroll
                for (int e = 1; e < P; ++e) sq = fma2(x[e], x[e], sq);
                const float norm2 = row_sum<LPR>(total2(sq), lpr) + a.eps;
                float inv;
                asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(on ? norm2 : 1.f));
                int by = 0;
                const bool any = __any_sync(0xffffffffu, on && out_of_range(norm2));
                if (any) {
                    const Rescaled<W> q = rescale<T, VE>(px, norm2, a.eps, lpr);
                    if (on) px = q.row, inv = q.inv, by = q.by;
                    unpack<T, VE>(px, x);
                }
                const f32x2 inv2 = make2(inv, inv);
                const Piece<W>& mine = BWD ? pg : px;
                f32x2 in[P], other[P], out[P];
                unpack<T, VE>(mine, in);
                if (a.inter) {
#pragma unroll
                    for (int e = 0; e < P; ++e) other[e] = swap2(in[e]);
                } else {
                    Piece<W> far;
#pragma unroll
                    for (int i = 0; i < W; ++i) far.w[i] = __shfl_sync(0xffffffffu, mine.w[i], mate);
                    unpack<T, VE>(far, other);
                }
                if (BWD) {
                    f32x2 sum = 0;
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        out[e] = fma2(other[e], S[e], mul2(in[e], C[e]));  // du
                        x[e] = mul2(x[e], inv2);                           // xhat
                    }
                    if (a.w[z]) {
#pragma unroll
                        for (int e = 0; e < P; ++e) {
                            acc[e] = fma2(out[e], x[e], acc[e]);
                            out[e] = mul2(out[e], wc[e]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < P; ++e) sum = fma2(out[e], x[e], sum);  // g . xhat
                    const float along = -row_sum<LPR>(total2(sum), lpr);
                    const f32x2 along2 = make2(along, along);
#pragma unroll
                    for (int e = 0; e < P; ++e) out[e] = mul2(fma2(x[e], along2, out[e]), inv2);
                    if (any) {
#pragma unroll
                        for (int e = 0; e < P; ++e) {
                            const float2 f = split2(out[e]);
                            out[e] = make2(ldexpf(f.x, -by), ldexpf(f.y, -by));
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < P; ++e) out[e] = mul2(fma2(other[e], S[e], mul2(in[e], C[e])), inv2);
                }
                if (on) store_piece<W>(y, pack<T, VE>(out));
            }
            if (BWD && a.w[z]) {
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const float2 f = split2(acc[e]);
                    dw[z][tid][2 * e] += f.x;
                    dw[z][tid][2 * e + 1] += f.y;
                }
            }
        }
        __syncthreads();  // cs is free for the next tile
    }
    ptx::pdl_launch_dependents();
    if (BWD && a.dw) {  // the last barrier above stands between the sums and their readers
        for (int i = tid; i < 2 * a.d; i += 256) {
            const int z = i / a.d, e = i - z * a.d;
            float v = 0.f;
            for (int g = e / VE; g < 256; g += lpr) v += dw[z][g][e % VE];
            a.dw[(int64_t)blockIdx.x * 2 * a.d + i] = v;
        }
    }
}

template <typename T, bool BWD>
using QkKernel = void (*)(QkArgs, int, int, int, int);

// 16-byte pieces with the row's lanes known at compile time, narrower ones
// (rows of odd lengths or alignment) with the count at run time.
template <typename T, bool BWD>
QkKernel<T, BWD> qk_vec(int ve, int lpr) {
    constexpr int full = 16 / (int)sizeof(T);
    if (ve == full) {
        switch (lpr) {
            case 1: return qk_vec_kernel<T, full, 1, BWD>;
            case 2: return qk_vec_kernel<T, full, 2, BWD>;
            case 4: return qk_vec_kernel<T, full, 4, BWD>;
            case 8: return qk_vec_kernel<T, full, 8, BWD>;
            default: return qk_vec_kernel<T, full, 64 / full, BWD>;
        }
    }
    if (ve == 4) return qk_vec_kernel<T, 4, 0, BWD>;
    return qk_vec_kernel<T, 2, 0, BWD>;
}

// dw[z][c] = sum of the CTAs' partials, 32 columns a CTA: warp w takes every
// 32nd partial sum from w on, then the warps' sums are joined, in this order.
__global__ void __launch_bounds__(1024)
qk_weight_grad_kernel(const float* __restrict__ part, int parts, int d, float* dqw, float* dkw) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    ptx::pdl_wait_primary();
    float v = 0.f;
    if (col < 2 * d) {
#pragma unroll 8
        for (int i = warp; i < parts; i += 32) v += part[(int64_t)i * 2 * d + col];
    }
    red[warp][lane] = v;
    __syncthreads();
    const int c = blockIdx.x * 32 + warp;
    v = warp_sum(red[lane][warp]);
    if (lane == 0 && c < 2 * d) {
        float* out = c < d ? dqw : dkw;
        if (out) out[c < d ? c : c - d] = v;
    }
}

// Whether the rows can be moved in pieces of VE entries: their length, the
// distance between the two entries of a pair, and every address.
template <typename T, bool BWD>
bool in_pieces(const QkArgs& a, int VE) {
    const size_t bytes = VE * sizeof(T);
    if (a.d % VE != 0 || (!a.inter && (a.rot / 2) % VE != 0)) return false;
    for (int z = 0; z < 2; ++z) {
        if (a.H[z] == 0) continue;
        if (!entry::aligned(a.x[z], bytes) || !entry::aligned(a.y[z], bytes)) return false;
        if (BWD && !entry::aligned(a.dy[z], bytes)) return false;
        for (int i = 0; i < 3; ++i)
            if (a.xs[z][i] % VE != 0 || (BWD && a.ys[z][i] % VE != 0)) return false;
    }
    return true;
}

struct QkPlan {
    int ve, lpr, tok, slices;
    int64_t grid;
};

template <typename T, bool BWD>
QkPlan plan_qk(const QkArgs& a, bool weights) {
    const int sms = entry::num_sms();
    const int64_t tokens = (int64_t)a.B * a.N;
    const int heads = a.H[0] > a.H[1] ? a.H[0] : a.H[1];
    QkPlan p = {};
    for (int ve = 16 / (int)sizeof(T); ve >= 2 && !p.ve; ve /= 2)
        if (in_pieces<T, BWD>(a, ve)) p.ve = ve;
    if (!p.ve) {
        // enough warps to fill the GPU before a warp takes several heads
        p.lpr = 2;
        while (p.lpr < 32 && p.lpr < a.d) p.lpr *= 2;
        const int64_t groups = (tokens + 32 / p.lpr - 1) / (32 / p.lpr);
        p.slices = 1;
        while (p.slices < heads && groups * p.slices < (int64_t)sms * 16) p.slices *= 2;
        if (p.slices > heads) p.slices = heads;
        p.grid = (groups * p.slices + 7) / 8;
        if (p.grid > (int64_t)sms * 8) p.grid = (int64_t)sms * 8;
        return p;
    }
    p.lpr = 1;
    while (p.lpr * p.ve < a.d) p.lpr *= 2;
    // a thread walks all heads of a token where that fills the GPU (the more
    // heads, the less the angles cost: 58 us at one slice, 62 us at two, 73 us
    // at four on 32,768 tokens of 16 + 16 heads), else a slice of them, up to
    // one wave of CTAs
    p.slices = 1;
    while (p.slices * p.lpr < 256 && p.slices < heads && tokens * p.lpr * p.slices * 2 <= (int64_t)sms * kCtas * 256)
        p.slices *= 2;
    p.tok = 256 / (p.lpr * p.slices);
    p.grid = (tokens + p.tok - 1) / p.tok;
    // with weight gradients, as many CTAs as fit at once: fewer partial sums
    // to join
    if (weights && p.grid > (int64_t)sms * kBackCtas) p.grid = (int64_t)sms * kBackCtas;
    return p;
}

template <typename T, bool BWD>
cudaError_t launch_qk(QkArgs& a, float* dqw, float* dkw, cudaStream_t stream) {
    const bool weights = BWD && (dqw || dkw);
    const QkPlan p = plan_qk<T, BWD>(a, weights);
    const unsigned grid = (unsigned)p.grid;
    if (weights) {
        const cudaError_t e = workspace_alloc(reinterpret_cast<void**>(&a.dw), (size_t)grid * 2 * a.d * 4, stream);
        if (e != cudaSuccess) return e;
    }
    if (!p.ve) {
        TA_TIMED(stream, "qk_any_kernel", qk_any<T, BWD>(a.d)<<<grid, 256, 0, stream>>>(a, p.slices));
    } else {
        const int tiles = (int)(((int64_t)a.B * a.N + p.tok - 1) / p.tok);
        const QkKernel<T, BWD> kernel = qk_vec<T, BWD>(p.ve, p.lpr);
        TA_TIMED(stream, "qk_vec_kernel", kernel<<<grid, 256, 0, stream>>>(a, p.lpr, p.tok, p.slices, tiles));
    }
    cudaError_t e = cudaGetLastError();
    if (weights) {
        if (e == cudaSuccess) {
            // its launch overlaps the end of the kernel before
            TA_TIMED(stream, "qk_weight_grad_kernel",
                     e = launch_maybe_pdl(qk_weight_grad_kernel, dim3((2 * a.d + 31) / 32), dim3(1024), 0, stream, true,
                                          static_cast<const float*>(a.dw), (int)grid, a.d, dqw, dkw));
        }
        const cudaError_t f = workspace_free(a.dw, stream);
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
