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

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "entry.h"
#include "feature_table.cuh"
#include "internal.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace ta {

namespace {

constexpr int kMaxSplits = 32;            // shares of the features

struct PrefixArgs {
    const void *q, *k, *v;
    const float* state;       // [H][stride]
    void *kc, *vc;            // [B][H][cap][d], [B][H][cap][dv]
    const int32_t* lengths;   // [B]
    float* out;               // [B][H][dv]
    float* part;              // workspace: the shared part's shares [splits][H][B][dv + 4]
    unsigned int* err;
    int64_t F, stride;
    int B, H, cap, d, dv, n;
    float tau;
};

// ------------------------------------------------------------ the shared part
// Y = (c (.) Phi(Q)) S for one head: a product of [queries x F] by [F x d_v + 1],
// its left side formed feature by feature from q.  A CTA takes MB queries, 64
// columns (and z, the column of ones) and a share of the features, 64 a step;
// the shares' sums go to the workspace and are joined by the kernel below.
//
// Outputs are fp32 and the numerator's terms cancel, so the product has to be
// one of fp32: both sides are split into two tf32 parts, x = hi + lo, and
// hi hi + hi lo + lo hi goes to the tensor cores (m16n8k8), 22 bits a factor,
// fp32 sums.  A warp has 16 queries and every n-th group of eight features; it
// forms its part of Phi in the registers that the instruction reads, each
// feature once.  On FMA units the operands' way through shared memory bound
// it: 4 x 4 outputs a thread took 2.2 to 3 us a step of 32 features.
constexpr int kFeats = 64;    // features a step
constexpr int kCols = 64;     // columns a CTA
constexpr int kPitch = 72;    // floats of a feature's row: the columns, z, zeros; 8 k + n covers the banks
constexpr int kSteps = 3;     // steps of the state in shared memory, two of them on their way

template <typename T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Span {
    T v[N];
};
template <typename T, int N>
__device__ __forceinline__ void to_floats(const Span<T, N>& p, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_float(p.v[i]);
}

// x = hi + lo, hi the upper 11 significant bits (which the tensor cores take
// as they are; of lo they take as many).
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T, int MB, int NF>
__global__ void __launch_bounds__(256, 2)
prefix_state_kernel(const __grid_constant__ PrefixArgs a, int splits, int ctiles, int btiles, int steps) {
    constexpr int MT = MB / 16, KS = 8 / MT, SLICES = kFeats / 8 / KS;  // query tiles; warps of one; slices of a step
    constexpr int NT = kPitch / 8, XP = MB + 8;
    extern __shared__ __align__(16) float dyn[];
    float(*st)[kFeats][kPitch] = reinterpret_cast<float(*)[kFeats][kPitch]>(dyn);  // [kSteps]
    float(*xs)[XP] = reinterpret_cast<float(*)[XP]>(dyn + kSteps * kFeats * kPitch);  // q by entry, row d is 1
    __shared__ uint2 desc[256];  // factors (8 bits each) and weight of four steps' features
    __shared__ float coef[kMaxN];
    ptx::pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int at = blockIdx.x;
    const int split = at % splits;
    at /= splits;
    const int ct = at % ctiles;
    at /= ctiles;
    const int b0 = at % btiles * MB, h = at / btiles;
    const int c0 = ct * kCols, ncol = min(kCols, a.dv - c0), nq = min(MB, a.B - b0);
    const int64_t f0 = (int64_t)split * steps * kFeats;
    const int64_t f1 = min64(a.F, f0 + (int64_t)steps * kFeats);
    const float* S = a.state + (int64_t)h * a.stride;
    const PackedFeat* tab = feat_table(a.d, a.n);

    auto load = [&](int64_t step) {  // 64 features of the state and of z; past f1: zeros
        const int64_t f = f0 + step * kFeats;
        const int buf = (int)(step % kSteps);
        if (f < f1) {
#pragma unroll
            for (int i = tid; i < kFeats * (kCols / 4); i += 256) {
                const int r = i / (kCols / 4), c = i % (kCols / 4) * 4;
                const bool in = f + r < f1 && c < ncol;
                ptx::cp_async16(&st[buf][r][c], in ? S + (f + r) * a.dv + c0 + c : S, in ? 16 : 0);
            }
            if (tid < kFeats) {
                const bool in = f + tid < f1;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(&st[buf][tid][kCols])),
                             "l"(in ? S + a.F * a.dv + f + tid : S), "r"(in ? 4 : 0)
                             : "memory");
            }
        }
        ptx::cp_async_commit();
    };
    for (int i = 0; i < kSteps - 1; ++i) load(i);
    for (int i = tid; i < kSteps * kFeats * (kPitch - kCols - 1); i += 256) {
        const int r = i / (kPitch - kCols - 1), c = kCols + 1 + i % (kPitch - kCols - 1);
        dyn[r * kPitch + c] = 0.f;
    }
    if (tid < a.n) coef[tid] = query_coeff(tid, a.tau);
    if (a.d * sizeof(T) % 16 == 0) {
        constexpr int E = 16 / sizeof(T);
        const int per = a.d / E;
        for (int i = tid; i < MB * per; i += 256) {
            const int m = i % MB, e = i / MB * E;
            Span<T, E> p = {};
            if (m < nq) p = *reinterpret_cast<const Span<T, E>*>(static_cast<const T*>(a.q) + ((int64_t)(b0 + m) * a.H + h) * a.d + e);
#pragma unroll
            for (int j = 0; j < E; ++j) xs[e + j][m] = to_float(p.v[j]);
        }
    } else {
        for (int i = tid; i < MB * a.d; i += 256) {
            const int m = i % MB, e = i / MB;
            xs[e][m] = m < nq ? to_float(static_cast<const T*>(a.q)[((int64_t)(b0 + m) * a.H + h) * a.d + e]) : 0.f;
        }
    }
    for (int m = tid; m < MB; m += 256) xs[a.d][m] = 1.f;
    __syncthreads();
    auto describe = [&](int64_t f) {  // feature f, one a thread
        FeatDesc fd = {};  // weight 0 past the last feature
        if (f < f1) fd = get_desc(tab, a.d, a.n, f, a.tau, coef, true);
        uint32_t packed = 0;  // factors past the degree point at the row of ones
#pragma unroll
        for (int p = 0; p < kMaxN - 1; ++p)
            packed |= (p < fd.m ? (fd.packed >> (8 * p)) & 0xffu : (uint32_t)a.d) << (8 * p);
        desc[tid] = make_uint2(packed, __float_as_uint(fd.w));
    };
    const int g = lane >> 2, t = lane & 3;  // the instruction's row group and column
    const int mt = warp % MT, ks = warp / MT, m0 = mt * 16;
    float acc[NT][4] = {};
    describe(f0 + tid);
    int64_t step = 0;
    for (int64_t f = f0; f < f1; f += kFeats, ++step) {
        const int buf = (int)(step % kSteps), group = (int)(step & 3) * kFeats;
        ptx::cp_async_wait<kSteps - 2>();
        __syncthreads();  // this step's state and descriptors are there, the last step's are free
        load(step + kSteps - 1);
#pragma unroll
        for (int i = 0; i < SLICES; ++i) {
            const int k0 = (i * KS + ks) * 8;
            float v[4];  // queries g, g + 8 by features t, t + 4
            const uint2 d0 = desc[group + k0 + t], d1 = desc[group + k0 + t + 4];
            v[0] = v[1] = __uint_as_float(d0.y);
            v[2] = v[3] = __uint_as_float(d1.y);
#pragma unroll
            for (int e = 0; e < NF; ++e) {
                const float* x0 = xs[(d0.x >> (8 * e)) & 0xffu] + m0 + g;
                const float* x1 = xs[(d1.x >> (8 * e)) & 0xffu] + m0 + g;
                v[0] *= x0[0];
                v[1] *= x0[8];
                v[2] *= x1[0];
                v[3] *= x1[8];
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_tf32(v[e], hi[e], lo[e]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t bh0, bl0, bh1, bl1;
                split_tf32(st[buf][k0 + t][n * 8 + g], bh0, bl0);
                split_tf32(st[buf][k0 + t + 4][n * 8 + g], bh1, bl1);
                mma_tf32(acc[n], lo, bh0, bh1);
                mma_tf32(acc[n], hi, bl0, bl1);
                mma_tf32(acc[n], hi, bh0, bh1);
            }
        }
        if (group == 3 * kFeats && f + kFeats < f1) {
            __syncthreads();  // every warp has read the descriptors
            describe(f + kFeats + tid);
        }
    }
    // the warps of one query tile join in shared memory, where the state was
    ptx::cp_async_wait<0>();
    __syncthreads();
    float(*part)[MB][kPitch] = reinterpret_cast<float(*)[MB][kPitch]>(dyn);  // [KS]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float2*>(&part[ks][m0 + g][n * 8 + 2 * t]) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2*>(&part[ks][m0 + g + 8][n * 8 + 2 * t]) = make_float2(acc[n][2], acc[n][3]);
    }
    __syncthreads();
    const int pitch = a.dv + 4;
    float* Y = a.part + (((int64_t)split * a.H + h) * a.B + b0) * pitch;
    for (int i = tid; i < nq * (kCols / 4 + 1); i += 256) {
        const int m = i / (kCols / 4 + 1), c = i % (kCols / 4 + 1) * 4;
        float4 v = *reinterpret_cast<const float4*>(&part[0][m][c]);
#pragma unroll
        for (int k = 1; k < KS; ++k) {
            const float4 w = *reinterpret_cast<const float4*>(&part[k][m][c]);
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        if (c < ncol) *reinterpret_cast<float4*>(Y + (int64_t)m * pitch + c0 + c) = v;
        else if (c == kCols && ct == 0) Y[(int64_t)m * pitch + a.dv] = v.x;
    }
}

// ------------------------------------------------------------ the own tokens
// One cluster of CTAs per sequence and head (one CTA but for long suffixes of
// few heads).  Eight lanes take a token: each multiplies its share of q and k,
// three shuffles make the score, and with the weight K(tau q.k) each adds its
// share of v.  Rows are read once, in pieces of up to 16 bytes, by asynchronous
// copies into slots that one lane alone reads, several steps ahead.  The sums
// of the lanes, warps and CTAs and the shared part's shares are joined in an
// order that depends on the sizes alone.
//
// The cache's bytes bound it: 64 sequences of 16 heads, d 64 and 64, up to
// 1,024 own tokens (144 MB) take 40 us on the device with the shared part beside
// them, 3.6 TB/s; tokens in registers 68 us, with selects on every token 55 us.  What is
// left is the start and end of each CTA (2 to 4 us of some 15).
constexpr int kUnroll = 2;  // tokens of eight lanes in a step

// Bytes of a token that one lane keeps in shared memory, and the steps that
// fit into 256 bytes a thread (two at least; three at most, so that seven CTAs
// of four warps stay on an SM where a lane keeps 32 bytes or less).
template <typename T, int KV, int VV, int J>
constexpr int kLaneBytes = (KV + J * VV) * (int)sizeof(T);
template <typename T, int KV, int VV, int J>
constexpr int ahead() {
    constexpr int fit = 256 / (kUnroll * kLaneBytes<T, KV, VV, J>);
    return fit < 2 ? 2 : fit > 3 ? 3 : fit;
}

// CTAs of NW warps that the compiler is to leave registers for on an SM: seven
// of four warps or three of eight, one where a lane's 32 columns and more need
// them, and no more than fit into 228 KB with their rings, sums (below) and the
// 1 KB that each CTA costs.  fp32, d_v 128 lets four or five CTAs of four warps
// in; held to seven's 72 registers it took 22.6 us (64 sequences of 16 heads, d
// 20, up to 200 tokens) and 23.8 us (d 64), with 86 and 96 registers 21.6 and
// 23.5 us.
template <typename T, int KV, int VV, int J, int NW>
constexpr int resident() {
    constexpr int sums = (NW * (kMaxDv + 4) + kMaxDv + 1) * (int)sizeof(float);
    constexpr int ring = 32 * NW * kUnroll * ahead<T, KV, VV, J>() * kLaneBytes<T, KV, VV, J>;
    constexpr int fit = 228 * 1024 / (ring + sums + 1024), want = J * VV > 16 ? 1 : NW == 4 ? 7 : 3;
    return fit < want ? fit : want;
}

template <typename T, int N>
__device__ __forceinline__ void to_pairs(const Span<T, N>& p, f32x2 (&x)[N / 2]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) x[i] = make2(p.v[2 * i], p.v[2 * i + 1]);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) x[i] = make2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}
template <int BYTES>
__device__ __forceinline__ void fetch_async(void* dst, const void* src) {
    if constexpr (BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < BYTES; i += 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(static_cast<char*>(dst) + i)),
                         "l"(static_cast<const char*>(src) + i)
                         : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "n"(BYTES)
                     : "memory");
    }
}

__device__ __forceinline__ float load_remote(const float* mine, int rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// KV: entries of k a lane reads at once (0: one by one, any d_k); VV: columns
// of v it reads at once, J times.
template <typename T, int KV, int VV, int J, int NW>
__global__ void __launch_bounds__(32 * NW, resident<T, KV, VV, J, NW>())
prefix_own_kernel(const __grid_constant__ PrefixArgs a, int splits, int cluster) {
    constexpr int KE = KV ? KV : kMaxDk / 8, THREADS = 32 * NW, TOKENS = 4 * NW * kUnroll;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __align__(16) float red[NW][kMaxDv + 4];
    __shared__ float tot[kMaxDv + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & 7, grp = lane >> 3;
    const int rank = blockIdx.x % cluster, bh = blockIdx.x / cluster, b = bh / a.H, h = bh - b * a.H;
    const T* k = static_cast<const T*>(a.k) + (int64_t)bh * a.d;
    const T* v = static_cast<const T*>(a.v) + (int64_t)bh * a.dv;
    T* kc = static_cast<T*>(a.kc) + (int64_t)bh * a.cap * a.d;
    T* vc = static_cast<T*>(a.vc) + (int64_t)bh * a.cap * a.dv;
    const int L = a.lengths[b];
    if (L < 0 || L >= a.cap) {  // the same in every CTA of the cluster
        ptx::pdl_wait_primary();
        if (rank == 0)
            for (int c = tid; c < a.dv; c += THREADS) a.out[(int64_t)bh * a.dv + c] = nanf("");
        if (rank == 0 && tid == 0) atomicOr(a.err, kErrPrefixLength);
        return;
    }
    f32x2 q[KE / 2];
    {
        float qf[KE];
        if constexpr (KV > 0) {
            const Span<T, KV> p = *reinterpret_cast<const Span<T, KV>*>(static_cast<const T*>(a.q) + (int64_t)bh * a.d + sub * KV);
            to_floats<T, KV>(p, qf);
        } else {
#pragma unroll
            for (int e = 0; e < KE; ++e)
                qf[e] = sub + 8 * e < a.d ? to_float(static_cast<const T*>(a.q)[(int64_t)bh * a.d + sub + 8 * e]) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < KE / 2; ++e) q[e] = make2(qf[2 * e], qf[2 * e + 1]);
    }
    // the series' coefficients tau^m / m!, 0 from degree n on
    float c1 = a.n > 1 ? query_coeff(1, a.tau) : 0.f, c2 = a.n > 2 ? query_coeff(2, a.tau) : 0.f;
    float c3 = a.n > 3 ? query_coeff(3, a.tau) : 0.f, c4 = a.n > 4 ? query_coeff(4, a.tau) : 0.f;

    f32x2 y[J][VV / 2] = {};
    float z = 0.f;
    // tokens ahead, each lane's share in slots that it alone reads
    constexpr int A = ahead<T, KV, VV, J>();
    Span<T, VV>* vring = reinterpret_cast<Span<T, VV>*>(ring);                                  // [A][kUnroll][J][THREADS]
    Span<T, KE>* kring = reinterpret_cast<Span<T, KE>*>(vring + A * kUnroll * J * THREADS);         // [A][kUnroll][THREADS]
    const int stride = cluster * TOKENS, mine = warp * 4 + grp, start = rank * TOKENS;
    // rows of the next step to fetch
    const T* kp = kc + (int64_t)(start + mine) * a.d + sub * KV;
    const T* vp = vc + (int64_t)(start + mine) * a.dv + sub * VV;
    int jf = start;
    const int64_t kstep = (int64_t)stride * a.d, vstep = (int64_t)stride * a.dv;
    const int ku = 4 * NW * a.d, vu = 4 * NW * a.dv;
    const bool wide = J * 8 * VV == a.dv;  // every lane's columns exist
    auto fetch = [&](int slot) {
        Span<T, KE>* kt = &kring[slot * kUnroll * THREADS + tid];
        Span<T, VV>* vt = &vring[slot * kUnroll * J * THREADS + tid];
        if (jf + TOKENS <= L && wide) {  // a whole step of cached tokens
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if constexpr (KV > 0) fetch_async<KV * sizeof(T)>(kt + u * THREADS, kp + u * ku);
#pragma unroll
                for (int i = 0; i < J; ++i) fetch_async<VV * sizeof(T)>(vt + (u * J + i) * THREADS, vp + u * vu + i * 8 * VV);
            }
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int j = jf + u * 4 * NW + mine;
                if (j <= L) {  // the new token comes from k and v
                    if constexpr (KV > 0) fetch_async<KV * sizeof(T)>(kt + u * THREADS, j < L ? kp + u * ku : k + sub * KV);
#pragma unroll
                    for (int i = 0; i < J; ++i) {
                        const int c = (i * 8 + sub) * VV;
                        if (c < a.dv)
                            fetch_async<VV * sizeof(T)>(vt + (u * J + i) * THREADS, j < L ? vp + u * vu + i * 8 * VV : v + c);
                    }
                }
            }
        }
        ptx::cp_async_commit();
        jf += stride;
        kp += kstep;
        vp += vstep;
    };
    auto consume = [&](auto whole, int j0, int slot) {
        Span<T, KE> kr[kUnroll];
        Span<T, VV> vr[kUnroll][J];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int j = j0 + u * 4 * NW + mine;
            const bool in = whole || j <= L;
            kr[u] = {};
            if constexpr (KV > 0) {
                if (in) kr[u] = kring[(slot * kUnroll + u) * THREADS + tid];
            } else {
                const T* krow = j < L ? kc + (int64_t)j * a.d : k;
#pragma unroll
                for (int e = 0; e < KE; ++e)
                    if (in && sub + 8 * e < a.d) kr[u].v[e] = krow[sub + 8 * e];
            }
#pragma unroll
            for (int i = 0; i < J; ++i) {
                vr[u][i] = {};
                if (whole || (in && (i * 8 + sub) * VV < a.dv)) vr[u][i] = vring[((slot * kUnroll + u) * J + i) * THREADS + tid];
            }
        }
        float x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            f32x2 kf[KE / 2], dot;
            to_pairs<T, KE>(kr[u], kf);
            dot = mul2(q[0], kf[0]);
#pragma unroll
            for (int e = 1; e < KE / 2; ++e) dot = fma2(q[e], kf[e], dot);
            const float2 f = split2(dot);
            x[u] = f.x + f.y;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) x[u] += __shfl_xor_sync(0xffffffffu, x[u], o);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float w = fmaf(x[u], fmaf(x[u], fmaf(x[u], fmaf(x[u], c4, c3), c2), c1), 1.f);
            if (!whole && j0 + u * 4 * NW + mine > L) w = 0.f;
            z += w;
            const f32x2 ww = make2(w, w);
#pragma unroll
            for (int i = 0; i < J; ++i) {
                f32x2 vf[VV / 2];
                to_pairs<T, VV>(vr[u][i], vf);
#pragma unroll
                for (int e = 0; e < VV / 2; ++e) y[i][e] = fma2(ww, vf[e], y[i][e]);
            }
        }
    };
#pragma unroll 1
    for (int i = 0; i < A - 1; ++i) fetch(i);
    if (rank == 0) {  // append the new token, whose row of the cache nobody reads here
        for (int c = tid; c < a.dv; c += THREADS) vc[(int64_t)L * a.dv + c] = v[c];
        if (tid < a.d) kc[(int64_t)L * a.d + tid] = k[tid];
    }
    int slot = 0;
#pragma unroll 1
    for (int j0 = start; j0 <= L; j0 += stride) {
        fetch(slot == 0 ? A - 1 : slot - 1);
        ptx::cp_async_wait<A - 1>();
        if (j0 + TOKENS <= L && wide) consume(std::true_type{}, j0, slot);
        else consume(std::false_type{}, j0, slot);
        if (++slot == A) slot = 0;
    }
    // the warp's four token groups
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
        for (int i = 0; i < J; ++i)
#pragma unroll
            for (int e = 0; e < VV / 2; ++e) {
                float2 f = split2(y[i][e]);
                f.x += __shfl_xor_sync(0xffffffffu, f.x, o);
                f.y += __shfl_xor_sync(0xffffffffu, f.y, o);
                y[i][e] = make2(f.x, f.y);
            }
    }
    if (grp == 0) {
#pragma unroll
        for (int i = 0; i < J; ++i)
#pragma unroll
            for (int e = 0; e < VV / 2; ++e) {
                const int c = (i * 8 + sub) * VV + 2 * e;
                if (c < a.dv) *reinterpret_cast<float2*>(&red[warp][c]) = split2(y[i][e]);
            }
        if (sub == 0) red[warp][a.dv] = z;
    }
    __syncwarp();
    if (rank == 0) {  // the shared part's shares, warp by warp
        ptx::pdl_wait_primary();
        const int pitch = a.dv + 4;
        const int64_t heads = (int64_t)a.B * a.H;
        for (int c = lane * 4; c <= a.dv; c += 128) {
            float4 s = *reinterpret_cast<float4*>(&red[warp][c]);
            const float* from = a.part + ((int64_t)h * a.B + b) * pitch + c;
            const int64_t share = heads * pitch;
            for (int i0 = warp; i0 < splits; i0 += 4 * NW) {  // four loads in flight
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[i] = i0 + i * NW < splits ? __ldcg(reinterpret_cast<const float4*>(from + (i0 + i * NW) * share))
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) s.x += p[i].x, s.y += p[i].y, s.z += p[i].z, s.w += p[i].w;
            }
            *reinterpret_cast<float4*>(&red[warp][c]) = s;
        }
    }
    __syncthreads();
    for (int c = tid; c <= a.dv; c += THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += red[w][c];
        tot[c] = s;
    }
    if (cluster > 1) {
        cluster_barrier();
        if (rank == 0)
            for (int c = tid; c <= a.dv; c += THREADS) {
                float s = tot[c];
                for (int i = 1; i < cluster; ++i) s += load_remote(&tot[c], i);
                tot[c] = s;
            }
        cluster_barrier();  // the others' sums are read before they leave
    }
    __syncthreads();
    if (rank == 0) {
        for (int c = tid; c < a.dv; c += THREADS) a.out[(int64_t)bh * a.dv + c] = tot[c] / tot[a.dv];
    }
}

struct OwnKernel {
    void (*run)(PrefixArgs, int, int);
    int smem;
    std::atomic<uint64_t>* done;
};
template <typename T, int KV, int VV, int J, int NW>
OwnKernel own_of() {
    static std::atomic<uint64_t> done{0};
    return {prefix_own_kernel<T, KV, VV, J, NW>, 32 * NW * kUnroll * ahead<T, KV, VV, J>() * kLaneBytes<T, KV, VV, J>,
            &done};
}
template <typename T, int KV, int NW, int VV>
OwnKernel own_kernel_j(int dv) {
    const int j = (dv + 8 * VV - 1) / (8 * VV);
    if (j <= 1) return own_of<T, KV, VV, 1, NW>();
    if (j <= 2) return own_of<T, KV, VV, 2, NW>();
    if constexpr (VV == 4)
        if (j > 4) return own_of<T, KV, 4, 8, NW>();
    return own_of<T, KV, VV, 4, NW>();
}
template <typename T, int KV, int NW>
OwnKernel own_kernel_v(int dv) {
    // 16-byte pieces of v where its rows hold whole ones for all lanes
    if constexpr (sizeof(T) == 2)
        if (dv % 64 == 0) return own_kernel_j<T, KV, NW, 8>(dv);
    return own_kernel_j<T, KV, NW, 4>(dv);
}
template <typename T, int NW>
OwnKernel own_kernel(int d, int dv) {
    if (d == 64) return own_kernel_v<T, 8, NW>(dv);
    if (d == 32) return own_kernel_v<T, 4, NW>(dv);
    if (d == 16) return own_kernel_v<T, 2, NW>(dv);
    return own_kernel_v<T, 0, NW>(dv);
}

struct StateKernel {
    void (*run)(PrefixArgs, int, int, int, int);
    std::atomic<uint64_t>* done;
};
template <typename T, int MB, int NF>
StateKernel state_of() {
    static std::atomic<uint64_t> done{0};
    return {prefix_state_kernel<T, MB, NF>, &done};
}
template <typename T, int MB>
StateKernel state_kernel_n(int n) {
    switch (n) {
        case 1: return state_of<T, MB, 0>();
        case 2: return state_of<T, MB, 1>();
        case 3: return state_of<T, MB, 2>();
        case 4: return state_of<T, MB, 3>();
        default: return state_of<T, MB, 4>();
    }
}
template <typename T>
StateKernel state_kernel(int MB, int n) {
    return MB == 16 ? state_kernel_n<T, 16>(n) : MB == 32 ? state_kernel_n<T, 32>(n) : state_kernel_n<T, 64>(n);
}
constexpr int state_smem(int MB, int d) { return (kSteps * kFeats * kPitch + (d + 1) * (MB + 8)) * (int)sizeof(float); }

template <typename T>
cudaError_t launch_prefix(PrefixArgs& a, cudaStream_t stream) {
    const int sms = entry::num_sms();
    // the shared part: a CTA an SM, a share of at least 64 features each (twice
    // as many gain nothing: their sums have to be joined)
    const int MB = a.B <= 16 ? 16 : a.B <= 32 ? 32 : 64;
    const int btiles = (a.B + MB - 1) / MB, ctiles = (a.dv + kCols - 1) / kCols;
    const int64_t tiles = (int64_t)a.H * btiles * ctiles, all = (a.F + kFeats - 1) / kFeats;
    int64_t splits = sms / tiles;
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (splits > all) splits = all;
    if (splits < 1) splits = 1;
    const int64_t steps = (all + splits - 1) / splits;
    splits = (all + steps - 1) / steps;
    // the own tokens: four warps a sequence and head where there are many and
    // none is long (more CTAs stay in flight while some begin and others end:
    // 1,024 heads of up to 512 tokens, d 16, 17.0 us, at eight warps 19; 4,096 of
    // up to 512, d 64, 90 and 99 us), else eight (a long one would still run
    // when the others are done: 1,024 of up to 1,024, d 64, 44 and 39 us), and
    // while that leaves each 256 tokens a cluster of CTAs.  The lengths lie on the
    // device, so the capacity stands for the longest: a cache of four times that
    // costs up to a quarter (1,024 heads of up to 512, d 16, 17.3 and 19.2 us;
    // 4,096 of up to 256, d 64, 65 and 81 us; 136 of up to 300, n 5 in fp32, 15.3
    // and 18.2 us)
    const int64_t heads = (int64_t)a.B * a.H;
    const bool many = heads >= 2 * (int64_t)sms && (int64_t)a.cap * (a.d + a.dv) * (int64_t)sizeof(T) <= 192 * 1024;
    int64_t cluster = (int64_t)sms * 4 / heads, room = ((int64_t)a.cap + 255) / 256;
    if (cluster > room) cluster = room;
    if (cluster > 8) cluster = 8;
    if (cluster < 1 || many) cluster = 1;

    const size_t bytes = (size_t)splits * heads * (a.dv + 4) * sizeof(float);
    cudaError_t e = workspace_alloc(reinterpret_cast<void**>(&a.part), bytes, stream);
    if (e != cudaSuccess) return e;
    const StateKernel state = state_kernel<T>(MB, a.n);
    const OwnKernel own = many ? own_kernel<T, 4>(a.d, a.dv) : own_kernel<T, 8>(a.d, a.dv);
    if ((e = entry::allow_smem(state.run, state_smem(MB, kMaxDk), *state.done)) != cudaSuccess ||
        (e = entry::allow_smem(own.run, own.smem, *own.done)) != cudaSuccess) {
        workspace_free(a.part, stream);
        return e;
    }
    TA_TIMED(stream, "prefix_state_kernel",
             state.run<<<(unsigned)(tiles * splits), 256, state_smem(MB, a.d), stream>>>(a, (int)splits, ctiles, btiles,
                                                                                         (int)steps));
    e = cudaGetLastError();
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(heads * cluster));
        cfg.blockDim = dim3(many ? 128 : 256);
        cfg.dynamicSmemBytes = own.smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 1 ? 2 : 1;
        TA_TIMED(stream, "prefix_own_kernel",
                 e = cudaLaunchKernelEx(&cfg, own.run, a, (int)splits, (int)cluster));
    }
    const cudaError_t f = workspace_free(a.part, stream);
    return e == cudaSuccess ? f : e;
}

template <typename T>
int prefix_entry(const T* q, const T* k, const T* v, const float* state, T* kc, T* vc, const int32_t* lengths,
                 float* out, int B, int H, int cap, int d, int dv, int n, float tau, cudaStream_t stream) {
    if (B < 0 || H < 0 || cap < 0 || d < 0 || dv < 0 || n < 0 || !isfinite(tau)) return TAYLOR_ERR_INVALID_ARG;
    if (n < 1 || n > kMaxN || d < 1 || d > kMaxDk || dv < 4 || dv > kMaxDv || dv % 4 != 0) return TAYLOR_ERR_UNSUPPORTED;
    if ((int64_t)B * H >= ((int64_t)1 << 24) || cap > (1 << 30)) return TAYLOR_ERR_UNSUPPORTED;
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
