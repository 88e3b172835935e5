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
//
// The gradient takes h_{t-1} as it is stored, so beside bf16 tensors dgate
// carries half a step of h next to its own rounding (dx and dh0 do not depend
// on h).  Norm of dgate's error against 64 bits, B2 N4096 D1024 bf16: coupled
// 1.75e-3, not coupled 2.34e-3, from fp32 states 1.66e-3 both.  Those would
// have to be stored beside h, twice its bytes written and read again, or formed
// by a second forward pass, 50 us more on the 87 us of B4 N8192 D1024.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "entry.h"
#include "internal.h"
#include "pairs.cuh"
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

// a = sigmoid(g) and 1 - a.  The exponential is capped so that e a is finite:
// a gate of -inf leaves a < 2^-125 of the state and 1 - a = 1.  NaN stays NaN.
// Beside bf16 gates and outputs the hardware's approximate exponential and
// reciprocal (2 and 1 steps off) do; with fp32 tensors a memory of hundreds of
// tokens would show their errors, so exponential and division are full ones.
// The fp32 states beside bf16 tensors carry the approximate ones: the last state
// of B2 N4096 D1024 is off by 1.6e-7 of its norm coupled and 6.0e-7 not, 1.3e-7
// and 3.6e-7 with full ones.
template <typename T>
__device__ __forceinline__ void gates(float g, float& a, float& keep) {
    float e;
    if constexpr (sizeof(T) == 2) {
        float t = g * -1.4426950408889634f;
        asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(t));  // 126
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(1.0f + e));
    } else {
        float t = -g;
        asm("min.NaN.f32 %0, %0, 0f42AE0000;" : "+f"(t));  // 87
        e = expf(t);
        a = __frcp_rn(1.0f + e);
    }
    keep = e * a;
}

template <typename T>
__device__ __forceinline__ void gates(f32x2 g, f32x2& a, f32x2& keep) {
    if constexpr (sizeof(T) == 2) {
        float2 t = split2(mul2(g, make2(-1.4426950408889634f, -1.4426950408889634f))), e;
        asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(t.x));
        asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(t.y));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
        const f32x2 e2 = make2(e.x, e.y);
        t = split2(add2(e2, make2(1.0f, 1.0f)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
        a = make2(e.x, e.y);
        keep = mul2(e2, a);
    } else {
        const float2 x = split2(g);
        float2 al, kp;
        gates<T>(x.x, al.x, kp.x);
        gates<T>(x.y, al.y, kp.y);
        a = make2(al.x, al.y);
        keep = make2(kp.x, kp.y);
    }
}

template <typename T>
__device__ __forceinline__ T round_to(float x);
template <>
__device__ __forceinline__ float round_to<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// The scan.  A CTA takes 32 channels and a chunk of tokens, a cluster of CTAs
// neighbouring chunks; it walks the sequence (backwards for the gradient) in
// strides of a cluster's chunks.  Over tokens in walking order both directions
// are c <- A c + b: forward A = a, b = s x, c = h; backward A = a, b = a dh,
// c = a G.  A thread holds V channels of R neighbouring tokens in registers
// and
//   1. forms (prod A, the end from c = 0) of its tokens,
//   2. joins it with its warp's other token groups by shuffles, with the other
//      warps through shared memory, with the cluster's other CTAs through
//      theirs: each CTA sends its total to all of them by stores that count
//      their bytes on the receiver's barrier, so no fence waits for outputs,
//   3. folds what precedes it into the carried state, in an order that depends
//      on the sizes alone, and walks its tokens again to write the outputs.
// So each input is read and each output written once, whatever the length.
// The tokens arrive by asynchronous copies, two chunks deep, each thread's
// into slots that it alone reads; only pieces under 4 bytes (single bf16
// channels, where width or alignment is odd) are loaded into registers, a round
// ahead.
//
// Memory bounds the operator, 6 B a value forward and 12 B backward in bf16;
// this kernel is bound by instructions and the latency of its rounds: 25 and
// 49 instructions a value, issue slots 58 to 61 % taken at 14 warps an SM.
// B4 N8192 D1024 bf16: 50 us forward (4.0 TB/s), 87 us backward (4.6 TB/s),
// replayed from a graph over two sets of buffers in turn (fp32 93 and 149 us).
// As single launches 52 and 91 us; with checks on every token, scalar
// arithmetic and a cluster barrier a round 73 and 126 us; one thread a channel
// 9.8 ms for both.  A third stage in flight, or 16-byte copies shared by two
// lanes, gain nothing.
//
// The CTAs of a cluster run at the same time, and each sends before it waits.
// The totals' buffers alternate: a CTA sends those of round i + 2 only after it
// has those of round i + 1, which every CTA sends after a CTA barrier behind
// its reads of round i.  A CTA whose wait ran out (never in a sound run) takes
// no further part in the exchange, sets the error word and walks on without
// waiting; it stays until the others are through, since they may still send
// to it.
constexpr int kTile = 32;     // channels of a CTA
constexpr int kStages = 2;
constexpr int kMaxCluster = 8;  // portable; 16 gain a tenth on few tiles and cost as much on many
constexpr uint32_t kWait = 1u << 24;  // polls of a cluster's totals

template <typename T, int V>
struct alignas(V * sizeof(T)) Chans {
    T v[V];
};

// V channels in arithmetic: pairs, or one value.
template <int V>
struct Lanes {
    f32x2 e[V / 2];
};
template <>
struct Lanes<1> {
    float e[1];
};
template <int V>
constexpr int kPairs = V == 1 ? 1 : V / 2;

__device__ __forceinline__ void spread(float v, float& out) { out = v; }
__device__ __forceinline__ void spread(float v, f32x2& out) { out = make2(v, v); }

template <int V>
__device__ __forceinline__ Lanes<V> lanes_of(float v) {
    Lanes<V> r;
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) spread(v, r.e[i]);
    return r;
}
template <int V>
__device__ __forceinline__ void unpack(const Chans<float, V>& p, Lanes<V>& r) {
    if constexpr (V == 1) {
        r.e[0] = p.v[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.e[i] = make2(p.v[2 * i], p.v[2 * i + 1]);
    }
}
template <int V>
__device__ __forceinline__ void unpack(const Chans<__nv_bfloat16, V>& p, Lanes<V>& r) {
    if constexpr (V == 1) {
        r.e[0] = __bfloat162float(p.v[0]);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.e[i] = make2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}
template <int V>
__device__ __forceinline__ void values(const Lanes<V>& r, float (&x)[V]) {
    if constexpr (V == 1) {
        x[0] = r.e[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 f = split2(r.e[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}
template <int V>
__device__ __forceinline__ Lanes<V> lanes_of(const float (&x)[V]) {
    Lanes<V> r;
    if constexpr (V == 1) {
        r.e[0] = x[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.e[i] = make2(x[2 * i], x[2 * i + 1]);
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ Chans<T, V> pack(const Lanes<V>& r) {
    float x[V];
    values<V>(r, x);
    Chans<T, V> p;
    if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) *reinterpret_cast<__nv_bfloat162*>(&p.v[i]) = __floats2bfloat162_rn(x[i], x[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p.v[i] = round_to<T>(x[i]);
    }
    return p;
}

template <int BYTES>
__device__ __forceinline__ void fetch_async(void* dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "n"(BYTES)
                     : "memory");
}

// Stores to the same shared-memory address of CTA `rank` of the cluster and
// counts the bytes on that CTA's barrier.
__device__ __forceinline__ void send(float2* mine, uint64_t* bar, int rank, float2 v) {
    uint32_t at, to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(mine)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(ptx::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
                 "f"(v.x), "f"(v.y), "r"(to)
                 : "memory");
}

// Waits for the totals of one parity.  The stores that complete the barrier
// come from other CTAs and release at the cluster's scope, which is where they
// have to be acquired.
__device__ __forceinline__ bool totals_here(uint64_t* bar, uint32_t phase) {
    for (uint32_t i = 0; i < kWait; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n"
            "  .reg .pred p;\n"
            "  mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            "  selp.u32 %0, 1, 0, p;\n"
            "}\n"
            : "=r"(ok)
            : "r"(ptx::smem_u32(bar)), "r"(phase)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// Elements (tokens x channels) of a thread and chunk: 128 bytes of tokens a
// thread and stage, which sixteen warps of 128 registers a thread hold on an
// SM.  Half as many, at twenty-four warps, cost a fifth more time: what a round
// costs whatever its length (the joins, the wait for the cluster) counts twice
// as often.  Single bf16 channels hold half as many, and the next round's
// beside them (B4 N8192 D1023: 79 and 178 us; loaded in the round itself 127
// and 277).
template <typename T, int V, bool BWD>
constexpr int elements() {
    return 32 / (int)sizeof(T) / (BWD ? 2 : 1) * (V * sizeof(T) < 4 ? 1 : 2);
}
constexpr int kSmWarps = 16;  // warps an SM holds

template <typename T, int V, bool BWD, int W>
__global__ void __launch_bounds__(32 * W, kSmWarps / W)
scan_kernel(const __grid_constant__ ScanArgs a, int tiles, int cluster, int rounds, unsigned int* err) {
    constexpr int LC = kTile / V, GROUPS = 32 / LC;   // lanes of a token; token groups of a warp
    constexpr int R = elements<T, V, BWD>() / V;         // tokens of a thread
    constexpr int CT = W * GROUPS * R;                // tokens of a chunk
    constexpr int K = BWD ? 4 : 2;                    // gate, x, h before, dh
    constexpr int P = kPairs<V>, kThreads = 32 * W;
    constexpr bool kAsync = V * sizeof(T) >= 4;
    using Piece = Chans<T, V>;
    extern __shared__ __align__(16) unsigned char raw[];
    Piece* slots = reinterpret_cast<Piece*>(raw);     // [stage][array][token][thread]
    __shared__ float2 warps[2][W][kTile];             // a warp's (A, b), per parity of the round
    __shared__ float2 ctas[2][kMaxCluster][kTile];    // a CTA's, sent by it to every CTA
    __shared__ __align__(8) uint64_t bars[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % cluster;
    const int tile = blockIdx.x / cluster % tiles, b = blockIdx.x / cluster / tiles;
    const int d0 = tile * kTile;
    // V divides D.  Lanes past the last channels compute what nobody uses: they
    // fetch and write nothing (many copies of one word into as many slots take
    // as many passes), their direct loads take the last channels
    const int ch = lane % LC * V, d = min(d0 + ch, a.D - V);
    const bool own = d == d0 + ch;
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
    const int first = (warp * GROUPS + lane / LC) * R;  // of this thread's tokens in the chunk, in walking order

    // lane l of every warp carries channel d0 + l of the state; read before the
    // cluster's barrier, since the last state may be written over the first
    const bool chan = d0 + lane < a.D;
    const int64_t state = (int64_t)b * a.D + d0 + lane;
    const float* init = BWD ? a.last : a.first;
    float run = init && chan ? init[state] : 0.f;
    if (cluster > 1) {
        if (tid == 0) {
            ptx::mbar_init(&bars[0], 1);
            ptx::mbar_init(&bars[1], 1);
            ptx::fence_mbar_init();
        }
        // no CTA sends to one that has not started
        __syncthreads();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    bool lost = false;  // a wait of this thread ran out

    const T* src[K];
    int64_t step[K];
    src[0] = static_cast<const T*>(a.gate) + b * a.gs[0] + d, step[0] = a.gs[1];
    src[1] = static_cast<const T*>(a.x) + b * a.xs[0] + d, step[1] = a.xs[1];
    const int64_t dense = (int64_t)b * a.N * a.D + d;
    if constexpr (BWD) {
        src[2] = static_cast<const T*>(a.h) + dense - a.D, step[2] = a.D;
        src[3] = static_cast<const T*>(a.dh) + dense, step[3] = a.D;
    }
    constexpr int DIR = BWD ? -1 : 1;
    // the token that walks first in this thread's run
    auto token = [&](int round) {
        const unsigned s = ((unsigned)round * cluster + rank) * CT + first;  // past 2^31 in the last round at most
        return (int)(BWD ? (unsigned)a.N - 1u - s : s);
    };
    // whether every token of this CTA's chunk exists, and (backward) has one
    // before it
    auto whole = [&](int round) {
        const int64_t s = ((int64_t)round * cluster + rank) * CT;
        return BWD ? a.N - s <= len && a.N - s - CT >= 1 : s + CT <= len;
    };
    auto used = [&](int t, int k) { return t >= (k == 2 ? 1 : 0) && t < len; };
    auto inside = [&](int t) { return (unsigned)t < (unsigned)a.N; };
    auto fetch = [&](int round) {
        if constexpr (kAsync) {
            if (round < rounds) {
                Piece* to = slots + (round % kStages) * K * R * kThreads + tid;
                const int t0 = token(round);
                const bool all = whole(round);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const T* p = src[k] + t0 * step[k];
                    if (all) {
                        if (own) {
#pragma unroll
                            for (int r = 0; r < R; ++r, p += DIR * step[k]) fetch_async<sizeof(Piece)>(to + (k * R + r) * kThreads, p);
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < R; ++r, p += DIR * step[k])
                            if (used(t0 + DIR * r, k)) fetch_async<sizeof(Piece)>(to + (k * R + r) * kThreads, p);
                    }
                }
            }
            ptx::cp_async_commit();
        }
    };
    // single bf16 channels: the next round's, in registers
    Piece next[kAsync ? 1 : K][kAsync ? 1 : R];
    auto read = [&](int round) {
        if constexpr (!kAsync) {
            const int t0 = token(round);
            const bool all = round < rounds && whole(round);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const T* p = src[k] + t0 * step[k];
#pragma unroll
                for (int r = 0; r < R; ++r, p += DIR * step[k]) {
                    next[k][r] = Piece{};
                    if (all || (round < rounds && used(t0 + DIR * r, k))) next[k][r] = *reinterpret_cast<const Piece*>(p);
                }
            }
        }
    };
    read(0);
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    for (int round = 0; round < rounds; ++round) {
        const int par = round & 1;
        if (cluster > 1 && tid == 0 && !lost) ptx::mbar_arrive_expect_tx(&bars[par], cluster * kTile * 8);
        fetch(round + kStages - 1);
        ptx::cp_async_wait<kStages - 1>();
        const int t0 = token(round);
        const Piece* mine = slots + (round % kStages) * K * R * kThreads + tid;
        auto piece = [&](int k, int r) {
            if constexpr (kAsync) return mine[(k * R + r) * kThreads];
            else return next[k][r];
        };
        const bool all = whole(round);
        // 1. this thread's tokens: A and b of each, and their join
        Lanes<V> A[R], Bv[R], keep[BWD ? R : 1];
        Lanes<V> pa = lanes_of<V>(1.f), pb = lanes_of<V>(0.f);
        auto gather = [&](auto every) {
            Piece g[R], q[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                g[r] = q[r] = Piece{};
                if (every || used(t0 + DIR * r, 0)) g[r] = piece(0, r), q[r] = piece(BWD ? 3 : 1, r);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool u = every || used(t0 + DIR * r, 0);
                Lanes<V> gv, qv;
                unpack(g[r], gv);
                unpack(q[r], qv);
                if (!u) A[r] = lanes_of<V>(1.f), Bv[r] = lanes_of<V>(0.f);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    auto& kp = keep[BWD ? r : 0].e[i];
                    if (u) {
                        gates<T>(gv.e[i], A[r].e[i], kp);
                        Bv[r].e[i] = !BWD && a.coupled ? mul2(kp, qv.e[i]) : qv.e[i];
                    } else if (BWD) {
                        spread(0.f, kp);
                    }
                    pb.e[i] = BWD ? mul2(A[r].e[i], add2(Bv[r].e[i], pb.e[i])) : fma2(A[r].e[i], pb.e[i], Bv[r].e[i]);
                    pa.e[i] = mul2(pa.e[i], A[r].e[i]);
                }
            }
        };
        if (all) gather(std::true_type{});
        else gather(std::false_type{});
        [[maybe_unused]] Piece kept[2][kAsync || !BWD ? 1 : R];  // x and h before, which are used again below
        if constexpr (!kAsync && BWD) {
#pragma unroll
            for (int r = 0; r < R; ++r) kept[0][r] = next[1][r], kept[1][r] = next[2][r];
        }
        read(round + 1);
        // 2. within the warp, over its token groups (by shuffles: through shared memory it
        // took 61 us instead of 55, B4 N8192 D1024 bf16)
        float ea[V], eb[V];
        values<V>(pa, ea);
        values<V>(pb, eb);
#pragma unroll
        for (int o = LC; o < 32; o <<= 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float ba = __shfl_up_sync(0xffffffffu, ea[v], o), bb = __shfl_up_sync(0xffffffffu, eb[v], o);
                if (lane >= o) {
                    eb[v] = fmaf(ea[v], bb, eb[v]);
                    ea[v] *= ba;
                }
            }
        }
        if (lane >= 32 - LC) {
#pragma unroll
            for (int v = 0; v < V; ++v) warps[par][warp][ch + v] = make_float2(ea[v], eb[v]);
        }
        __syncthreads();
        // across warps and CTAs, lane l for channel l: c is the state before this warp's tokens
        float c = run;
        if (cluster > 1) {
            if (warp == 0 && !lost) {
                float2 total = warps[par][0][lane];
#pragma unroll
                for (int w = 1; w < W; ++w) {
                    const float2 p = warps[par][w][lane];
                    total = make_float2(total.x * p.x, fmaf(p.x, total.y, p.y));
                }
                for (int i = 0; i < cluster; ++i) send(&ctas[par][rank][lane], &bars[par], i, total);
            }
            float2 before[W - 1];
#pragma unroll
            for (int w = 0; w < W - 1; ++w) before[w] = w < warp ? warps[par][w][lane] : make_float2(1.f, 0.f);
            if (!lost && !totals_here(&bars[par], (round >> 1) & 1)) {
                lost = true;  // the outputs from here on are not to be used
                if (lane == 0) atomicOr(err, kErrScanWait);
            }
            for (int i = 0; i < cluster; ++i) {
                if (i == rank) c = run;
                const float2 p = ctas[par][i][lane];
                run = fmaf(p.x, run, p.y);
            }
#pragma unroll
            for (int w = 0; w < W - 1; ++w) c = fmaf(before[w].x, c, before[w].y);
        } else {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w == warp) c = run;
                const float2 p = warps[par][w][lane];
                run = fmaf(p.x, run, p.y);
            }
        }
        // the state before this thread's tokens: where its predecessor group ends
        float sv[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float in = __shfl_sync(0xffffffffu, c, ch + v);
            sv[v] = in;
            if constexpr (GROUPS > 1) {
                const float end = __shfl_up_sync(0xffffffffu, fmaf(ea[v], in, eb[v]), LC);
                if (lane >= LC) sv[v] = end;
            }
        }
        // 3. the outputs
        Lanes<V> s = lanes_of<V>(sv);
        auto write = [&](auto every) {
            [[maybe_unused]] T *y = nullptr, *dg = nullptr, *dx = nullptr;
            if constexpr (BWD) {
                dg = static_cast<T*>(a.dgate) + b * a.dgs[0] + d + t0 * a.dgs[1];
                dx = static_cast<T*>(a.dx) + b * a.dxs[0] + d + t0 * a.dxs[1];
            } else {
                y = static_cast<T*>(a.y) + dense + (int64_t)t0 * a.D;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int t = t0 + DIR * r;
                const bool u = every || used(t, 0);
                if constexpr (!BWD) {
#pragma unroll
                    for (int i = 0; i < P; ++i) s.e[i] = fma2(A[r].e[i], s.e[i], Bv[r].e[i]);
                    if (own && (every || inside(t))) *reinterpret_cast<Piece*>(y) = u ? pack<T, V>(s) : Piece{};
                    y += a.D;
                } else {
                    Piece px{}, ph{};
                    if constexpr (kAsync) {
                        if (u) px = piece(1, r);
                        if (every || used(t, 2)) ph = piece(2, r);
                    } else {
                        px = kept[0][r], ph = kept[1][r];
                    }
                    Lanes<V> x, before, og, ox;
                    unpack(px, x);
                    unpack(ph, before);
                    if (!every && t == 0 && a.first) {
                        float f[V];
#pragma unroll
                        for (int v = 0; v < V; ++v) f[v] = a.first[(int64_t)b * a.D + d + v];
                        before = lanes_of<V>(f);
                    }
                    const Lanes<V> minus = lanes_of<V>(a.coupled ? -1.f : 0.f);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const auto G = add2(Bv[r].e[i], s.e[i]);
                        s.e[i] = mul2(A[r].e[i], G);
                        const auto diff = a.coupled ? fma2(x.e[i], minus.e[i], before.e[i]) : before.e[i];
                        og.e[i] = mul2(mul2(s.e[i], keep[r].e[i]), diff);
                        ox.e[i] = a.coupled ? mul2(G, keep[r].e[i]) : G;
                    }
                    if (own && (every || inside(t))) {
                        *reinterpret_cast<Piece*>(dg) = u ? pack<T, V>(og) : Piece{};
                        *reinterpret_cast<Piece*>(dx) = u ? pack<T, V>(ox) : Piece{};
                    }
                    dg -= a.dgs[1];
                    dx -= a.dxs[1];
                }
            }
        };
        if (all) write(std::true_type{});
        else write(std::false_type{});
    }
    if (a.end && rank == 0 && warp == 0 && chan) a.end[state] = run;
    if (lost) {  // until every thread of the cluster is here or gone
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    }
}

template <typename T, bool BWD>
bool in_pieces(const ScanArgs& a, int V) {
    const size_t bytes = V * sizeof(T);
    if (a.D % V != 0) return false;
    const void* p[] = {a.gate, a.x, a.h, a.dh, a.y, a.dgate, a.dx};
    for (const void* q : p)
        if (q && !entry::aligned(q, bytes)) return false;
    for (int i = 0; i < 2; ++i)
        if (a.gs[i] % V || a.xs[i] % V || (BWD && (a.dgs[i] % V || a.dxs[i] % V))) return false;
    return true;
}

template <typename T, int V, bool BWD, int W>
cudaError_t launch_scan_w(const ScanArgs& a, cudaStream_t stream) {
    constexpr int CT = W * elements<T, V, BWD>();  // warps x 32 lanes x elements / 32 channels
    constexpr size_t smem = V * sizeof(T) >= 4 ? (size_t)kStages * (BWD ? 4 : 2) * elements<T, V, BWD>() * sizeof(T) * 32 * W : 0;
    const int64_t tiles = (a.D + kTile - 1) / kTile, work = tiles * a.B;
    const int64_t chunks = (a.N + CT - 1) / CT;
    // CTAs that fit at once share a sequence while there are more of them than
    // channel tiles
    int64_t cluster = (int64_t)entry::num_sms() * (kSmWarps / W) / work;
    if (cluster > chunks) cluster = chunks;
    if (cluster > kMaxCluster) cluster = kMaxCluster;
    if (cluster < 1) cluster = 1;
    if (work * cluster >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    const int rounds = (int)((chunks + cluster - 1) / cluster);
    unsigned int* err = device_error_word();
    if (!err) return cudaErrorUnknown;
    auto kernel = scan_kernel<T, V, BWD, W>;
    if (smem > 0) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = entry::allow_smem(kernel, (int)smem, done);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(work * cluster));
    cfg.blockDim = dim3(32 * W);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    TA_TIMED(stream, BWD ? "scan_kernel_backward" : "scan_kernel_forward",
             e = cudaLaunchKernelEx(&cfg, kernel, a, (int)tiles, (int)cluster, rounds, err));
    return e;
}

// Four warps a CTA where its channel tiles, or the chunks of a short sequence,
// make enough of them: four CTAs an SM wait for one another's joins less than
// two of eight (B4 N8192 D1024 bf16: 52 and 91 us, with eight 54 and 99).
// Eight where a cluster's size limits how many warps share a tile (B1 N65536
// D512: 98 and 180 us, with four 113 and 195).
template <typename T, int V, bool BWD>
cudaError_t launch_scan_v(const ScanArgs& a, cudaStream_t stream) {
    constexpr int CT = 4 * elements<T, V, BWD>();
    const int64_t work = (int64_t)((a.D + kTile - 1) / kTile) * a.B;
    const bool four = a.N <= kMaxCluster * CT || work * kMaxCluster >= 4 * (int64_t)entry::num_sms();
    return four ? launch_scan_w<T, V, BWD, 4>(a, stream) : launch_scan_w<T, V, BWD, 8>(a, stream);
}

template <typename T, bool BWD>
cudaError_t launch_scan(const ScanArgs& a, cudaStream_t stream) {
    if (in_pieces<T, BWD>(a, 4)) return launch_scan_v<T, 4, BWD>(a, stream);
    if (in_pieces<T, BWD>(a, 2)) return launch_scan_v<T, 2, BWD>(a, stream);
    return launch_scan_v<T, 1, BWD>(a, stream);
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
        alignas(16) T g[VE], v[VE], o[VE];
        alignas(16) float s[VE];
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
            gates<T>(to_float(g[e]), a, keep);
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
