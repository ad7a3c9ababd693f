// kda_token_logprobs: log probability of a given token, entropy and the top
// alternatives of each row of logits (sm_103a).  Contract in include/kda.h.
//
// Mathematics: one pass keeps a running maximum m and, with d = x - m, s =
// sum e^d and w = sum e^d d, rescaled when the maximum grows: from m to n, f =
// e^(m - n), w <- f (w + s (m - n)), s <- f s.  Then lse = m + ln s and the
// entropy is ln s - w / s.  The difference is formed before the factor log2 e
// of the exponential: x log2 e would overflow where masks hold the type's
// lowest value, and the difference of near values is exact.
//
// Alternatives without a second pass: each thread's running maximum is kept
// anyway, and those of 16 stretches of its elements beside it.  The k-th
// largest of the maxima of 64 groups of threads is a lower bound of the k-th
// largest logit, so only stretches whose maximum reaches it can hold one of
// the top k: little more than k of them.  (Of 32 groups the 32nd is too weak a
// bound, and the lists overflow: 32 alternatives of 131072 in 256 rows 78 us,
// not 24.)  Their elements are read once more (from L2), what reaches the
// bound becomes a candidate, and a candidate's place is the number of
// candidates before it.  (Reading all elements of the threads that
// reach it again took as long as the row itself for 20 alternatives.)  Where
// that leaves too many (rows of equal or masked values), warps insert what
// qualifies into lists sorted across the lanes: one more pass over the row and
// no more.
//
// HBM bounds the large calls: each logit is read once, by 16-byte loads (a
// row that does not start on 16 bytes has a few elements before and after
// them).  A row is taken by a cluster of 1 to 8 CTAs, joined over distributed
// shared memory in rank order: CTAs of 128 threads, up to 8 on an SM with 8
// loads a thread in flight, so that rows of any length and number fill the GPU
// evenly, and of 512 for the few rows that latency counts for.  4096 rows of
// 131072 in bf16: 157 us, the measured copy rate (184 with a CTA of 512 a row).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kda_async.cuh"
#include "kda_cache.cuh"

namespace {

using kda_cache::add_pair;
using kda_cache::both;
using kda_cache::exp2_fast;
using kda_cache::fma_pair;
using kda_cache::kFull;
using kda_cache::mul_pair;
using kda_cache::pair;

constexpr int kCandidates = 512;
constexpr int kStretches = 16;    // parts of a thread's elements whose maxima are kept
constexpr int kMaxima = 64;       // groups of threads whose maxima give the bound
constexpr int kFew = 64;          // keys of a cluster that are compared with each other
constexpr int kListed = 128;      // (thread, stretch) pairs that are read again
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kNever = -140.0f; // a distance whose weight e^d is 0 in fp32

struct Params {
    const char *logits;
    const int *tokens;
    float *logprob, *entropy, *lse, *top_logprob;
    int *top_index, *err;
    long long stride;             // elements
    int vocab, top, ctas;         // ctas: of a row's cluster
};

template <typename T>  // of 16 bits
__device__ __forceinline__ void unpack(uint4 u, float (&x)[8], T) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = kda_cache::unpack(w[i], T());
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void unpack(uint4 u, float (&x)[4], float) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
}

// The largest element of a vector; NaNs are passed over.
__device__ __forceinline__ float largest(uint4 u, __nv_bfloat16) {
    auto pair = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
    const __nv_bfloat162 m = __hmax2(__hmax2(pair(u.x), pair(u.y)), __hmax2(pair(u.z), pair(u.w)));
    return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ float largest(uint4 u, __half) {
    auto pair = [](uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); };
    const __half2 m = __hmax2(__hmax2(pair(u.x), pair(u.y)), __hmax2(pair(u.z), pair(u.w)));
    return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ float largest(uint4 u, float) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
                 fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}

// The vector with the type's lowest value in the place of -inf (NaNs stay).
__device__ __forceinline__ uint4 no_minus_infinity(uint4 u, __nv_bfloat16) {
    auto clamp = [](uint32_t w) {
        const uint32_t low = 0xff7fff7fu;
        const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&w),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&low));
        return *reinterpret_cast<const uint32_t *>(&m);
    };
    return make_uint4(clamp(u.x), clamp(u.y), clamp(u.z), clamp(u.w));
}

__device__ __forceinline__ uint4 no_minus_infinity(uint4 u, __half) {
    auto clamp = [](uint32_t w) {
        const uint32_t low = 0xfbfffbffu;
        const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2 *>(&w),
                                      *reinterpret_cast<const __half2 *>(&low));
        return *reinterpret_cast<const uint32_t *>(&m);
    };
    return make_uint4(clamp(u.x), clamp(u.y), clamp(u.z), clamp(u.w));
}

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

template <typename T>
__device__ __forceinline__ uint4 minus_infinity() {
    if constexpr (sizeof(T) == 4) {
        const uint32_t u = 0xff800000u;
        return make_uint4(u, u, u, u);
    } else {
        const uint32_t h = sizeof(T) == 2 && __is_same(T, __half) ? 0xfc00u : 0xff80u;
        const uint32_t u = h | (h << 16);
        return make_uint4(u, u, u, u);
    }
}

__device__ __forceinline__ uint4 load_once(const uint4 *ptr) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(ptr));
    return u;
}

// Running statistics: maximum m, s = sum e^(x - m), w = sum e^(x - m) (x - m).
struct Stats {
    float m, s, w;
};

__device__ __forceinline__ void rescale(Stats &a, float m) {  // m >= a.m
    if (a.m == -INFINITY) {  // nothing summed yet (or a NaN, kept in s)
        a.w = a.s;
    } else {
        const float d = a.m - m, f = exp2_fast(d * kLog2e);
        a.w = f * fmaf(a.s, fmaxf(d, kNever), a.w);
        a.s *= f;
    }
    a.m = m;
}

// Whether the lowest value of a 16-bit type has the weight 0 at this base (a
// row that is masked by that value may have no larger one), and no distance
// from base overflows.
template <typename T>
__device__ __forceinline__ bool far_from_lowest(float base) {
    constexpr float kAbove = sizeof(T) == 2 && __is_same(T, __half) ? -65504.0f + 200.0f : -1e30f;
    return base > kAbove && base < 1e30f;
}

// Adds a vector's elements to s and w (even and odd elements apart), as
// distances from base.  A masked element (-inf) has the weight 0 but an
// infinite distance, whose product is no number: kClamp bounds the distance;
// without it the element is the type's lowest value instead, one instruction
// for two elements, which weighs nothing either where base is far above it
// (`far_from_lowest`).  The pairs
// and that took 12 instructions an element to 8, where some 11 keep up with
// HBM: 256 x 131072 with 8 alternatives 21.2 -> 19.6 us.
template <typename T, bool kClamp>
__device__ __forceinline__ void accumulate(uint4 u, float base, unsigned long long &s,
                                           unsigned long long &w) {
    constexpr int kN = 16 / (int)sizeof(T);
    float f[kN];
    if constexpr (kClamp)
        unpack(u, f, T());
    else
        unpack(no_minus_infinity(u, T()), f, T());
    const unsigned long long shift = pair(-base, -base), scale = pair(kLog2e, kLog2e);
#pragma unroll
    for (int e = 0; e < kN; e += 2) {
        unsigned long long d = add_pair(pair(f[e], f[e + 1]), shift);
        const float2 y = both(mul_pair(d, scale));
        const unsigned long long z = pair(exp2_fast(y.x), exp2_fast(y.y));
        if constexpr (kClamp) {
            const float2 x = both(d);
            d = pair(fmaxf(x.x, kNever), fmaxf(x.y, kNever));
        }
        s = add_pair(s, z);
        w = fma_pair(z, d, w);
    }
}

__device__ __forceinline__ Stats join(Stats a, Stats b) {
    const float m = fmaxf(a.m, b.m);
    if (a.m != m) rescale(a, m);
    if (b.m != m) rescale(b, m);
    return Stats{m, a.s + b.s, a.w + b.w};
}

// The statistics of a warp's 32 lanes together, in every lane.
__device__ __forceinline__ Stats warp_join(Stats a) {
    float m = a.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (a.m != m) rescale(a, m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(kFull, a.s, o);
        a.w += __shfl_xor_sync(kFull, a.w, o);
    }
    return Stats{m, a.s, a.w};
}

// A logit and its index as one number that orders by value, then by the lower
// index; a NaN counts as -inf, and 0 comes after every logit.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t b = __float_as_uint((v == v ? v : -INFINITY) + 0.0f);
    return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of_order(uint32_t order) {
    return __uint_as_float((order >> 31) != 0 ? order & 0x7fffffffu : ~order);
}

__device__ __forceinline__ unsigned long long key_of(float v, int i) {
    return (unsigned long long)order_of(v) << 32 | (uint32_t)~i;
}

__device__ __forceinline__ float value_of(unsigned long long key) {
    return value_of_order((uint32_t)(key >> 32));
}

__device__ __forceinline__ int index_of(unsigned long long key) { return (int)~(uint32_t)key; }

// A list of up to 32 keys, the best in lane 0.
struct TopList {
    unsigned long long key;
    // Offer each lane's key (0: none); only the first k places count.
    __device__ __forceinline__ void offer(unsigned long long offered, int k, int lane) {
        const unsigned long long last = __shfl_sync(kFull, key, k - 1);
        unsigned todo = __ballot_sync(kFull, offered > last);
        while (todo != 0) {
            const int src = __ffs(todo) - 1;
            todo &= todo - 1;
            const unsigned long long in = __shfl_sync(kFull, offered, src);
            const int place = __popc(__ballot_sync(kFull, key > in));
            const unsigned long long up = __shfl_up_sync(kFull, key, 1);
            if (lane == place)
                key = in;
            else if (lane > place)
                key = up;
        }
    }
};

template <int kWarps, bool kTop>
struct Shared {
    Stats stats[kWarps];
    Stats row;                        // this CTA's, for the cluster
    alignas(16) uint32_t maxima[kMaxima];
    float bound;                      // a lower bound of the k-th largest logit
    int listed;                       // pairs that reach the bound
    int candidates;
    int list[kListed];                // thread * kStretches + stretch
    alignas(16) unsigned long long candidate[kCandidates];
    unsigned long long top[KDA_MAX_TOP];  // this CTA's top k
    float stretch[kTop ? kStretches : 1][32 * kWarps];  // each thread's maxima
};

// The top k of the n candidates in shared memory, each placed by the number
// of candidates before it.
template <int kWarps>
__device__ __forceinline__ void place(Shared<kWarps, true> &sh, int n, int k) {
    const int tid = threadIdx.x;
    if (tid < k) sh.top[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += 32 * kWarps) {
        const unsigned long long key = sh.candidate[i];
        int rank = 0;
#pragma unroll 4
        for (int c = 0; c + 1 < n; c += 2) {
            const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(&sh.candidate[c]);
            rank += (two.x > key ? 1 : 0) + (two.y > key ? 1 : 0);
        }
        if (n % 2 != 0) rank += sh.candidate[n - 1] > key ? 1 : 0;
        if (rank < k) sh.top[rank] = key;
    }
    __syncthreads();
}

// The top k of the lists of `ctas` CTAs, k sorted keys each (0: none), in
// shared memory: a key's place is its own and those of the keys before it in
// the other lists, found by bisection: 8 lists of 32 take 0.5 to 2 us less than
// by comparing it with each, as `place` does, which takes 0.8 us less for 8
// lists of 8.
template <int kWarps>
__device__ __forceinline__ void merge(Shared<kWarps, true> &sh, int ctas, int k) {
    const int tid = threadIdx.x;
    __syncthreads();
    for (int i = tid; i < ctas * k; i += 32 * kWarps) {
        const unsigned long long key = sh.candidate[i];
        if (key == 0) continue;
        int at[8] = {};
#pragma unroll
        for (int step = KDA_MAX_TOP; step > 0; step >>= 1)
            if (step <= k)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c < ctas && at[c] + step <= k &&
                        sh.candidate[c * k + at[c] + step - 1] > key)
                        at[c] += step;
        int rank = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) rank += at[c];  // of its own list: its place there
        if (rank < k) sh.top[rank] = key;
    }
    __syncthreads();
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Address of a shared variable in CTA `rank` of the cluster, and loads from it.
__device__ __forceinline__ uint32_t remote(const void *ptr, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"(kda::smem_u32(ptr)), "r"(rank));
    return a;
}

__device__ __forceinline__ float remote_f32(const float *ptr, int rank) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(remote(ptr, rank)) : "memory");
    return x;
}

__device__ __forceinline__ unsigned long long remote_u64(const unsigned long long *ptr, int rank) {
    unsigned long long x;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(remote(ptr, rank)) : "memory");
    return x;
}

template <typename T, int kWarps, bool kTop>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 4 ? 8 : 3)
    logprobs_kernel(const Params p) {
    constexpr int kN = 16 / (int)sizeof(T), kThreads = 32 * kWarps;
    constexpr int kUnroll = kWarps == 4 ? 8 : 4;  // 16-byte loads in flight per thread
    __shared__ Shared<kWarps, kTop> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / p.ctas, rank = blockIdx.x % p.ctas;
    kda_cache::grid_dependents_launch();
    if (tid == 0) sh.listed = sh.candidates = 0;
    kda_cache::grid_dependency_wait();
    const int token = p.tokens[row];
    if (token >= p.vocab) {  // uniform over the cluster
        if (tid == 0 && rank == 0) kda_cache::flag(p.err, KDA_ROW_BAD_TOKEN);
        return;
    }
    const T *x = reinterpret_cast<const T *>(p.logits) + row * p.stride;
    float x_token = 0.0f;
    if (tid == 0 && token >= 0) x_token = to_float(x[token]);
    // head elements up to a 16-byte boundary, whole vectors, tail elements
    const int head = min(p.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) /
                                      (int)sizeof(T));
    const int vectors = (p.vocab - head) / kN;
    const int tail = p.vocab - head - vectors * kN;
    const uint4 *body = reinterpret_cast<const uint4 *>(x + head);
    const int begin = (int)((long long)vectors * rank / p.ctas);
    const int end = (int)((long long)vectors * (rank + 1) / p.ctas);
    // the single element before or after the vectors that a thread adds
    auto extra_of = [&](int thread) {
        if (rank != 0) return -1;
        if (thread < head) return thread;
        return thread - head < tail ? vectors * kN + thread : -1;
    };

    Stats st{-INFINITY, 0.0f, 0.0f};
    float base = 0.0f;  // st.m, the thread's largest logit, or 0 while that is -inf
    const int extra = extra_of(tid);
    if (extra >= 0) {
        const float v = to_float(x[extra]);
        st.m = fmaxf(v, -INFINITY);
        base = st.m == -INFINITY ? 0.0f : st.m;
        const float d = v - base;
        st.s = exp2_fast(d * kLog2e);
        st.w = st.s * fmaxf(d, kNever);
    }
    // rounds of kUnroll vectors a thread, and rounds of a stretch
    const int rounds = (end - begin + kUnroll * kThreads - 1) / (kUnroll * kThreads);
    const int stretch = (rounds + kStretches - 1) / kStretches;
    float stretch_most = -INFINITY;
    int stretch_left = stretch, stretch_at = 0;
    for (int j = begin + tid; j < end; j += kUnroll * kThreads) {
        uint4 u[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            u[i] = j + i * kThreads < end ? load_once(body + j + i * kThreads)
                                          : minus_infinity<T>();
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) top = fmaxf(top, largest(u[i], T()));
        if constexpr (kTop) {
            stretch_most = fmaxf(stretch_most, top);
            if (--stretch_left == 0) {
                sh.stretch[stretch_at++][tid] = stretch_most;
                stretch_most = -INFINITY;
                stretch_left = stretch;
            }
        }
        if (top > st.m) {
            rescale(st, top);
            base = top;
        }
        unsigned long long s = 0, w = 0;  // pairs of 0
        if (sizeof(T) == 2 && far_from_lowest<T>(base)) {
            if constexpr (sizeof(T) == 2)
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) accumulate<T, false>(u[i], base, s, w);
        } else {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) accumulate<T, true>(u[i], base, s, w);
        }
        const float2 s2 = both(s), w2 = both(w);
        st.s += s2.x + s2.y;
        st.w += w2.x + w2.y;
    }

    const Stats of_warp = warp_join(st);
    if (lane == 0) sh.stats[warp] = of_warp;
    if constexpr (kTop) {
        constexpr int kEach = kThreads / kMaxima;  // threads of a group
        float v = st.m;
#pragma unroll
        for (int o = 1; o < kEach; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
        // the group's number in the last bits makes them differ; what they
        // held only lowers the bound
        if (lane % kEach == 0)
            sh.maxima[tid / kEach] = (order_of(v) & ~(uint32_t)(kMaxima - 1)) | (tid / kEach);
    }
    __syncthreads();
    if (warp == 0) {
        const Stats a =
            warp_join(lane < kWarps ? sh.stats[lane] : Stats{-INFINITY, 0.0f, 0.0f});
        if (lane == 0) sh.row = a;
    }
    if constexpr (kTop) {
        if (warp >= kWarps - kMaxima / 32) {  // the k-th largest of the maxima
            const uint32_t mine = sh.maxima[tid - (kThreads - kMaxima)];
            int rank[4] = {};
#pragma unroll
            for (int c = 0; c < kMaxima; c += 4) {
                const uint4 four = *reinterpret_cast<const uint4 *>(&sh.maxima[c]);
                rank[0] += four.x > mine ? 1 : 0;
                rank[1] += four.y > mine ? 1 : 0;
                rank[2] += four.z > mine ? 1 : 0;
                rank[3] += four.w > mine ? 1 : 0;
            }
            if (rank[0] + rank[1] + rank[2] + rank[3] == p.top - 1) {
                const uint32_t order = mine & ~(uint32_t)(kMaxima - 1);
                sh.bound = order <= order_of(-INFINITY) ? -INFINITY : value_of_order(order);
            }
        }
        __syncthreads();
        const float bound = sh.bound;
        auto push = [&](float v, int i) {
            if (!(v < bound)) {  // (a NaN counts as -inf, which may be the bound)
                if (v != v && bound != -INFINITY) return;
                const int c = atomicAdd(&sh.candidates, 1);
                if (c < kCandidates) sh.candidate[c] = key_of(v, i);
            }
        };
        // which stretches reach it
        if (st.m >= bound) {
            if (extra >= 0) push(to_float(x[extra]), extra);
            for (int i = 0; i <= stretch_at; ++i) {
                const float v = i < stretch_at ? sh.stretch[i][tid] : stretch_most;
                if (v >= bound && i * stretch < rounds) {
                    const int c = atomicAdd(&sh.listed, 1);
                    if (c < kListed) sh.list[c] = tid * kStretches + i;
                }
            }
        }
        __syncthreads();
        // their elements again, as candidates
        const int listed = sh.listed, each = stretch * kUnroll;
        if (listed <= kListed) {
            constexpr int kBatch = 2;  // loads in flight together
            for (int i0 = tid; i0 < listed * each; i0 += kBatch * kThreads) {
                uint4 u[kBatch];
                int j[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int i = i0 + b * kThreads;
                    j[b] = end;
                    if (i < listed * each) {
                        const int who = sh.list[i / each], n = who % kStretches * each + i % each;
                        j[b] = begin + who / kStretches + n * kThreads;
                    }
                    if (j[b] < end) u[b] = body[j[b]];
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    if (j[b] >= end) continue;
                    float f[kN];
                    unpack(u[b], f, T());
#pragma unroll
                    for (int e = 0; e < kN; ++e) push(f[e], head + j[b] * kN + e);
                }
            }
        }
        __syncthreads();
        if (listed > kListed || sh.candidates > kCandidates) {  // uniform over the CTA
            TopList best{0};
            best.offer(extra >= 0 ? key_of(to_float(x[extra]), extra) : 0, p.top, lane);
            for (int j0 = begin + warp * 32; j0 < end; j0 += kThreads) {
                const int j = j0 + lane;
                float f[kN];
                unpack(j < end ? body[j] : minus_infinity<T>(), f, T());
#pragma unroll
                for (int e = 0; e < kN; ++e)
                    best.offer(j < end ? key_of(f[e], head + j * kN + e) : 0, p.top, lane);
            }
            __syncthreads();
            if (tid == 0) sh.candidates = 32 * kWarps;
            sh.candidate[tid] = lane < p.top ? best.key : 0;
            __syncthreads();
        }
        place(sh, sh.candidates, p.top);
    }

    if (p.ctas > 1) {
        cluster_sync();
        if (rank == 0) {
            if (kTop)
                for (int i = tid; i < p.ctas * p.top; i += kThreads)  // at most 8 * 32
                    sh.candidate[i] = remote_u64(&sh.top[i % p.top], i / p.top);
            if (tid == 0) {
                Stats a = sh.row;
                for (int c = 1; c < p.ctas; ++c)
                    a = join(a, Stats{remote_f32(&sh.row.m, c), remote_f32(&sh.row.s, c),
                                      remote_f32(&sh.row.w, c)});
                sh.row = a;
            }
        }
        cluster_sync();
        if (rank != 0) return;
        if constexpr (kTop) {
            if (p.ctas * p.top <= kFew)
                place(sh, p.ctas * p.top, p.top);
            else
                merge(sh, p.ctas, p.top);
        }
    } else if (!kTop) {
        __syncthreads();
    }

    const Stats a = sh.row;
    const float log_s = kLn2 * log2f(a.s);
    const float lse = a.s == 0.0f ? -INFINITY : a.m + log_s;
    if (tid == 0) {
        p.logprob[row] = token < 0 ? 0.0f : (lse == -INFINITY ? lse : x_token - lse);
        if (p.entropy != nullptr) p.entropy[row] = a.s == 0.0f ? 0.0f : log_s - a.w / a.s;
        if (p.lse != nullptr) p.lse[row] = lse;
    }
    if (kTop && tid < p.top) {
        const long long at = (long long)row * p.top + tid;
        const unsigned long long key = sh.top[tid];
        p.top_logprob[at] = lse == -INFINITY ? lse : value_of(key) - lse;
        p.top_index[at] = index_of(key);
    }
}

template <typename T, int kWarps>
kda_status launch_logprobs(const Params &p, int rows, void *stream) {
    void (*kernel)(const Params) =
        p.top > 0 ? logprobs_kernel<T, kWarps, true> : logprobs_kernel<T, kWarps, false>;
    return kda_cache::launch(kernel, dim3((unsigned)rows * (unsigned)p.ctas), dim3(32 * kWarps), 0,
                             p.ctas, stream, p);
}

template <typename T>
kda_status launch_rows(Params &p, int rows, void *stream) {
    // CTAs of 512 threads for few rows: one of 131072 8.1 us (9.9 with 128
    // threads), 40 of 115069 39 us (19).  More CTAs a row up to some four an
    // SM, each with enough elements to be worth its part of the join: 256 rows
    // of 131072 with 2, 4 or 8 CTAs 28, 21 and 27 us, 517 of 100003 in fp32
    // with 1, 2 or 4 44, 39 and 47 us.
    const bool wide = rows * 8ll <= 304;
    p.ctas = 1;
    while (p.ctas < 8 && (long long)rows * p.ctas < 600 && p.vocab / (2 * p.ctas) >= 16384)
        p.ctas *= 2;
    return wide ? launch_logprobs<T, 16>(p, rows, stream) : launch_logprobs<T, 4>(p, rows, stream);
}

}  // namespace

extern "C" kda_status kda_token_logprobs(const void *logits, int32_t dtype, int64_t stride_row,
                                         int32_t rows, int32_t vocab, const int32_t *tokens,
                                         int32_t num_top, float *logprob, float *entropy,
                                         float *lse_out, float *top_logprob, int32_t *top_index,
                                         int32_t *error_word, void *stream) {
    using kda_cache::aligned;
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP16 && dtype != KDA_DTYPE_FP32)
        return KDA_ERR_INVALID_ARG;
    if (rows < 0 || vocab < 1 || stride_row < 0 || num_top < 0 || num_top > vocab)
        return KDA_ERR_INVALID_ARG;
    if (num_top > KDA_MAX_TOP || rows > (1 << 27)) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;  // nothing to do; no pointer is inspected
    if (!logits || !tokens || !logprob || (num_top > 0 && (!top_logprob || !top_index)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == KDA_DTYPE_FP32 ? 4 : 2) || !aligned(tokens, 4) ||
        !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse_out, 4) ||
        !aligned(error_word, 4) ||
        (num_top > 0 && (!aligned(top_logprob, 4) || !aligned(top_index, 4))))
        return KDA_ERR_INVALID_ARG;
    Params p;
    p.logits = static_cast<const char *>(logits);
    p.tokens = tokens;
    p.logprob = logprob;
    p.entropy = entropy;
    p.lse = lse_out;
    p.top_logprob = top_logprob;
    p.top_index = top_index;
    p.err = error_word;
    p.stride = stride_row;
    p.vocab = vocab;
    p.top = num_top;
    if (dtype == KDA_DTYPE_BF16) return launch_rows<__nv_bfloat16>(p, rows, stream);
    if (dtype == KDA_DTYPE_FP16) return launch_rows<__half>(p, rows, stream);
    return launch_rows<float>(p, rows, stream);
}

extern "C" kda_status kda_token_logprobs_packed(const kda_logprobs_args *a) {
    if (a == nullptr) return KDA_ERR_INVALID_ARG;
    return kda_token_logprobs(a->logits, a->dtype, a->stride_row, a->rows, a->vocab, a->tokens,
                              a->num_top, a->logprob, a->entropy, a->lse_out, a->top_logprob,
                              a->top_index, a->error_word, a->stream);
}
