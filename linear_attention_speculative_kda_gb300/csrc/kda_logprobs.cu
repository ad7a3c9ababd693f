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
// anyway.  The k-th largest of them is a lower bound of the k-th largest
// logit, so only threads whose maximum reaches it can hold one of the top k:
// about k of 512.  Their elements are read once more (from L2), and warps
// insert what qualifies into a list sorted across the lanes.  Rows of equal
// values, where every thread qualifies, cost one more pass and no more.
//
// HBM bounds the large calls: each logit is read once, by 16-byte loads (a
// row that does not start on 16 bytes has a few elements before and after
// them).  A CTA takes a row; where there are fewer rows than CTAs fill the
// GPU, a cluster of 2 to 8 CTAs shares a row and joins over distributed
// shared memory, in rank order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kda_async.cuh"
#include "kda_cache.cuh"

namespace {

using kda_cache::kFull;

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnroll = 4;        // 16-byte loads in flight per thread
constexpr int kTopOfWarp = 4;     // thread maxima of a warp that the bound looks at
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

__device__ __forceinline__ float exp2_fast(float x) {  // within 2 ulp, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void unpack(uint4 u, float (&x)[8], __nv_bfloat16) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void unpack(uint4 u, float (&x)[8], __half) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
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

__device__ __forceinline__ Stats join(Stats a, Stats b) {
    const float m = fmaxf(a.m, b.m);
    if (a.m != m) rescale(a, m);
    if (b.m != m) rescale(b, m);
    return Stats{m, a.s + b.s, a.w + b.w};
}

__device__ __forceinline__ Stats shuffle_xor(Stats a, int o) {
    return Stats{__shfl_xor_sync(kFull, a.m, o), __shfl_xor_sync(kFull, a.s, o),
                 __shfl_xor_sync(kFull, a.w, o)};
}

// Whether (v, i) comes before (u, j): larger, or equal at the lower index.
__device__ __forceinline__ bool before(float v, int i, float u, int j) {
    return v > u || (v == u && i < j);
}

// A list of up to 32 (value, index) pairs, the best in lane 0.
struct TopList {
    float v;
    int i;
    __device__ __forceinline__ void clear() {
        v = -INFINITY;
        i = 0x7fffffff;
    }
    // Offer each lane's (x, at) where `offered`; only the first k places count.
    __device__ __forceinline__ void offer(float x, int at, bool offered, int k, int lane) {
        float kv = __shfl_sync(kFull, v, k - 1);
        int ki = __shfl_sync(kFull, i, k - 1);
        unsigned todo = __ballot_sync(kFull, offered && before(x, at, kv, ki));
        while (todo != 0) {
            const int src = __ffs(todo) - 1;
            todo &= todo - 1;
            const float nv = __shfl_sync(kFull, x, src);
            const int ni = __shfl_sync(kFull, at, src);
            const int place = __popc(__ballot_sync(kFull, before(v, i, nv, ni)));
            const float uv = __shfl_up_sync(kFull, v, 1);
            const int ui = __shfl_up_sync(kFull, i, 1);
            if (lane == place) {
                v = nv;
                i = ni;
            } else if (lane > place) {
                v = uv;
                i = ui;
            }
        }
    }
};

struct Shared {
    Stats stats[kWarps];
    Stats row;                        // this CTA's, for the cluster
    float maxima[kWarps * kTopOfWarp];
    float bound;
    int threads;                      // threads that reach the bound
    int candidates;
    int list[kThreads];
    float cand_v[kThreads];
    int cand_i[kThreads];
    float top_v[KDA_MAX_TOP];         // this CTA's top k
    int top_i[KDA_MAX_TOP];
};

// The top k of the n candidates in shared memory, each placed by the number
// of candidates before it.
__device__ __forceinline__ void place(Shared &sh, int n, int k) {
    const int tid = threadIdx.x;
    if (tid < k) {
        sh.top_v[tid] = -INFINITY;
        sh.top_i[tid] = 0x7fffffff;
    }
    float v = 0.0f;
    int i = 0, rank = k;
    if (tid < n) {
        v = sh.cand_v[tid];
        i = sh.cand_i[tid];
        rank = 0;
        for (int c = 0; c < n; ++c) rank += before(sh.cand_v[c], sh.cand_i[c], v, i) ? 1 : 0;
    }
    __syncthreads();
    if (rank < k) {
        sh.top_v[rank] = v;
        sh.top_i[rank] = i;
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

__device__ __forceinline__ int remote_s32(const int *ptr, int rank) {
    int x;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(remote(ptr, rank)) : "memory");
    return x;
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 3) logprobs_kernel(const Params p) {
    constexpr int kN = 16 / (int)sizeof(T);
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / p.ctas, rank = blockIdx.x % p.ctas;
    kda_cache::grid_dependents_launch();
    kda_cache::grid_dependency_wait();
    const int token = p.tokens[row];
    if (token >= p.vocab) {  // uniform over the cluster
        if (tid == 0 && rank == 0) kda_cache::flag(p.err, KDA_ROW_BAD_TOKEN);
        return;
    }
    const T *x = reinterpret_cast<const T *>(p.logits) + row * p.stride;
    // head elements up to a 16-byte boundary, whole vectors, tail elements
    const int head = min(p.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) /
                                      (int)sizeof(T));
    const int vectors = (p.vocab - head) / kN;
    const int tail = p.vocab - head - vectors * kN;
    const uint4 *body = reinterpret_cast<const uint4 *>(x + head);
    const int begin = (int)((long long)vectors * rank / p.ctas);
    const int end = (int)((long long)vectors * (rank + 1) / p.ctas);
    // the single element before or after the vectors that this thread adds
    int extra = -1;
    if (rank == 0) {
        if (tid < head) extra = tid;
        else if (tid - head < tail) extra = head + vectors * kN + (tid - head);
    }

    Stats st{-INFINITY, 0.0f, 0.0f};
    float base = 0.0f;  // st.m, the thread's largest logit, or 0 while that is -inf
    if (extra >= 0) {
        const float v = to_float(x[extra]);
        st.m = fmaxf(v, -INFINITY);
        base = st.m == -INFINITY ? 0.0f : st.m;
        const float d = v - base;
        st.s = exp2_fast(d * kLog2e);
        st.w = st.s * fmaxf(d, kNever);
    }
    for (int j = begin + tid; j < end; j += kUnroll * kThreads) {
        uint4 u[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            u[i] = j + i * kThreads < end ? load_once(body + j + i * kThreads)
                                          : minus_infinity<T>();
        float f[kUnroll][kN];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            unpack(u[i], f[i], T());
#pragma unroll
            for (int e = 0; e < kN; ++e) top = fmaxf(top, f[i][e]);
        }
        if (top > st.m) {
            rescale(st, top);
            base = top;
        }
        float s[2] = {0.0f, 0.0f}, w[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const float d = f[i][e] - base;
                const float z = exp2_fast(d * kLog2e);
                s[e & 1] += z;
                w[e & 1] = fmaf(z, fmaxf(d, kNever), w[e & 1]);
            }
        st.s += s[0] + s[1];
        st.w += w[0] + w[1];
    }

    Stats all = st;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all = join(all, shuffle_xor(all, o));
    if (lane == 0) sh.stats[warp] = all;
    if constexpr (kTop) {
        // the warp's thread maxima in descending order (a bitonic network)
        float v = st.m;
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
            for (int o = size >> 1; o > 0; o >>= 1) {
                const float u = __shfl_xor_sync(kFull, v, o);
                const bool larger = ((lane & size) == 0) == ((lane & o) == 0);
                v = larger ? fmaxf(v, u) : fminf(v, u);
            }
        if (lane < kTopOfWarp) sh.maxima[warp * kTopOfWarp + lane] = v;
        if (tid == 0) sh.threads = sh.candidates = 0;
    }
    __syncthreads();
    if (warp == 0) {
        Stats a = lane < kWarps ? sh.stats[lane] : Stats{-INFINITY, 0.0f, 0.0f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = join(a, shuffle_xor(a, o));
        if (lane == 0) sh.row = a;
    }
    if constexpr (kTop) {
        constexpr int kMaxima = kWarps * kTopOfWarp;
        if (warp == 1) {  // the k-th largest of the maxima kept
            float bound = -INFINITY;
            for (int c = lane; c < kMaxima; c += 32) {
                const float v = sh.maxima[c];
                int ge = 0;
                for (int d = 0; d < kMaxima; ++d) ge += sh.maxima[d] >= v ? 1 : 0;
                if (ge >= p.top) bound = fmaxf(bound, v);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                bound = fmaxf(bound, __shfl_xor_sync(kFull, bound, o));
            if (lane == 0) sh.bound = bound;
        }
        __syncthreads();
        const float bound = sh.bound;
        if (st.m >= bound) sh.list[atomicAdd(&sh.threads, 1)] = tid;
        __syncthreads();
        // read those threads' elements again
        TopList best;
        best.clear();
        for (int c = warp; c < sh.threads; c += kWarps) {
            const int who = sh.list[c];
            int who_extra = -1;
            if (rank == 0) {
                if (who < head) who_extra = who;
                else if (who - head < tail) who_extra = head + vectors * kN + (who - head);
            }
            if (who_extra >= 0) {
                float v = to_float(x[who_extra]);
                v = v == v ? v : -INFINITY;
                best.offer(v, who_extra, lane == 0 && v >= bound, p.top, lane);
            }
            for (int j0 = begin + who; j0 < end; j0 += 32 * kThreads) {
                const int j = j0 + lane * kThreads;
                const bool in = j < end;
                float f[kN];
                unpack(in ? body[j] : minus_infinity<T>(), f, T());
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    const float v = f[e] == f[e] ? f[e] : -INFINITY;
                    best.offer(v, head + j * kN + e, in && v >= bound, p.top, lane);
                }
            }
        }
        if (lane < p.top && best.i != 0x7fffffff) {
            const int c = atomicAdd(&sh.candidates, 1);
            sh.cand_v[c] = best.v;
            sh.cand_i[c] = best.i;
        }
        __syncthreads();
        place(sh, sh.candidates, p.top);
    }

    if (p.ctas > 1) {
        cluster_sync();
        if (rank == 0) {
            if (kTop && tid < p.ctas * p.top) {  // at most 8 * 32
                sh.cand_v[tid] = remote_f32(&sh.top_v[tid % p.top], tid / p.top);
                sh.cand_i[tid] = remote_s32(&sh.top_i[tid % p.top], tid / p.top);
            }
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
        if constexpr (kTop) place(sh, p.ctas * p.top, p.top);
    } else {
        __syncthreads();
    }

    const Stats a = sh.row;
    const float log_s = kLn2 * log2f(a.s);
    const float lse = a.s == 0.0f ? -INFINITY : a.m + log_s;
    if (tid == 0) {
        p.logprob[row] = token < 0 ? 0.0f
                                   : (lse == -INFINITY ? lse : to_float(x[token]) - lse);
        if (p.entropy != nullptr)
            p.entropy[row] = a.s == 0.0f ? 0.0f : log_s - a.w / a.s;
        if (p.lse != nullptr) p.lse[row] = lse;
    }
    if (kTop && tid < p.top) {
        const long long at = (long long)row * p.top + tid;
        p.top_logprob[at] = lse == -INFINITY ? lse : to_float(x[sh.top_i[tid]]) - lse;
        p.top_index[at] = sh.top_i[tid];
    }
}

template <typename T>
kda_status launch_logprobs(const Params &p, int rows, void *stream) {
    void (*kernel)(const Params) = p.top > 0 ? logprobs_kernel<T, true> : logprobs_kernel<T, false>;
    return kda_cache::launch(kernel, dim3((unsigned)rows * (unsigned)p.ctas), dim3(kThreads), 0,
                             p.ctas, stream, p);
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
    // CTAs of a row: enough to fill the SMs, each with two rounds of loads
    p.ctas = 1;
    while (p.ctas < 8 && (long long)rows * p.ctas * 2 <= 304 && vocab / (p.ctas * 2) >= 8192)
        p.ctas *= 2;
    if (dtype == KDA_DTYPE_BF16) return launch_logprobs<__nv_bfloat16>(p, rows, stream);
    if (dtype == KDA_DTYPE_FP16) return launch_logprobs<__half>(p, rows, stream);
    return launch_logprobs<float>(p, rows, stream);
}
