// Row metadata of the paged key/value cache, shared by the append and the
// window attention, and small helpers of both (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda_cache {

constexpr unsigned kFull = 0xffffffffu;

// Division of a position (0 <= n < 2^31) by the block size: with s =
// ceil(log2 d) and m = ceil(2^(31 + s) / d), n * m >> (31 + s) is exact,
// because m exceeds 2^(31 + s) / d by less than 1 and n / 2^(31 + s) < 1 / d.
struct Divider {
    uint32_t mul, shift;
};

inline Divider make_divider(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    const uint64_t m = ((1ull << (31 + s)) + d - 1) / d;
    return Divider{(uint32_t)m, 31 + s};
}

__host__ __device__ __forceinline__ int divide(int n, const Divider &d) {
    return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
}

// ------------------------------------------------------------- arithmetic --

__device__ __forceinline__ float exp2_fast(float x) {  // within 2 ulp, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of fp32 operations in one instruction, each as its scalar form rounds.
__device__ __forceinline__ unsigned long long pair(float x, float y) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ float2 both(unsigned long long v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__device__ __forceinline__ unsigned long long add_pair(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ unsigned long long mul_pair(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ unsigned long long fma_pair(unsigned long long a, unsigned long long b,
                                                       unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Two values of a 16-bit type side by side, the first in the low half.
__device__ __forceinline__ float2 unpack(uint32_t u, __nv_bfloat16) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

__device__ __forceinline__ float2 unpack(uint32_t u, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

__device__ __forceinline__ uint32_t pack(float lo, float hi, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi, __half) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// ------------------------------------------------------------------- rows --

// The rows' side of a call: where each row's tokens lie and which request's
// table it reads.
struct Rows {
    const int *cu_seqlens;
    const int *block_table, *num_computed, *request_indices;
    long long bt_stride;
    int B, num_tokens, bt_width, block_size, num_requests, num_blocks;
    Divider by_block;
    int *err;
};

struct Row {
    int first, tokens;  // first token, token count (0: nothing to do)
    int computed;       // position of the first token
    int request;
};

__device__ __forceinline__ void flag(int *err, int bits) {
    if (err != nullptr) atomicOr(err, bits);
}

// Row b, checked; `bits` collects what is wrong with it (the row is then
// empty).  most: the largest token count allowed.  Every load is issued before
// any is looked at: one way to memory, two with request_indices.
__device__ __forceinline__ Row read_row(const Rows &r, int b, int most, int &bits) {
    const int first = r.cu_seqlens[b], end = r.cu_seqlens[b + 1];
    const int request = r.request_indices != nullptr ? r.request_indices[b] : b;
    const bool known = request >= 0 && request < r.num_requests;
    const int computed = r.num_computed[known ? request : 0];
    Row row{first, 0, computed, request};
    const long long n = (long long)end - first, last = (long long)computed + n - 1;
    if (n == 0) return row;
    if (n < 0 || n > most || first < 0 || end > r.num_tokens)
        bits |= KDA_ROW_BAD_LENGTH;
    else if (!known || computed < 0 || last > 0x7ffffff0LL ||
             divide((int)last, r.by_block) >= r.bt_width)
        bits |= KDA_ROW_BAD_BLOCK;
    else
        row.tokens = (int)n;
    return row;
}

__device__ __forceinline__ void grid_dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void grid_dependents_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------- host --

inline bool aligned(const void *ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0;
}

inline bool stride_ok(int64_t s) { return s >= 1 && (s & 7) == 0; }

// Host checks of what the append and the attention share.
inline kda_status check_config(const kda_cache_config *c) {
    if (c == nullptr) return KDA_ERR_INVALID_ARG;
    if (c->q_heads < 1 || c->kv_heads < 1 || c->q_heads % c->kv_heads != 0 || c->num_blocks < 1)
        return KDA_ERR_INVALID_ARG;
    if (c->dtype != KDA_DTYPE_BF16 && c->dtype != KDA_DTYPE_FP16) return KDA_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return KDA_ERR_UNSUPPORTED;
    if (c->q_heads > KDA_MAX_HEADS) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(c->stride_block) || !stride_ok(c->stride_token) || !stride_ok(c->stride_head))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

inline kda_status set_rows(const kda_cache_config *c, const kda_align *al, const int32_t *cu_seqlens,
                           int32_t B, int32_t num_tokens, int32_t *error_word, Rows &r) {
    if (al == nullptr || al->reserved != 0) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens || !al->block_table || !al->num_computed) return KDA_ERR_INVALID_ARG;
    if (al->block_table_width < 1 || al->block_table_stride < al->block_table_width ||
        al->num_requests < 1 || al->block_size < 1 || al->block_size > (1 << 30))
        return KDA_ERR_INVALID_ARG;
    if (!aligned(cu_seqlens, 4) || !aligned(al->block_table, 4) || !aligned(al->num_computed, 4) ||
        (al->request_indices != nullptr && !aligned(al->request_indices, 4)) ||
        (error_word != nullptr && !aligned(error_word, 4)))
        return KDA_ERR_INVALID_ARG;
    if (al->request_indices == nullptr && B > al->num_requests) return KDA_ERR_INVALID_ARG;
    r.cu_seqlens = cu_seqlens;
    r.block_table = al->block_table;
    r.num_computed = al->num_computed;
    r.request_indices = al->request_indices;
    r.bt_stride = al->block_table_stride;
    r.B = B;
    r.num_tokens = num_tokens;
    r.bt_width = al->block_table_width;
    r.block_size = al->block_size;
    r.num_requests = al->num_requests;
    r.num_blocks = c->num_blocks;
    r.by_block = make_divider((uint32_t)al->block_size);
    r.err = error_word;
    return KDA_OK;
}

inline int sm_count() {
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) cache[dev] = n;
    return n;
}

// Launch with programmatic dependent launch: the kernel may start its set-up
// while the one before it in the stream drains; it waits for it
// (grid_dependency_wait) before it touches memory.
template <typename... P, typename... A>
inline kda_status launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster,
                         void *stream, A... args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        lc.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&lc, kernel, args...) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda_cache
