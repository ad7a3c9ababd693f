// kda_kv_append: rotate the new tokens' queries and keys by position and
// write keys and values to the paged cache (sm_103a), and kda_kv_norm_append,
// which norms each head's queries and keys first.  Contracts in include/kda.h.
//
// Mathematics.  Pair i of a head at position p turns by the angle p * f_i.
// Only the angle modulo a full turn counts, so the phase is kept in turns:
// u_i = (f_i / 2 pi mod 1) * 2^64 as a whole number, and p * u_i mod 2^64 is
// the fraction of a turn exactly; the rounding of u_i, 2^-63 of it, is all
// that grows with p.  Its top 32 bits, signed, give the angle in [-pi, pi)
// for sincospif.  u_i is made from f_i's bits in whole numbers too: with fp64
// arithmetic, some 2 lanes a clock on an SM here, 256 tokens took 6.4 us and
// not 4.2.
//
// Every value is read and written once and the arithmetic is 3 flops per
// rotated channel, so HBM bounds the large calls and latency the small ones.
// A warp takes part of one token: a lane moves units of 16 channels of a head
// (two 16-byte chunks: the two halves of its 8 pairs).  Where a unit lies
// does not depend on the row, so a warp's first unit is loaded before the
// row's metadata is read and the sines are made (once per warp, in shared
// memory), and each later unit before the one ahead of it is written.
#include "kda_cache.cuh"

namespace {

using kda_cache::pack;
using kda_cache::Rows;
using kda_cache::unpack;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxPairs = 64;
// Pair 8 j + i of a token (unit j's i-th) is kept at kTurn i + j: the lanes that
// read the i-th side by side find it side by side.
constexpr int kTurn = 8;

// With 64 registers a thread for heads of 128 channels and 48 for 64.  Measured
// (us, 4 | 5 CTAs an SM): 256 tokens 4.2 | 4.9 and 13.7k tokens 45 | 48 with
// 128 channels (16k interleaved ones 53 | 51), 10k tokens 7.4 | 6.8 and 56k
// tokens 22 | 20 with 64.
// The norm takes 62 and spills with 48: 14k tokens of 64 channels 34 us, not 39.
constexpr int ctas_per_sm(int dim, bool norm) { return dim == 128 || norm ? 4 : 5; }

struct Params {
    Rows rows;
    const char *q, *k, *v;
    char *q_out, *key_cache, *value_cache;
    const double *inv_freq;
    long long stride_q, stride_k, stride_v;              // elements
    long long stride_block, stride_token, stride_head;   // elements
    int q_heads, kv_heads, num_tokens;
    int pairs;        // rotary_dim / 2
    int interleaved;
    int parts;        // warps that share a token
    int rounds;       // rounds of 32 units (one a lane) each of them takes
    int token_blocks; // CTAs that take tokens; those behind them check the rows
    const void *q_weight, *k_weight;   // of the norms (nullptr: ones)
    int weight_dtype;
    float eps;
};

// The row that owns token t (the last one that starts at or before t), found
// by a warp in steps of 32; -1 when t lies before every row.
__device__ __forceinline__ int find_row(const int *cu, int B, int t, int lane) {
    int lo = 0, n = B;
    for (;;) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool starts = lane * step < n && cu[i] <= t;
        const unsigned mask = __ballot_sync(kda_cache::kFull, starts);
        if (mask == 0) return -1;
        const int skip = (31 - __clz(mask)) * step;
        lo += skip;
        n = min(step, n - skip);
        if (n <= 1) return lo;
    }
}

// f / 2 pi modulo 1 as a 64-bit fraction of a turn: with f = M 2^(e - 63),
// 2^63 <= M < 2^64, and C = 2^66 / 2 pi, it is f / 2 pi 2^64 =
// (M C / 2^64) 2^(e - 1).
__device__ __forceinline__ unsigned long long turns_per_position(double f) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
    const int e = (int)((bits >> 52) & 0x7ff) - 1023;
    if (e == -1023) return 0;  // 0, or too small to turn anything
    const unsigned long long m = (bits << 11) | 0x8000000000000000ull;
    const unsigned long long h = __umul64hi(m, 0xa2f9836e4e44152aull);
    const int right = 1 - e;
    const unsigned long long u =
        right >= 64 || right <= -64 ? 0 : right >= 0 ? h >> right : h << -right;
    return (bits >> 63) != 0 ? 0 - u : u;
}

// Two pairs of one head: p and r hold them as halves (p.x with r.x) or side by
// side (p.x with p.y), i = 0..3 of a unit's chunks.
__device__ __forceinline__ void rotate_pairs(float2 &p, float2 &r, const float2 *turn, int i,
                                             bool interleaved) {
    if (interleaved) {
        const float2 s = turn[kTurn * i], t = turn[kTurn * (4 + i)];
        p = make_float2(p.x * s.x - p.y * s.y, p.x * s.y + p.y * s.x);
        r = make_float2(r.x * t.x - r.y * t.y, r.x * t.y + r.y * t.x);
    } else {
        const float2 s = turn[kTurn * 2 * i], t = turn[kTurn * (2 * i + 1)];
        const float2 u = p;
        p = make_float2(u.x * s.x - r.x * s.y, u.y * t.x - r.y * t.y);
        r = make_float2(u.x * s.y + r.x * s.x, u.y * t.y + r.y * t.x);
    }
}

// 8 pairs of one head: chunk a and chunk b hold them as halves (a[e], b[e])
// or side by side (a[2e], a[2e+1], then b).
template <typename T>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float2 *turn, bool interleaved) {
    uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 p = unpack(x[i], T()), r = unpack(y[i], T());
        rotate_pairs(p, r, turn, i, interleaved);
        x[i] = pack(p.x, p.y, T());
        y[i] = pack(r.x, r.y, T());
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
    b = make_uint4(y[0], y[1], y[2], y[3]);
}

// Element i of a weight as fp32.
__device__ __forceinline__ float weight_at(const void *w, int dtype, int i) {
    if (w == nullptr) return 1.0f;
    if (dtype == KDA_DTYPE_FP32) return static_cast<const float *>(w)[i];
    return dtype == KDA_DTYPE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i])
                                   : __half2float(static_cast<const __half *>(w)[i]);
}

// The same behind the norm of the head, which kUnits lanes beside each other
// hold (all of them get here).  weight: the unit's, four fourths kUnits apart.
template <typename T, int kUnits>
__device__ __forceinline__ void norm_rotate(uint4 &a, uint4 &b, const float4 *weight,
                                            float eps, const float2 *turn, bool turned,
                                            bool interleaved, int lane) {
    uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    unsigned long long p[4], r[4], squares = kda_cache::pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = unpack(x[i], T()), v = unpack(y[i], T());
        p[i] = kda_cache::pair(u.x, u.y);
        r[i] = kda_cache::pair(v.x, v.y);
        squares = kda_cache::fma_pair(p[i], p[i], kda_cache::fma_pair(r[i], r[i], squares));
    }
    const float2 both = kda_cache::both(squares);
    float sum = both.x + both.y;
    const unsigned group = ((1u << kUnits) - 1) << (lane & ~(kUnits - 1));
#pragma unroll
    for (int o = kUnits / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(group, sum, o);
    const float root = rsqrtf(fmaf(sum, 1.0f / (16 * kUnits), eps));
    const unsigned long long f = kda_cache::pair(root, root);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (two weights are a half of a fourth)
        const ulonglong2 *w = reinterpret_cast<const ulonglong2 *>(weight + (i >> 1) * kUnits);
        const ulonglong2 *z = reinterpret_cast<const ulonglong2 *>(weight + (2 + (i >> 1)) * kUnits);
        float2 u = kda_cache::both(
            kda_cache::mul_pair(kda_cache::mul_pair(p[i], f), (i & 1) ? w->y : w->x));
        float2 v = kda_cache::both(
            kda_cache::mul_pair(kda_cache::mul_pair(r[i], f), (i & 1) ? z->y : z->x));
        if (turned) rotate_pairs(u, v, turn, i, interleaved);
        x[i] = pack(u.x, u.y, T());
        y[i] = pack(v.x, v.y, T());
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
    b = make_uint4(y[0], y[1], y[2], y[3]);
}

// Where the two chunks of a head's unit j start: the same pairs in both
// halves, or 16 channels side by side.
__device__ __forceinline__ int2 chunks_of(const Params &p, bool turned, int j) {
    return turned && !p.interleaved ? make_int2(j * 8, p.pairs + j * 8)
                                    : make_int2(j * 16, j * 16 + 8);
}

template <typename T, int kDim, bool kNorm>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kDim, kNorm))
    append_kernel(const Params p) {
    constexpr int kUnits = kDim / 16;  // units of a head
    __shared__ float2 turns[kWarps][kMaxPairs];
    // of q and of k: fourths of a unit's weights, so that the units that read one
    // lie side by side
    __shared__ float4 weights[kNorm ? 2 : 1][kNorm ? 4 * kUnits : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    kda_cache::grid_dependents_launch();
    kda_cache::grid_dependency_wait();
    if ((int)blockIdx.x >= p.token_blocks) {  // these check the rows
        const long long r = ((long long)blockIdx.x - p.token_blocks) * kThreads + threadIdx.x;
        int bits = 0;
        if (r < p.rows.B) kda_cache::read_row(p.rows, (int)r, 0x7fffffff, bits);
        if (bits != 0) kda_cache::flag(p.rows.err, bits);
        return;
    }
    const long long item = (long long)blockIdx.x * kWarps + warp;
    const int t = (int)(item / p.parts), part = (int)(item % p.parts);
    const int first_k = p.q_heads, first_v = p.q_heads + p.kv_heads;
    const int begin = part * p.rounds * 32;
    const int end = min((first_v + p.kv_heads) * kUnits, begin + p.rounds * 32);

    auto load = [&](int u, uint4 &x, uint4 &y) {
        if (u >= end || t >= p.num_tokens) return;
        const int head = u / kUnits, j = u % kUnits;
        const T *src;
        if (head < first_k)
            src = reinterpret_cast<const T *>(p.q) + t * p.stride_q + head * kDim;
        else if (head < first_v)
            src = reinterpret_cast<const T *>(p.k) + t * p.stride_k + (head - first_k) * kDim;
        else
            src = reinterpret_cast<const T *>(p.v) + t * p.stride_v + (head - first_v) * kDim;
        const int2 at = chunks_of(p, head < first_v && j * 8 < p.pairs, j);
        // read and written once here: marked to leave the caches first, which
        // takes 2 of 53 us off 16k tokens
        x = __ldcs(reinterpret_cast<const uint4 *>(src + at.x));
        y = __ldcs(reinterpret_cast<const uint4 *>(src + at.y));
    };
    uint4 x[2], y[2];
    load(begin + lane, x[0], y[0]);
    if constexpr (kNorm) {  // while the first units are on their way
        for (int i = threadIdx.x; i < 2 * kDim; i += kThreads) {
            const int which = i / kDim, quarter = i / (4 * kUnits) & 3, j = i / 4 % kUnits;
            const int2 at = chunks_of(p, j * 8 < p.pairs, j);
            reinterpret_cast<float *>(weights)[i] =
                weight_at(which == 0 ? p.q_weight : p.k_weight, p.weight_dtype,
                          (quarter < 2 ? at.x : at.y) + (quarter & 1) * 4 + (i & 3));
        }
        __syncthreads();
    }
    if (t >= p.num_tokens) return;
    const int b = find_row(p.rows.cu_seqlens, p.rows.B, t, lane);
    if (b < 0) return;
    int bits = 0;  // flagged where the rows are checked
    const kda_cache::Row row = kda_cache::read_row(p.rows, b, 0x7fffffff, bits);
    if (t - row.first >= row.tokens) return;  // between rows, or a row that is skipped
    const int pos = row.computed + (t - row.first);
    const int col = kda_cache::divide(pos, p.rows.by_block);
    int block = p.rows.block_table[row.request * p.rows.bt_stride + col];
    if (block >= p.rows.num_blocks) {
        if (lane == 0) kda_cache::flag(p.rows.err, KDA_ROW_BAD_SLOT);
        block = 0;
    }
    for (int i = lane; i < p.pairs; i += 32) {
        const double f = p.inv_freq[i];
        const int phase = (int)((turns_per_position(f) * (unsigned long long)pos) >> 32);
        float2 cs;
        sincospif((float)phase * 0x1p-31f, &cs.y, &cs.x);
        if ((__double2hiint(f) & 0x7ff00000) == 0x7ff00000)  // infinite or a NaN: no angle
            cs = make_float2(NAN, NAN);
        turns[warp][kTurn * (i & 7) + (i >> 3)] = cs;
    }
    __syncwarp();
    const long long slot = (long long)max(block, 0) * p.stride_block +
                           (long long)(pos - col * p.rows.block_size) * p.stride_token;

    auto store = [&](int u, uint4 &x, uint4 &y) {
        if (u >= end) return;
        const int head = u / kUnits, j = u % kUnits;
        T *dst;
        if (head < first_k)
            dst = reinterpret_cast<T *>(p.q_out) + ((long long)t * p.q_heads + head) * kDim;
        else if (head < first_v)
            dst = reinterpret_cast<T *>(p.key_cache) + slot + (head - first_k) * p.stride_head;
        else
            dst = reinterpret_cast<T *>(p.value_cache) + slot + (head - first_v) * p.stride_head;
        const bool turned = head < first_v && j * 8 < p.pairs;
        const int2 at = chunks_of(p, turned, j);
        if constexpr (kNorm) {
            if (head < first_v)
                norm_rotate<T, kUnits>(x, y, &weights[head < first_k ? 0 : 1][j], p.eps,
                                       &turns[warp][j], turned, p.interleaved != 0, lane);
        } else {
            if (turned) rotate<T>(x, y, &turns[warp][j], p.interleaved != 0);
        }
        if (head < first_k || block > 0) {
            __stcs(reinterpret_cast<uint4 *>(dst + at.x), x);
            __stcs(reinterpret_cast<uint4 *>(dst + at.y), y);
        }
    };
    for (int u = begin + lane; u < end; u += 64) {
        load(u + 32, x[1], y[1]);
        store(u, x[0], y[0]);
        load(u + 64, x[0], y[0]);
        store(u + 32, x[1], y[1]);
    }
}

template <bool kNorm>
void (*kernel_for(bool bf16, bool small))(const Params) {
    if (bf16)
        return small ? append_kernel<__nv_bfloat16, 64, kNorm> : append_kernel<__nv_bfloat16, 128, kNorm>;
    return small ? append_kernel<__half, 64, kNorm> : append_kernel<__half, 128, kNorm>;
}

}  // namespace

namespace {

// The norm of a call: none, or its weights and eps.
struct Norm {
    const void *q_weight, *k_weight;
    int dtype;
    float eps;
};

kda_status append(const kda_cache_config *cfg, const void *q, const void *k, const void *v,
                  void *q_out, void *key_cache, void *value_cache, const double *inv_freq,
                  const int32_t *cu_seqlens, int32_t B, int32_t num_tokens, const kda_align *align,
                  int32_t *error_word, void *stream, const Norm *norm) {
    using kda_cache::aligned;
    using kda_cache::stride_ok;
    kda_status st = kda_cache::check_config(cfg);
    if (st != KDA_OK) return st;
    if (B < 0 || num_tokens < 0) return KDA_ERR_INVALID_ARG;
    if (cfg->rotary_dim < 0 || cfg->rotary_dim > cfg->head_dim || (cfg->rotary_dim & 15) != 0 ||
        (cfg->interleaved != 0 && cfg->interleaved != 1))
        return KDA_ERR_INVALID_ARG;
    if (norm != nullptr) {
        // 0 is a choice too; a sum of squares that it leaves at 0 gives 0 / 0
        if (!(norm->eps >= 0.0f && isfinite(norm->eps))) return KDA_ERR_INVALID_ARG;
        if (norm->dtype != cfg->dtype && norm->dtype != KDA_DTYPE_FP32) return KDA_ERR_INVALID_ARG;
    }
    if (B == 0 || num_tokens == 0) return KDA_OK;  // nothing to do; no pointer is inspected
    Params p{};
    st = kda_cache::set_rows(cfg, align, cu_seqlens, B, num_tokens, error_word, p.rows);
    if (st != KDA_OK) return st;
    if (!k || !v || !key_cache || !value_cache || (q != nullptr && !q_out) ||
        (cfg->rotary_dim > 0 && !inv_freq))
        return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(key_cache, 16) ||
        !aligned(value_cache, 16) || (q != nullptr && !aligned(q_out, 16)) ||
        (cfg->rotary_dim > 0 && !aligned(inv_freq, 8)))
        return KDA_ERR_INVALID_ARG;
    if ((q != nullptr && !stride_ok(cfg->stride_q_t)) || !stride_ok(cfg->stride_k_t) ||
        !stride_ok(cfg->stride_v_t))
        return KDA_ERR_INVALID_ARG;
    if (norm != nullptr) {
        if (!aligned(norm->q_weight, 16) || !aligned(norm->k_weight, 16))
            return KDA_ERR_INVALID_ARG;
        p.q_weight = norm->q_weight;
        p.k_weight = norm->k_weight;
        p.weight_dtype = norm->dtype;
        p.eps = norm->eps;
    }
    p.q = static_cast<const char *>(q);
    p.k = static_cast<const char *>(k);
    p.v = static_cast<const char *>(v);
    p.q_out = static_cast<char *>(q_out);
    p.key_cache = static_cast<char *>(key_cache);
    p.value_cache = static_cast<char *>(value_cache);
    p.inv_freq = inv_freq;
    p.stride_q = cfg->stride_q_t;
    p.stride_k = cfg->stride_k_t;
    p.stride_v = cfg->stride_v_t;
    p.stride_block = cfg->stride_block;
    p.stride_token = cfg->stride_token;
    p.stride_head = cfg->stride_head;
    p.q_heads = q != nullptr ? cfg->q_heads : 0;
    p.kv_heads = cfg->kv_heads;
    p.num_tokens = num_tokens;
    p.pairs = cfg->rotary_dim / 2;
    p.interleaved = cfg->interleaved;
    const int rounds =
        ((p.q_heads + 2 * p.kv_heads) * (cfg->head_dim / 16) + 31) / 32;  // of a whole token
    // A warp that takes a whole token makes its sines once and keeps its loads
    // ahead of its stores, one that takes a round of it leaves more warps for
    // few tokens.  Measured (us, a round | a token of 10 or 12): 256 tokens
    // 4.2 | 7.1, 16k tokens 75 | 53.  So rounds grow once two full sets of
    // resident warps have one each.
    const long long most =
        (long long)kda_cache::sm_count() * ctas_per_sm(cfg->head_dim, norm != nullptr) * kWarps * 2;
    if (most <= 0) return KDA_ERR_CUDA;
    const long long wanted = (long long)num_tokens * rounds / most;
    p.rounds = wanted < 1 ? 1 : wanted > rounds ? rounds : (int)wanted;
    p.parts = (rounds + p.rounds - 1) / p.rounds;
    const long long items = (long long)num_tokens * p.parts;
    const long long token_blocks = (items + kWarps - 1) / kWarps;
    // CTAs of their own check the rows, each once, a thread a row: a row that is
    // wrong may have no token that leads to it, and where it has, every warp of
    // its tokens would report it.
    const long long grid =
        token_blocks + (error_word != nullptr ? ((long long)B + kThreads - 1) / kThreads : 0);
    if (grid > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    p.token_blocks = (int)token_blocks;
    void (*kernel)(const Params) =
        norm != nullptr ? kernel_for<true>(cfg->dtype == KDA_DTYPE_BF16, cfg->head_dim == 64)
                        : kernel_for<false>(cfg->dtype == KDA_DTYPE_BF16, cfg->head_dim == 64);
    return kda_cache::launch(kernel, dim3((unsigned)grid), dim3(kThreads), 0, 1, stream, p);
}

}  // namespace

extern "C" kda_status kda_kv_append(const kda_cache_config *cfg, const void *q, const void *k,
                                    const void *v, void *q_out, void *key_cache,
                                    void *value_cache, const double *inv_freq,
                                    const int32_t *cu_seqlens, int32_t B, int32_t num_tokens,
                                    const kda_align *align, int32_t *error_word, void *stream) {
    return append(cfg, q, k, v, q_out, key_cache, value_cache, inv_freq, cu_seqlens, B, num_tokens,
                  align, error_word, stream, nullptr);
}

extern "C" kda_status kda_kv_norm_append(const kda_cache_config *cfg, const void *q, const void *k,
                                         const void *v, const void *q_weight, const void *k_weight,
                                         int32_t weight_dtype, float eps, void *q_out,
                                         void *key_cache, void *value_cache,
                                         const double *inv_freq, const int32_t *cu_seqlens,
                                         int32_t B, int32_t num_tokens, const kda_align *align,
                                         int32_t *error_word, void *stream) {
    const Norm norm{q_weight, k_weight, weight_dtype, eps};
    return append(cfg, q, k, v, q_out, key_cache, value_cache, inv_freq, cu_seqlens, B, num_tokens,
                  align, error_word, stream, &norm);
}

extern "C" kda_status kda_kv_norm_append_packed(const kda_norm_append_args *n) {
    if (n == nullptr) return KDA_ERR_INVALID_ARG;
    const kda_append_args *a = &n->append;
    return kda_kv_norm_append(&a->config, a->q, a->k, a->v, n->q_weight, n->k_weight,
                              n->weight_dtype, n->eps, a->q_out, a->key_cache, a->value_cache,
                              a->inv_freq, a->cu_seqlens, a->B, a->num_tokens, &a->align,
                              a->error_word, a->stream);
}

extern "C" kda_status kda_kv_append_packed(const kda_append_args *a) {
    if (a == nullptr) return KDA_ERR_INVALID_ARG;
    return kda_kv_append(&a->config, a->q, a->k, a->v, a->q_out, a->key_cache, a->value_cache,
                         a->inv_freq, a->cu_seqlens, a->B, a->num_tokens, &a->align, a->error_word,
                         a->stream);
}
