// kda_kv_append: rotate the new tokens' queries and keys by position and
// write keys and values to the paged cache (sm_103a).  Contract in
// include/kda.h.
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

// With 64 registers a thread for heads of 128 channels and 48 for 64.  Measured
// (us, 4 | 5 CTAs an SM): 256 tokens 4.2 | 4.9 and 13.7k tokens 45 | 48 with
// 128 channels (16k interleaved ones 53 | 51), 10k tokens 7.4 | 6.8 and 56k
// tokens 22 | 20 with 64.
constexpr int ctas_per_sm(int dim) { return dim == 128 ? 4 : 5; }

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

// 8 pairs of one head: chunk a and chunk b hold them as halves (a[e], b[e])
// or side by side (a[2e], a[2e+1], then b).
template <typename T>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float2 *turn, bool interleaved) {
    uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 p = unpack(x[i], T()), r = unpack(y[i], T());
        if (interleaved) {
            const float2 s = turn[i], t = turn[4 + i];
            p = make_float2(p.x * s.x - p.y * s.y, p.x * s.y + p.y * s.x);
            r = make_float2(r.x * t.x - r.y * t.y, r.x * t.y + r.y * t.x);
        } else {
            const float2 s = turn[2 * i], t = turn[2 * i + 1];
            const float2 u = p;
            p = make_float2(u.x * s.x - r.x * s.y, u.y * t.x - r.y * t.y);
            r = make_float2(u.x * s.y + r.x * s.x, u.y * t.y + r.y * t.x);
        }
        x[i] = pack(p.x, p.y, T());
        y[i] = pack(r.x, r.y, T());
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

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kDim)) append_kernel(const Params p) {
    constexpr int kUnits = kDim / 16;  // units of a head
    __shared__ float2 turns[kWarps][kMaxPairs];
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
    if (t >= p.num_tokens) return;
    const int first_k = p.q_heads, first_v = p.q_heads + p.kv_heads;
    const int begin = part * p.rounds * 32;
    const int end = min((first_v + p.kv_heads) * kUnits, begin + p.rounds * 32);

    auto load = [&](int u, uint4 &x, uint4 &y) {
        if (u >= end) return;
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
        turns[warp][i] = cs;
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
        if (turned) rotate<T>(x, y, &turns[warp][j * 8], p.interleaved != 0);
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

}  // namespace

extern "C" kda_status kda_kv_append(const kda_cache_config *cfg, const void *q, const void *k,
                                    const void *v, void *q_out, void *key_cache,
                                    void *value_cache, const double *inv_freq,
                                    const int32_t *cu_seqlens, int32_t B, int32_t num_tokens,
                                    const kda_align *align, int32_t *error_word, void *stream) {
    using kda_cache::aligned;
    using kda_cache::stride_ok;
    kda_status st = kda_cache::check_config(cfg);
    if (st != KDA_OK) return st;
    if (B < 0 || num_tokens < 0) return KDA_ERR_INVALID_ARG;
    if (cfg->rotary_dim < 0 || cfg->rotary_dim > cfg->head_dim || (cfg->rotary_dim & 15) != 0 ||
        (cfg->interleaved != 0 && cfg->interleaved != 1))
        return KDA_ERR_INVALID_ARG;
    if (B == 0 || num_tokens == 0) return KDA_OK;  // nothing to do; no pointer is inspected
    Params p;
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
        (long long)kda_cache::sm_count() * ctas_per_sm(cfg->head_dim) * kWarps * 2;
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
        cfg->dtype == KDA_DTYPE_BF16
            ? (cfg->head_dim == 64 ? append_kernel<__nv_bfloat16, 64>
                                   : append_kernel<__nv_bfloat16, 128>)
            : (cfg->head_dim == 64 ? append_kernel<__half, 64> : append_kernel<__half, 128>);
    return kda_cache::launch(kernel, dim3((unsigned)grid), dim3(kThreads), 0, 1, stream, p);
}

extern "C" kda_status kda_kv_append_packed(const kda_append_args *a) {
    if (a == nullptr) return KDA_ERR_INVALID_ARG;
    return kda_kv_append(&a->config, a->q, a->k, a->v, a->q_out, a->key_cache, a->value_cache,
                         a->inv_freq, a->cu_seqlens, a->B, a->num_tokens, &a->align, a->error_word,
                         a->stream);
}
