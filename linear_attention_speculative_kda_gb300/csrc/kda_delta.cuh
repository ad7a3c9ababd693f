// Rows of the delta rule's own calls (kda_prefill, kda_decode): metadata,
// host checks and the parameters they share (sm_103a).  Contracts in
// include/kda.h.
#pragma once

#include "kda_cache.cuh"
#include "kda_device.cuh"

namespace kda_delta {

using kda::kD;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kTile = kD * kD;   // elements of a head's state

struct Params {
    const __nv_bfloat16 *q, *k, *v, *g, *beta;
    long long stride_q, stride_k, stride_v, stride_g, stride_beta;   // elements
    const float *A_log, *g_bias;
    float *pool;
    const int *cu_seqlens;   // nullptr: one token a row
    const int *state_indices, *initial_indices;
    __nv_bfloat16 *out;
    int *err;
    int H, S, B, num_tokens;
    int bounded;
    float lower_bound, scale;
    int least, most;   // token counts of the rows that the kernel takes
};

struct Row {
    int first, tokens;   // first token, token count (0: nothing to do)
    int from, to;        // slots of the state before (<= 0: none, zeros) and after
};

// Row b, checked; `bits` collects what is wrong with it (the row is then
// empty).
__device__ __forceinline__ Row read_row(const Params &p, int b, int &bits) {
    const int to = p.state_indices[b];
    const int from = p.initial_indices != nullptr ? p.initial_indices[b] : to;
    int first = b, end = b + 1;
    if (p.cu_seqlens != nullptr) {
        first = p.cu_seqlens[b];
        end = p.cu_seqlens[b + 1];
    }
    Row row{first, 0, from, to};
    const long long n = (long long)end - first;
    if (to <= 0 || n == 0) return row;   // padding, or nothing new
    if (n < 0 || first < 0 || end > p.num_tokens)
        bits |= KDA_ROW_BAD_LENGTH;
    else if (to >= p.S || from >= p.S)
        bits |= KDA_ROW_BAD_SLOT;
    else if (n >= p.least && n <= p.most)
        row.tokens = (int)n;
    return row;
}

// ------------------------------------------------------------------- host --

// The rows of p.least to p.most tokens, token by token (kda_decode.cu).
kda_status launch_recurrent(const Params &p, void *stream);

inline kda_status set_params(const kda_config *c, const void *q, const void *k, const void *v,
                             const void *g_raw, const void *beta_raw, const float *A_log,
                             const float *g_bias, float *pool, const int32_t *state_indices,
                             const int32_t *initial_indices, int32_t B, int32_t num_tokens,
                             void *out, int32_t *error_word, Params &p) {
    using kda_cache::aligned;
    if (!q || !k || !v || !g_raw || !beta_raw || !A_log || !g_bias || !pool || !state_indices ||
        !out)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 8) || !aligned(k, 8) || !aligned(v, 8) || !aligned(g_raw, 8) ||
        !aligned(beta_raw, 2) || !aligned(A_log, 4) || !aligned(g_bias, 16) || !aligned(pool, 16) ||
        !aligned(state_indices, 4) || !aligned(initial_indices, 4) || !aligned(out, 16) ||
        !aligned(error_word, 4))
        return KDA_ERR_INVALID_ARG;
    for (const int64_t s : {c->stride_q_t, c->stride_k_t, c->stride_v_t, c->stride_g_t})
        if (s < 1 || (s & 3) != 0) return KDA_ERR_INVALID_ARG;
    if (c->stride_beta_t < 1) return KDA_ERR_INVALID_ARG;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.g = static_cast<const __nv_bfloat16 *>(g_raw);
    p.beta = static_cast<const __nv_bfloat16 *>(beta_raw);
    p.stride_q = c->stride_q_t;
    p.stride_k = c->stride_k_t;
    p.stride_v = c->stride_v_t;
    p.stride_g = c->stride_g_t;
    p.stride_beta = c->stride_beta_t;
    p.A_log = A_log;
    p.g_bias = g_bias;
    p.pool = pool;
    p.state_indices = state_indices;
    p.initial_indices = initial_indices;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.err = error_word;
    p.H = c->num_heads;
    p.S = c->num_slots;
    p.B = B;
    p.num_tokens = num_tokens;
    p.bounded = c->use_lower_bound;
    p.lower_bound = c->lower_bound;
    p.scale = c->scale;
    p.least = 1;
    p.most = 0x7fffffff;
    return KDA_OK;
}

// The parts of the config that these calls read (its window and records are
// the verify's).
inline kda_status check_config(const kda_config *c) {
    if (c == nullptr || c->num_heads < 1 || c->num_slots < 1 || c->reserved != 0)
        return KDA_ERR_INVALID_ARG;
    if (c->head_dim != KDA_HEAD_DIM || c->num_heads > KDA_MAX_HEADS) return KDA_ERR_UNSUPPORTED;
    if (c->use_lower_bound != 0 && c->use_lower_bound != 1) return KDA_ERR_INVALID_ARG;
    if (c->use_lower_bound == 1 && !(c->lower_bound < 0.0f && isfinite(c->lower_bound)))
        return KDA_ERR_INVALID_ARG;
    return isfinite(c->scale) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

}  // namespace kda_delta
