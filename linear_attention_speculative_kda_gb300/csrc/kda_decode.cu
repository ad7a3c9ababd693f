// kda_decode: the gated delta rule for one token a row, and kda_prefill's rows
// of a few tokens, token by token (sm_103a).  Contracts in include/kda.h.
//
// Mathematics, a head's state S [V, K] and a token:
//   S' = S diag(e),  u = S' k^,  v' = beta (v - u),  S <- S' + v' k^T,  o = S q^.
// With z = S' q^ the output is o = z + v' (k^ . q^), so both products of a
// token read S' and one round of sums serves them.
//
// HBM bounds the call: the state once each way.  Rows of S (values' channels)
// do not meet, so a CTA has half of the rows of one head of one row, 32 KiB in
// registers: lane 8 g + j of warp w has the rows 16 w + 4 g + i and of each the
// columns 32 m + 4 j + c (i, m, c = 0..3), so a load or store of a warp moves
// whole 128-byte lines and a row's sums stay in 8 lanes.  All its loads are
// issued before the token's vectors are made, and the four CTAs of an SM start
// and end at different times: 1024 rows x 16 heads take 325 us (99% of the
// measured copy rate), 357 with a whole head a CTA and two of them an SM, 332
// with a quarter.  Loads that are not marked to leave the caches first took 318
// there, but 45 us for 64 rows x 32 heads and not 44.
#include "kda_delta.cuh"

namespace {

using kda_delta::kD;
using kda_delta::kFull;
using kda_delta::Params;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

struct Token {
    float q[kD], k[kD], e[kD], v[kD];
};

__device__ __forceinline__ float sum8(float x) {  // over the 8 lanes of a row
    x += __shfl_xor_sync(kFull, x, 4);
    x += __shfl_xor_sync(kFull, x, 2);
    return x + __shfl_xor_sync(kFull, x, 1);
}

__global__ void __launch_bounds__(kThreads, 4) recurrent_kernel(const Params p) {
    __shared__ __align__(16) Token token;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = blockIdx.x & 1, tile = blockIdx.x >> 1;
    const int b = tile / p.H, h = tile % p.H;
    kda_cache::grid_dependents_launch();
    kda_cache::grid_dependency_wait();
    int bits = 0;
    const kda_delta::Row row = kda_delta::read_row(p, b, bits);
    if (bits != 0 && h == 0 && half == 0 && tid == 0) kda_cache::flag(p.err, bits);
    if (row.tokens == 0) return;
    const int r0 = 64 * half + 16 * warp + 4 * (lane >> 3), c0 = 4 * (lane & 7);
    float4 s[4][4];
    if (row.from > 0) {
        const float *src =
            p.pool + ((long long)row.from * p.H + h) * kda_delta::kTile + r0 * kD + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m)
                s[i][m] = __ldcs(reinterpret_cast<const float4 *>(src + i * kD + 32 * m));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m) s[i][m] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    const float a = __expf(p.A_log[h]);
    for (int n = 0; n < row.tokens; ++n) {
        const long long t = row.first + n;
        // a warp each: q and k normalised, the decays, v; four channels a lane
        {
            const __nv_bfloat16 *src = warp == 0   ? p.q + t * p.stride_q
                                       : warp == 1 ? p.k + t * p.stride_k
                                       : warp == 2 ? p.g + t * p.stride_g
                                                   : p.v + t * p.stride_v;
            float4 x = kda::bf16x4_to_float4(
                __ldg(reinterpret_cast<const uint2 *>(src + (long long)h * kD + 4 * lane)));
            if (warp < 2) {
                const float r = kda::inv_l2(kda::warp_allsum(kda::dot4(x, x)));
                x = make_float4(x.x * r, x.y * r, x.z * r, x.w * r);
            } else if (warp == 2) {
                const float4 bias = kda::ld4(p.g_bias + (long long)h * kD + 4 * lane);
                x = make_float4(
                    kda::decay_factor(x.x + bias.x, a, p.bounded, p.lower_bound),
                    kda::decay_factor(x.y + bias.y, a, p.bounded, p.lower_bound),
                    kda::decay_factor(x.z + bias.z, a, p.bounded, p.lower_bound),
                    kda::decay_factor(x.w + bias.w, a, p.bounded, p.lower_bound));
            }
            float *dst = warp == 0 ? token.q : warp == 1 ? token.k : warp == 2 ? token.e : token.v;
            *reinterpret_cast<float4 *>(dst + 4 * lane) = x;
        }
        const float beta = kda::sigmoidf_rn(__bfloat162float(p.beta[t * p.stride_beta + h]));
        __syncthreads();
        float u[4] = {}, z[4] = {}, kq = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 e = kda::ld4(token.e + c0 + 32 * m), k = kda::ld4(token.k + c0 + 32 * m);
            const float4 q = kda::ld4(token.q + c0 + 32 * m);
            kq += kda::dot4(k, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i][m] = kda::mul4(s[i][m], e);
                u[i] += kda::dot4(s[i][m], k);
                z[i] += kda::dot4(s[i][m], q);
            }
        }
        kq = sum8(kq);
        float o = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float d = beta * (token.v[r0 + i] - sum8(u[i]));
            const float y = sum8(z[i]) + d * kq;
            if ((lane & 7) == i) o = y;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float4 k = kda::ld4(token.k + c0 + 32 * m);
                s[i][m].x = fmaf(d, k.x, s[i][m].x);
                s[i][m].y = fmaf(d, k.y, s[i][m].y);
                s[i][m].z = fmaf(d, k.z, s[i][m].z);
                s[i][m].w = fmaf(d, k.w, s[i][m].w);
            }
        }
        if ((lane & 7) < 4)
            p.out[(t * p.H + h) * kD + r0 + (lane & 7)] = __float2bfloat16_rn(o * p.scale);
        __syncthreads();
    }
    float *dst = p.pool + ((long long)row.to * p.H + h) * kda_delta::kTile + r0 * kD + c0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m)
            __stcs(reinterpret_cast<float4 *>(dst + i * kD + 32 * m), s[i][m]);
}

}  // namespace

kda_status kda_delta::launch_recurrent(const Params &p, void *stream) {
    const long long tiles = (long long)p.B * p.H;
    if (tiles > 0x3fffffffLL) return KDA_ERR_UNSUPPORTED;
    return kda_cache::launch(recurrent_kernel, dim3((unsigned)(2 * tiles)), dim3(kThreads), 0, 1,
                             stream, p);
}

extern "C" kda_status kda_decode(const kda_config *cfg, const void *q, const void *k,
                                 const void *v, const void *g_raw, const void *beta_raw,
                                 const float *A_log, const float *g_bias, float *state_pool,
                                 const int32_t *state_indices, const int32_t *initial_indices,
                                 int32_t B, void *out, int32_t *error_word, void *stream) {
    kda_status st = kda_delta::check_config(cfg);
    if (st != KDA_OK) return st;
    if (B < 0) return KDA_ERR_INVALID_ARG;
    if (B == 0) return KDA_OK;  // nothing to do; no pointer is inspected
    Params p{};
    st = kda_delta::set_params(cfg, q, k, v, g_raw, beta_raw, A_log, g_bias, state_pool,
                               state_indices, initial_indices, B, B, out, error_word, p);
    return st != KDA_OK ? st : kda_delta::launch_recurrent(p, stream);
}

extern "C" kda_status kda_decode_packed(const kda_delta_args *a) {
    if (a == nullptr) return KDA_ERR_INVALID_ARG;
    return kda_decode(&a->config, a->q, a->k, a->v, a->g_raw, a->beta_raw, a->A_log, a->g_bias,
                      a->state_pool, a->state_indices, a->initial_indices, a->B, a->out,
                      a->error_word, a->stream);
}
