// kda_prefill: the gated delta rule over rows of any length, chunked
// (sm_103a).  Contract in include/kda.h.
//
// Mathematics.  A head's state S [V, K], a chunk of C = 16 tokens, e_t the
// token's decays, P_t = prod_{i<=t} e_i within the chunk, all norms taken:
//   A_ts = sum_c k_t k_s prod_{s<i<=t} e_i   (s < t)
//   B_ts = sum_c q_t k_s prod_{s<i<=t} e_i   (s <= t)
//   T    = (1 + diag(beta) A)^-1 diag(beta)                      [C, C]
//   V'   = T (V - (K P) S^T),   O = (Q P) S^T + B V'
//   S   <- S diag(P_C) + V'^T (K P_C / P_t)
// All factors are products of decays behind one another, never quotients, so
// none is above 1 and strong decays underflow to what they are.
//
// Every product with S and V' runs on mma.sync m16n8k16 in fp16 with fp32
// sums.  An fp32 operand x is two fp16 numbers, hi = fp16(x) and lo =
// fp16(x - hi), 22 bits, and a product is hi hi + hi lo + lo hi: what is left
// out is below 2^-22 of it.  Only O takes hi alone: it is rounded to bf16,
// 2^-9, anyway.  Decayed keys and queries are at most 1 and scaled by powers of
// two; the rows of S and V, whose sizes are the caller's, are held times a
// power of two of their own that puts the larger of the two near 2^7, as
// fp16's range needs it.
//
// Layout.  Rows of S (values' channels) never meet each other, so a consumer
// warp owns 16 of them and all 128 columns as the fp32 accumulators of 16
// n-tiles, for the whole row: no exchange between warps, and an accumulator
// pair is an operand pair of the next product.  The operands that all rows
// share (K P, Q P, K P_C / P_t, T, B, P_C) are made by producer warps, a chunk
// each, in fragment order in a ring of stages.  Tokens of a chunk are numbered
// for the products in the order 0 7 1 6 2 5 3 4, 8 15 9 14 ...: a lane of the
// producer that steps along the chunk has four tokens, {g, 7 - g, 8 + g, 15 - g},
// whose work is then equal, and they are a lane's pairs of the fragments.
#include <cuda_fp16.h>

#include "kda_delta.cuh"

namespace {

using kda_cache::add_pair;
using kda_cache::both;
using kda_cache::fma_pair;
using kda_cache::mul_pair;
using kda_cache::pair;
using kda_delta::kD;
using kda_delta::kFull;
using kda_delta::Params;
using kda_delta::Row;
typedef unsigned long long u64;

constexpr int kC = 16;           // tokens of a chunk
constexpr int kProducers = 4;    // warps, one a sub-core
constexpr int kStages = 6;
constexpr int kMaxConsumers = 8; // warps of 16 rows of S
constexpr int kMaxThreads = 32 * (kProducers + kMaxConsumers);

#ifdef KDA_TEST_PREFILL_WAIT_BUDGET  // a test build: a wait that runs out, soon
constexpr long long kWaitBudget = KDA_TEST_PREFILL_WAIT_BUDGET;
#else
constexpr long long kWaitBudget = 4000000000LL;   // clock cycles (about 2 s)
#endif

// Powers of two on the operands: products of S with keys and queries carry
// kKeyScale, V' and the keys that update S carry inverse ones.
constexpr float kKeyScale = 1024.0f;      // K P, Q P
constexpr float kTScale = 1024.0f;        // T
constexpr float kUpdateScale = 32.0f;     // K P_C / P_t; V' carries 1 / 32
constexpr float kBScale = 32768.0f;       // B: kKeyScale * 32

// One chunk's operands, in fragment order (16 bytes a lane).
constexpr int kKeyStep = 1024 + 64;       // bytes of a k step of K P, padded against bank conflicts
constexpr int kQueryStep = 512 + 64;
struct __align__(128) Stage {
    unsigned char key[8 * kKeyStep];      // [k step][n tile][lane]: hi b0 b1, lo b0 b1
    unsigned char query[8 * kQueryStep];  // [k step][lane]: n tile 0 b0 b1, 1 b0 b1
    uint4 update[16][32];                 // [n tile][slot]: hi b0 b1, lo b0 b1
    uint4 t[2][32];                       // [n tile][lane]: hi b0 b1, lo b0 b1
    uint4 b[32];                          // [lane]: n tile 0 b0 b1, 1 b0 b1
    float decay[kD];                      // P_C
    uint4 v[kC][16];                      // bf16 [token][channel], 16-byte units swizzled
};

struct __align__(16) Scratch {            // of a producer warp
    float e[4][kD], k[4][kD], q[4][kD];   // four tokens
    float a[kC][kC + 4], b[kC][kC + 4];
    float beta[kC];
};

struct Shared {
    Stage stage[kStages];
    Scratch scratch[kProducers];
    unsigned char out[kMaxConsumers][kC * 48];
    uint64_t full[kStages], empty[kStages];
    int gave_up;
};

// The place of token t in the products' order, and the token at a place.
__host__ __device__ constexpr int place_of(int t) {
    return (t & 8) + ((t & 7) < 4 ? 2 * (t & 7) : 2 * (7 - (t & 7)) + 1);
}
__device__ __forceinline__ int token_at(int n) {
    return (n & 8) + ((n & 1) ? 7 - ((n & 7) >> 1) : (n & 7) >> 1);
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half_pair(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// x and y as pairs of fp16: the numbers, and what is left of them.
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = half_pair(x, y);
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    lo = half_pair(x - h.x, y - h.y);
}

// Bounded wait of a warp: it gives up, as a whole, after the budget, or when
// another warp has.
__device__ __forceinline__ bool wait(Shared &sh, uint64_t *bar, uint32_t parity, int *err) {
    bool done = kda::mbar_try_wait(bar, parity);
    if (!done) {
        const long long t0 = clock64();
        while (!(done = kda::mbar_try_wait(bar, parity))) {
            if (*reinterpret_cast<volatile int *>(&sh.gave_up) != 0) break;
            if (clock64() - t0 > kWaitBudget) {
                *reinterpret_cast<volatile int *>(&sh.gave_up) = 1;
                kda_cache::flag(err, KDA_ERR_WAIT_TIMEOUT);
                break;
            }
        }
    }
    return __all_sync(kFull, done);
}

struct Work {   // one row and head's share of a CTA
    Row row;
    int head, part;
};

__device__ __forceinline__ Work work_at(const Params &p, long long item, int parts, int &bits) {
    Work w;
    w.part = (int)(item % parts);
    const long long tile = item / parts;
    w.head = (int)(tile % p.H);
    w.row = kda_delta::read_row(p, (int)(tile / p.H), bits);
    return w;
}

// ---------------------------------------------------------------- producer --

// 2^x, within 2 ulp, 0 far below.
__device__ __forceinline__ float exp2_of(float x) { return kda_cache::exp2_fast(x); }

constexpr float kLog2e = 1.4426950408889634f;

// The decays of two channels, exp(g): as kda::decay_factor, two at a time.
// x: gate inputs with their bias; gate: -exp(A_log) log2 e for the softplus
// gate, and for the bounded one.
template <bool kBounded>
__device__ __forceinline__ u64 decays(u64 x, float gate, float bound) {
    const float2 v = both(x);
    if constexpr (kBounded) {
        // bound / (1 + exp(-a x)), in powers of two
        const float2 y = both(mul_pair(x, pair(gate, gate)));
        const float2 g = make_float2(__fdividef(bound, 1.0f + exp2_of(y.x)),
                                     __fdividef(bound, 1.0f + exp2_of(y.y)));
        return pair(exp2_of(g.x), exp2_of(g.y));
    } else {
        // softplus(x) = max(x, 0) + log1p(z), z = exp(-|x|); log1p(z) = z P(z)
        // with the polynomial of kda::softplus
        constexpr float c[10] = {0x1p+0f,        -0x1.ffffcp-2f,  0x1.554c9cp-2f, -0x1.ff11c2p-3f,
                                 0x1.930202p-3f, -0x1.399642p-3f, 0x1.b2c2a2p-4f, -0x1.d3784ep-5f,
                                 0x1.4628bp-6f,  -0x1.aad1eep-9f};
        const u64 z = pair(exp2_of(-fabsf(v.x) * kLog2e), exp2_of(-fabsf(v.y) * kLog2e));
        u64 r = pair(c[9], c[9]);
#pragma unroll
        for (int i = 8; i >= 0; --i) r = fma_pair(r, z, pair(c[i], c[i]));
        const u64 sp = fma_pair(z, r, pair(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
        const float2 g = both(mul_pair(sp, pair(gate, gate)));
        return pair(exp2_of(g.x), exp2_of(g.y));
    }
}

struct Raw {   // four tokens' channels 4 lane .. 4 lane + 3
    uint2 q[4], k[4], g[4];
};

__device__ __forceinline__ void load_raw(const Params &p, Raw &raw, long long first, int valid,
                                         long long at) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const long long t = first + u;
        raw.q[u] = raw.k[u] = raw.g[u] = make_uint2(0u, 0u);
        if (u < valid) {
            raw.q[u] = __ldg(reinterpret_cast<const uint2 *>(p.q + t * p.stride_q + at));
            raw.k[u] = __ldg(reinterpret_cast<const uint2 *>(p.k + t * p.stride_k + at));
            raw.g[u] = __ldg(reinterpret_cast<const uint2 *>(p.g + t * p.stride_g + at));
        }
    }
}

__device__ __forceinline__ void pairs_of(uint2 x, u64 &a, u64 &b) {
    const float4 f = kda::bf16x4_to_float4(x);
    a = pair(f.x, f.y);
    b = pair(f.z, f.w);
}

// Sums 8 values over lanes 8 i .. 8 i + 7 of a warp: lane l ends with the sum
// of value l & 7 over its 8 lanes.
__device__ __forceinline__ float reduce8(float (&x)[8], int lane) {
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) {
        const bool upper = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = upper ? x[i] : x[i + w];
            const float keep = upper ? x[i + w] : x[i];
            x[i] = keep + __shfl_xor_sync(kFull, send, w);
        }
    }
    return x[0];
}

template <bool kBounded>
__device__ __forceinline__ void produce(const Params &p, Stage &st, Scratch &sc, const Row &row,
                                        int head, int chunk, int lane) {
    const long long first = (long long)row.first + (long long)chunk * kC;
    const int valid = min(kC, row.tokens - chunk * kC);
    const long long at = (long long)head * kD + 4 * lane;
    Raw raw;
    load_raw(p, raw, first, valid, at);
    // the values as they are
#pragma unroll
    for (int t = 0; t < kC; ++t) {
        unsigned char *dst = reinterpret_cast<unsigned char *>(&st.v[t][(lane >> 1) ^ (t & 7)]) +
                             (lane & 1) * 8;
        if (t < valid)
            kda::cp_async8(dst, p.v + (first + t) * p.stride_v + at);
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(0u, 0u);
    }
    kda::cp_async_commit();
    if (lane < kC)
        sc.beta[lane] =
            lane < valid ? kda::sigmoidf_rn(__bfloat162float(
                               p.beta[(first + lane) * p.stride_beta + head]))
                         : 0.0f;
    const float a = __expf(p.A_log[head]);
    const float gate = -a * kLog2e, bound = p.lower_bound * kLog2e;
    u64 bias[2];
    {
        const float4 f = kda::ld4(p.g_bias + at);
        bias[0] = pair(f.x, f.y);
        bias[1] = pair(f.z, f.w);
    }
    const int group = lane >> 3, sub = lane & 7;   // tokens and channels of the steps along the chunk
    u64 w[4][8];                                   // [slot][channel pair]: k_s prod_{s<i<=t} e_i
    u64 reach[2] = {pair(kKeyScale, kKeyScale), pair(kKeyScale, kKeyScale)};   // P_t
#pragma unroll
    for (int block = 0; block < 4; ++block) {
        Raw now = raw;
        if (block < 3) load_raw(p, raw, first + 4 * (block + 1), valid - 4 * (block + 1), at);
        // norms of four tokens
        float sums[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            u64 x, y;
            pairs_of(now.k[u], x, y);
            float2 s = both(fma_pair(x, x, mul_pair(y, y)));
            sums[u] = s.x + s.y;
            pairs_of(now.q[u], x, y);
            s = both(fma_pair(x, x, mul_pair(y, y)));
            sums[4 + u] = s.x + s.y;
        }
        float norm = reduce8(sums, lane);
        norm += __shfl_xor_sync(kFull, norm, 8);
        norm += __shfl_xor_sync(kFull, norm, 16);
        norm = kda::inv_l2(norm);
        __syncwarp();   // the block before has been read
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = 4 * block + u;
            const float rk = __shfl_sync(kFull, norm, u), rq = __shfl_sync(kFull, norm, 4 + u);
            u64 e[2], k[2], q[2];
            pairs_of(now.g[u], e[0], e[1]);
            pairs_of(now.k[u], k[0], k[1]);
            pairs_of(now.q[u], q[0], q[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // tokens behind the row's end do not decay
                e[i] = t < valid ? decays<kBounded>(add_pair(e[i], bias[i]), gate, bound)
                                 : pair(1.0f, 1.0f);
                reach[i] = mul_pair(reach[i], e[i]);
                k[i] = mul_pair(k[i], pair(rk, rk));
                q[i] = mul_pair(q[i], pair(rq, rq));
            }
            *reinterpret_cast<ulonglong2 *>(&sc.e[u][4 * lane]) = make_ulonglong2(e[0], e[1]);
            *reinterpret_cast<ulonglong2 *>(&sc.k[u][4 * lane]) = make_ulonglong2(k[0], k[1]);
            *reinterpret_cast<ulonglong2 *>(&sc.q[u][4 * lane]) = make_ulonglong2(q[0], q[1]);
            // K P and Q P: channels 4 lane .. + 3 are b0 and b1 of k step lane / 4
            constexpr int kTiles = 2;
            const int n = place_of(t) & 7, tile = place_of(t) >> 3;
            const int slot = n * 4 + (lane & 3);
            uint4 f;
            float2 x = both(mul_pair(k[0], reach[0]));
            split(x.x, x.y, f.x, f.z);
            x = both(mul_pair(k[1], reach[1]));
            split(x.x, x.y, f.y, f.w);
            *reinterpret_cast<uint4 *>(st.key + (lane >> 2) * kKeyStep + (tile * 32 + slot) * 16) =
                f;
            uint2 h;
            x = both(mul_pair(q[0], reach[0]));
            h.x = half_pair(x.x, x.y);
            x = both(mul_pair(q[1], reach[1]));
            h.y = half_pair(x.x, x.y);
            *reinterpret_cast<uint2 *>(st.query + (lane >> 2) * kQueryStep +
                                       (slot * kTiles + tile) * 8) = h;
        }
        __syncwarp();
        // along the block: slot i's token is s, its channels 32 m + 4 sub + 0..3
#pragma unroll
        for (int i = 0; i <= block; ++i) {
            const int s = (i & 1) ? 8 * (i >> 1) + 7 - group : 8 * (i >> 1) + group;
            float x[8];   // (A, B) of four tokens
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                u64 sa = pair(0.0f, 0.0f), sb = sa;
                const u64 starts = i == block && 4 * block + u == s ? pair(1.0f, 1.0f)
                                                                    : pair(0.0f, 0.0f);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int c = 32 * m + 4 * sub;
                    const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(&sc.e[u][c]);
                    const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(&sc.k[u][c]);
                    const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(&sc.q[u][c]);
                    u64 &w0 = w[i][2 * m], &w1 = w[i][2 * m + 1];
                    if (i == block) {   // the token itself lies in this block
                        w0 = u == 0 ? mul_pair(k.x, starts)
                                    : fma_pair(k.x, starts, mul_pair(w0, e.x));
                        w1 = u == 0 ? mul_pair(k.y, starts)
                                    : fma_pair(k.y, starts, mul_pair(w1, e.y));
                    } else {
                        w0 = mul_pair(w0, e.x);
                        w1 = mul_pair(w1, e.y);
                    }
                    sa = fma_pair(k.x, w0, sa);
                    sa = fma_pair(k.y, w1, sa);
                    sb = fma_pair(q.x, w0, sb);
                    sb = fma_pair(q.y, w1, sb);
                }
                float2 f = both(sa);
                x[2 * u] = f.x + f.y;
                f = both(sb);
                x[2 * u + 1] = f.x + f.y;
            }
            const float sum = reduce8(x, lane);
            (sub & 1 ? sc.b : sc.a)[4 * block + (sub >> 1)][s] = sum;
        }
    }
    // P_C
    {
        const u64 back = pair(1.0f / kKeyScale, 1.0f / kKeyScale);
        *reinterpret_cast<ulonglong2 *>(&st.decay[4 * lane]) =
            make_ulonglong2(mul_pair(reach[0], back), mul_pair(reach[1], back));
    }
    // K P_C / P_t: tokens (group, 7 - group) and (8 + group, 15 - group) are b0 and b1
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = both(mul_pair(w[i][2 * m + h], pair(kUpdateScale, kUpdateScale)));
                x[i][0] = f.x;
                x[i][1] = f.y;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint4 f;
                split(x[0][u], x[1][u], f.x, f.z);
                split(x[2][u], x[3][u], f.y, f.w);
                // channel 32 m + 4 sub + 2 h + u
                const int tile = 2 * (2 * m + (sub >> 2)) + h, line = sub & 3;
                st.update[tile][line * 8 + ((u * 4 + group) ^ (line | ((tile >> 1) & 1) << 2))] =
                    f;
            }
        }
    __syncwarp();
    // T, column lane & 15 in a lane: T_t = beta_t (1_t - sum_{j<t} A_tj T_j)
    {
        const int s = lane & 15;
        float col[kC];
#pragma unroll
        for (int t = 0; t < kC; ++t) {
            float x = t == s ? 1.0f : 0.0f, y = 0.0f;
#pragma unroll
            for (int j = 0; j < t; ++j) {
                const float n = sc.a[t][j];
                if (j & 1)
                    y = fmaf(-n, col[j], y);
                else
                    x = fmaf(-n, col[j], x);
            }
            col[t] = sc.beta[t] * (x + y);
        }
        __syncwarp();
        if (lane < 16)
#pragma unroll
            for (int t = 0; t < kC; ++t) sc.a[t][s] = col[t] * kTScale;
    }
    __syncwarp();
    {
        const int j = lane & 3, g = lane >> 2;
        uint4 f;
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
            const int t = token_at(8 * tile + g);
            uint4 x;
            split(sc.a[t][j], sc.a[t][7 - j], x.x, x.z);
            split(sc.a[t][8 + j], sc.a[t][15 - j], x.y, x.w);
            st.t[tile][lane] = x;
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = (i & 1) ? 8 * (i >> 1) + 7 - j : 8 * (i >> 1) + j;
                y[i] = s <= t ? sc.b[t][s] * kBScale : 0.0f;
            }
            (tile ? f.z : f.x) = half_pair(y[0], y[1]);
            (tile ? f.w : f.y) = half_pair(y[2], y[3]);
        }
        st.b[lane] = f;
    }
    kda::cp_async_wait_all();
    __syncwarp();
}

// ---------------------------------------------------------------- consumer --

__device__ __forceinline__ void scale4(float (&x)[4], float lower, float upper) {
    x[0] *= lower;
    x[1] *= lower;
    x[2] *= upper;
    x[3] *= upper;
}

// floor(log2 |x|) of x (-10000 for 0, subnormals and what is not finite).
__device__ __forceinline__ int exponent_of(float x) {
    const int e = (int)((__float_as_uint(x) >> 23) & 0xff);
    return e == 0 || e == 255 ? -10000 : e - 127;
}

__device__ __forceinline__ float power_of_two(int e) {   // -126 <= e <= 127
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
    return fmaxf(x, __shfl_xor_sync(kFull, x, 2));
}

__device__ __forceinline__ void load_v(const Stage &st, int warp_v, int lane, uint32_t (&v)[4]) {
    const int t = token_at((lane >> 4) * 8 + (lane & 7));
    const uint4 *src = &st.v[t][(2 * warp_v + ((lane >> 3) & 1)) ^ (t & 7)];
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(kda::smem_u32(src)));
}

// What a consumer warp holds of a row: 16 rows of S, those of lane / 4 and
// lane / 4 + 8, times powers of two of their own.
struct Held {
    float s[16][4];
    int ex[2];          // exponents: held = value * 2^ex
    float most[2];      // bound of the rows' norms as held
};

// Looks at the sizes of the rows of S and takes new powers of two, by them and
// by the largest values to come: the larger of the two is held in [2^7, 2^8).
__device__ __forceinline__ void rescale(Held &h, float vmax0, float vmax1) {
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < 16; ++n) {
        m[0] = fmaxf(m[0], fmaxf(fabsf(h.s[n][0]), fabsf(h.s[n][1])));
        m[1] = fmaxf(m[1], fmaxf(fabsf(h.s[n][2]), fabsf(h.s[n][3])));
    }
    int step[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        m[i] = quad_max(m[i]);
        const int most = max(exponent_of(m[i]) - h.ex[i], exponent_of(i ? vmax1 : vmax0));
        // within 2^-120 .. 2^120, so that the way back is a power that fp32 has
        const int ex = most < -5000 ? h.ex[i] : max(-120, min(120, 7 - most));
        step[i] = ex - h.ex[i];
        h.ex[i] = ex;
    }
    // in two powers: a step may be twice as far
    const float a0 = power_of_two(step[0] / 2), b0 = power_of_two(step[0] - step[0] / 2);
    const float a1 = power_of_two(step[1] / 2), b1 = power_of_two(step[1] - step[1] / 2);
    if (__any_sync(kFull, (step[0] | step[1]) != 0))
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            scale4(h.s[n], a0, a1);
            scale4(h.s[n], b0, b1);
        }
    h.most[0] = 11.4f * m[0] * a0 * b0;   // sqrt(128) of the largest
    h.most[1] = 11.4f * m[1] * a1 * b1;
}

__device__ __forceinline__ void consume(const Params &p, const Stage &st, unsigned char *out_tile,
                                        Held &h, const Row &row, int head, int chunk, int warp_v,
                                        int lane) {
    const int j = lane & 3;
    uint32_t v[4];
    load_v(st, warp_v, lane, v);
    // [n tile][row g: 2, row g + 8: 2]
    float x[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const float2 lower = kda::bf16x2_to_float2(v[2 * n]);
        const float2 upper = kda::bf16x2_to_float2(v[2 * n + 1]);
        x[n][0] = lower.x;
        x[n][1] = lower.y;
        x[n][2] = upper.x;
        x[n][3] = upper.y;
    }
    const float vmax0 = quad_max(fmaxf(fmaxf(fabsf(x[0][0]), fabsf(x[0][1])),
                                       fmaxf(fabsf(x[1][0]), fabsf(x[1][1]))));
    const float vmax1 = quad_max(fmaxf(fmaxf(fabsf(x[0][2]), fabsf(x[0][3])),
                                       fmaxf(fabsf(x[1][2]), fabsf(x[1][3]))));
    // What V - U and V' can come to, as held, has to stay inside fp16: a row's
    // norm grows by at most |v| a token.  Every fourth chunk the sizes are
    // looked at anyway, as rows may have shrunk.
    const bool grows = h.most[0] + 17.0f * vmax0 * power_of_two(h.ex[0]) > 60000.0f ||
                       h.most[1] + 17.0f * vmax1 * power_of_two(h.ex[1]) > 60000.0f;
    if ((chunk & 3) == 0 || __any_sync(kFull, grows)) rescale(h, vmax0, vmax1);
    const float down0 = power_of_two(h.ex[0]), down1 = power_of_two(h.ex[1]);
    h.most[0] += 16.0f * vmax0 * down0;
    h.most[1] += 16.0f * vmax1 * down1;
    // U = S (K P)^T and O = S (Q P)^T; S takes its decay on the way
    float u[2][4] = {}, u2[2][4] = {}, o[2][4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t hi[4], lo[4];
        split(h.s[2 * i][0], h.s[2 * i][1], hi[0], lo[0]);
        split(h.s[2 * i][2], h.s[2 * i][3], hi[1], lo[1]);
        split(h.s[2 * i + 1][0], h.s[2 * i + 1][1], hi[2], lo[2]);
        split(h.s[2 * i + 1][2], h.s[2 * i + 1][3], hi[3], lo[3]);
        const uint4 k0 = *reinterpret_cast<const uint4 *>(st.key + i * kKeyStep + lane * 16);
        const uint4 k1 = *reinterpret_cast<const uint4 *>(st.key + i * kKeyStep + 512 + lane * 16);
        const uint4 q = *reinterpret_cast<const uint4 *>(st.query + i * kQueryStep + lane * 16);
        mma(u[0], hi, k0.x, k0.y);
        mma(u[1], hi, k1.x, k1.y);
        mma(o[0], hi, q.x, q.y);
        mma(o[1], hi, q.z, q.w);
        mma(u2[0], hi, k0.z, k0.w);
        mma(u2[1], hi, k1.z, k1.w);
        mma(u2[0], lo, k0.x, k0.y);
        mma(u2[1], lo, k1.x, k1.y);
        const float4 d = kda::ld4(&st.decay[16 * i + 4 * j]);
        h.s[2 * i][0] *= d.x;
        h.s[2 * i][1] *= d.y;
        h.s[2 * i][2] *= d.x;
        h.s[2 * i][3] *= d.y;
        h.s[2 * i + 1][0] *= d.z;
        h.s[2 * i + 1][1] *= d.w;
        h.s[2 * i + 1][2] *= d.z;
        h.s[2 * i + 1][3] *= d.w;
    }
    // V - U, then V' = T (V - U)
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        scale4(x[n], down0, down1);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[n][c] = fmaf(u[n][c] + u2[n][c], -1.0f / kKeyScale, x[n][c]);
        split(x[n][0], x[n][1], hi[2 * n], lo[2 * n]);
        split(x[n][2], x[n][3], hi[2 * n + 1], lo[2 * n + 1]);
    }
    float d[2][4] = {}, d2[2][4] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const uint4 t = st.t[n][lane];
        mma(d[n], hi, t.x, t.y);
        mma(d2[n], hi, t.z, t.w);
        mma(d2[n], lo, t.x, t.y);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        constexpr float f = 1.0f / (kTScale * kUpdateScale);
#pragma unroll
        for (int c = 0; c < 4; ++c) d[n][c] = (d[n][c] + d2[n][c]) * f;
        split(d[n][0], d[n][1], hi[2 * n], lo[2 * n]);
        split(d[n][2], d[n][3], hi[2 * n + 1], lo[2 * n + 1]);
    }
    const uint4 b = st.b[lane];
    mma(o[0], hi, b.x, b.y);
    mma(o[1], hi, b.z, b.w);
    // S += V'^T (K P_C / P_t)
#pragma unroll
    for (int n = 0; n < 16; ++n) {
        const uint4 k =
            st.update[n][(lane & 24) | ((lane & 7) ^ ((lane >> 3) | ((n >> 1) & 1) << 2))];
        mma(h.s[n], hi, k.x, k.y);
        mma(h.s[n], hi, k.z, k.w);
        mma(h.s[n], lo, k.x, k.y);
    }
    // the outputs, [token][16 channels] in shared memory first
    const float up0 = power_of_two(-h.ex[0]) * (p.scale / kKeyScale);
    const float up1 = power_of_two(-h.ex[1]) * (p.scale / kKeyScale);
    uint32_t y[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        scale4(o[n], up0, up1);
        y[2 * n] = kda_cache::pack(o[n][0], o[n][1], __nv_bfloat16());
        y[2 * n + 1] = kda_cache::pack(o[n][2], o[n][3], __nv_bfloat16());
    }
    const int t = token_at((lane >> 4) * 8 + (lane & 7));
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     kda::smem_u32(out_tile + t * 48 + ((lane >> 3) & 1) * 16)),
                 "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                 : "memory");
    __syncwarp();
    const int token = chunk * kC + (lane >> 1);
    if (token < row.tokens)
        *reinterpret_cast<uint4 *>(p.out + ((long long)(row.first + token) * p.H + head) * kD +
                                   16 * warp_v + 8 * (lane & 1)) =
            *reinterpret_cast<const uint4 *>(out_tile + (lane >> 1) * 48 + (lane & 1) * 16);
    __syncwarp();
}

// ------------------------------------------------------------------ kernel --

template <bool kBounded>
__global__ void __launch_bounds__(kMaxThreads, 1)
    prefill_kernel(const Params p, long long items, int parts) {
    extern __shared__ unsigned char raw_smem[];
    Shared &sh = *reinterpret_cast<Shared *>(
        (reinterpret_cast<uintptr_t>(raw_smem) + 127) & ~(uintptr_t)127);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int consumers = kMaxConsumers / parts;
    if (threadIdx.x == 0) {
        sh.gave_up = 0;
        for (int i = 0; i < kStages; ++i) {
            kda::mbar_init(&sh.full[i], 1);
            kda::mbar_init(&sh.empty[i], consumers);
        }
    }
    kda_cache::grid_dependents_launch();
    __syncthreads();
    kda_cache::grid_dependency_wait();
    unsigned count = 0;   // chunks so far, of all items
    if (warp < kProducers) {
        for (long long item = blockIdx.x; item < items; item += gridDim.x) {
            int bits = 0;
            const Work w = work_at(p, item, parts, bits);
            if (bits != 0 && w.head == 0 && w.part == 0 && threadIdx.x == 0)
                kda_cache::flag(p.err, bits);
            const int chunks = (w.row.tokens + kC - 1) / kC;
            for (int c = 0; c < chunks; ++c, ++count) {
                if (count % kProducers != (unsigned)warp) continue;
                const unsigned stage = count % kStages, turn = count / kStages;
                if (!wait(sh, &sh.empty[stage], (turn & 1) ^ 1, p.err)) return;
                produce<kBounded>(p, sh.stage[stage], sh.scratch[warp], w.row, w.head, c, lane);
                if (lane == 0) kda::mbar_arrive(&sh.full[stage]);
            }
        }
        return;
    }
    const int me = warp - kProducers;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        int bits = 0;
        const Work w = work_at(p, item, parts, bits);
        if (w.row.tokens == 0) continue;
        const int warp_v = w.part * consumers + me;   // of the 8 sixteenths of a state's rows
        const long long tile = (long long)w.head * kda_delta::kTile +
                               (16 * warp_v + (lane >> 2)) * kD + 4 * (lane & 3);
        const long long slot = (long long)p.H * kda_delta::kTile;
        Held h;
        h.ex[0] = h.ex[1] = 0;
        h.most[0] = h.most[1] = 0.0f;
        if (w.row.from > 0) {
            const float *src = p.pool + w.row.from * slot + tile;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 a = __ldcs(reinterpret_cast<const float4 *>(src + 16 * i));
                const float4 b = __ldcs(reinterpret_cast<const float4 *>(src + 8 * kD + 16 * i));
                h.s[2 * i][0] = a.x;
                h.s[2 * i][1] = a.y;
                h.s[2 * i][2] = b.x;
                h.s[2 * i][3] = b.y;
                h.s[2 * i + 1][0] = a.z;
                h.s[2 * i + 1][1] = a.w;
                h.s[2 * i + 1][2] = b.z;
                h.s[2 * i + 1][3] = b.w;
            }
        } else {
#pragma unroll
            for (int n = 0; n < 16; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) h.s[n][c] = 0.0f;
        }
        const int chunks = (w.row.tokens + kC - 1) / kC;
        for (int c = 0; c < chunks; ++c, ++count) {
            const unsigned stage = count % kStages, turn = count / kStages;
            if (!wait(sh, &sh.full[stage], turn & 1, p.err)) return;
            consume(p, sh.stage[stage], sh.out[me], h, w.row, w.head, c, warp_v, lane);
            if (lane == 0) kda::mbar_arrive(&sh.empty[stage]);
        }
        float *dst = p.pool + w.row.to * slot + tile;
        const float up0 = power_of_two(-h.ex[0]), up1 = power_of_two(-h.ex[1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            __stcs(reinterpret_cast<float4 *>(dst + 16 * i),
                   make_float4(h.s[2 * i][0] * up0, h.s[2 * i][1] * up0, h.s[2 * i + 1][0] * up0,
                               h.s[2 * i + 1][1] * up0));
            __stcs(reinterpret_cast<float4 *>(dst + 8 * kD + 16 * i),
                   make_float4(h.s[2 * i][2] * up1, h.s[2 * i][3] * up1, h.s[2 * i + 1][2] * up1,
                               h.s[2 * i + 1][3] * up1));
        }
    }
}

}  // namespace

extern "C" kda_status kda_prefill(const kda_config *cfg, const void *q, const void *k,
                                  const void *v, const void *g_raw, const void *beta_raw,
                                  const float *A_log, const float *g_bias, float *state_pool,
                                  const int32_t *cu_seqlens, const int32_t *state_indices,
                                  const int32_t *initial_indices, int32_t B, int32_t num_tokens,
                                  void *out, int32_t *error_word, void *stream) {
    kda_status st = kda_delta::check_config(cfg);
    if (st != KDA_OK) return st;
    if (B < 0 || num_tokens < 0) return KDA_ERR_INVALID_ARG;
    if (B == 0 || num_tokens == 0) return KDA_OK;  // nothing to do; no pointer is inspected
    if (!cu_seqlens || !kda_cache::aligned(cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    Params p{};
    st = kda_delta::set_params(cfg, q, k, v, g_raw, beta_raw, A_log, g_bias, state_pool,
                               state_indices, initial_indices, B, num_tokens, out, error_word, p);
    if (st != KDA_OK) return st;
    p.cu_seqlens = cu_seqlens;
    const long long tiles = (long long)B * p.H;
    const int sms = kda_cache::sm_count();
    if (sms <= 0) return KDA_ERR_CUDA;
    // A state's rows can go to several CTAs, each of which makes the shared
    // operands for itself: where there are few states, that is better than
    // idle SMs.
    int parts = 1;
    while (parts < 4 && tiles * parts * 2 <= sms) parts *= 2;
    const long long items = tiles * parts;
    const int smem = (int)sizeof(Shared) + 128;
    void (*kernel)(const Params, long long, int) =
        p.bounded ? prefill_kernel<true> : prefill_kernel<false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return KDA_ERR_CUDA;
    return kda_cache::launch(kernel, dim3((unsigned)(items < sms ? items : sms)),
                             dim3(32 * (kProducers + kMaxConsumers / parts)), smem, 1, stream, p,
                             items, parts);
}

extern "C" kda_status kda_prefill_packed(const kda_delta_args *a) {
    if (a == nullptr) return KDA_ERR_INVALID_ARG;
    return kda_prefill(&a->config, a->q, a->k, a->v, a->g_raw, a->beta_raw, a->A_log, a->g_bias,
                       a->state_pool, a->cu_seqlens, a->state_indices, a->initial_indices, a->B,
                       a->num_tokens, a->out, a->error_word, a->stream);
}
