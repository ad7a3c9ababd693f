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
// for the products in the order 0 8 1 9 2 10 3 11, 4 12 ... 7 15: the pairs of
// tokens that a producer's lane has are then the pairs of the fragments.
//
// A and B.  Two producer warps make a chunk's operands, the first the tokens'
// vectors, the second the products between tokens.  Four tokens t at a time
// meet all s before and among them: k_s decayed to the block's first token
// times k_t, q_t decayed from it.  Among the four that is k_s / R_s, R_s the
// decays from the first, a quotient.  There, and in K P_C / P_t, a decay below
// 2^-40 counts as 2^-40, so that three of them fit fp32: what that adds is
// 2^-40 beside factors of 1.  The operands keep fp32's range: tf32, hi and lo
// as above.
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
constexpr int kPairs = 4;        // pairs of producer warps, a chunk each
constexpr int kProducers = 2 * kPairs;
constexpr int kStages = 5;
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

// What the first warp of a pair hands to the second, four tokens at a time.
// Their decays are products from the first of them, R_u = prod_{0<i<=u} e_i.
constexpr int kRow = kD + 16;             // floats, padded against bank conflicts
struct __align__(16) Block {
    float ahead[8][kRow];                 // k_u R_u, then q_u R_u
    float back[4][kRow];                  // k_u / R_u
    float since[kD];                      // decays since the block before's first token
    float end[kD];                        // R_3
};

struct __align__(16) Scratch {            // of a pair of producer warps
    Block block[2];
    float a[kC][kC + 4], b[kC][kC + 4];
    float beta[kC];
    uint64_t ready[2], taken[2];
};

struct Shared {
    Stage stage[kStages];
    Scratch scratch[kPairs];
    unsigned char out[kMaxConsumers][kC * 48];
    float zeros[kD];
    uint64_t full[kStages], empty[kStages];
    int gave_up;
};

// The place of token t in the products' order, and the token at a place.
__host__ __device__ constexpr int place_of(int t) {
    return ((t & 4) << 1) + 2 * (t & 3) + (t >> 3);
}
__device__ __forceinline__ int token_at(int n) {
    return ((n & 8) >> 1) + ((n & 7) >> 1) + ((n & 1) << 3);
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first product of a sum.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// The same for k steps of 8 in tf32.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x and y as two tf32 numbers each, 11 bits each: the low 13 bits of an operand
// are not looked at.
__device__ __forceinline__ void split_tf32(u64 xy, uint32_t &hi_x, uint32_t &hi_y, uint32_t &lo_x,
                                           uint32_t &lo_y) {
    const float2 v = both(xy);
    hi_x = __float_as_uint(v.x) & 0xffffe000u;
    hi_y = __float_as_uint(v.y) & 0xffffe000u;
    lo_x = __float_as_uint(v.x - __uint_as_float(hi_x));
    lo_y = __float_as_uint(v.y - __uint_as_float(hi_y));
}

__device__ __forceinline__ uint32_t half_pair(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// x and y as pairs of fp16: the numbers, and what is left of them.
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = half_pair(x, y);
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    u64 rest;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(rest) : "l"(pair(x, y)), "l"(pair(h.x, h.y)));
    const float2 r = both(rest);
    lo = half_pair(r.x, r.y);
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

// parts: 2^part_bits CTAs share a row and head.
__device__ __forceinline__ Work work_at(const Params &p, unsigned item, int part_bits, int &bits) {
    Work w;
    w.part = (int)(item & ((1u << part_bits) - 1));
    const unsigned tile = item >> part_bits, b = tile / (unsigned)p.H;
    w.head = (int)(tile - b * (unsigned)p.H);
    w.row = kda_delta::read_row(p, (int)b, bits);
    return w;
}

// Keeps the compiler from fetching operands so far ahead that registers run out.
__device__ __forceinline__ void no_further_ahead() { asm volatile("" ::: "memory"); }

// Registers a thread from here on, of all four warps of a warpgroup.  The
// shares of the launch's 128 a thread: 4 warps of 96, 4 of 128 and 8 of 144
// are 16 times 128 (with 4 consumers 12 times 123).
template <int kRegisters>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegisters));
}
template <int kRegisters>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegisters));
}

// x, in a way that keeps addresses made from it from being held in registers
// for longer than the caller's turn of a loop: beside the states there is no
// room, and what is spilled to local memory comes back from L2, as shared
// memory leaves L1 little.
__device__ __forceinline__ int made_anew(int x) {
    asm volatile("" : "+r"(x));
    return x;
}

// ---------------------------------------------------------------- producer --

// 2^x, within 2 ulp, 0 far below.
__device__ __forceinline__ float exp2_of(float x) { return kda_cache::exp2_fast(x); }

constexpr float kLog2e = 1.4426950408889634f;

// log2 of a channel's decay, as kda::decay_factor has it.  x: the gate's input
// with its bias; gate: -exp(A_log) log2 e; bound: lower_bound log2 e.
template <bool kBounded>
__device__ __forceinline__ float log2_decay(float x, float gate, float bound) {
    if constexpr (kBounded) {
        return __fdividef(bound, 1.0f + exp2_of(gate * x));
    } else {
        // softplus(x) = max(x, 0) + log1p(z), z = exp(-|x|); log1p(z) = z P(z)
        // with the polynomial of kda::softplus
        constexpr float c[10] = {0x1p+0f,        -0x1.ffffcp-2f,  0x1.554c9cp-2f, -0x1.ff11c2p-3f,
                                 0x1.930202p-3f, -0x1.399642p-3f, 0x1.b2c2a2p-4f, -0x1.d3784ep-5f,
                                 0x1.4628bp-6f,  -0x1.aad1eep-9f};
        const float z = exp2_of(-fabsf(x) * kLog2e);
        float r = c[9];
#pragma unroll
        for (int i = 8; i >= 0; --i) r = fmaf(r, z, c[i]);
        return gate * fmaf(z, r, fmaxf(x, 0.0f));
    }
}

struct Raw {   // a token's channels 4 lane .. 4 lane + 3
    uint2 q, k, g;
};

__device__ __forceinline__ void pairs_of(uint2 x, u64 &a, u64 &b) {
    const float4 f = kda::bf16x4_to_float4(x);
    a = pair(f.x, f.y);
    b = pair(f.z, f.w);
}

__device__ __forceinline__ void put(float *dst, u64 a, u64 b) {
    *reinterpret_cast<ulonglong2 *>(dst) = make_ulonglong2(a, b);
}

__device__ __forceinline__ float squares(u64 a, u64 b) {
    const float2 s = both(fma_pair(a, a, mul_pair(b, b)));
    return s.x + s.y;
}

__device__ __forceinline__ float reciprocal(float x) {   // within 1 ulp
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Where a warp reads a row's activations, four channels a lane.
struct Inputs {
    const __nv_bfloat16 *q, *k, *g;
};

__device__ __forceinline__ Raw load_raw(const Params &p, Inputs &in, bool valid) {
    Raw raw;
    raw.q = raw.k = raw.g = make_uint2(0u, 0u);
    if (valid) {
        raw.q = __ldg(reinterpret_cast<const uint2 *>(in.q));
        raw.k = __ldg(reinterpret_cast<const uint2 *>(in.k));
        raw.g = __ldg(reinterpret_cast<const uint2 *>(in.g));
    }
    in.q += p.stride_q;
    in.k += p.stride_k;
    in.g += p.stride_g;
    return raw;
}

// The tokens' vectors of a chunk, by the first warp of a pair.  blocks: how
// many blocks of four tokens the pair has had.
template <bool kBounded>
__device__ __forceinline__ bool produce_tokens(const Params &p, Shared &sh, Stage &st, Scratch &sc,
                                               const Row &row, int head, int chunk, int lane,
                                               unsigned &blocks) {
    lane = made_anew(lane);
    const long long first = (long long)row.first + (long long)chunk * kC;
    const int valid = min(kC, row.tokens - chunk * kC);
    const long long at = (long long)head * kD + 4 * lane;
    Inputs in{p.q + first * p.stride_q + at, p.k + first * p.stride_k + at,
              p.g + first * p.stride_g + at};
    Raw next[2];
    next[0] = load_raw(p, in, true);
    next[1] = load_raw(p, in, 1 < valid);
    {   // the values as they are
        const __nv_bfloat16 *src = p.v + first * p.stride_v + at;
#pragma unroll 4
        for (int t = 0; t < kC; ++t, src += p.stride_v) {
            unsigned char *dst =
                reinterpret_cast<unsigned char *>(&st.v[t][(lane >> 1) ^ (t & 7)]) + (lane & 1) * 8;
            if (t < valid)
                kda::cp_async8(dst, src);
            else
                *reinterpret_cast<uint2 *>(dst) = make_uint2(0u, 0u);
        }
    }
    kda::cp_async_commit();
    const float gate = -__expf(p.A_log[head]) * kLog2e, bound = p.lower_bound * kLog2e;
    const float4 bias = kda::ld4(p.g_bias + at);
    u64 reach[2] = {pair(kKeyScale, kKeyScale), pair(kKeyScale, kKeyScale)};   // P_t
    u64 total[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};                       // log2 P_t
    u64 r[2] = {pair(1.0f, 1.0f), pair(1.0f, 1.0f)};                            // R
    unsigned char *key = st.key + (lane >> 2) * kKeyStep + (lane & 3) * 16;
    unsigned char *query = st.query + (lane >> 2) * kQueryStep + (lane & 3) * 16;
    // two tokens a turn, the next two on their way
#pragma unroll 1
    for (int t0 = 0; t0 < kC; t0 += 2) {
        const Raw now[2] = {next[0], next[1]};
        next[0] = load_raw(p, in, t0 + 2 < valid);
        next[1] = load_raw(p, in, t0 + 3 < valid);
        Block &out = sc.block[blocks & 1];
        if ((t0 & 2) == 0 && !wait(sh, &sc.taken[blocks & 1], ((blocks >> 1) & 1) ^ 1, p.err)) {
            kda::cp_async_wait_all();
            return false;
        }
        // norms: lane bits 4 and 3 choose among the sums of k and q of both tokens
        float norm;
        {
            u64 x, y;
            float s[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                pairs_of(now[u].k, x, y);
                s[2 * u] = squares(x, y);
                pairs_of(now[u].q, x, y);
                s[2 * u + 1] = squares(x, y);
            }
            const bool b4 = (lane & 16) != 0, b3 = (lane & 8) != 0;
            s[0] = (b4 ? s[2] : s[0]) + __shfl_xor_sync(kFull, b4 ? s[0] : s[2], 16);
            s[1] = (b4 ? s[3] : s[1]) + __shfl_xor_sync(kFull, b4 ? s[1] : s[3], 16);
            norm = (b3 ? s[1] : s[0]) + __shfl_xor_sync(kFull, b3 ? s[0] : s[1], 8);
            norm += __shfl_xor_sync(kFull, norm, 4);
            norm += __shfl_xor_sync(kFull, norm, 2);
            norm += __shfl_xor_sync(kFull, norm, 1);
            norm = kda::inv_l2(norm);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = t0 + u;
            const float rk = __shfl_sync(kFull, norm, 16 * u);
            const float rq = __shfl_sync(kFull, norm, 16 * u + 8);
            float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // behind the row's end nothing decays
            if (t < valid) {
                const float4 x = kda::bf16x4_to_float4(now[u].g);
                y[0] = log2_decay<kBounded>(x.x + bias.x, gate, bound);
                y[1] = log2_decay<kBounded>(x.y + bias.y, gate, bound);
                y[2] = log2_decay<kBounded>(x.z + bias.z, gate, bound);
                y[3] = log2_decay<kBounded>(x.w + bias.w, gate, bound);
            }
            total[0] = add_pair(total[0], pair(y[0], y[1]));
            total[1] = add_pair(total[1], pair(y[2], y[3]));
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = exp2_of(y[c]);
            const u64 e[2] = {pair(y[0], y[1]), pair(y[2], y[3])};
            u64 k[2], q[2];
            pairs_of(now[u].k, k[0], k[1]);
            pairs_of(now[u].q, q[0], q[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                reach[i] = mul_pair(reach[i], e[i]);
                k[i] = mul_pair(k[i], pair(rk, rk));
                q[i] = mul_pair(q[i], pair(rq, rq));
            }
            if (u == 0 && (t0 & 2) == 0) {   // a block's first token
                put(&out.since[4 * lane], mul_pair(r[0], e[0]), mul_pair(r[1], e[1]));
                r[0] = r[1] = pair(1.0f, 1.0f);
            } else {
                r[0] = mul_pair(r[0], pair(fmaxf(y[0], 0x1p-40f), fmaxf(y[1], 0x1p-40f)));
                r[1] = mul_pair(r[1], pair(fmaxf(y[2], 0x1p-40f), fmaxf(y[3], 0x1p-40f)));
            }
            float *ahead = &out.ahead[t & 3][4 * lane];
            put(ahead, mul_pair(k[0], r[0]), mul_pair(k[1], r[1]));
            put(ahead + 4 * kRow, mul_pair(q[0], r[0]), mul_pair(q[1], r[1]));
            const float2 r0 = both(r[0]), r1 = both(r[1]);
            put(&out.back[t & 3][4 * lane], mul_pair(k[0], pair(reciprocal(r0.x), reciprocal(r0.y))),
                mul_pair(k[1], pair(reciprocal(r1.x), reciprocal(r1.y))));
            // K P and Q P: channels 4 lane .. + 3 are b0 and b1 of k step lane / 4
            const int place = place_of(t), slot = (place & 7) * 4, tile = place >> 3;
            uint4 f;
            float2 x = both(mul_pair(k[0], reach[0]));
            split(x.x, x.y, f.x, f.z);
            x = both(mul_pair(k[1], reach[1]));
            split(x.x, x.y, f.y, f.w);
            *reinterpret_cast<uint4 *>(key + (tile * 32 + slot) * 16) = f;
            uint2 h;
            x = both(mul_pair(q[0], reach[0]));
            h.x = half_pair(x.x, x.y);
            x = both(mul_pair(q[1], reach[1]));
            h.y = half_pair(x.x, x.y);
            *reinterpret_cast<uint2 *>(query + slot * 16 + tile * 8) = h;
        }
        if ((t0 & 2) != 0) {
            put(&out.end[4 * lane], r[0], r[1]);
            __syncwarp();
            if (lane == 0) kda::mbar_arrive(&sc.ready[blocks & 1]);
            ++blocks;
        }
    }
    // P_C decays the state chunk after chunk, so its error adds up: from the sum
    // of the logarithms, within 1 ulp also near 1, not as a product
    {
        const float2 x = both(total[0]), y = both(total[1]);
        float f[4] = {x.x, x.y, y.x, y.y};
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            const float v = f[0];
            f[0] = f[1];
            f[1] = f[2];
            f[2] = f[3];
            f[3] = 1.0f + expm1f(v * 0.693147180559945309f);
        }
        *reinterpret_cast<float4 *>(&st.decay[4 * lane]) = make_float4(f[0], f[1], f[2], f[3]);
    }
    kda::cp_async_wait_all();
    __syncwarp();
    return true;
}

// The products between tokens, by the second warp of a pair.
__device__ __forceinline__ bool produce_products(const Params &p, Shared &sh, Stage &st,
                                                 Scratch &sc, const Row &row, int head, int chunk,
                                                 int lane, unsigned &blocks) {
    lane = made_anew(lane);
    const long long first = (long long)row.first + (long long)chunk * kC;
    const int valid = min(kC, row.tokens - chunk * kC);
    if (lane < kC)
        sc.beta[lane] =
            lane < valid ? kda::sigmoidf_rn(__bfloat162float(
                               p.beta[(first + lane) * p.stride_beta + head]))
                         : 0.0f;
    // lane 4 g + j: tokens s = g and g + 8, channels 16 m + 4 j + 0..3: k_s decayed to where the
    // block in work needs it
    u64 w[2][16];
#pragma unroll
    for (int c = 0; c < 16; ++c) w[0][c] = w[1][c] = pair(0.0f, 0.0f);
    // (one copy of the code for all blocks: it has to stay in the instruction cache
    // beside that of the other warps)
#pragma unroll 1
    for (int block = 0; block < 4; ++block, ++blocks) {
        if (!wait(sh, &sc.ready[blocks & 1], (blocks >> 1) & 1, p.err)) return false;
        const Block &in = sc.block[blocks & 1];
        const int at = made_anew(lane), j = at & 3, g = at >> 2;
        // the block's own tokens join, the others decay; zeros for what does neither
        const bool own = (g >> 2) == (block & 1);
        const float *back0 = own && block < 2 ? in.back[g & 3] : sh.zeros;
        const float *back1 = own && block >= 2 ? in.back[g & 3] : sh.zeros;
        float d[2][4] = {};   // sums of hi hi, and of the others
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const int c = 16 * m + 4 * j;
            no_further_ahead();
            const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(&in.since[c]);
            const ulonglong2 k0 = *reinterpret_cast<const ulonglong2 *>(&back0[c]);
            const ulonglong2 k1 = *reinterpret_cast<const ulonglong2 *>(&back1[c]);
            const ulonglong2 n = *reinterpret_cast<const ulonglong2 *>(&in.ahead[g][c]);
            w[0][2 * m] = fma_pair(w[0][2 * m], f.x, k0.x);
            w[0][2 * m + 1] = fma_pair(w[0][2 * m + 1], f.y, k0.y);
            w[1][2 * m] = fma_pair(w[1][2 * m], f.x, k1.x);
            w[1][2 * m + 1] = fma_pair(w[1][2 * m + 1], f.y, k1.y);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t hi[4], lo[4], b[2], bl[2];
                split_tf32(h ? n.y : n.x, b[0], b[1], bl[0], bl[1]);
                split_tf32(w[0][2 * m + h], hi[0], hi[2], lo[0], lo[2]);
                split_tf32(w[1][2 * m + h], hi[1], hi[3], lo[1], lo[3]);
                mma_tf32(d[0], hi, b[0], b[1]);
                mma_tf32(d[1], hi, bl[0], bl[1]);
                mma_tf32(d[1], lo, b[0], b[1]);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            // column 2 j (+ 1): the block's k 0..3, q 0..3; tokens s behind the block are
            // not looked at
            const float x = d[0][c] + d[1][c];
            (j < 2 ? sc.a : sc.b)[4 * block + 2 * (j & 1) + (c & 1)][g + 4 * (c & 2)] = x;
        }
        if (block == 3) {   // K P_C / P_t, in units of the update
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                no_further_ahead();
                const float4 f = kda::ld4(&in.end[16 * m + 4 * j]);
                const u64 scale = pair(kUpdateScale, kUpdateScale);
                const u64 e[2] = {mul_pair(pair(f.x, f.y), scale), mul_pair(pair(f.z, f.w), scale)};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float2 y = both(mul_pair(w[0][2 * m + (u >> 1)], e[u >> 1]));
                    const float2 z = both(mul_pair(w[1][2 * m + (u >> 1)], e[u >> 1]));
                    uint2 x;
                    split(u & 1 ? y.y : y.x, u & 1 ? z.y : z.x, x.x, x.y);
                    // channel 16 m + 4 j + u; tokens (g, g + 8) are b0 for g < 4, else b1
                    const int tile = 2 * m + (u >> 1), spot = (u & 1) * 4 + (g & 3);
                    uint32_t *dst = reinterpret_cast<uint32_t *>(
                                        &st.update[tile][8 * j + (spot ^ ((j & 1) << 2))]) +
                                    (g >> 2);
                    dst[0] = x.x;
                    dst[2] = x.y;
                }
            }
        }
        __syncwarp();
        if (lane == 0) kda::mbar_arrive(&sc.taken[blocks & 1]);
    }
    // T, column lane & 15 in a lane: T_t = beta_t (1_t - sum_{j<t} A_tj T_j)
    {
        lane = made_anew(lane);
        const int s = lane & 15;
        float col[kC];
#pragma unroll
        for (int t = 0; t < kC; ++t) {
            float x = t == s ? 1.0f : 0.0f, y = 0.0f;
            if ((t & 3) == 0) no_further_ahead();
#pragma unroll
            for (int i = 0; i < t; i += 4) {
                const float4 n = kda::ld4(&sc.a[t][i]);
                x = fmaf(-n.x, col[i], x);
                if (i + 1 < t) y = fmaf(-n.y, col[i + 1], y);
                if (i + 2 < t) x = fmaf(-n.z, col[i + 2], x);
                if (i + 3 < t) y = fmaf(-n.w, col[i + 3], y);
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
            split(sc.a[t][j], sc.a[t][j + 8], x.x, x.z);
            split(sc.a[t][j + 4], sc.a[t][j + 12], x.y, x.w);
            st.t[tile][lane] = x;
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = j + 8 * (i & 1) + 4 * (i >> 1);
                y[i] = s <= t ? sc.b[t][s] * kBScale : 0.0f;
            }
            (tile ? f.z : f.x) = half_pair(y[0], y[1]);
            (tile ? f.w : f.y) = half_pair(y[2], y[3]);
        }
        st.b[lane] = f;
    }
    __syncwarp();
    return true;
}

// ---------------------------------------------------------------- consumer --

__device__ __forceinline__ void times(float &x, float &y, u64 f) {
    const float2 r = both(mul_pair(pair(x, y), f));
    x = r.x;
    y = r.y;
}

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
    lane = made_anew(lane);
    const int j = lane & 3;
    uint32_t v[4];   // [n tile][rows g, rows g + 8], two tokens each
    load_v(st, warp_v, lane, v);
    float vmax0 = 0.0f, vmax1 = 0.0f;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const float2 lower = kda::bf16x2_to_float2(v[2 * n]);
        const float2 upper = kda::bf16x2_to_float2(v[2 * n + 1]);
        vmax0 = fmaxf(vmax0, fmaxf(fabsf(lower.x), fabsf(lower.y)));
        vmax1 = fmaxf(vmax1, fmaxf(fabsf(upper.x), fabsf(upper.y)));
    }
    vmax0 = quad_max(vmax0);
    vmax1 = quad_max(vmax1);
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
    float u[2][4], o[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        no_further_ahead();
        uint32_t hi[4], lo[4];
        split(h.s[2 * i][0], h.s[2 * i][1], hi[0], lo[0]);
        split(h.s[2 * i][2], h.s[2 * i][3], hi[1], lo[1]);
        split(h.s[2 * i + 1][0], h.s[2 * i + 1][1], hi[2], lo[2]);
        split(h.s[2 * i + 1][2], h.s[2 * i + 1][3], hi[3], lo[3]);
        const uint4 k0 = *reinterpret_cast<const uint4 *>(st.key + i * kKeyStep + lane * 16);
        const uint4 k1 = *reinterpret_cast<const uint4 *>(st.key + i * kKeyStep + 512 + lane * 16);
        const uint4 q = *reinterpret_cast<const uint4 *>(st.query + i * kQueryStep + lane * 16);
        if (i == 0) {
            mma_first(u[0], hi, k0.x, k0.y);
            mma_first(u[1], hi, k1.x, k1.y);
            mma_first(o[0], hi, q.x, q.y);
            mma_first(o[1], hi, q.z, q.w);
        } else {
            mma(u[0], hi, k0.x, k0.y);
            mma(u[1], hi, k1.x, k1.y);
            mma(o[0], hi, q.x, q.y);
            mma(o[1], hi, q.z, q.w);
        }
        mma(u[0], hi, k0.z, k0.w);
        mma(u[1], hi, k1.z, k1.w);
        mma(u[0], lo, k0.x, k0.y);
        mma(u[1], lo, k1.x, k1.y);
        const ulonglong2 d = *reinterpret_cast<const ulonglong2 *>(&st.decay[16 * i + 4 * j]);
        times(h.s[2 * i][0], h.s[2 * i][1], d.x);
        times(h.s[2 * i][2], h.s[2 * i][3], d.x);
        times(h.s[2 * i + 1][0], h.s[2 * i + 1][1], d.y);
        times(h.s[2 * i + 1][2], h.s[2 * i + 1][3], d.y);
    }
    // V - U, then V' = T (V - U)
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const float2 lower = kda::bf16x2_to_float2(v[2 * n]);
        const float2 upper = kda::bf16x2_to_float2(v[2 * n + 1]);
        float x[4] = {lower.x, lower.y, upper.x, upper.y};
        scale4(x, down0, down1);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = fmaf(u[n][c], -1.0f / kKeyScale, x[c]);
        split(x[0], x[1], hi[2 * n], lo[2 * n]);
        split(x[2], x[3], hi[2 * n + 1], lo[2 * n + 1]);
    }
    float d[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const uint4 t = st.t[n][lane];
        mma_first(d[n], hi, t.x, t.y);
        mma(d[n], hi, t.z, t.w);
        mma(d[n], lo, t.x, t.y);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        constexpr float f = 1.0f / (kTScale * kUpdateScale);
#pragma unroll
        for (int c = 0; c < 4; ++c) d[n][c] *= f;
        split(d[n][0], d[n][1], hi[2 * n], lo[2 * n]);
        split(d[n][2], d[n][3], hi[2 * n + 1], lo[2 * n + 1]);
    }
    const uint4 b = st.b[lane];
    mma(o[0], hi, b.x, b.y);
    mma(o[1], hi, b.z, b.w);
    // S += V'^T (K P_C / P_t)
#pragma unroll
    for (int n = 0; n < 16; ++n) {
        if ((n & 1) == 0) no_further_ahead();
        const uint4 k = st.update[n][lane ^ (((lane >> 3) & 1) << 2)];
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

// A producer warp: the tokens' vectors (kTokens) or the products between them
// of every kPairs-th chunk of the CTA's work.
template <bool kBounded, bool kTokens>
__device__ __forceinline__ void produce(const Params &p, Shared &sh, unsigned items, int part_bits,
                                        int warp, int lane) {
    const unsigned pair_of = warp % kPairs;
    unsigned count = 0, blocks = 0;
    for (unsigned item = blockIdx.x; item < items; item += gridDim.x) {
        int bits = 0;
        const Work w = work_at(p, item, part_bits, bits);
        if (bits != 0 && w.head == 0 && w.part == 0 && threadIdx.x == 0)
            kda_cache::flag(p.err, bits);
        const unsigned chunks = (unsigned)(w.row.tokens + kC - 1) / kC;
        for (unsigned c = (pair_of - count) % kPairs; c < chunks; c += kPairs) {
            const unsigned stage = (count + c) % kStages, turn = (count + c) / kStages;
            if (!wait(sh, &sh.empty[stage], (turn & 1) ^ 1, p.err)) return;
            Stage &st = sh.stage[stage];
            Scratch &sc = sh.scratch[pair_of];
            bool made;
            if constexpr (kTokens)
                made = produce_tokens<kBounded>(p, sh, st, sc, w.row, w.head, c, lane, blocks);
            else
                made = produce_products(p, sh, st, sc, w.row, w.head, c, lane, blocks);
            if (!made) return;
            if (lane == 0) kda::mbar_arrive(&sh.full[stage]);
        }
        count += chunks;
    }
}

template <bool kBounded>
__global__ void __launch_bounds__(kMaxThreads, 1)
    prefill_kernel(const Params p, unsigned items, int part_bits) {
    extern __shared__ unsigned char raw_smem[];
    Shared &sh = *reinterpret_cast<Shared *>(
        (reinterpret_cast<uintptr_t>(raw_smem) + 127) & ~(uintptr_t)127);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int consumers = kMaxConsumers >> part_bits;
    if (threadIdx.x < kD) sh.zeros[threadIdx.x] = 0.0f;
    if (threadIdx.x == 0) {
        sh.gave_up = 0;
        for (int i = 0; i < kStages; ++i) {
            kda::mbar_init(&sh.full[i], 2);
            kda::mbar_init(&sh.empty[i], consumers);
        }
        for (int i = 0; i < 2 * kPairs; ++i) {
            kda::mbar_init(&sh.scratch[i >> 1].ready[i & 1], 1);
            kda::mbar_init(&sh.scratch[i >> 1].taken[i & 1], 1);
        }
    }
    kda_cache::grid_dependents_launch();
    __syncthreads();
    kda_cache::grid_dependency_wait();
    unsigned count = 0;   // chunks so far, of all items
    if (warp < kProducers) {
        if (warp < kPairs) {
            fewer_registers<96>();
            produce<kBounded, true>(p, sh, items, part_bits, warp, lane);
        } else {
            produce<kBounded, false>(p, sh, items, part_bits, warp, lane);
        }
        return;
    }
    more_registers<144>();
    const int me = warp - kProducers;
    if (me >= consumers) return;   // there to make up a warpgroup
    for (unsigned item = blockIdx.x; item < items; item += gridDim.x) {
        int bits = 0;
        const Work w = work_at(p, item, part_bits, bits);
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
    int part_bits = 0;
    while (part_bits < 2 && (tiles << (part_bits + 1)) <= sms) ++part_bits;
    const long long items = tiles << part_bits;
    if (items > 0x7fffffffLL - sms) return KDA_ERR_UNSUPPORTED;
    const int smem = (int)sizeof(Shared) + 128;
    void (*kernel)(const Params, unsigned, int) =
        p.bounded ? prefill_kernel<true> : prefill_kernel<false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return KDA_ERR_CUDA;
    return kda_cache::launch(kernel, dim3((unsigned)(items < sms ? items : sms)),
                             dim3(32 * (kProducers + (part_bits == 0 ? 8 : 4))), smem, 1, stream,
                             p, (unsigned)items, part_bits);
}

extern "C" kda_status kda_prefill_packed(const kda_delta_args *a) {
    if (a == nullptr) return KDA_ERR_INVALID_ARG;
    return kda_prefill(&a->config, a->q, a->k, a->v, a->g_raw, a->beta_raw, a->A_log, a->g_bias,
                       a->state_pool, a->cu_seqlens, a->state_indices, a->initial_indices, a->B,
                       a->num_tokens, a->out, a->error_word, a->stream);
}
