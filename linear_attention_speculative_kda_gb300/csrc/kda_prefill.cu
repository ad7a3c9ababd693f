// kda_prefill: the gated delta rule over rows of any length, chunked
// (sm_103a).  Contract in include/kda.h.
//
// Mathematics.  A head's state S [V, K], a chunk of C = 16 tokens, e_t the
// token's decays, P_t = prod_{i<=t} e_i within the chunk, all norms taken:
//   A_ts = sum_c k_t k_s prod_{s<i<=t} e_i   (s < t)
//   B_ts = sum_c q_t k_s prod_{s<i<=t} e_i   (s <= t)
//   T    = (1 + diag(beta) A)^-1 diag(beta)                      [C, C]
//   X    = V - (K P) S^T,  V' = T X,  O = (Q P) S^T + B V' = (Q P) S^T + (B T) X
//   S   <- S diag(P_C) + V'^T (K P_C / P_t)
//
// Precision.  States are fp32 and the products with them have to be: every
// product with S, and of V' into S, runs on tcgen05.mma in fp16 with fp32 sums,
// an fp32 operand x as two fp16 numbers, hi = fp16(x) and lo = fp16(x - hi), 22
// bits, and a product as hi hi + hi lo + lo hi; what is left out is below 2^-22
// of it.  fp16's range needs powers of two, and each is from what it scales, not
// from a bound that knows no decay or no beta: a row of S has its own, moved with
// its values; a token's K P and Q P have one of the largest P that is left, and
// its K P_C / P_t one of their largest, which V' takes; a row of V', so taken, has
// its own.  What decays leave, and what weak betas write, is so as exact as what
// was there before, but for one thing: an entry of S far below its row's largest
// has 2^-23 of that, in the chunk at whose start it is.
//   V' = T X and (B T) X are 136 fp32 products a row each, made where X lies.  O is
// rounded once, to bf16 (with hi alone in its products, 11 bits, the outputs were
// 1e-3 off those of fp32 products, not 5e-5).  Behind the diagonals nothing is
// multiplied: 0 times what is not finite would reach the tokens before it.
//
// A and B.  Four tokens t at a time meet all s before and among them: k_s
// decayed to the block's first token times k_t, q_t decayed from it, all of
// them products of decays, which strong decays may take to 0.  Among the four
// that is k_s / R_s, R_s the decays from the first.  There, and in K P_C / P_t,
// a decay below 2^-40 counts as 2^-40, so that three of them fit fp32 (and a
// product over blocks that fp32 does not have as 0): what that adds or takes is
// 2^-40 beside factors of 1.  The operands keep fp32's range: mma.sync in tf32, hi
// and lo as above (5% of the tensor pipe's time).
//
// Layout.  A CTA has one row and head at a time: the chunks of a row follow
// one another, so rows and heads are what runs side by side.  S lies in tensor
// memory, in fp32 and, split, as the A operand of the products.  Of the
// eight consumer warps two threads have a row of it, each half of its columns,
// where they add what the chunk brought and split it, and half of the chunk's
// tokens, of which they make V', split it and write the outputs.  The operands
// that all rows share (K P, Q P, K P_C / P_t, T, B T, P_C) are made by eight
// producer warps, a pair a chunk, in two rings: the first warp of a pair makes
// the tokens' vectors, the second the products between them.
//   Rows and heads are dealt out to the CTAs by their lengths, or in turn where each
// CTA has many (make_plan, and the rule at the launch).
//   Where fewer rows and heads than SMs have many tokens, a cluster of two CTAs
// shares one (kSplit): the warps of the second produce, seven pairs, and write
// their operands into the first's rings (mapa), all warps of the first
// consume, four threads a row of S.
//
// What bounds it.  Neither HBM (15% of its rate over 64 rows of 1024 tokens x
// 32 heads, 2.86 ms) nor the tensor cores (14%), but instructions: some 15,900 a
// chunk, 57% of the issue slots.  A consumer's turn is 6,400 clocks (S 2,000, its
// products 1,400, V' 1,000, outputs 1,300, barriers 700), of which it waits some
// 400 for the tensor cores and 200 for operands; the producers are idle for a
// quarter and a third of it.
//   Code that lies in the way counts too: 2.4 KB more of it in the pass over S cost
// 10%, so loops are short where all roles share an SM (63 KB of code: 6% of the
// instruction fetches miss, 13% of 69 KB).
//   On the way here, the same 64 rows: token by token in fp32 13.3 ms (the decay,
// two dot products and the update are 8 fp32 operations an element of S: 3.2 ms at
// the least); consumers on mma.sync with S in their registers 3.8; 80 KB of
// straight code 4.6; both halves of a row on V' and the outputs, and shared memory
// addressed as such, 2.7, with outputs of 11 bits and powers of two from bounds
// that missed (see above); with neither 3.3, and with less code 2.9.  CTAs that
// take over others' rows as they finish (cluster launch control) were 9% slower
// over 256 rows of 1 to 45 tokens x 32 heads than rows dealt out in turn.
//   A single long row is a chain: a turn a chunk, 2.6 us where two CTAs share it
// (32 heads x 16001 tokens 2.58 ms), 3.1 in one.  All warps' hand-backs to the other
// CTA, each with a release of its own, took 1,000 clocks a turn: one warp's does.
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
constexpr int kThreads = 512;
// Pairs of producer warps, a chunk each, and places of their rings, with 8
// consumer warps beside them, or 16 in another CTA (kSplit).  A chunk's operands
// lie in two rings: what the products with the state read is written from the
// chunk's first token on and done with in the middle of the consumers' turn, the
// rest is written at the end and done with a turn later.
template <bool kSplit>
constexpr int kPairs = kSplit ? 7 : 4;
template <bool kSplit>
constexpr int kReaches = kSplit ? 7 : 5;
template <bool kSplit>
constexpr int kUpdates = kSplit ? 7 : 4;
// A pair waits for a place to be empty by the parity of its turn: all that was
// taken from it before that is done when the pair's last chunk was begun.
static_assert(kPairs<true> <= kReaches<true> && kPairs<false> <= kReaches<false> &&
                  kPairs<true> <= kUpdates<true> && kPairs<false> <= kUpdates<false>,
              "a wait for a place is never two turns ahead");

#ifdef KDA_TEST_PREFILL_WAIT_BUDGET  // a test build: a wait that runs out, soon
constexpr long long kWaitBudget = KDA_TEST_PREFILL_WAIT_BUDGET;
#else
constexpr long long kWaitBudget = 4000000000LL;   // clock cycles (about 2 s)
#endif

// Powers of two on the operands.
constexpr int kKeyExponent = 14;          // K P, Q P: of the largest P
constexpr float kKeyLeast = 0x1p10f;      // below which it is moved there again
constexpr int kUpdateExponent = 13;       // of a token's largest K P_C / P_t

// One chunk's operands: fp16 matrices of rows of 128 bytes with the 128-byte
// swizzle (16-byte unit u of row r at u ^ (r & 7)), two blocks of 64 channels.
constexpr int kTall = 4 * kC;             // rows: K P hi, Q P hi, K P lo, Q P lo
struct __align__(1024) Reach {
    // [64 channels][row]: channels along K, the tokens of Q P in the order of V'
    unsigned char reach[2][kTall * 128];
    __nv_bfloat16 v[kC][kD];
};
struct __align__(1024) Update {
    unsigned char update[2][2][kC * 128]; // K P_C / P_t, [hi, lo][64 channels][token's place]
    float inner[kC][2 * kC];              // [token t]: (B T)_t, then T_t
    float decay[kD];                      // P_C
    float given[kC];                      // [token's place]: about its largest K P_C / P_t
    float undo[2][kC];                    // K P and Q P are held times 1 / undo: [token], [place]
};

// Consumer threads that share a row of S: each has its part of the columns and
// of the tokens.
template <bool kSplit>
constexpr int kParts = kSplit ? 4 : 2;

// A part's i-th token, in order along V'.  All parts have the same to do: the T
// of their tokens have as many entries up to the diagonal's group of four (0 3
// 4 7 8 11 12 15 and 1 2 5 6 9 10 13 14 of two parts; 0 7 8 15, 1 6 9 14 ... of
// four).
template <bool kSplit>
__device__ __forceinline__ int token_of(int part, int i) {
    const int group = kSplit ? i : i >> 1;
    return 4 * group + ((i & 1) ? 3 - part : part);
}

// The place along V' of token t.
template <bool kSplit>
__device__ __forceinline__ int order_of(int t) {
    const int group = t >> 2, off = t & 3;
    if (kSplit) return 4 * ((group & 1) ? 3 - off : off) + group;
    const int part = off == 0 || off == 3 ? 0 : 1;
    return 8 * part + 2 * group + (off >> 1);
}

// Byte offset of channel c (even, of 64) of row r.
__device__ __forceinline__ int place(int r, int c) {
    return r * 128 + ((((c >> 3) ^ r) & 7) << 4) + (c & 7) * 2;
}

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
    float a[kC][kC + 4], b[kC][kC + 4], t[kC][kC];
    float beta[kC];
    uint64_t ready[2], taken[2];
};

template <bool kSplit>
struct Work_space {
    Reach reach[kReaches<false>];
    Update update[kUpdates<false>];
    Scratch scratch[kPairs<false>];
};
template <>
struct Work_space<true> {
    union {
        struct {                          // of the CTA that consumes
            Reach reach[kReaches<true>];
            Update update[kUpdates<true>];
        };
        Scratch scratch[kPairs<true>];    // of the other
    };
};

// The rows and heads of a CTA: one, and more of those that are left (make_plan;
// dealt out in turn where it makes none).
constexpr unsigned kNone = 0xffffffffu;
constexpr int kPlanRows = kThreads;
struct Plan {
    unsigned short row[kPlanRows];
    unsigned rest, end;                        // places of the CTA's items
    unsigned down, across;                     // items of a column, columns
    int planned;                               // 0: dealt out in turn
};

template <bool kSplit>
struct Shared : Work_space<kSplit> {
    Plan plan;
    // (what is read 16 bytes at a time)
    __align__(16) float most[kParts<kSplit>][kD];  // largest of each part of a row of S
    __align__(16) float sum[kParts<kSplit>][kD];   // of |V'| as given, of each part's tokens
    __align__(16) float zeros[kD], ones[kD];
    uint64_t full[kReaches<kSplit>];      // both operands
    uint64_t reach_empty[kReaches<kSplit>], update_empty[kUpdates<kSplit>];
    uint64_t u_done, s_done;              // products of a chunk
    uint64_t drained;
    int gave_up;
    uint32_t tmem;
};

static_assert(sizeof(Shared<true>) <= 227 * 1024 && sizeof(Shared<false>) <= 227 * 1024,
              "a CTA's shared memory");

// Columns of tensor memory.
constexpr uint32_t kColState = 0;         // S, fp32, 128
constexpr uint32_t kColS = 128;           // S as fp16: 64 of hi, 64 of lo, two channels each
constexpr uint32_t kColUpdate = 256;      // V'^T (K P_C / P_t), 128
constexpr uint32_t kColReach = 384;       // S (K P | Q P | K P lo | Q P lo)^T, 64
constexpr uint32_t kColLow = 448;         // lo of S with hi of K P and of Q P, 32
constexpr uint32_t kColY = 480;           // V': 8 of hi, 8 of lo
constexpr uint32_t kTmemColumns = 512;

// D += A B for k steps of 8 in tf32.
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

// floor(log2 |x|) of x, at least -110 (0 and the like), 127 for what is not
// finite.
__device__ __forceinline__ int exponent_of(float x) {
    const int e = (int)((__float_as_uint(x) >> 23) & 0xff) - 127;
    return max(-110, min(127, e));
}

__device__ __forceinline__ float power_of_two(int e) {   // -126 <= e <= 127
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float larger(float m, u64 xy) {   // of m >= 0, |x| and |y|
    const float2 v = both(xy);
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v.x), "f"(v.y));
    return m;
}

// Where two CTAs share a row and head (kSplit), the first consumes and the
// second produces: its operands and its arrivals go to the first's shared
// memory, as the consumers' arrivals come to it.
__device__ __forceinline__ uint32_t rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

template <typename T>
__device__ __forceinline__ T &at_rank(T &x, uint32_t r) {
    uint64_t y;
    asm("mapa.u64 %0, %1, %2;" : "=l"(y) : "l"(reinterpret_cast<uint64_t>(&x)), "r"(r));
    return *reinterpret_cast<T *>(y);
}

__device__ __forceinline__ void arrive_at(uint64_t *bar, uint32_t r) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(
            kda::smem_u32(bar)),
        "r"(r)
        : "memory");
}

__device__ __forceinline__ void meet_cluster() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}

// Whether the phase is over; across CTAs, with what was written before it.
template <bool kAcross>
__device__ __forceinline__ bool try_wait(uint64_t *bar, uint32_t parity) {
    if constexpr (!kAcross) return kda::mbar_try_wait(bar, parity);
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(kda::smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// The rest of a wait that is not over at once.
template <bool kAcross>
__device__ __noinline__ bool wait_on(int &gave_up, uint64_t *bar, uint32_t parity, int *err) {
    bool done = false;
    const long long t0 = clock64();
    while (!(done = try_wait<kAcross>(bar, parity))) {
        if (*reinterpret_cast<volatile int *>(&gave_up) != 0) break;
        if (clock64() - t0 > kWaitBudget) {
            *reinterpret_cast<volatile int *>(&gave_up) = 1;
            kda_cache::flag(err, KDA_ERR_WAIT_TIMEOUT);
            break;
        }
    }
    return __all_sync(kFull, done);
}

// Bounded wait of a warp: it gives up, as a whole, after the budget, or when
// another warp has.
template <bool kAcross = false, typename S>
__device__ __forceinline__ bool wait(S &sh, uint64_t *bar, uint32_t parity, int *err) {
    if (__all_sync(kFull, try_wait<kAcross>(bar, parity))) return true;
    return wait_on<kAcross>(sh.gave_up, bar, parity, err);
}

struct Work {   // one row and head
    Row row;
    int head;
};

template <bool kPlanned>
__device__ __forceinline__ Work work_at(const Params &p, const Plan &plan, unsigned item,
                                        int &bits) {
    const unsigned at = item / (unsigned)p.H;
    Work w;
    w.head = (int)(item - at * (unsigned)p.H);
    w.row = kda_delta::read_row(p, kPlanned && plan.planned ? plan.row[at] : (int)at, bits);
    return w;
}

// Keeps the compiler from fetching operands so far ahead that registers run out.
__device__ __forceinline__ void no_further_ahead() { asm volatile("" ::: "memory"); }

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

// The polynomial of kda::softplus, log1p(z) = z P(z), as pairs of fp32.
struct Poly {
    u64 c[10];
};
__device__ __forceinline__ Poly softplus_poly() {
    constexpr float c[10] = {0x1p+0f,        -0x1.ffffcp-2f,  0x1.554c9cp-2f, -0x1.ff11c2p-3f,
                             0x1.930202p-3f, -0x1.399642p-3f, 0x1.b2c2a2p-4f, -0x1.d3784ep-5f,
                             0x1.4628bp-6f,  -0x1.aad1eep-9f};
    Poly p;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        p.c[i] = pair(c[i], c[i]);
        asm volatile("" : "+l"(p.c[i]));   // in registers, not made anew at each use
    }
    return p;
}

// log2 of two channels' decays, as kda::decay_factor has them.  x: the gate's
// inputs with their bias; gate: -exp(A_log) log2 e; bound: lower_bound log2 e.
template <bool kBounded>
__device__ __forceinline__ u64 log2_decays(u64 x, float gate, float bound, const Poly &poly) {
    if constexpr (kBounded) {
        const float2 y = both(mul_pair(x, pair(gate, gate)));
        return pair(__fdividef(bound, 1.0f + exp2_of(y.x)), __fdividef(bound, 1.0f + exp2_of(y.y)));
    } else {
        // softplus(x) = max(x, 0) + log1p(z), z = exp(-|x|)
        const float2 v = both(x);
        const u64 z = pair(exp2_of(-fabsf(v.x) * kLog2e), exp2_of(-fabsf(v.y) * kLog2e));
        u64 r = poly.c[9];
#pragma unroll
        for (int i = 8; i >= 0; --i) r = fma_pair(r, z, poly.c[i]);
        const u64 sp = fma_pair(z, r, pair(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
        return mul_pair(sp, pair(gate, gate));
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

// 1 / sqrt(sum + 1e-6), as kda::inv_l2 (the sum is never subnormal).
__device__ __forceinline__ float inverse_norm(float sum) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(sum + 1e-6f));
    return y;
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

// The place of chunk n of a CTA, and the wait for it to be empty.
template <bool kSplit>
__device__ __forceinline__ Update &update_of(Shared<kSplit> &sh, unsigned n) {
    Update &up = sh.update[n % kUpdates<kSplit>];
    return kSplit ? at_rank(up, 0) : up;
}

template <bool kSplit>
__device__ __forceinline__ bool wait_for_update(Shared<kSplit> &sh, unsigned n, int *err) {
    return wait<kSplit>(sh, &sh.update_empty[n % kUpdates<kSplit>],
                        ((n / kUpdates<kSplit>) & 1) ^ 1, err);
}

// The tokens' vectors of a chunk, by the first warp of a pair.  blocks: how
// many blocks of four tokens the pair has had.
template <bool kBounded, bool kSplit>
__device__ __forceinline__ bool produce_tokens(const Params &p, Shared<kSplit> &sh, Reach &st,
                                               unsigned n, Scratch &sc,
                                               const Row &row, int head, int chunk, int lane,
                                               unsigned &blocks) {
    lane = made_anew(lane);
    const long long first = (long long)row.first + (long long)chunk * kC;
    const int valid = min(kC, row.tokens - chunk * kC);
    const long long at = (long long)head * kD + 4 * lane;
    Inputs in{p.q + first * p.stride_q + at, p.k + first * p.stride_k + at,
              p.g + first * p.stride_g + at};
    Raw next = load_raw(p, in, true), later = load_raw(p, in, 1 < valid);
    {   // the values as they are
        const __nv_bfloat16 *src = p.v + first * p.stride_v + at;
#pragma unroll kSplit ? 8 : 1
        for (int t = 0; t < kC; ++t, src += p.stride_v) {
            if (!kSplit && t < valid)
                kda::cp_async8(&st.v[t][4 * lane], src);
            else
                *reinterpret_cast<uint2 *>(&st.v[t][4 * lane]) =
                    t < valid ? __ldg(reinterpret_cast<const uint2 *>(src)) : make_uint2(0u, 0u);
        }
    }
    kda::cp_async_commit();
    const float gate = -__expf(p.A_log[head]) * kLog2e, bound = p.lower_bound * kLog2e;
    const ulonglong2 biases = *reinterpret_cast<const ulonglong2 *>(p.g_bias + at);
    const u64 bias[2] = {biases.x, biases.y};
    Poly poly;
    if constexpr (!kBounded) poly = softplus_poly();
    const float start = power_of_two(kKeyExponent);
    u64 reach[2] = {pair(start, start), pair(start, start)};                   // P_t
    float undo = 1.0f, mine = 1.0f;   // of P_t, and of token `lane`'s
    u64 total[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};                       // log2 P_t
    u64 r[2] = {pair(1.0f, 1.0f), pair(1.0f, 1.0f)};                            // R
    unsigned char *reached = st.reach[lane >> 4];
    // two tokens a turn, the next two on their way
#pragma unroll 1
    for (int t0 = 0; t0 < kC; t0 += 2) {
        const Raw now[2] = {next, later};
        next = load_raw(p, in, t0 + 2 < valid);
        later = load_raw(p, in, t0 + 3 < valid);
        Block &out = sc.block[blocks & 1];
        if ((t0 & 2) == 0 && !wait(sh, &sc.taken[blocks & 1], ((blocks >> 1) & 1) ^ 1, p.err)) {
            kda::cp_async_wait_all();
            return false;
        }
        u64 k[2][2], q[2][2];
        float norm;   // lane bits 4 and 3 choose the token, and k or q
        {
            float s[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                pairs_of(now[u].k, k[u][0], k[u][1]);
                pairs_of(now[u].q, q[u][0], q[u][1]);
                s[2 * u] = squares(k[u][0], k[u][1]);
                s[2 * u + 1] = squares(q[u][0], q[u][1]);
            }
            const bool b4 = (lane & 16) != 0, b3 = (lane & 8) != 0;
            s[0] = (b4 ? s[2] : s[0]) + __shfl_xor_sync(kFull, b4 ? s[0] : s[2], 16);
            s[1] = (b4 ? s[3] : s[1]) + __shfl_xor_sync(kFull, b4 ? s[1] : s[3], 16);
            norm = (b3 ? s[1] : s[0]) + __shfl_xor_sync(kFull, b3 ? s[0] : s[1], 8);
            norm += __shfl_xor_sync(kFull, norm, 4);
            norm += __shfl_xor_sync(kFull, norm, 2);
            norm += __shfl_xor_sync(kFull, norm, 1);
            norm = inverse_norm(norm);
        }
        // one copy of the code for both where other warps' code lies beside it
        uint2 gates = now[0].g;
#pragma unroll kSplit ? 2 : 1
        for (int u = 0; u < 2; ++u) {
            const int t = t0 + u;
            u64 y[2] = {0ull, 0ull};   // behind the row's end nothing decays
            if (t < valid) {
                u64 x[2];
                pairs_of(gates, x[0], x[1]);
                y[0] = log2_decays<kBounded>(add_pair(x[0], bias[0]), gate, bound, poly);
                y[1] = log2_decays<kBounded>(add_pair(x[1], bias[1]), gate, bound, poly);
            }
            total[0] = add_pair(total[0], y[0]);
            total[1] = add_pair(total[1], y[1]);
            const float2 e0 = both(y[0]), e1 = both(y[1]);
            const float e[4] = {exp2_of(e0.x), exp2_of(e0.y), exp2_of(e1.x), exp2_of(e1.y)};
            reach[0] = mul_pair(reach[0], pair(e[0], e[1]));
            reach[1] = mul_pair(reach[1], pair(e[2], e[3]));
            const float most = larger(larger(0.0f, reach[0]), reach[1]);
            if (!__any_sync(kFull, most >= kKeyLeast)) {   // no channel has much left
                const int up = kKeyExponent - exponent_of(__uint_as_float(
                                   __reduce_max_sync(kFull, __float_as_uint(most))));
                const float f = power_of_two(min(up, 120));
                reach[0] = mul_pair(reach[0], pair(f, f));
                reach[1] = mul_pair(reach[1], pair(f, f));
                undo *= power_of_two(-min(up, 120));
            }
            if (lane == t) mine = undo;
            const float nk = __shfl_sync(kFull, norm, 16 * u);
            const float nq = __shfl_sync(kFull, norm, 16 * u + 8);
            const u64 rk = pair(nk, nk), rq = pair(nq, nq);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                k[0][i] = mul_pair(k[0][i], rk);
                q[0][i] = mul_pair(q[0][i], rq);
            }
            if (u == 0 && (t0 & 2) == 0) {   // a block's first token
                put(&out.since[4 * lane], mul_pair(r[0], pair(e[0], e[1])),
                    mul_pair(r[1], pair(e[2], e[3])));
                r[0] = r[1] = pair(1.0f, 1.0f);
            } else {
                r[0] = mul_pair(r[0], pair(fmaxf(e[0], 0x1p-40f), fmaxf(e[1], 0x1p-40f)));
                r[1] = mul_pair(r[1], pair(fmaxf(e[2], 0x1p-40f), fmaxf(e[3], 0x1p-40f)));
            }
            float *ahead = &out.ahead[t & 3][4 * lane];
            put(ahead, mul_pair(k[0][0], r[0]), mul_pair(k[0][1], r[1]));
            put(ahead + 4 * kRow, mul_pair(q[0][0], r[0]), mul_pair(q[0][1], r[1]));
            const float2 r0 = both(r[0]), r1 = both(r[1]);
            put(&out.back[t & 3][4 * lane],
                mul_pair(k[0][0], pair(reciprocal(r0.x), reciprocal(r0.y))),
                mul_pair(k[0][1], pair(reciprocal(r1.x), reciprocal(r1.y))));
            int to = place(t, 4 * (lane & 15));   // (rows 16 and 32 further swizzle alike)
            uint2 hi, lo;
            float2 x = both(mul_pair(k[0][0], reach[0]));
            split(x.x, x.y, hi.x, lo.x);
            x = both(mul_pair(k[0][1], reach[1]));
            split(x.x, x.y, hi.y, lo.y);
            *reinterpret_cast<uint2 *>(reached + to) = hi;
            *reinterpret_cast<uint2 *>(reached + to + 2 * kC * 128) = lo;
            to = place(kC + order_of<kSplit>(t), 4 * (lane & 15));
            x = both(mul_pair(q[0][0], reach[0]));
            split(x.x, x.y, hi.x, lo.x);
            x = both(mul_pair(q[0][1], reach[1]));
            split(x.x, x.y, hi.y, lo.y);
            *reinterpret_cast<uint2 *>(reached + to) = hi;
            *reinterpret_cast<uint2 *>(reached + to + 2 * kC * 128) = lo;
            gates = now[1].g;
#pragma unroll
            for (int i = 0; i < 2; ++i) k[0][i] = k[1][i], q[0][i] = q[1][i];
        }
        if ((t0 & 2) != 0) {
            put(&out.end[4 * lane], r[0], r[1]);
            __syncwarp();
            if (lane == 0) kda::mbar_arrive(&sc.ready[blocks & 1]);
            ++blocks;
        }
    }
    // P_C decays the state chunk after chunk, so its error adds up: from the sum
    // of the logarithms, not as a product; within 1 ulp also near 1, and as exact
    // beside itself where little is left (2^x has 2 ulp and the rounding of x)
    {
        const float2 x = both(total[0]), y = both(total[1]);
        float f[4] = {x.x, x.y, y.x, y.y};
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            const float v = f[0];
            f[0] = f[1];
            f[1] = f[2];
            f[2] = f[3];
            f[3] = v > -1.0f ? 1.0f + expm1f(v * 0.693147180559945309f) : exp2_of(v);
        }
        kda::cp_async_wait_all();
        if (!wait_for_update(sh, n, p.err)) return false;
        Update &up = update_of(sh, n);
        *reinterpret_cast<float4 *>(&up.decay[4 * lane]) = make_float4(f[0], f[1], f[2], f[3]);
        if (lane < kC) up.undo[0][lane] = up.undo[1][order_of<kSplit>(lane)] = mine;
    }
    __syncwarp();
    return true;
}

// The products between tokens, by the second warp of a pair.
template <bool kSplit>
__device__ __forceinline__ bool produce_products(const Params &p, Shared<kSplit> &sh, unsigned n,
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
    // lane 4 g + j: tokens s = g and g + 8, channels 16 m + 4 j + 0..3: k_s decayed
    // to where the block in work needs it
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
            const ulonglong2 n = *reinterpret_cast<const ulonglong2 *>(&in.ahead[g][c]);
            w[0][2 * m] = fma_pair(w[0][2 * m], f.x, k0.x);
            w[0][2 * m + 1] = fma_pair(w[0][2 * m + 1], f.y, k0.y);
            uint32_t hi[2][4] = {}, lo[2][4] = {};
            if (block >= 2) {   // tokens 8..15 come in here
                const ulonglong2 k1 = *reinterpret_cast<const ulonglong2 *>(&back1[c]);
                w[1][2 * m] = fma_pair(w[1][2 * m], f.x, k1.x);
                w[1][2 * m + 1] = fma_pair(w[1][2 * m + 1], f.y, k1.y);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    split_tf32(w[1][2 * m + h], hi[h][1], hi[h][3], lo[h][1], lo[h][3]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t b[2], bl[2];
                split_tf32(h ? n.y : n.x, b[0], b[1], bl[0], bl[1]);
                split_tf32(w[0][2 * m + h], hi[h][0], hi[h][2], lo[h][0], lo[h][2]);
                mma_tf32(d[0], hi[h], b[0], b[1]);
                mma_tf32(d[1], hi[h], bl[0], bl[1]);
                mma_tf32(d[1], lo[h], b[0], b[1]);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            // column 2 j (+ 1): the block's k 0..3, q 0..3; tokens s behind the block are
            // not looked at
            const float x = d[0][c] + d[1][c];
            (j < 2 ? sc.a : sc.b)[4 * block + 2 * (j & 1) + (c & 1)][g + 4 * (c & 2)] = x;
        }
        if (block == 3) {   // K P_C / P_t
            if (!wait_for_update(sh, n, p.err)) return false;
            Update &up = update_of(sh, n);
            float most[2] = {};
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                no_further_ahead();
                const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(&in.end[16 * m + 4 * j]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {   // tokens g and g + 8
                    w[i][2 * m] = mul_pair(w[i][2 * m], f.x);
                    w[i][2 * m + 1] = mul_pair(w[i][2 * m + 1], f.y);
                    most[i] = larger(larger(most[i], w[i][2 * m]), w[i][2 * m + 1]);
                }
            }
            // A token's are held beside their own largest, whose power of two V' takes:
            // what the chunk's decays leave of a token is as exact as what they leave of
            // the others, however large its value was.
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                most[i] = fmaxf(most[i], __shfl_xor_sync(kFull, most[i], 1));
                most[i] = fmaxf(most[i], __shfl_xor_sync(kFull, most[i], 2));
                const int e = exponent_of(most[i]), row = order_of<kSplit>(g + 8 * i);
                const float f = power_of_two(kUpdateExponent - e);
                if (j == 0) up.given[row] = power_of_two(e);
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    const float2 y = both(mul_pair(w[i][2 * m], pair(f, f)));
                    const float2 z = both(mul_pair(w[i][2 * m + 1], pair(f, f)));
                    uint2 hi, lo;
                    split(y.x, y.y, hi.x, lo.x);
                    split(z.x, z.y, hi.y, lo.y);
                    const int to = place(row, 16 * (m & 3) + 4 * j);
                    *reinterpret_cast<uint2 *>(up.update[0][m >> 2] + to) = hi;
                    *reinterpret_cast<uint2 *>(up.update[1][m >> 2] + to) = lo;
                }
            }
        }
        __syncwarp();
        if (lane == 0) kda::mbar_arrive(&sc.taken[blocks & 1]);
    }
    // T and B T, column s in a lane of each half of the warp, four rows at a time:
    // T_t = beta_t (1_t - sum_{j<t} A_tj T_j),  (B T)_t = sum_{j<=t} B_tj T_j
    {
        lane = made_anew(lane);
        const int s = lane & 15;
        const bool second = lane >= 16;   // B T
        Update &up = update_of(sh, n);
        const float(*const m)[kC + 4] = second ? sc.b : sc.a;
#pragma unroll 1
        for (int t = 0; t < kC; t += 4) {
            float x[4] = {};
#pragma unroll 1
            for (int i = 0; i < t; i += 4) {
                float y[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) y[u] = sc.t[i + u][s];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 n = kda::ld4(&m[t + u][i]);
                    x[u] = fmaf(n.x, y[0], x[u]);
                    x[u] = fmaf(n.y, y[1], x[u]);
                    x[u] = fmaf(n.z, y[2], x[u]);
                    x[u] = fmaf(n.w, y[3], x[u]);
                }
            }
            float y[4];   // T
            {
                const float4 b = kda::ld4(&sc.beta[t]);
                const float4 n1 = kda::ld4(&sc.a[t + 1][t]), n2 = kda::ld4(&sc.a[t + 2][t]);
                const float4 n3 = kda::ld4(&sc.a[t + 3][t]);
#pragma unroll
                for (int u = 0; u < 4; ++u) y[u] = (t + u == s ? 1.0f : 0.0f) - x[u];
                y[0] *= b.x;
                y[1] = b.y * fmaf(-n1.x, y[0], y[1]);
                y[2] = b.z * fmaf(-n2.y, y[1], fmaf(-n2.x, y[0], y[2]));
                y[3] = b.w * fmaf(-n3.z, y[2], fmaf(-n3.y, y[1], fmaf(-n3.x, y[0], y[3])));
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) y[u] = __shfl_sync(kFull, y[u], s);
            // (what lies above the diagonal of B is not looked at)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 n = kda::ld4(&sc.b[t + u][t]);
                float z = fmaf(n.x, y[0], x[u]);
                if (u > 0) z = fmaf(n.y, y[1], z);
                if (u > 1) z = fmaf(n.z, y[2], z);
                if (u > 2) z = fmaf(n.w, y[3], z);
                if (!second) sc.t[t + u][s] = z = y[u];
                up.inner[t + u][second ? s : kC + s] = z;
            }
            __syncwarp();
        }
    }
    return true;
}

// ---------------------------------------------------------------- consumer --

// Instruction descriptor of kind::f16: fp16 operands, fp32 sums, 128 rows, A
// along K, B along K or along N.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_along_n) {
    return (1u << 4) | ((b_along_n ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}

// B along N with the 128-byte swizzle: 64-column blocks `block` bytes apart,
// groups of 8 along K 1024 bytes apart.
__device__ __forceinline__ uint64_t along_n(uint32_t addr, uint32_t block) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)(block >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// D [+]= A B^T of one K step of 16, A from tensor memory; by one lane.
__device__ __forceinline__ void umma(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u)
        : "memory");
}

// One lane of the warp.
__device__ __forceinline__ bool elected() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// 16 or 8 columns of the warp's lanes; they are there behind arrived().
__device__ __forceinline__ void arrived(uint32_t (&u)[16]) {
    kda::tmem_wait_ld();
    asm volatile(""
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]),
                   "+r"(u[6]), "+r"(u[7]), "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]),
                   "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void arrived(uint32_t (&u)[8]) {
    kda::tmem_wait_ld();
    asm volatile(""
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]),
                   "+r"(u[6]), "+r"(u[7])
                 :
                 : "memory");
}

__device__ __forceinline__ void arrived(uint32_t (&u)[4]) {
    kda::tmem_wait_ld();
    asm volatile("" : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]) : : "memory");
}

__device__ __forceinline__ void load(uint32_t from, uint32_t (&u)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                 : "r"(from)
                 : "memory");
}

__device__ __forceinline__ void load(uint32_t from, uint32_t (&u)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7])
        : "r"(from)
        : "memory");
}

__device__ __forceinline__ void store8(uint32_t to, const uint32_t (&u)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(to),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
        : "memory");
}

__device__ __forceinline__ void store(uint32_t to, const uint32_t (&u)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
                 : "memory");
}

__device__ __forceinline__ void store(uint32_t to, const uint32_t (&u)[2]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(to), "r"(u[0]),
                 "r"(u[1])
                 : "memory");
}

__device__ __forceinline__ u64 pair_of(uint32_t x, uint32_t y) {
    return pair(__uint_as_float(x), __uint_as_float(y));
}

// The product of x, all tokens' of a chunk, with the row of a triangular matrix
// that is the part's i-th token's.  Behind the diagonal x counts as 0, whatever it
// is: 0 in the matrix would not do where it is not finite.
template <bool kSplit>
__device__ __forceinline__ float dot_row(const float *row, int i, int part,
                                         const u64 (&x)[kC / 2]) {
    const int last = kSplit ? i : i >> 1, off = (i & 1) ? 3 - part : part;   // token_of
    u64 sum = 0ull;
#pragma unroll
    for (int n = 0; n < last; ++n) {   // four entries each
        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(row + 4 * n);
        sum = n == 0 ? mul_pair(f.x, x[0]) : fma_pair(f.x, x[2 * n], sum);
        sum = fma_pair(f.y, x[2 * n + 1], sum);
    }
    const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(row + 4 * last);
    const float2 u = both(x[2 * last]), v = both(x[2 * last + 1]);
    const u64 w = kSplit || !(i & 1) ? pair(u.x, off > 0 ? u.y : 0.0f) : x[2 * last];
    sum = last == 0 ? mul_pair(f.x, w) : fma_pair(f.x, w, sum);
    if (kSplit)
        sum = fma_pair(f.y, pair(off > 1 ? v.x : 0.0f, off > 2 ? v.y : 0.0f), sum);
    else if (i & 1)
        sum = fma_pair(f.y, pair(v.x, off > 2 ? v.y : 0.0f), sum);
    const float2 y = both(sum);
    return y.x + y.y;
}

// Named barriers of the consumers.
template <int kId, int kMembers>
__device__ __forceinline__ void meet() {
    asm volatile("bar.sync %0, %1;" ::"n"(kId), "n"(kMembers) : "memory");
}

template <int kN>
__device__ __forceinline__ void undo_pairs(u64 (&x)[kN], const float *undo) {
    asm volatile("" ::: "memory");   // (a branch, not predicated loads)
#pragma unroll
    for (int n = 0; n < kN; n += 2) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(undo + 2 * n);
        x[n] = mul_pair(x[n], f.x);
        x[n + 1] = mul_pair(x[n + 1], f.y);
    }
}

// Those that share 32 rows of S.
template <int kOf>
__device__ __forceinline__ void meet_row(int me) {
    asm volatile("bar.sync %0, %1;" ::"r"(3 + (me & 3)), "n"(32 * kOf) : "memory");
}

// 16 channels of a row of S, as they are and as two fp16 numbers each, to
// tensor memory: state and halves are the columns of the first.
__device__ __forceinline__ void store_state(uint32_t state, uint32_t halves, const u64 (&s)[8]) {
    uint32_t x[16], hi[8], lo[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float2 y = both(s[c]);
        x[2 * c] = __float_as_uint(y.x);
        x[2 * c + 1] = __float_as_uint(y.y);
        split(y.x, y.y, hi[c], lo[c]);
    }
    kda::tmem_st16(state, x);
    store8(halves, hi);
    store8(halves + 64, lo);
}

// 2 kPairsOf values times `scale` as two fp16 numbers each: hi to as many
// columns, lo to those that are 8 further.
template <int kPairsOf>
__device__ __forceinline__ void store_split(uint32_t to, const u64 (&x)[kPairsOf], float scale) {
    uint32_t hi[kPairsOf], lo[kPairsOf];
    const u64 f = pair(scale, scale);
#pragma unroll
    for (int c = 0; c < kPairsOf; ++c) {
        const float2 y = both(mul_pair(x[c], f));
        split(y.x, y.y, hi[c], lo[c]);
    }
    store(to, hi);
    store(to + 8, lo);
}

// S is held times 2^ex, a power of its row.  As held, a bound of the row's largest
// stays below 2^15, so that fp16 has it, and the largest above 2^-2, so that what
// is left out of two fp16 numbers, 2^-25, is below 2^-23 of it; else the row moves
// to 2^8.  (Rows gain and lose some powers of two from chunk to chunk where strong
// decays leave the last tokens' values alone: moving costs a twentieth of a turn.)
constexpr int kHeld = 8, kLeast = -2, kMost = 14, kMostExponent = 119;

__device__ __forceinline__ int state_exponent(float bound, int ex) {
    const int e = exponent_of(bound);
    return e + ex > kMost || e + ex < kLeast ? min(kHeld - e, kMostExponent) : ex;
}

// The products of a chunk, by one warp each.
__device__ __forceinline__ void issue_reach(const Reach &st, uint32_t tmem) {
    const uint64_t b = kda::sw128_desc(kda::smem_u32(st.reach[0]));
#pragma unroll
    for (int k = 0; k < 8; ++k)
        umma(tmem + kColReach, tmem + kColS + 8 * k,
             b + (((k >> 2) * kTall * 128 + (k & 3) * 32) >> 4), idesc(kTall, false), k > 0);
}

// (columns of their own: products of different shapes are not kept in order)
__device__ __forceinline__ void issue_low(const Reach &st, uint32_t tmem) {
    const uint64_t b = kda::sw128_desc(kda::smem_u32(st.reach[0]));
#pragma unroll
    for (int k = 0; k < 8; ++k)
        umma(tmem + kColLow, tmem + kColS + 64 + 8 * k,
             b + (((k >> 2) * kTall * 128 + (k & 3) * 32) >> 4), idesc(2 * kC, false), k > 0);
}

__device__ __forceinline__ void issue_update(const Update &st, uint32_t tmem) {
    constexpr uint32_t kAll = idesc(kD, true);
    const uint64_t hi = along_n(kda::smem_u32(st.update[0][0]), kC * 128);
    const uint64_t lo = along_n(kda::smem_u32(st.update[1][0]), kC * 128);
    umma(tmem + kColUpdate, tmem + kColY, hi, kAll, false);
    umma(tmem + kColUpdate, tmem + kColY, lo, kAll, true);
    umma(tmem + kColUpdate, tmem + kColY + 8, hi, kAll, true);
}

// ------------------------------------------------------------------ kernel --

// The sum over the CTA's threads up to this one.
__device__ __forceinline__ u64 sum_up_to(u64 *sums, u64 sum) {
    const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int o = 1; o < 32; o *= 2) {
        const u64 x = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += x;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
#pragma unroll 1
    for (unsigned i = 0; i < warp; ++i) sum += sums[i];
    return sum;
}

// A CTA's rows and heads by cost: a chunk is 2, a state 5 (its way in and out
// takes as long as some 2.5 chunks).  In the order of falling cost each CTA takes
// one of the first.  What is left goes to the CTAs whose first is below the level
// that this fills them up to, D of them: dealt out to as many columns in turn, the
// columns lie one behind the other on a line, and the CTAs take of it, in turn, as
// much as their firsts leave room for.  An item is the CTA's that its middle falls
// to, so a CTA is over the level by half an item at most, or by its first one.
// All CTAs come to the same.
__device__ __forceinline__ void make_plan(const Params &p, Shared<false> &sh, unsigned items) {
    Plan &plan = sh.plan;
    unsigned *key = reinterpret_cast<unsigned *>(sh.reach[0].reach);   // not in use yet
    unsigned *cost = key + kPlanRows;
    u64 *sums = reinterpret_cast<u64 *>(cost + kPlanRows);
    u64 *column = sums + kThreads / 32;   // where it starts
    u64 *start = column + kThreads + 1;   // of a row's cost for a head, falling
    static_assert(2 * 4 * kPlanRows + 8 * (kThreads / 32 + kThreads + 1 + kPlanRows + 2) <=
                      sizeof(Reach::reach),
                  "what the plan is made of");
    const unsigned tid = threadIdx.x, B = (unsigned)p.B, H = (unsigned)p.H, G = gridDim.x;
    unsigned mine = 0;
    if (tid < B) {
        int bits = 0;   // flagged where the row's turn comes
        const unsigned n = (unsigned)kda_delta::read_row(p, (int)tid, bits).tokens;
        mine = n == 0 ? 1 : min(2 * ((n + kC - 1) / kC) + 5, (1u << 23) - 1);
    }
    u64 sum = sum_up_to(sums, mine);
    if (tid == kThreads - 1) column[0] = sum;
    __syncthreads();
    // Where no row is long beside a CTA's share, dealing out in turn does as well (256
    // rows of 1 to 45 tokens x 32 heads: 770 us in turn, 763 planned) and needs no plan.
    if (__syncthreads_or((u64)mine * G * 8 > column[0] * H) == 0) {
        if (tid == 0) plan.planned = 0;
        return;
    }
    const unsigned my_key = mine * kPlanRows + (kPlanRows - 1 - tid);
    key[tid] = my_key;   // (those behind the last row are below all others)
    cost[tid] = 0;
    __syncthreads();
    unsigned place = 0;
#pragma unroll 1
    for (unsigned r = 0; r < B; r += 4) {
        const uint4 c = *reinterpret_cast<const uint4 *>(key + r);
        place += (unsigned)(c.x > my_key) + (unsigned)(c.y > my_key) + (unsigned)(c.z > my_key) +
                 (unsigned)(c.w > my_key);
    }
    if (tid < B) {
        plan.row[place] = (unsigned short)tid;
        cost[place] = mine;
    }
    __syncthreads();
    sum = sum_up_to(sums, cost[tid]);
    start[tid + 1] = sum;
    if (tid == 0) start[0] = 0;
    if (tid == kThreads - 1) start[kPlanRows + 1] = sum;
    __syncthreads();
    auto cost_of = [&](unsigned n) { return start[n / H + 1] - start[n / H]; };
    auto start_of = [&](unsigned n) { return start[n / H] * H + n % H * cost_of(n); };
    const u64 total = start_of(items);
    // The CTAs whose first item alone is over the level of it and those behind it.
    const unsigned full = (unsigned)__syncthreads_count(
        tid < G && cost_of(tid) * (G - tid) > total - start_of(tid));
    const unsigned share = G - full, left = items - G;
    const unsigned across = min(share, left), down = (left + across - 1) / across;
    const unsigned row_step = across / H, head_step = across % H;
    // Down column x from the top: whether `stop` at an item of cost c behind a sum.
    auto walk = [&](unsigned x, u64 &sum, auto stop) {
        unsigned n = G + x, y = 0, k = n / H, h = n % H;
#pragma unroll 1
        for (; n < items; n += across, ++y) {
            const unsigned c = cost[k];
            if (stop(sum, c)) return y;
            sum += c;
            k += row_step;
            h += head_step;
            if (h >= H) h -= H, ++k;
        }
        return down;
    };
    sum = 0;
    if (tid < across) walk(tid, sum, [](u64, unsigned) { return false; });
    sum = sum_up_to(sums, sum);
    column[tid + 1] = sum;
    if (tid == 0) column[0] = 0;
    __syncthreads();
#pragma unroll 1
    for (unsigned i = 0; i < 2; ++i) {   // where this CTA's part of the line starts and ends
        const unsigned j = blockIdx.x + i;
        // (times D)
        const u64 edge = j <= full ? 0 : (total - start_of(full)) * (j - full) -
                                             share * (start_of(j) - start_of(full));
        const unsigned x =
            (unsigned)__syncthreads_count(tid < across && column[tid] * share <= edge) - 1;
        if (tid == 0) {
            sum = column[x];
            (i == 0 ? plan.rest : plan.end) =   // the first item with its middle behind it
                x * down + walk(x, sum, [&](u64 at, unsigned c) {
                    return (2 * at + c) * share >= 2 * edge;
                });
        }
    }
    if (tid == 0) {
        plan.down = down;
        plan.across = across;
        plan.planned = 1;
    }
}

template <bool kSplit>
__device__ __forceinline__ unsigned first_item() {
    return kSplit ? blockIdx.x >> 1 : blockIdx.x;
}

// The CTA's item behind this one; in a plan the one at place i, or the next one behind
// it.
template <bool kPlanned, bool kSplit>
__device__ __forceinline__ unsigned next_item(const Plan &plan, unsigned item, unsigned &i,
                                              unsigned items) {
    const unsigned in_turn = item + (kSplit ? gridDim.x >> 1 : gridDim.x);
    if constexpr (kPlanned) {
        if (!plan.planned) return in_turn;
        while (i < plan.end) {
            const unsigned x = i / plan.down, n = gridDim.x + (i - x * plan.down) * plan.across + x;
            ++i;
            if (n < items) return n;
        }
        return kNone;
    }
    return in_turn;
}

// A producer warp: the tokens' vectors (the first kPairs) or the products
// between them of every kPairs-th chunk of the CTA's work.
template <bool kBounded, bool kSplit, bool kPlanned>
__device__ __forceinline__ void produce(const Params &p, Shared<kSplit> &sh, unsigned items,
                                        int warp, int lane) {
    const unsigned pair_of = warp % kPairs<kSplit>;
    unsigned count = 0, blocks = 0;
    for (unsigned next = kPlanned ? sh.plan.rest : 0, item = first_item<kSplit>(); item < items;
         item = next_item<kPlanned, kSplit>(sh.plan, item, next, items)) {
        int bits = 0;
        const Work w = work_at<kPlanned>(p, sh.plan, item, bits);
        if (bits != 0 && w.head == 0 && threadIdx.x == 0) kda_cache::flag(p.err, bits);
        if (warp == 0 && lane == 0 && w.row.tokens > 0 && w.row.from > 0)
            // the state is on its way to L2 before a consumer asks for it
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             p.pool + ((long long)w.row.from * p.H + w.head) * kda_delta::kTile),
                         "r"(kda_delta::kTile * 4)
                         : "memory");
        const unsigned chunks = (unsigned)(w.row.tokens + kC - 1) / kC;
        for (unsigned c = (pair_of + kPairs<kSplit> - count % kPairs<kSplit>) % kPairs<kSplit>;
             c < chunks; c += kPairs<kSplit>) {
            const unsigned n = count + c;
            Reach &reach = kSplit ? at_rank(sh.reach[n % kReaches<kSplit>], 0)
                                  : sh.reach[n % kReaches<kSplit>];
            Scratch &sc = sh.scratch[pair_of];
            bool made;
            if (warp < kPairs<kSplit>)
                made = (kSplit ? wait_for_update(sh, n, p.err)
                               : wait<kSplit>(sh, &sh.reach_empty[n % kReaches<kSplit>],
                                              ((n / kReaches<kSplit>) & 1) ^ 1, p.err)) &&
                       produce_tokens<kBounded, kSplit>(p, sh, reach, n, sc, w.row, w.head, c, lane, blocks);
            else
                made = produce_products<kSplit>(p, sh, n, sc, w.row, w.head, c, lane, blocks);
            if (!made) return;
            // the tensor cores read it
            if (kSplit)
                asm volatile("fence.proxy.async;" ::: "memory");
            else
                kda::fence_proxy_async_smem();
            __syncwarp();
#ifdef KDA_TEST_PREFILL_WAIT_BUDGET
            if (item == 0) continue;   // the first row and head's operands are never handed over
#endif
            if (lane == 0) {
                if (kSplit)
                    arrive_at(&sh.full[n % kReaches<kSplit>], 0);
                else
                    kda::mbar_arrive(&sh.full[n % kReaches<kSplit>]);
            }
        }
        count += chunks;
    }
}

// The largest of a row's parts.
template <int kOf>
__device__ __forceinline__ float largest_of(const float (&x)[kOf][kD], int r) {
    float m = fmaxf(x[0][r], x[1][r]);
    if constexpr (kOf > 2) m = fmaxf(m, fmaxf(x[2][r], x[3][r]));
    return m;
}

// The warp is done with a place of a ring.
__device__ __forceinline__ void hand_back(uint64_t *empty, int lane) {
    __syncwarp();
    if (lane == 0) kda::mbar_arrive(empty);
}

// The consumer warps.  A wait that runs out ends nothing by itself: from then
// on the warp, and soon all of them, go through the same barriers without
// waiting, issuing or writing, so that no barrier is left with too few.
template <bool kSplit, bool kPlanned>
__device__ __forceinline__ void consume(const Params &p, Shared<kSplit> &sh, unsigned items, int me,
                                        int lane) {
    constexpr int kOf = kParts<kSplit>, kCols = kD / kOf, kTokens = kC / kOf;
    const int part = me >> 2, r = 32 * (me & 3) + lane;   // columns of S, and the row
    const uint32_t tmem = sh.tmem + ((uint32_t)(32 * (me & 3)) << 16);
    const uint32_t state = tmem + kColState + kCols * part;
    const uint32_t halves = tmem + kColS + kCols / 2 * part;
    bool ok = true;
    unsigned count = 0;
    for (unsigned next = kPlanned ? sh.plan.rest : 0, item = first_item<kSplit>(); item < items;
         item = next_item<kPlanned, kSplit>(sh.plan, item, next, items)) {
        int bits = 0;
        const Work w = work_at<kPlanned>(p, sh.plan, item, bits);
        if (w.row.tokens == 0) continue;
        const long long slot = (long long)p.H * kda_delta::kTile;
        const long long at = (long long)w.head * kda_delta::kTile + r * kD + kCols * part;
        float bound;   // the largest of the row's values, or above it
        int ex;
        {
            const float *src = p.pool + max(w.row.from, 0) * slot + at;
            u64 s[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i) {
                ulonglong2 y = make_ulonglong2(0ull, 0ull);
                if (w.row.from > 0) y = *reinterpret_cast<const ulonglong2 *>(src + 4 * i);
                s[2 * i] = y.x;
                s[2 * i + 1] = y.y;
            }
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) most = larger(most, s[i]);
            sh.most[part][r] = most;
#pragma unroll
            for (int i = 0; i < kCols / 16; ++i) {
                uint32_t y[16];
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float2 z = both(s[8 * i + n]);
                    y[2 * n] = __float_as_uint(z.x);
                    y[2 * n + 1] = __float_as_uint(z.y);
                }
                kda::tmem_st16(state + 16 * i, y);
            }
            kda::tmem_wait_st();
            meet_row<kOf>(me);
            bound = largest_of<kOf>(sh.most, r);
            ex = min(kHeld - exponent_of(bound), kMostExponent);
            const u64 f = pair(power_of_two(ex), power_of_two(ex));
#pragma unroll 1
            for (int i = 0; i < kCols / 16; ++i) {   // (one copy of the code)
                uint32_t x[16];
                kda::tmem_ld16(state + 16 * i, x);
                arrived(x);
                u64 y[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) y[n] = mul_pair(pair_of(x[2 * n], x[2 * n + 1]), f);
                store_state(state + 16 * i, halves + 8 * i, y);
            }
        }
        const int chunks = (w.row.tokens + kC - 1) / kC;
        int step = 0;                               // of ex, due with the next addition
        float added = 0.0f;
        const int token = p.H * kD;
        uint16_t *const out = reinterpret_cast<uint16_t *>(p.out) +
                              (long long)w.row.first * token + w.head * kD + r;
        uint32_t result[kTokens / 2] = {};   // outputs of the last chunk
        // turn c adds what chunk c - 1 brought, makes chunk c's V' and writes its outputs
        for (int c = 0; c <= chunks; ++c) {
            if (c > 0) {
                const unsigned before = count - 1;
                ok &= wait(sh, &sh.s_done, before & 1, p.err);
                kda::tc_fence_after();
                const float *decay = &sh.update[before % kUpdates<kSplit>].decay[kCols * part];
                bool all = (c & 3) == 0;   // look at all columns, not at some
                for (;;) {
                    float most = 0.0f;
                    const u64 factor = pair(added, added);
                    const bool moved = __any_sync(kFull, step != 0);
                    // (16 columns at a time: code of 32 took longer, see the kernel's size)
#pragma unroll 1
                    for (int i = 0; i < kCols / 16; ++i) {
                        uint32_t u[16], x[16];
                        kda::tmem_ld16(tmem + kColUpdate + kCols * part + 16 * i, u);
                        kda::tmem_ld16(state + 16 * i, x);
                        arrived(u);
                        arrived(x);
                        u64 s[8];
#pragma unroll
                        for (int n = 0; n < 8; ++n) s[n] = pair_of(x[2 * n], x[2 * n + 1]);
                        if (moved) {   // in two powers: a step may be twice as far as one goes
                            const float g = power_of_two(step / 2);
                            const float g2 = power_of_two(step - step / 2);
#pragma unroll
                            for (int n = 0; n < 8; ++n)
                                s[n] = mul_pair(mul_pair(s[n], pair(g, g)), pair(g2, g2));
                        }
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const ulonglong2 d =
                                *reinterpret_cast<const ulonglong2 *>(decay + 16 * i + 4 * n);
                            s[2 * n] = fma_pair(pair_of(u[4 * n], u[4 * n + 1]), factor,
                                                mul_pair(s[2 * n], d.x));
                            s[2 * n + 1] = fma_pair(pair_of(u[4 * n + 2], u[4 * n + 3]), factor,
                                                    mul_pair(s[2 * n + 1], d.y));
                        }
                        most = larger(larger(most, s[0]), s[1]);
                        if (all)
#pragma unroll
                            for (int n = 2; n < 8; ++n) most = larger(most, s[n]);
                        store_state(state + 16 * i, halves + 8 * i, s);
                    }
                    if (c == chunks) break;
                    // The bound knows of no decay.  Where the row is far below it, the columns
                    // that were looked at are: then all are, and the row moves.
                    sh.most[part][r] = most;
                    meet_row<kOf>(me);
                    most = largest_of<kOf>(sh.most, r);
                    if (all) bound = most * power_of_two(-ex);
                    const bool low = bound > 0.0f && exponent_of(most) < kLeast;
                    step = low && all ? min(kHeld - exponent_of(most), kMostExponent - ex) : 0;
                    ex += step;
                    if (!__any_sync(kFull, low && !(all && step == 0))) break;
                    all = true;
                    added = 0.0f;   // (it is there)
                    decay = sh.ones;
                    kda::tmem_wait_st();
                    meet_row<kOf>(me);   // before `most` is written again
                }
            }
            if (c < chunks) {
                ok &= wait<kSplit>(sh, &sh.full[count % kReaches<kSplit>],
                                   (count / kReaches<kSplit>) & 1, p.err);
                kda::tmem_wait_st();
                kda::tc_fence_before();
                meet<1, 128 * kOf>();
                if (ok && me == 0 && elected()) {
                    kda::tc_fence_after();
                    if (kSplit) kda::fence_proxy_async_smem();
                    issue_reach(sh.reach[count % kReaches<kSplit>], sh.tmem);
                    kda::umma_commit(&sh.u_done);
                }
                __syncwarp();
                if (ok && me == 4 && elected()) {
                    kda::tc_fence_after();
                    if (kSplit) kda::fence_proxy_async_smem();
                    issue_low(sh.reach[count % kReaches<kSplit>], sh.tmem);
                    kda::umma_commit(&sh.u_done);
                }
                __syncwarp();
            }
            if (c > 0) {
                uint64_t *empty = &sh.update_empty[(count - 1) % kUpdates<kSplit>];
                if constexpr (kSplit) {
                    // (one for all, who have met: its release takes some 1000 clocks)
                    if (c == chunks) meet<1, 128 * kOf>();
                    if (me == 4 * kOf - 1 && lane == 0) arrive_at(empty, 1);
                    __syncwarp();
                } else {
                    hand_back(empty, lane);
                }
                // (behind that, which would wait for what was written before it)
                const int n = ok ? w.row.tokens - (c - 1) * kC : 0;
                uint16_t *to = out + (long long)(c - 1) * kC * token;
                uint16_t *even = to + part * token, *odd = to + (3 - part) * token;   // token_of
                const int step = 4 * token, evens = n - part, odds = n - (3 - part);
#pragma unroll
                for (int i = 0; i < kTokens; i += 2) {
                    const int g = kSplit ? i : i >> 1, h = kSplit ? i + 1 : g;   // fours of tokens
                    if (4 * g < evens) even[g * step] = (uint16_t)result[i / 2];
                    if (4 * h < odds) odd[h * step] = (uint16_t)(result[i / 2] >> 16);
                }
            }
            if (c == chunks) break;
            const unsigned parity = count & 1;
            const Reach &st = sh.reach[count % kReaches<kSplit>];
            const Update &up = sh.update[count % kUpdates<kSplit>];
            u64 x[kC / 2];
#pragma unroll
            for (int n = 0; n < kC / 2; ++n)
                x[n] = pair(__bfloat162float(st.v[2 * n][r]), __bfloat162float(st.v[2 * n + 1][r]));
            const float fx = -power_of_two(-ex) / (float)(1 << kKeyExponent);
            const bool undo = up.undo[0][kC - 1] != 1.0f;   // (of some token, then of the last)
            ok &= wait(sh, &sh.u_done, parity, p.err);
            kda::tc_fence_after();
            {
                uint32_t u[16], y[16], z[16];
                u64 s[kC / 2];
                kda::tmem_ld16(tmem + kColReach, u);
                kda::tmem_ld16(tmem + kColReach + 2 * kC, y);
                kda::tmem_ld16(tmem + kColLow, z);
                arrived(u);
                arrived(y);
                arrived(z);
#pragma unroll
                for (int n = 0; n < kC / 2; ++n)
                    s[n] = add_pair(pair_of(u[2 * n], u[2 * n + 1]),
                                    add_pair(pair_of(y[2 * n], y[2 * n + 1]),
                                             pair_of(z[2 * n], z[2 * n + 1])));
                if (undo) undo_pairs(s, up.undo[0]);
#pragma unroll
                for (int n = 0; n < kC / 2; ++n) x[n] = fma_pair(s[n], pair(fx, fx), x[n]);
            }
            if (!kSplit) hand_back(&sh.reach_empty[count % kReaches<kSplit>], lane);
            float sum = 0.0f, back;   // of |V'| as given, of the row's tokens
            {
                u64 y[kTokens / 2];   // V' of the part's tokens, times what is given of them
#pragma unroll
                for (int i = 0; i < kTokens; i += 2) {
                    const float *f = up.inner[token_of<kSplit>(part, i)] + kC;
                    const float *f1 = up.inner[token_of<kSplit>(part, i + 1)] + kC;
                    y[i / 2] = mul_pair(
                        pair(dot_row<kSplit>(f, i, part, x),
                             dot_row<kSplit>(f1, i + 1, part, x)),
                        *reinterpret_cast<const u64 *>(&up.given[kTokens * part + i]));
                    const float2 z = both(y[i / 2]);
                    sum += fabsf(z.x) + fabsf(z.y);
                }
                // the power of two is from V' itself, so that weakly written tokens keep
                // their bits (a bound by the values and the state does not know beta)
                sh.sum[part][r] = sum;
                meet_row<kOf>(me);
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kOf; ++i) sum += sh.sum[i][r];
                const int ey = 13 - exponent_of(sum);
                store_split(tmem + kColY + kTokens / 2 * part, y, power_of_two(ey));
                back = power_of_two(-ey);
            }
            kda::tmem_wait_st();
            kda::tc_fence_before();
            meet<2, 128 * kOf>();
            if (ok && me == 0 && elected()) {
                kda::tc_fence_after();
                issue_update(up, sh.tmem);
                kda::umma_commit(&sh.s_done);
            }
            __syncwarp();
            {   // outputs, from the state and from the chunk itself, while S is updated
                u64 o[kTokens / 2];
                {
                    uint32_t hi[kTokens], lo[kTokens], low[kTokens];
                    load(tmem + kColReach + kC + kTokens * part, hi);
                    load(tmem + kColReach + 3 * kC + kTokens * part, lo);
                    load(tmem + kColLow + kC + kTokens * part, low);
                    arrived(hi);
                    arrived(lo);
                    arrived(low);
                    const float f = power_of_two(-ex) * (p.scale / (float)(1 << kKeyExponent));
#pragma unroll
                    for (int i = 0; i < kTokens; i += 2)
                        o[i / 2] = mul_pair(add_pair(pair_of(hi[i], hi[i + 1]),
                                                     add_pair(pair_of(lo[i], lo[i + 1]),
                                                              pair_of(low[i], low[i + 1]))),
                                            pair(f, f));
                    if (undo) undo_pairs(o, &up.undo[1][kTokens * part]);
                }
                const u64 f = pair(p.scale, p.scale);
#pragma unroll
                for (int i = 0; i < kTokens; i += 2)
                    o[i / 2] = fma_pair(
                        pair(dot_row<kSplit>(up.inner[token_of<kSplit>(part, i)], i, part, x),
                             dot_row<kSplit>(up.inner[token_of<kSplit>(part, i + 1)], i + 1, part,
                                             x)),
                        f, o[i / 2]);
#pragma unroll
                for (int i = 0; i < kTokens / 2; ++i) {
                    const float2 z = both(o[i]);
                    result[i] = kda_cache::pack(z.x, z.y, __nv_bfloat16());
                }
            }
            // S is at most what it was and all that is added to it
            bound += 2.0f * sum;
            const int moved = state_exponent(bound, ex);
            step = moved - ex;
            ex = moved;
            added = back / (float)(1 << kUpdateExponent) * power_of_two(ex);
            ++count;
        }
        kda::tmem_wait_st();
        if (ok) {
            float *dst = p.pool + w.row.to * slot + at;
            const u64 f = pair(power_of_two(-ex), power_of_two(-ex));
#pragma unroll 1
            for (int i = 0; i < kCols / 16; ++i) {
                uint32_t x[16];
                kda::tmem_ld16(state + 16 * i, x);
                arrived(x);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<ulonglong2 *>(dst + 16 * i + 4 * c) =
                        make_ulonglong2(mul_pair(pair_of(x[4 * c], x[4 * c + 1]), f),
                                        mul_pair(pair_of(x[4 * c + 2], x[4 * c + 3]), f));
            }
        }
        __syncwarp();
    }
}

template <bool kBounded, bool kSplit, bool kPlanned>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const Params p, unsigned items) {
    extern __shared__ __align__(1024) unsigned char smem[];
    Shared<kSplit> &sh = *reinterpret_cast<Shared<kSplit> *>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < kD) sh.zeros[threadIdx.x] = 0.0f, sh.ones[threadIdx.x] = 1.0f;
    if (threadIdx.x == 0) {
        sh.gave_up = 0;
        for (int i = 0; i < kReaches<kSplit>; ++i) {
            kda::mbar_init(&sh.full[i], 2);
            kda::mbar_init(&sh.reach_empty[i], 4 * kParts<kSplit>);
        }
        for (int i = 0; i < kUpdates<kSplit>; ++i)
            kda::mbar_init(&sh.update_empty[i], kSplit ? 1 : 4 * kParts<kSplit>);
        if (!kSplit || rank() == 1)
            for (int i = 0; i < 2 * kPairs<kSplit>; ++i) {
                kda::mbar_init(&sh.scratch[i >> 1].ready[i & 1], 1);
                kda::mbar_init(&sh.scratch[i >> 1].taken[i & 1], 1);
            }
        kda::mbar_init(&sh.u_done, 2);
        kda::mbar_init(&sh.s_done, 1);
        kda::mbar_init(&sh.drained, 2);
        kda::fence_mbar_init();
    }
    const bool consumes = !kSplit || rank() == 0, produces = !kSplit || rank() == 1;
    constexpr int kFirst = kSplit ? 0 : 2 * kPairs<kSplit>;   // of the consumers
    if (consumes && warp == kFirst) {
        kda::tmem_alloc(&sh.tmem, kTmemColumns);
        kda::tc_fence_before();
    }
    // (Two CTAs a head leave SMs free: what follows would sit there, and what follows
    // that, and the clusters of a long run of calls would end up scattered.)
    if (!kSplit) kda_cache::grid_dependents_launch();
    __syncthreads();
    if (kSplit) meet_cluster();   // the barriers of both are there
    kda::tc_fence_after();
    kda_cache::grid_dependency_wait();
    if constexpr (kPlanned) {
        make_plan(p, sh, items);
        __syncthreads();
    }
    if (consumes && warp >= kFirst)
        consume<kSplit, kPlanned>(p, sh, items, warp - kFirst, lane);
    else if (produces && warp < 2 * kPairs<kSplit>)
        produce<kBounded, kSplit, kPlanned>(p, sh, items, warp, lane);
    if (kSplit) kda_cache::grid_dependents_launch();
    if (consumes && (warp == kFirst || warp == kFirst + 4)) {
        // no product may outlive the memory, whatever became of who waited for it
        if (elected()) kda::umma_commit(&sh.drained);
        kda::mbar_wait_bounded(&sh.drained, 0, kWaitBudget);
    }
    __syncthreads();
    if (kSplit) meet_cluster();   // neither's memory goes while the other may still use it
    if (consumes && warp == kFirst) {
        kda::tc_fence_after();
        kda::tmem_dealloc(sh.tmem, kTmemColumns);
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
    if (tiles > 0x7fffffffLL - sms) return KDA_ERR_UNSUPPORTED;
    // Where SMs would be idle and rows are long, two SMs share a row and head, one
    // that produces and one that consumes: a row of 16001 tokens x 32 heads takes
    // 2.59 ms, not 3.12, one of 512 x 16 103 us, not 115, of 256 62, not 66, but of 64
    // 28, not 27 (it starts later).  (Pairs of SMs: not every SM has another beside it,
    // so no more than a third of them.)
    constexpr int kLong = 256;
    const bool split = 3 * tiles <= sms && num_tokens >= (long long)kLong * B;
    // A plan costs some us, and little is gained where each CTA has many rows and
    // heads: 256 rows of 1 to 45 tokens x 32 heads (54 each) take 770 us either way.
    // 200 rows, 30 of them of 300 to 1501 tokens, x 16 heads (21 each) take 1035 planned
    // and 1118 in turn, 13 rows of 1 to 2501 x 16 heads 468 and 834; where all are
    // alike a plan costs 1% at most (19 rows of 512 x 16 heads 231 us, not 228), and
    // only the device knows.  With up to 20 tokens for an SM it costs as much as it
    // gives, with 70 to 150 it takes off a fifth to a third (100 rows of 1 to 150 x 2
    // heads 57 us, not 72).
    const bool planned = !split && tiles > sms && tiles <= 32LL * sms && B <= kPlanRows &&
                         sms <= kThreads && (long long)num_tokens * p.H >= 64LL * sms;
    void (*kernel)(const Params, unsigned) =
        split     ? (p.bounded ? prefill_kernel<true, true, false> : prefill_kernel<false, true, false>)
        : planned ? (p.bounded ? prefill_kernel<true, false, true> : prefill_kernel<false, false, true>)
                  : (p.bounded ? prefill_kernel<true, false, false> : prefill_kernel<false, false, false>);
    const int smem = (int)(split ? sizeof(Shared<true>) : sizeof(Shared<false>));
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return KDA_ERR_CUDA;
    // Rows of up to kShort tokens go token by token where most rows can be such
    // (512 rows x 16 heads: 228 us with 1 token, 347 with 4, 441 with 6, and 550
    // as a chunk each; states from the slots that they go to).  Elsewhere the second
    // launch costs more than it gives: 256 rows of 1 to 45 tokens x 32 heads took 789
    // us, not 770.
    constexpr int kShort = 6;
    if (num_tokens <= (long long)kShort * B) {
        p.most = kShort;
        st = kda_delta::launch_recurrent(p, stream);
        if (st != KDA_OK || num_tokens <= kShort) return st;
        p.least = kShort + 1;
        p.most = 0x7fffffff;
    }
    const long long grid = split ? 2 * tiles : tiles < sms ? tiles : sms;
    return kda_cache::launch(kernel, dim3((unsigned)grid), dim3(kThreads), smem, split ? 2 : 1,
                             stream, p, (unsigned)tiles);
}

extern "C" kda_status kda_prefill_packed(const kda_delta_args *a) {
    if (a == nullptr) return KDA_ERR_INVALID_ARG;
    return kda_prefill(&a->config, a->q, a->k, a->v, a->g_raw, a->beta_raw, a->A_log, a->g_bias,
                       a->state_pool, a->cu_seqlens, a->state_indices, a->initial_indices, a->B,
                       a->num_tokens, a->out, a->error_word, a->stream);
}
