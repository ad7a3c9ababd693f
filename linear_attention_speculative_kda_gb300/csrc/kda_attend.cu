// kda_window_attention: softmax attention of a window of 1..8 new tokens per
// row over a paged key/value cache (sm_103a).  Contract in include/kda.h.
//
// Mathematics.  The R = T * G query rows of one row and kv head (T tokens, G
// query heads per kv head, row t * G + g) share its keys and values, which
// are read once: S = Q K^T, and with a running maximum m and sum l per query
// row, P = 2^(S' - m), l += sum P, O += P V (S' = S * scale * log2 e).  When
// a row's maximum grows by more than 2^8, O and l are scaled down to the new
// one; smaller growth stays in m's old units (P <= 2^8), which changes no
// result, only how often O is rescaled.
//
// S, m, l and O are fp32.  P is rounded to the storage type for P V, because the
// matrix instructions take both operands in one type: half a step of it a
// weight, relative, where a second product with what the rounding left would
// cost as much as the first, and give NaN for a weight without a rest times an
// infinite value.  l adds the weights as they were.  In fp16 P and l are held
// times 2^7: weights would be subnormal from 2^-14 of the largest one on, and
// vanish below 2^-25, where half of the sum can lie if one key leads the others
// far enough; so they keep their bits down to 2^-21, and the largest, 2^15 with
// the slack, stays below 65504.
//
// Work split.  The unit is a tile of 64 keys of one (row, kv head); all tiles
// of the call, in row, head, key order, are cut into equal runs, one per CTA
// of the two or three that fit an SM.  Each CTA finds its run from the rows'
// lengths by itself.  A run may cut a (row, head) segment: the pieces leave
// (m, l, O) in fp32 in the workspace, and a second, short kernel joins them in
// a fixed order.
//
// Two forms.  HBM bounds both where there are keys to read (each once: 256
// bytes of 64 channels' K and V a key and head, 512 of 128).
//
// - attend_kernel, for up to 32 query rows (64 at 64 channels): 4 warps in
//   groups of kMW.  A group's warps hold different query rows (16 * kMT each)
//   of the same keys; the 4 / kMW groups take different keys of each tile.
//   Keys and values arrive by 16-byte cp.async in a ring of tiles, each warp
//   loading its own 16 keys, so with kMW = 1 no warp waits for another inside
//   a segment.  The products are mma.sync m16n8k16 on fragments that ldmatrix
//   reads from XOR-swizzled rows.  64 requests of 4 tokens over up to 8192
//   keys, 16 rows: 188 to 192 us, 93% to 95% of the measured HBM rate.
// - tc::attend_tc_kernel, for more: tcgen05.mma with S and O in tensor memory
//   and tensor-map TMA loads (below).  128 requests of 8 tokens over up to
//   12000 keys, 64 rows: 573 to 578 us, 91% (698 with the first form).  A
//   sliding window is a template parameter of it (launch_rows says why).  Its
//   128 registers a thread, for two CTAs on an SM, leave 56 to 72 bytes of
//   spills, of values that a segment uses once.
#include <cuda.h>

#include "kda_async.cuh"
#include "kda_cache.cuh"
#include "kda_tc.cuh"

namespace {

using kda_cache::exp2_fast;
using kda_cache::kFull;
using kda_cache::pack;
using kda_cache::Row;
using kda_cache::Rows;
using kda_cache::unpack;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 64;             // keys of a tile
constexpr int kMaxCtas = 512;         // bound of the grid, for the workspace
constexpr float kLazy = 8.0f;         // log2 of the growth a stale maximum may have
template <typename T>                 // log2 of the factor that P and l are held times
constexpr float kLift = __is_same(T, __half) ? 7.0f : 0.0f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

struct alignas(16) Cut {     // a segment first cut at the start of this CTA's run
    int pieces;              // 0: none
    int first_slot;          // partial slot of the first piece
    int first_token, tokens, head;
    int pad[3];
};

struct Params {
    Rows rows;
    const char *q, *key_cache, *value_cache;
    char *out;
    float *lse;
    float *partials;         // [2 * grid][slot_size]
    Cut *cuts;               // [grid]
    long long stride_q, stride_block, stride_token, stride_head;  // elements
    int q_heads, kv_heads, group, window, left_window, most_rows;
    int by_group;            // 2^16 / group, rounded up
    kda_cache::Divider by_heads, by_grid;
    int box;                 // tokens of a tensor-map box
    long long slot_size;     // floats of a partial slot: O, the maxima, the sums
    float scale_log2;        // |scale| log2 e
    uint32_t flip;           // sign bits of a pair of queries when scale < 0
};

// ------------------------------------------------------------ instructions --

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1, __nv_bfloat16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1, __half) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether either half of u is a NaN or an infinity.
__device__ __forceinline__ bool not_finite(uint32_t u, __nv_bfloat16) {
    return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ bool not_finite(uint32_t u, __half) {
    return (u & 0x7c00u) == 0x7c00u || (u & 0x7c000000u) == 0x7c000000u;
}

// 16-byte cp.async that writes zeros instead when `there` is false.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <int kMW>
__device__ __forceinline__ void group_sync(int group) {
    if constexpr (kMW == 1)
        __syncwarp();
    else if constexpr (kMW == kWarps)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * kMW) : "memory");
}

// ------------------------------------------------------------------- plan --

// The first key that a query of the row sees.  What lies before it in its tile
// is never read, or zeroed: its weights are 0, but 0 times a NaN is one.
__device__ __forceinline__ int first_key(const Params &p, const Row &row) {
    return p.left_window > 0 ? max(0, row.computed + 1 - p.left_window) : 0;
}

// The tiles a row's keys span: [first, end).
__device__ __forceinline__ void row_tiles(const Params &p, const Row &row, int &first, int &end) {
    first = end = 0;
    if (row.tokens == 0) return;
    first = first_key(p, row) / kTile;
    end = (row.computed + row.tokens - 1) / kTile + 1;
}

// Where a CTA's run stands: tile `tile` of kv head `head` of row `b`.
struct Cursor {
    Row row;
    int b, head, tile, first, end;

    __device__ __forceinline__ void set_row(const Params &p, int row_index, int &bits) {
        b = row_index;
        row = kda_cache::read_row(p.rows, b, p.window, bits);
        row_tiles(p, row, first, end);
        tile = first;
        head = 0;
    }
    __device__ __forceinline__ void next_segment(const Params &p) {
        if (++head < p.kv_heads) {
            tile = first;
            return;
        }
        int bits = 0;
        do {
            if (b + 1 >= p.rows.B) return;  // past the last unit; never read
            set_row(p, b + 1, bits);
        } while (end == first);
    }
};

struct Run {
    long long units, begin, end;  // of the call; this CTA's [begin, end)
    long long before_row;         // units before the starting row
    long long each;               // units of a run; the first `more` runs have one more
    int more, ctas;               // CTAs with work
};

// a / b of whole numbers >= 0: nearly always in 32 bits, in a third of the time.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

__device__ __forceinline__ long long quotient(long long a, int b, const kda_cache::Divider &by) {
    return (a >> 31) == 0 ? kda_cache::divide((int)a, by) : a / b;
}

// First unit of CTA i's run, and the CTA whose run holds unit u.
__device__ __forceinline__ long long run_begin(const Run &run, int i) {
    return i * run.each + min(i, run.more);
}

__device__ __forceinline__ int cta_of(const Run &run, long long u) {
    const long long split = run.more * (run.each + 1);
    return u < split ? (int)quotient(u, run.each + 1)
                     : run.more + (int)quotient(u - split, run.each);
}

// Every CTA adds up the rows' tiles itself: thread i takes a run of rows, a
// scan over the threads gives the units before it, and the thread whose rows
// hold the CTA's first unit finds the row.
struct PlanScratch {
    long long sums[8];
    long long before;
    Cursor row;
};

template <int kWarpCount>
__device__ __forceinline__ Run plan(const Params &p, PlanScratch &sc) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kCount = 32 * kWarpCount;
    const int per = (p.rows.B + kCount - 1) / kCount;
    const int b0 = min(p.rows.B, tid * per), b1 = min(p.rows.B, b0 + per);
    long long mine = 0;
    int bits = 0;
    Cursor own = {};  // the thread's first row
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {  // the loads overlap
        Cursor c;
        c.set_row(p, b, bits);
        mine += c.end - c.first;
        if (b == b0) own = c;
    }
    if (bits != 0 && blockIdx.x == 0) kda_cache::flag(p.rows.err, bits);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long other = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += other;
    }
    if (lane == 31) sc.sums[warp] = upto;
    __syncthreads();
    long long before = upto - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarpCount; ++w) {
        if (w < warp) before += sc.sums[w];
        total += sc.sums[w];
    }
    Run run;
    run.units = total * p.kv_heads;
    run.ctas = (int)min((long long)gridDim.x, run.units);
    run.each = quotient(run.units, gridDim.x, p.by_grid);
    run.more = (int)(run.units - run.each * gridDim.x);
    run.begin = run.end = 0;
    if ((int)blockIdx.x >= run.ctas) return run;  // uniform over the CTA
    run.begin = run_begin(run, blockIdx.x);
    run.end = run_begin(run, blockIdx.x + 1);
    const long long at = quotient(run.begin, p.kv_heads, p.by_heads);  // the first tile, counted over rows
    if (at >= before && at < before + mine) {
        while (at >= before + own.end - own.first) {
            before += own.end - own.first;
            own.set_row(p, own.b + 1, bits);
        }
        sc.row = own;
        sc.before = before * p.kv_heads;
    }
    __syncthreads();
    run.before_row = sc.before;
    return run;
}

// Where the CTA's run begins.
__device__ __forceinline__ Cursor run_start(const Run &run, const PlanScratch &sc) {
    Cursor at = sc.row;
    const long long in_row = run.begin - run.before_row;
    const int n = at.end - at.first;
    at.head = (int)quotient(in_row, n);
    at.tile += (int)(in_row - (long long)at.head * n);
    return at;
}

// The join's work item of a CTA whose run starts at `at`: the segment that is
// first cut there, if there is one.
__device__ __forceinline__ Cut first_cut(const Run &run, const Cursor &at, int cta) {
    Cut cut = {};
    const int n = at.end - at.first;
    const long long s = run.before_row + (long long)at.head * n;
    if (s < run.begin) {
        const long long before = run_begin(run, cta - 1);
        if (s >= before) {
            cut.pieces = cta_of(run, s + n - 1) - cta + 2;
            cut.first_slot = 2 * (cta - 1) + (before < s ? 1 : 0);
            cut.first_token = at.row.first;
            cut.tokens = at.row.tokens;
            cut.head = at.head;
        }
    }
    return cut;
}

// Row r of a segment's queries is query head r % group of token r / group
// (r < 128, group <= 128: the product with 2^16 / group, rounded up, is exact).
__device__ __forceinline__ int token_of(const Params &p, int r) { return (r * p.by_group) >> 16; }

// ---------------------------------------------------------------- layout --

template <int kDim, int kMT, int kMW, int kCtas>
struct Layout {
    static constexpr int kRows = 16 * kMT * kMW;       // query rows, padded
    static constexpr int kGroups = kWarps / kMW;
    static constexpr int kKeys = kTile / kGroups;      // keys of a group's step
    static constexpr int kRowBytes = kDim * 2;
    static constexpr int kHalfTile = kTile * kRowBytes;
    static constexpr int kStage = 2 * kHalfTile;       // keys, then values
    static constexpr int kQuery = kRows * kRowBytes;
    static constexpr int kStats = kGroups * kRows * 8;
    static constexpr int kFixed = kQuery + kStats;
    // the SM's 228 KB, less 1 KB a CTA that the system takes and the static part
    static constexpr int kBudget = 233472 / kCtas - 1024 - 1280;
    static constexpr int kStages = (kBudget - kFixed) / kStage < 6 ? (kBudget - kFixed) / kStage : 6;
    static constexpr int kBytes = kFixed + kStages * kStage;
    static_assert(kGroups == 1 || kMT == 1, "a group hands over one tile of rows a warp");
    static_assert(kStages >= 2, "the ring needs two tiles");
};

// Byte offset of 16-byte chunk c of row r in a swizzled tile.
template <int kDim>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    return (uint32_t)(r * kDim * 2 + ((c ^ (r & 7)) << 4));
}

// ---------------------------------------------------------------- kernel --

template <typename T, int kDim, int kMT, int kMW, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) attend_kernel(const Params p) {
    using L = Layout<kDim, kMT, kMW, kCtas>;
    constexpr int kNB = L::kKeys / 16;      // blocks of 16 keys in a group's step
    constexpr int kDT = kDim / 8;           // 8-channel tiles of O
    constexpr int kOwn = 8 / L::kGroups;    // of each 8 of them, a group's share of the sum
    constexpr int kChunks = kDim / 8;       // 16-byte chunks of a cache row
    constexpr int kPerInstr = 32 / kChunks; // cache rows one cp.async of a warp covers
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint32_t there[kStages][kWarps];  // keys of each warp's 16 that are in the cache
    unsigned char *ring = smem;
    unsigned char *query_area = smem + kStages * L::kStage;
    float *stat_m = reinterpret_cast<float *>(query_area + L::kQuery);
    float *stat_l = stat_m + L::kGroups * L::kRows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = warp / kMW, mwarp = warp % kMW;
    const int qr = lane >> 2, qc = lane & 3;  // row and column pair inside a fragment

    kda_cache::grid_dependents_launch();
    kda_cache::grid_dependency_wait();
    __shared__ PlanScratch plan_scratch;
    const Run run = plan<kWarps>(p, plan_scratch);
    const int cta = blockIdx.x;
    if (cta >= run.ctas) {
        if (tid == 0) p.cuts[cta].pieces = 0;
        return;
    }

    // cursor of the tile to compute and of the tile to load
    Cursor at = run_start(run, plan_scratch);
    Cursor ld = at;
    long long left = run.end - run.begin;       // tiles to compute
    long long to_load = left;

    // Load one tile into ring slot `slot`: this warp's 16 keys and values.
    // Lane l looks up key l mod 16; the address goes to the loading lanes by
    // shuffle.  Keys behind a sliding window, past the row's end and in null
    // blocks become zeros.
    auto load_tile = [&](int slot) {
        if (to_load > 0) {
            const int pos = ld.tile * kTile + 16 * warp + (lane & 15);
            int block = 0;
            long long off = 0;
            if (pos >= first_key(p, ld.row) && pos < ld.row.computed + ld.row.tokens) {
                const int col = kda_cache::divide(pos, p.rows.by_block);
                block = p.rows.block_table[ld.row.request * p.rows.bt_stride + col];
                if (block >= p.rows.num_blocks) {
                    kda_cache::flag(p.rows.err, KDA_ROW_BAD_SLOT);
                    block = 0;
                }
                if (block > 0)
                    off = block * p.stride_block +
                          (long long)(pos - col * p.rows.block_size) * p.stride_token +
                          ld.head * p.stride_head;
            }
            const unsigned mask = __ballot_sync(kFull, block > 0) & 0xffffu;
            if (lane == 0) there[slot][warp] = mask;
            const uint32_t dst = kda::smem_u32(ring + slot * L::kStage);
            const int chunk = lane % kChunks;
#pragma unroll
            for (int i = 0; i < 16 / kPerInstr; ++i) {
                const int r = i * kPerInstr + lane / kChunks;
                const long long o = (__shfl_sync(kFull, off, r) + chunk * 8) * 2;
                const bool ok = (mask >> r) & 1u;
                const uint32_t d = dst + swizzled<kDim>(16 * warp + r, chunk);
                cp_async16_or_zero(d, p.key_cache + o, ok);
                cp_async16_or_zero(d + L::kHalfTile, p.value_cache + o, ok);
            }
            if (--to_load > 0 && ++ld.tile == ld.end) ld.next_segment(p);
        }
        kda::cp_async_commit();
    };

    // A segment's queries (rows past the last one: zeros), a batch of loads in
    // flight together: one after the other they took most of the 10 us that 64
    // rows cost beside their tiles.
    constexpr int kEach = L::kRows * kChunks / kThreads, kBatch = kEach < 8 ? kEach : 8;
    constexpr int kBatches = kEach / kBatch;
    constexpr bool kAhead = kEach <= 4;
    uint4 queries[kBatch];
    auto fetch_queries = [&](const Cursor &c, int batch) {
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            const int i = (batch * kBatch + n) * kThreads + tid, r = i / kChunks;
            queries[n] = make_uint4(0, 0, 0, 0);
            if (r < c.row.tokens * p.group) {
                const int t = token_of(p, r), h = c.head * p.group + r - t * p.group;
                queries[n] = __ldg(reinterpret_cast<const uint4 *>(
                    reinterpret_cast<const T *>(p.q) + (c.row.first + t) * p.stride_q +
                    (long long)h * kDim + i % kChunks * 8));
            }
        }
    };
    auto store_queries = [&](int batch) {
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            const int i = (batch * kBatch + n) * kThreads + tid;
            const uint4 x = queries[n];
            *reinterpret_cast<uint4 *>(query_area + swizzled<kDim>(i / kChunks, i % kChunks)) =
                make_uint4(x.x ^ p.flip, x.y ^ p.flip, x.z ^ p.flip, x.w ^ p.flip);
        }
    };

    if (kAhead) fetch_queries(at, 0);
    for (int i = 0; i < kStages - 1; ++i) load_tile(i);
    if (tid == 0) p.cuts[cta] = first_cut(run, at, cta);

    int slot = 0;            // ring slot of the tile to compute
    int piece_first = 1;     // whether the segment is this run's first
    while (left > 0) {
        // ------------------------------------------------- a segment's piece
        const int tiles = (int)min(left, (long long)(at.end - at.tile));
        const bool whole = at.tile == at.first && tiles == at.end - at.first;
        const int partial_slot = 2 * cta + (piece_first ? 0 : 1);
        const int rows = at.row.tokens * p.group;
        const bool busy = mwarp * 16 * kMT < rows;  // whether this warp has query rows
        // queries to shared memory; few enough are here already, fetched while
        // the segment before was joined
        if (!kAhead) fetch_queries(at, 0);
        store_queries(0);
#pragma unroll 1
        for (int batch = 1; batch < kBatches; ++batch) {
            fetch_queries(at, batch);
            store_queries(batch);
        }
        __syncthreads();
        const uint32_t q_addr = kda::smem_u32(query_area);
        const int q_row = mwarp * 16 * kMT + (lane & 15);
        uint32_t qf[kMT == 1 ? kDim / 16 : 1][4];
        if constexpr (kMT == 1) {
#pragma unroll
            for (int k = 0; k < kDim / 16; ++k)
                ldmatrix4(qf[k], q_addr + swizzled<kDim>(q_row, 2 * k + (lane >> 4)));
        }
        // the keys each of this thread's rows sees: (lo, hi]
        int lo[kMT][2], hi[kMT][2];
        float m[kMT][2], l[kMT][2];
        float o[kMT][kDT][4];
#pragma unroll
        for (int a = 0; a < kMT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = (mwarp * kMT + a) * 16 + qr + 8 * h;
                hi[a][h] = at.row.computed + min(token_of(p, r), at.row.tokens - 1);
                lo[a][h] = p.left_window > 0 ? hi[a][h] - p.left_window : -1;
                m[a][h] = -INFINITY;
                l[a][h] = 0.0f;
            }
#pragma unroll
        for (int a = 0; a < kMT; ++a)
#pragma unroll
            for (int d = 0; d < kDT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[a][d][e] = 0.0f;

        for (int done = 0; done < tiles; ++done) {
            cp_async_wait<kStages - 2>();
            group_sync<kMW>(group);  // the tile is here, and the one before is done with
            load_tile(slot == 0 ? kStages - 1 : slot - 1);
            const uint32_t k_addr = kda::smem_u32(ring + slot * L::kStage) +
                                    group * L::kKeys * L::kRowBytes;
            const uint32_t v_addr = k_addr + L::kHalfTile;
            const int key0 = (at.tile + done) * kTile + group * L::kKeys;
            unsigned long long seen = 0;  // keys of the step that are in the cache
#pragma unroll
            for (int w = 0; w < kMW; ++w)
                seen |= (unsigned long long)there[slot][group * kMW + w] << (16 * w);

            // a step that some row does not see whole: at the window's own
            // keys, at a sliding window's start, at null blocks
            constexpr unsigned long long kAll = kNB == 4 ? ~0ull : (1ull << (16 * kNB % 64)) - 1;
            const bool edge =
                key0 + L::kKeys - 1 > at.row.computed || seen != kAll ||
                (p.left_window > 0 && key0 <= at.row.computed + at.row.tokens - 1 - p.left_window);
            float s[kMT][2 * kNB][4];
#pragma unroll
            for (int a = 0; a < kMT; ++a)
#pragma unroll
                for (int n = 0; n < 2 * kNB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[a][n][e] = 0.0f;
            if (busy) {
#pragma unroll
                for (int k = 0; k < kDim / 16; ++k) {
                    uint32_t af[kMT][4];
#pragma unroll
                    for (int a = 0; a < kMT; ++a) {
                        if constexpr (kMT == 1) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) af[a][e] = qf[k][e];
                        } else {
                            ldmatrix4(af[a], q_addr + swizzled<kDim>(q_row + 16 * a,
                                                                     2 * k + (lane >> 4)));
                        }
                    }
#pragma unroll
                    for (int n = 0; n < kNB; ++n) {
                        uint32_t bf[4];
                        ldmatrix4(bf, k_addr + swizzled<kDim>(16 * n + ((lane >> 4) << 3) + (lane & 7),
                                                              2 * k + ((lane >> 3) & 1)));
#pragma unroll
                        for (int a = 0; a < kMT; ++a) {
                            mma(s[a][2 * n], af[a], bf[0], bf[1], T());
                            mma(s[a][2 * n + 1], af[a], bf[2], bf[3], T());
                        }
                    }
                }

                if (edge) {
#pragma unroll
                    for (int a = 0; a < kMT; ++a)
#pragma unroll
                        for (int n = 0; n < 2 * kNB; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = 8 * n + 2 * qc + (e & 1);
                                const int pos = key0 + j;
                                if (!((seen >> j) & 1ull) || pos > hi[a][e >> 1] ||
                                    pos <= lo[a][e >> 1])
                                    s[a][n][e] = -INFINITY;
                            }
                }

                // running maximum; O is rescaled only when it grew past the slack
                float top[kMT][2];
                bool grew = false;
#pragma unroll
                for (int a = 0; a < kMT; ++a)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x = -INFINITY;
#pragma unroll
                        for (int n = 0; n < 2 * kNB; ++n)
                            x = fmaxf(x, fmaxf(s[a][n][2 * h], s[a][n][2 * h + 1]));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 2)) * p.scale_log2;
                        top[a][h] = x;
                        grew |= x > m[a][h] + kLazy;
                    }
                if (__any_sync(kFull, grew)) {
#pragma unroll
                    for (int a = 0; a < kMT; ++a)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float now = fmaxf(m[a][h], top[a][h]);
                            const float f = now == -INFINITY ? 1.0f : exp2_fast(m[a][h] - now);
                            m[a][h] = now;
                            l[a][h] *= f;
#pragma unroll
                            for (int d = 0; d < kDT; ++d) {
                                o[a][d][2 * h] *= f;
                                o[a][d][2 * h + 1] *= f;
                            }
                        }
                }
#pragma unroll
                for (int a = 0; a < kMT; ++a)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float base = m[a][h] == -INFINITY ? 0.0f : kLift<T> - m[a][h];
                        unsigned long long sum = 0;  // a pair of 0
#pragma unroll
                        for (int n = 0; n < 2 * kNB; ++n) {
                            const float2 x = kda_cache::both(kda_cache::fma_pair(
                                kda_cache::pair(s[a][n][2 * h], s[a][n][2 * h + 1]),
                                kda_cache::pair(p.scale_log2, p.scale_log2),
                                kda_cache::pair(base, base)));
                            s[a][n][2 * h] = exp2_fast(x.x);
                            s[a][n][2 * h + 1] = exp2_fast(x.y);
                            sum = kda_cache::add_pair(
                                sum, kda_cache::pair(s[a][n][2 * h], s[a][n][2 * h + 1]));
                        }
                        const float2 two = kda_cache::both(sum);
                        l[a][h] += two.x + two.y;
                    }

            }

            // A value that is not finite must not reach the rows that do not
            // see its key (0 * inf is NaN in the product): where rows see
            // different keys, such values are added by hand to the rows that
            // do and zeroed for the product.
            // (That can only be the window's own keys but the first, and as
            // many at a sliding window's start.)
            if (edge && at.row.tokens > 1) {
                const int own = at.row.tokens - 1;
                unsigned long long odd = 0;
                for (int i = lane; i < (p.left_window > 0 ? 2 : 1) * own * kChunks; i += 32) {
                    const int k = i / kChunks;
                    const int key = (k < own ? at.row.computed + 1 + k
                                             : at.row.computed + 1 - p.left_window + k - own) -
                                    key0;
                    if (key < 0 || key >= L::kKeys) continue;
                    uint4 x;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                 : "r"(v_addr + swizzled<kDim>(key, i % kChunks))
                                 : "memory");
                    if (not_finite(x.x, T()) || not_finite(x.y, T()) || not_finite(x.z, T()) ||
                        not_finite(x.w, T()))
                        odd |= 1ull << key;
                }
                odd = (unsigned long long)__reduce_or_sync(kFull, (uint32_t)odd) |
                      (unsigned long long)__reduce_or_sync(kFull, (uint32_t)(odd >> 32)) << 32;
                if (odd != 0) {  // the same for every warp of the group
#pragma unroll
                    for (int n = 0; n < 2 * kNB; ++n) {
                        uint32_t bits = (uint32_t)(odd >> (8 * n)) & 0xffu;
                        while (bits != 0) {
                            const int j = __ffs(bits) - 1;
                            bits &= bits - 1;
                            const int src = (lane & ~3) | (j >> 1);
                            const int pos = key0 + 8 * n + j;
#pragma unroll
                            for (int a = 0; a < kMT; ++a) {
                                const float2 w0 = unpack(pack(s[a][n][0], s[a][n][1], T()), T());
                                const float2 w1 = unpack(pack(s[a][n][2], s[a][n][3], T()), T());
                                const float p0 = __shfl_sync(kFull, (j & 1) ? w0.y : w0.x, src);
                                const float p1 = __shfl_sync(kFull, (j & 1) ? w1.y : w1.x, src);
                                const bool see0 = pos <= hi[a][0] && pos > lo[a][0];
                                const bool see1 = pos <= hi[a][1] && pos > lo[a][1];
#pragma unroll
                                for (int d = 0; d < kDT; ++d) {
                                    uint32_t u;
                                    asm volatile("ld.shared.u32 %0, [%1];"
                                                 : "=r"(u)
                                                 : "r"(v_addr + swizzled<kDim>(8 * n + j, d) +
                                                       4 * qc));
                                    const float2 x = unpack(u, T());
                                    if (busy && see0) {
                                        o[a][d][0] = fmaf(p0, x.x, o[a][d][0]);
                                        o[a][d][1] = fmaf(p0, x.y, o[a][d][1]);
                                    }
                                    if (busy && see1) {
                                        o[a][d][2] = fmaf(p1, x.x, o[a][d][2]);
                                        o[a][d][3] = fmaf(p1, x.y, o[a][d][3]);
                                    }
                                }
                            }
                        }
                    }
                    group_sync<kMW>(group);
                    for (int i = lane; i < L::kKeys * kChunks; i += 32)
                        if ((odd >> (i / kChunks)) & 1ull)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             v_addr + swizzled<kDim>(i / kChunks, i % kChunks)),
                                         "r"(0)
                                         : "memory");
                    group_sync<kMW>(group);
                }
            }

            if (busy) {
#pragma unroll
                for (int n = 0; n < kNB; ++n) {
                    uint32_t pf[kMT][4];
#pragma unroll
                    for (int a = 0; a < kMT; ++a) {
                        pf[a][0] = pack(s[a][2 * n][0], s[a][2 * n][1], T());
                        pf[a][1] = pack(s[a][2 * n][2], s[a][2 * n][3], T());
                        pf[a][2] = pack(s[a][2 * n + 1][0], s[a][2 * n + 1][1], T());
                        pf[a][3] = pack(s[a][2 * n + 1][2], s[a][2 * n + 1][3], T());
                    }
#pragma unroll
                    for (int d = 0; d < kDim / 16; ++d) {
                        uint32_t bf[4];
                        ldmatrix4_trans(bf, v_addr + swizzled<kDim>(16 * n + (lane & 15),
                                                                    2 * d + (lane >> 4)));
#pragma unroll
                        for (int a = 0; a < kMT; ++a) {
                            mma(o[a][2 * d], pf[a], bf[0], bf[1], T());
                            mma(o[a][2 * d + 1], pf[a], bf[2], bf[3], T());
                        }
                    }
                }
            }
            slot = slot + 1 == kStages ? 0 : slot + 1;
        }

        // the next segment, and its queries on their way
        Cursor next = at;
        if (left > tiles) {
            next.next_segment(p);
            if (kAhead) fetch_queries(next, 0);
        }

        // ------------------------------------------- the groups' sums joined
#pragma unroll
        for (int a = 0; a < kMT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[a][h] += __shfl_xor_sync(kFull, l[a][h], 1);
                l[a][h] += __shfl_xor_sync(kFull, l[a][h], 2);
                m[a][h] -= kLift<T>;  // what l and O are relative to
            }
        if constexpr (L::kGroups > 1) {
#pragma unroll
            for (int a = 0; a < kMT; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (qc == 0) {
                        const int r = (mwarp * kMT + a) * 16 + qr + 8 * h;
                        stat_m[group * L::kRows + r] = m[a][h];
                        stat_l[group * L::kRows + r] = l[a][h];
                    }
            // Each group sums and writes its share of the channels.  The others
            // hand it theirs through the group's part of the ring slot of the
            // last tile, which is not loaded again before the next segment's
            // first barrier.
            const uint32_t area = kda::smem_u32(ring + (slot == 0 ? kStages - 1 : slot - 1) *
                                                           L::kStage) +
                                  8 * lane;
            auto place = [&](int g, int d, int h) {  // 256 bytes of a warp of group g
                constexpr int kHalf = kMW == 1 ? kDT : 2 * kDT;  // of keys, of values
                const int c = 2 * d + h, half = kMW == 1 ? c / kHalf : mwarp;
                return area + g * L::kKeys * L::kRowBytes + half * L::kHalfTile + c % kHalf * 256;
            };
            group_sync<kMW>(group);
#pragma unroll
            for (int d = 0; d < kDT; ++d)
                if (d % 8 / kOwn != group)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(place(group, d, h)),
                                     "f"(o[0][d][2 * h]), "f"(o[0][d][2 * h + 1])
                                     : "memory");
            __syncthreads();
            float f[2][L::kGroups];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = mwarp * 16 + qr + 8 * h;
                float all = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int g = 0; g < L::kGroups; ++g) all = fmaxf(all, stat_m[g * L::kRows + r]);
                const float base = all == -INFINITY ? 0.0f : all;
#pragma unroll
                for (int g = 0; g < L::kGroups; ++g) {
                    f[h][g] = exp2_fast(stat_m[g * L::kRows + r] - base);
                    sum += stat_l[g * L::kRows + r] * f[h][g];
                }
                m[0][h] = all;
                l[0][h] = sum;
            }
#pragma unroll
            for (int d = 0; d < kDT; ++d)
                if (d % 8 / kOwn == group)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float2 all = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int g = 0; g < L::kGroups; ++g) {
                            float2 x = make_float2(o[0][d][2 * h], o[0][d][2 * h + 1]);
                            if (g != group)
                                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                                             : "=f"(x.x), "=f"(x.y)
                                             : "r"(place(g, d, h))
                                             : "memory");
                            all.x = fmaf(x.x, f[h][g], all.x);
                            all.y = fmaf(x.y, f[h][g], all.y);
                        }
                        o[0][d][2 * h] = all.x;
                        o[0][d][2 * h + 1] = all.y;
                    }
        } else {
            __syncthreads();  // every warp is done with the queries
        }

        // ---------------------------------------------------------- results
#pragma unroll
            for (int a = 0; a < kMT; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (mwarp * kMT + a) * 16 + qr + 8 * h;
                    if (r >= rows) continue;
                    if (whole) {
                        const int t = token_of(p, r);
                        const long long row = (long long)(at.row.first + t) * p.q_heads +
                                              at.head * p.group + r - t * p.group;
                        const float f = l[a][h] == 0.0f ? 0.0f : 1.0f / l[a][h];
                        uint32_t *dst = reinterpret_cast<uint32_t *>(p.out) + row * (kDim / 2) + qc;
#pragma unroll
                        for (int d = 0; d < kDT; ++d)
                            if (d % 8 / kOwn == group)
                                dst[4 * d] = pack(o[a][d][2 * h] * f, o[a][d][2 * h + 1] * f, T());
                        if (p.lse != nullptr && qc == 0 && group == 0)
                            p.lse[row] = (m[a][h] + log2f(l[a][h])) * kLn2;
                    } else {
                        float *part = p.partials + partial_slot * p.slot_size;
                        float2 *dst = reinterpret_cast<float2 *>(part + r * kDim) + qc;
#pragma unroll
                        for (int d = 0; d < kDT; ++d)
                            if (d % 8 / kOwn == group)
                                dst[4 * d] = make_float2(o[a][d][2 * h], o[a][d][2 * h + 1]);
                        if (qc == 0 && group == 0) {
                            part[p.most_rows * kDim + r] = m[a][h];
                            part[p.most_rows * (kDim + 1) + r] = l[a][h];
                        }
                    }
                }
        left -= tiles;
        piece_first = 0;
        at = next;
    }
    cp_async_wait<0>();
}


// ------------------------------------------------------- tensor-core form --
//
// For more query rows: S = Q K^T and O += P V on the 5th-generation tensor
// cores, with 128 query rows (unused ones zero), S and O in tensor memory and
// P written over its S as the second product's A operand.  Two warps load
// keys and values (ring stages of 64 rows, keys and values in turn), a thread
// of one warp issues the products S and a thread of another O (one thread for
// both spent 1500 of a tile's 1950 clocks on issuing at 64 channels), four
// warps do the softmax, a thread or two per query row.  S of the next tile is
// made while the softmax of this one runs; two CTAs on an SM fill each
// other's gaps.
//
// Shared memory: rows of 128 bytes (64 channels) with the 128-byte swizzle,
// channel block after channel block.  The same rows are a K-major operand
// for S (queries and keys) and an MN-major one for O (values).
namespace tc {

constexpr int kSoftmaxWarps = 4;
constexpr int kLoadWarp = kSoftmaxWarps, kScoreWarp = kLoadWarp + 1;
constexpr int kOutWarp = kScoreWarp + 1, kQueryWarp = kOutWarp + 1;
constexpr int kWarpCount = kQueryWarp + 1;
constexpr int kThreadCount = 32 * kWarpCount;
constexpr int kRows = 128;
constexpr int kCtasPerSm = 2;
constexpr int kTmemColumns = 256;                 // two CTAs per SM share 512
#ifdef KDA_TEST_ATTENTION_WAIT_BUDGET  // a test build: a wait that runs out, soon
constexpr long long kWaitBudget = KDA_TEST_ATTENTION_WAIT_BUDGET;
#else
constexpr long long kWaitBudget = 4000000000LL;   // clock cycles (about 2 s)
#endif

template <int kDim, int kQRows>
struct Form {
    static constexpr int kBlocks = kDim / 64;                 // channel blocks of 128 bytes
    static constexpr int kQuery = kBlocks * kQRows * 128;
    static constexpr int kStage = kBlocks * kTile * 128;      // 64 keys, or their values
    static constexpr int kStages = kDim == 64 ? 10 : kQRows == 64 ? 6 : 5;
    static constexpr int kControl = 512;
    static constexpr int kBytes = kQuery + kStages * kStage + kControl;
    static constexpr int kS = 128;                            // column of the first S; O at 0
    // Stage 0 lies before the queries, the others behind them: with 64 query
    // rows the products read the 8 KB to either side of a block of them.
    __device__ static __forceinline__ uint32_t stage(uint32_t smem, int i) {
        return smem + i * kStage + (i > 0 ? kQuery : 0);
    }
    __device__ static __forceinline__ uint32_t query(uint32_t smem) { return smem + kStage; }
};

// The query rows' first lane.  Up to 64 rows take the softmax warps 0 and 1,
// or 2 and 3 in the second half of the grid, so that the two CTAs of an SM,
// which come from the two halves, share out its four schedulers and their
// exponentials (4 lanes a clock each): 1.48 us a tile and SM, not 1.54.  The
// products take what lies there for the other 64 rows; nothing reads what
// they make of it.
template <int kQRows>
__device__ __forceinline__ int first_lane() {
    return kQRows == 64 && blockIdx.x >= gridDim.x / 2 ? 64 : 0;
}

struct Control {
    PlanScratch plan;
    uint64_t full[10], empty[10];   // ring stages
    uint64_t s_full[2], p_full[2];  // S in tensor memory, P over it
    uint64_t o_done[2];             // the product of P with V is complete
    uint64_t q_full, q_empty;       // a segment's queries are in shared memory, are done with
    uint64_t meet;                  // the softmax warps' own barrier
    uint64_t drained[2];
    uint32_t there[8][2];           // keys of a tile that are in the cache
    int keep[2];                    // O was started by hand: add to it
    int abort;
    uint32_t tmem;
};

// Bounded wait: gives up after the budget, or when another warp has.
__device__ __forceinline__ bool wait(Control &c, uint64_t *bar, uint32_t parity, int *err) {
    if (kda::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!kda::mbar_try_wait(bar, parity)) {
        if (*reinterpret_cast<volatile int *>(&c.abort) != 0) return false;
        if (clock64() - t0 > kWaitBudget) {
            *reinterpret_cast<volatile int *>(&c.abort) = 1;
            kda_cache::flag(err, KDA_ERR_WAIT_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The same for a whole warp: every lane gets the same answer, converged.
__device__ __forceinline__ bool warp_wait(Control &c, uint64_t *bar, uint32_t parity, int *err) {
    return __all_sync(kFull, wait(c, bar, parity, err));
}

// 4-D tensor-map load of one box: 64 channels, some tokens, one head, one block.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap *map, int channel,
                                             int token, int head, int block, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(channel), "r"(token), "r"(head), "r"(block),
        "r"(kda::smem_u32(bar))
        : "memory");
}

// Instruction descriptor of kind::f16: fp32 accumulation, A and B of type T,
// A K-major, B K-major or MN-major.
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc(int m, int n, bool b_mn) {
    const uint32_t type = sizeof(T) == 2 && __is_same(T, __nv_bfloat16) ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// MN-major operand with the 128-byte swizzle: 64-element blocks along MN
// `block` bytes apart, 8-row groups along K 1024 bytes apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t block) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)(block >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(add)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(add)
        : "memory");
}

// The registers of a tensor-memory load are there only after its wait; this
// keeps the compiler from using them before it (a wait names no register).
__device__ __forceinline__ void landed(uint32_t (&u)[16]) {
    asm volatile(""
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]),
                   "+r"(u[6]), "+r"(u[7]), "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]),
                   "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&u)[16]) {
    kda::tmem_ld16(addr, u);
    kda::tmem_wait_ld();
    landed(u);
}

__device__ __forceinline__ uint32_t tmem_load1(uint32_t addr) {
    uint32_t u;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                 : "=r"(u)
                 : "r"(addr)
                 : "memory");
    kda::tmem_wait_ld();
    asm volatile("" : "+r"(u) : : "memory");
    return u;
}

__device__ __forceinline__ void store16(uint32_t addr, uint4 x) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x.x), "r"(x.y),
                 "r"(x.z), "r"(x.w)
                 : "memory");
}

__device__ __forceinline__ uint4 load16(uint32_t addr) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(addr)
                 : "memory");
    return x;
}

// Byte offset of 16-byte chunk c (of a row's kDim / 8) of row r, with `rows`
// rows in a channel block.
__device__ __forceinline__ uint32_t place(int r, int c, int rows) {
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Multiplies the warp's rows of O (kDim columns at `o`) by each thread's f.
template <int kDim>
__device__ __forceinline__ void scale_o(uint32_t o, float f) {
#pragma unroll
    for (int c = 0; c < kDim; c += 16) {
        uint32_t u[16];
        tmem_load16(o + c, u);
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * f);
        kda::tmem_st16(o + c, u);
    }
    kda::tmem_wait_st();
}

// ---- the loading warp -----------------------------------------------------
//
// A box is p.box keys, the greatest common divisor of the block size and the
// tile, so a tile is kTile / p.box boxes of each channel block, each inside
// one block of the cache.  A lane fetches the table entry of a box's block a
// tile ahead and asks for the box.  The null block, boxes past the row's end
// and boxes behind a sliding window are boxes past the tensor's last block,
// which arrive as zeros.

template <typename T, int kDim, int kQRows, bool kSliding>
__device__ __forceinline__ void run_loader(const Params &p, const Run &run, Control &c,
                                           uint32_t smem, int lane, const CUtensorMap *k_map,
                                           const CUtensorMap *v_map) {
    using F = Form<kDim, kQRows>;
    Cursor at = run_start(run, c.plan);
    const long long tiles = run.end - run.begin;
    const int boxes = kTile / p.box, mine = lane % boxes;
    const int channel_block = lane / boxes;
    int pos = 0, block = 0;
    auto look_up = [&]() {
        pos = at.tile * kTile + mine * p.box;
        block = 0;
        if ((!kSliding || first_key(p, at.row) - pos < p.box) &&
            pos < at.row.computed + at.row.tokens)
            block = p.rows.block_table[at.row.request * p.rows.bt_stride +
                                       kda_cache::divide(pos, p.rows.by_block)];
    };
    look_up();
    int stage = 0;
    uint32_t phase = 1;  // of the stage's empty barrier; the first use waits for nothing
    long long loaded = 0;
    bool ok = true;
    for (long long g = 0; ok && g < tiles; ++g) {
        if (block >= p.rows.num_blocks) {
            kda_cache::flag(p.rows.err, KDA_ROW_BAD_SLOT);
            block = 0;
        }
        const int token = pos - kda_cache::divide(pos, p.rows.by_block) * p.rows.block_size;
        const int from = block > 0 ? block : p.rows.num_blocks;
        const int head = at.head;
        const unsigned there = __ballot_sync(kFull, block > 0);
        if (lane == 0) {
            unsigned long long keys = 0;
            for (int i = 0; i < boxes; ++i)
                if ((there >> i) & 1u)
                    keys |= (p.box == 64 ? ~0ull : (1ull << p.box) - 1) << (i * p.box);
            c.there[g & 7][0] = (uint32_t)keys;
            c.there[g & 7][1] = (uint32_t)(keys >> 32);
        }
        if (g + 1 < tiles) {
            if (++at.tile == at.end) at.next_segment(p);
            look_up();
        }
        for (int half = 0; half < 2; ++half) {
            ok = warp_wait(c, &c.empty[stage], phase, p.rows.err);
            if (!ok) break;
            if (lane == 0) kda::mbar_arrive_expect_tx(&c.full[stage], F::kStage);
            __syncwarp();
            if (channel_block < F::kBlocks)
                tma_load_box(F::stage(smem, stage) + channel_block * kTile * 128 +
                                 mine * p.box * 128,
                             half == 0 ? k_map : v_map, channel_block * 64, token, head, from,
                             &c.full[stage]);
            ++loaded;
            if (++stage == F::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    // no copy may outlive the CTA, whatever became of its users
    for (long long j = loaded > F::kStages ? loaded - F::kStages : 0; j < loaded; ++j)
        kda::mbar_wait_bounded(&c.full[j % F::kStages], (uint32_t)((j / F::kStages) & 1),
                               kWaitBudget);
    __syncwarp();
}

// ---- the query warp -------------------------------------------------------
//
// Copies each segment's queries to shared memory as soon as the segment
// before has its last S.

template <typename T, int kDim, int kQRows>
__device__ __forceinline__ void run_queries(const Params &p, const Run &run, Control &c,
                                            uint32_t smem, int lane) {
    constexpr int kChunks = kDim / 8;
    const uint32_t query = Form<kDim, kQRows>::query(smem);
    Cursor at = run_start(run, c.plan);
    long long left = run.end - run.begin;
    for (uint32_t segment = 0;; ++segment) {
        if (!warp_wait(c, &c.q_empty, (segment & 1u) ^ 1u, p.rows.err)) break;
        const int rows = at.row.tokens * p.group;
        // the rows that make up whole warps of the softmax: zeros past the last
        for (int i = lane; i < (rows + 31) / 32 * 32 * kChunks; i += 32) {
            const int r = i / kChunks, ch = i % kChunks;
            const int t = token_of(p, r), h = at.head * p.group + r - t * p.group;
            const T *src = reinterpret_cast<const T *>(p.q);
            if (r < rows) src += (at.row.first + t) * p.stride_q + (long long)h * kDim + ch * 8;
            cp_async16_or_zero(query + place(r, ch, kQRows), src, r < rows);
        }
        kda::cp_async_commit();
        cp_async_wait<0>();
        kda::fence_proxy_async_smem();
        __syncwarp();
#ifdef KDA_TEST_ATTENTION_WAIT_BUDGET
        if (blockIdx.x == 0) break;  // CTA 0's queries are never handed over
#endif
        if (lane == 0) kda::mbar_arrive(&c.q_full);
        left -= min(left, (long long)(at.end - at.tile));
        if (left == 0) break;
        at.next_segment(p);
    }
}

// ---- the issuing threads --------------------------------------------------
//
// Neither relies on the order in which the tensor cores take up products of
// different shape: each waits until what it overwrites has been read.

// Nothing a thread issued may outlive the CTA's shared and tensor memory.
__device__ __forceinline__ void drain(uint64_t *bar) {
    kda::umma_commit(bar);
    kda::mbar_wait_bounded(bar, 0, kWaitBudget);
}

// S = Q K^T of every tile.
template <typename T, int kDim, int kQRows>
__device__ __forceinline__ void run_scores(const Params &p, const Run &run, Control &c,
                                           uint32_t smem, uint32_t tmem) {
    using F = Form<kDim, kQRows>;
    constexpr uint32_t kId = idesc<T>(kRows, kTile, false);
    Cursor at = run_start(run, c.plan);
    const long long tiles = run.end - run.begin;
    const uint64_t q_desc = kda::sw128_desc(F::query(smem) - first_lane<kQRows>() * 128);
    uint32_t phase = 0;
    int stage = 0;
    uint32_t segment = 0;
    for (long long g = 0; g < tiles; ++g) {
        if (g == 0 || at.tile == at.first) {
            if (!wait(c, &c.q_full, segment & 1u, p.rows.err)) break;
            ++segment;
        }
        // it goes where P(g - 2) was: that product has to be complete
        if (g >= 2 && !wait(c, &c.o_done[g & 1], (uint32_t)((g / 2 - 1) & 1), p.rows.err)) break;
        if (!wait(c, &c.full[stage], phase, p.rows.err)) break;
        kda::tc_fence_after();
        const uint64_t k_desc = kda::sw128_desc(F::stage(smem, stage));
        const uint32_t s = tmem + F::kS + (uint32_t)(g & 1) * kTile;
#pragma unroll
        for (int k = 0; k < kDim / 16; ++k)
            mma_ss(s, q_desc + (((k >> 2) * kQRows * 128 + (k & 3) * 32) >> 4),
                   k_desc + (((k >> 2) * kTile * 128 + (k & 3) * 32) >> 4), kId, k > 0);
        kda::umma_commit(&c.s_full[g & 1]);
        kda::umma_commit(&c.empty[stage]);
        if (g + 1 == tiles || at.tile + 1 == at.end) kda::umma_commit(&c.q_empty);
        stage += 2;
        if (stage >= F::kStages) {
            stage -= F::kStages;
            phase ^= 1u;
        }
        if (g + 1 < tiles && ++at.tile == at.end) at.next_segment(p);
    }
    drain(&c.drained[0]);
}

// O += P V of every tile.
template <typename T, int kDim, int kQRows>
__device__ __forceinline__ void run_outputs(const Params &p, const Run &run, Control &c,
                                            uint32_t smem, uint32_t tmem) {
    using F = Form<kDim, kQRows>;
    constexpr uint32_t kId = idesc<T>(kRows, kDim, true);
    Cursor at = run_start(run, c.plan);
    p.cuts[blockIdx.x] = first_cut(run, at, blockIdx.x);
    const long long tiles = run.end - run.begin;
    uint32_t phase = 0;
    int stage = 1;
    bool first = true;   // the segment's first tile
    for (long long g = 0; g < tiles; ++g) {
        const int b = (int)(g & 1);
        if (!wait(c, &c.p_full[b], (uint32_t)((g >> 1) & 1), p.rows.err)) break;
        if (!wait(c, &c.full[stage], phase, p.rows.err)) break;
        kda::tc_fence_after();
        uint32_t add = first ? 0u : 1u;
        volatile int *keep = &c.keep[b];
        if (*keep != 0) {
            add = 1;
            *keep = 0;
        }
        const uint64_t v_desc = mn_desc(F::stage(smem, stage), kTile * 128);
        const uint32_t pp = tmem + F::kS + (uint32_t)b * kTile;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
            mma_ts(tmem, pp + 8 * k, v_desc + (k * 2048 >> 4), kId, k > 0 ? 1u : add);
        kda::umma_commit(&c.o_done[b]);
        kda::umma_commit(&c.empty[stage]);
        stage += 2;
        if (stage >= F::kStages) {
            stage -= F::kStages;
            phase ^= 1u;
        }
        first = false;
        if (g + 1 < tiles && ++at.tile == at.end) {
            at.next_segment(p);
            first = true;
        }
    }
    drain(&c.drained[1]);
}

// ---- the softmax warps ----------------------------------------------------

template <typename T, int kDim, int kQRows, bool kSliding>
__device__ __forceinline__ void run_softmax(const Params &p, const Run &run, Control &c,
                                            uint32_t smem, uint32_t tmem_all, int cta, int warp,
                                            int lane) {
    using F = Form<kDim, kQRows>;
    constexpr int kChunks = kDim / 8;
    const int tid = warp * 32 + lane;
    const int row = tid - first_lane<kQRows>();                           // query row of this thread
    const uint32_t tmem = tmem_all + ((uint32_t)(warp * 32) << 16);  // the warp's lanes
    const float scale = p.flip != 0 ? -p.scale_log2 : p.scale_log2;
    Cursor at = run_start(run, c.plan);
    long long left = run.end - run.begin, g = 0;
    bool run_first = true;
    uint32_t meetings = 0;
    auto meet = [&]() -> bool {  // a barrier of the four warps
        __syncwarp();
        if (lane == 0) kda::mbar_arrive(&c.meet);
        return warp_wait(c, &c.meet, meetings++ & 1u, p.rows.err);
    };
    auto product_done = [&]() -> bool {  // of the tile before tile g
        return warp_wait(c, &c.o_done[(g - 1) & 1], (uint32_t)(((g - 1) >> 1) & 1), p.rows.err);
    };
    while (left > 0) {
        const int tiles = (int)min(left, (long long)(at.end - at.tile));
        const bool whole = at.tile == at.first && tiles == at.end - at.first;
        const int rows = at.row.tokens * p.group;
        const bool active = row - lane >= 0 && row - lane < rows;
        const bool mine = row >= 0 && row < rows;
        const int token = token_of(p, max(row, 0));
        const int hi = at.row.computed + min(token, at.row.tokens - 1);
        const int lo = kSliding ? hi - p.left_window : -1;
        float m = -INFINITY, l = 0.0f;
        for (int done = 0; done < tiles; ++done, ++g) {
            const int b = (int)(g & 1);
            const uint32_t s_col = tmem + F::kS + b * kTile;
            if (!warp_wait(c, &c.s_full[b], (uint32_t)((g >> 1) & 1), p.rows.err)) return;
            kda::tc_fence_after();
            const int key0 = (at.tile + done) * kTile;
            const unsigned long long seen =
                (unsigned long long)*reinterpret_cast<volatile uint32_t *>(&c.there[g & 7][0]) |
                (unsigned long long)*reinterpret_cast<volatile uint32_t *>(&c.there[g & 7][1]) << 32;
            // a tile that some row does not see whole
            const bool edge =
                key0 + kTile - 1 > at.row.computed || seen != ~0ull ||
                (kSliding && key0 <= at.row.computed + at.row.tokens - 1 - p.left_window);
            if (active) {
                float s[kTile];
                {
                    uint32_t u[kTile / 16][16];
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i) kda::tmem_ld16(s_col + 16 * i, u[i]);
                    kda::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i) {
                        landed(u[i]);
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[16 * i + e] = __uint_as_float(u[i][e]);
                    }
                }
                // scores as they are times mul: where all of a tile counts and
                // the scale is positive, the factor is part of the exponent
                float mul = scale;
                if (edge || p.flip != 0) {
                    mul = 1.0f;
                    // the row's keys of the tile: up to hi, past lo, in the cache
                    const int upto = hi - key0 + 1, from = lo - key0 + 1;
                    unsigned long long own = upto >= 64  ? ~0ull
                                             : upto > 0 ? (1ull << upto) - 1
                                                        : 0ull;
                    own &= from >= 64 ? 0ull : from > 0 ? ~0ull << from : ~0ull;
                    own &= seen;
                    const uint32_t half[2] = {(uint32_t)own, (uint32_t)(own >> 32)};
#pragma unroll
                    for (int i = 0; i < kTile; ++i)
                        s[i] = (half[i / 32] >> (i % 32)) & 1u ? s[i] * scale : -INFINITY;
                }
                float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < kTile; ++i) top[i & 3] = fmaxf(top[i & 3], s[i]);
                const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * mul;
                if (__any_sync(kFull, most > m + kLazy)) {
                    const float now = fmaxf(m, most);
                    const float f = now == -INFINITY ? 1.0f : exp2_fast(m - now);
                    if (done > 0) {
                        if (!product_done()) return;
                        kda::tc_fence_after();
                        scale_o<kDim>(tmem, f);
                    }
                    m = now;
                    l *= f;
                }
                const float base = m == -INFINITY ? 0.0f : m - kLift<T>;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < kTile; i += 32) {
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float x = exp2_fast(fmaf(s[i + e], mul, -base));
                        const float y = exp2_fast(fmaf(s[i + e + 1], mul, -base));
                        sum[e & 2] += x;
                        sum[(e & 2) + 1] += y;
                        u[e / 2] = pack(x, y, T());
                    }
                    kda::tmem_st16(s_col + i / 2, u);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                kda::tmem_wait_st();
            }
            // A value that is not finite must not reach the rows that do not
            // see its key (0 * inf is NaN in the product).  What lies past the
            // row's end or behind a sliding window is zeroed; of the other keys
            // only those matter that some rows see and others do not: the
            // window's own but the first, and as many at a sliding window's
            // start.
            const int tail = at.row.computed + at.row.tokens - key0;  // first key past the row
            if (edge && (at.row.tokens > 1 || kSliding || tail < kTile)) {
                const int j = (int)((2 * g + 1) % F::kStages);
                if (!warp_wait(c, &c.full[j], (uint32_t)(((2 * g + 1) / F::kStages) & 1),
                               p.rows.err))
                    return;
                const uint32_t values = F::stage(smem, j);
                const int front = kSliding ? first_key(p, at.row) - key0 : 0;  // first key seen
                for (int i = (front > 0 ? 0 : max(tail, 0) * kChunks) + tid; i < kTile * kChunks;
                     i += 32 * kSoftmaxWarps)
                    if (i / kChunks < front || i / kChunks >= tail)
                        store16(values + place(i / kChunks, i % kChunks, kTile),
                                make_uint4(0, 0, 0, 0));
                kda::fence_proxy_async_smem();
                const int own = at.row.tokens - 1;
                unsigned long long odd = 0;
                for (int i = lane; i < (kSliding ? 2 : 1) * own * kChunks; i += 32) {
                    const int k = i / kChunks;
                    const int key = (k < own ? at.row.computed + 1 + k
                                             : at.row.computed + 1 - p.left_window + k - own) -
                                    key0;
                    if (key < 0 || key >= kTile) continue;
                    const uint4 x = load16(values + place(key, i % kChunks, kTile));
                    if (not_finite(x.x, T()) || not_finite(x.y, T()) || not_finite(x.z, T()) ||
                        not_finite(x.w, T()))
                        odd |= 1ull << key;
                }
                odd = (unsigned long long)__reduce_or_sync(kFull, (uint32_t)odd) |
                      (unsigned long long)__reduce_or_sync(kFull, (uint32_t)(odd >> 32)) << 32;
                if (odd != 0) {  // the same for the four warps
                    if (active) {
                        // such values are added by hand to the rows that do
                        // see them, and zeroed for the product
                        if (done > 0) {
                            if (!product_done()) return;
                            kda::tc_fence_after();
                        } else {
                            uint32_t zero[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) zero[e] = 0;
#pragma unroll
                            for (int d = 0; d < kDim; d += 16) kda::tmem_st16(tmem + d, zero);
                            kda::tmem_wait_st();
                            *reinterpret_cast<volatile int *>(&c.keep[b]) = 1;
                        }
                        for (unsigned long long bits = odd; bits != 0; bits &= bits - 1) {
                            const int key = __ffsll((long long)bits) - 1;
                            const float2 both = unpack(tmem_load1(s_col + key / 2), T());
                            const float weight = (key & 1) ? both.y : both.x;
                            const bool sees = key0 + key <= hi && key0 + key > lo;
#pragma unroll 1
                            for (int d = 0; d < kDim; d += 16) {
                                uint32_t u[16];
                                tmem_load16(tmem + d, u);
#pragma unroll
                                for (int e = 0; e < 16; e += 8) {
                                    const uint4 x =
                                        load16(values + place(key, (d + e) / 8, kTile));
                                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                    for (int n = 0; n < 4; ++n) {
                                        const float2 v = unpack(w[n], T());
                                        float *a = reinterpret_cast<float *>(&u[e + 2 * n]);
                                        if (sees) {
                                            a[0] = fmaf(weight, v.x, a[0]);
                                            a[1] = fmaf(weight, v.y, a[1]);
                                        }
                                    }
                                }
                                __syncwarp();
                                kda::tmem_st16(tmem + d, u);
                                kda::tmem_wait_st();
                            }
                        }
                    }
                    if (!meet()) return;  // every warp has read them
                    for (int i = tid; i < kTile * kChunks; i += 32 * kSoftmaxWarps)
                        if ((odd >> (i / kChunks)) & 1ull)
                            store16(values + place(i / kChunks, i % kChunks, kTile),
                                    make_uint4(0, 0, 0, 0));
                    kda::fence_proxy_async_smem();
                }
            }
            // A warp sees every product's phase, one after the other: had it
            // skipped one, a later wait could take the parity of the phase
            // before for its own.  (The next product cannot start before this
            // one is complete, so nothing is lost here.)
            if (g > 0 && !product_done()) return;
            kda::tc_fence_before();
            __syncwarp();
            if (lane == 0) kda::mbar_arrive(&c.p_full[b]);
        }

        // the segment's place in the results, then on to the next one while
        // this one's last product is made
        const long long out_row = (long long)(at.row.first + token) * p.q_heads +
                                  at.head * p.group + row - token * p.group;
        float *piece = p.partials + (2ll * cta + (run_first ? 0 : 1)) * p.slot_size;
        left -= tiles;
        run_first = false;
        if (left > 0) at.next_segment(p);
        if (!product_done()) return;
        kda::tc_fence_after();
        m -= kLift<T>;  // what l and O are relative to
        if (active) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int d0 = 0; d0 < kDim; d0 += 32) {
                uint32_t u[2][16];
                kda::tmem_ld16(tmem + d0, u[0]);
                kda::tmem_ld16(tmem + d0 + 16, u[1]);
                kda::tmem_wait_ld();
                landed(u[0]);
                landed(u[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int d = d0 + 16 * i;
                    if (mine && whole) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = pack(__uint_as_float(u[i][2 * e]) * inv,
                                        __uint_as_float(u[i][2 * e + 1]) * inv, T());
                        uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<T *>(p.out) +
                                                               out_row * kDim + d);
                        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    } else if (mine) {
                        uint4 *dst = reinterpret_cast<uint4 *>(piece + row * kDim + d);
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            dst[e / 4] = make_uint4(u[i][e], u[i][e + 1], u[i][e + 2], u[i][e + 3]);
                    }
                }
                __syncwarp();
            }
        }
        if (mine) {
            if (!whole) {
                piece[p.most_rows * kDim + row] = m;
                piece[p.most_rows * (kDim + 1) + row] = l;
            } else if (p.lse != nullptr) {
                p.lse[out_row] = (m + log2f(l)) * kLn2;
            }
        }
        kda::tc_fence_before();
    }
}

template <typename T, int kDim, int kQRows, bool kSliding>
__global__ void __launch_bounds__(kThreadCount, kCtasPerSm)
    attend_tc_kernel(const Params p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
    using F = Form<kDim, kQRows>;
    extern __shared__ __align__(1024) unsigned char smem_tc[];
    Control &c = *reinterpret_cast<Control *>(smem_tc + F::kQuery + F::kStages * F::kStage);
    static_assert(sizeof(Control) <= F::kControl, "control area");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t smem = kda::smem_u32(smem_tc);
    kda_cache::grid_dependents_launch();
    if (tid == 0) {
        for (int i = 0; i < F::kStages; ++i) {
            kda::mbar_init(&c.full[i], 1);
            kda::mbar_init(&c.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            kda::mbar_init(&c.s_full[i], 1);
            kda::mbar_init(&c.p_full[i], kSoftmaxWarps);
            kda::mbar_init(&c.o_done[i], 1);
            c.keep[i] = 0;
        }
        kda::mbar_init(&c.q_full, 1);
        kda::mbar_init(&c.q_empty, 1);
        kda::mbar_init(&c.meet, kSoftmaxWarps);
        kda::mbar_init(&c.drained[0], 1);
        kda::mbar_init(&c.drained[1], 1);
        c.abort = 0;
        kda::fence_mbar_init();
    }
    if (warp == kScoreWarp) kda::tmem_alloc(&c.tmem, kTmemColumns);
    kda_cache::grid_dependency_wait();
    const Run run = plan<kWarpCount>(p, c.plan);
    const int cta = blockIdx.x;
    const bool busy = cta < run.ctas;
    if (!busy && tid == 0) p.cuts[cta].pieces = 0;
    kda::tc_fence_before();
    __syncthreads();
    kda::tc_fence_after();
    const uint32_t tmem = c.tmem;
    if (busy) {
        if (warp < kSoftmaxWarps) {
            run_softmax<T, kDim, kQRows, kSliding>(p, run, c, smem, tmem, cta, warp, lane);
        } else if (warp == kLoadWarp) {
            run_loader<T, kDim, kQRows, kSliding>(p, run, c, smem, lane, &k_map, &v_map);
        } else if (warp == kQueryWarp) {
            run_queries<T, kDim, kQRows>(p, run, c, smem, lane);
        } else if (lane == 0) {
            if (warp == kScoreWarp)
                run_scores<T, kDim, kQRows>(p, run, c, smem, tmem);
            else
                run_outputs<T, kDim, kQRows>(p, run, c, smem, tmem);
        }
        __syncwarp();
    }
    kda::tc_fence_before();
    __syncthreads();
    kda::tc_fence_after();
    if (warp == kScoreWarp) kda::tmem_dealloc(tmem, kTmemColumns);
}

}  // namespace tc

// Joins the pieces of the segments that runs cut: block (i, y) takes the
// segment first cut at the start of CTA i + 1's run, a warp its query rows
// 4 y + warp, then 4 gridDim.y on.  The pieces' maxima and sums are read one a
// lane, their O in batches of kBatch loads, the first batch in flight with
// them.
constexpr int kJoinRows = 16;   // blocks a cut, at most

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads) join_kernel(const Params p) {
    constexpr int kLanes = kDim / 4;           // lanes that hold a row
    constexpr int kSide = 32 / kLanes;         // pieces a warp reads side by side
    constexpr int kBatch = 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    kda_cache::grid_dependents_launch();
    kda_cache::grid_dependency_wait();
    const int cta = blockIdx.x + 1;
    const int4 head = __ldcg(reinterpret_cast<const int4 *>(&p.cuts[cta]));
    const int kv_head = __ldcg(&p.cuts[cta].head);
    const int pieces = head.x, tokens = head.w;
    if (pieces == 0) return;
    const float *first = p.partials + head.y * p.slot_size;
    const float *others = p.partials + 2 * (cta - 1) * p.slot_size;  // piece i > 0: 2 i slots on
    auto piece = [&](int i) { return i == 0 ? first : others + 2 * i * p.slot_size; };
    for (int r = blockIdx.y * kWarps + warp; r < tokens * p.group; r += gridDim.y * kWarps) {
        float m = -INFINITY, l = 0.0f;  // of the pieces so far, in every lane and per lane
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i0 = 0; i0 < pieces; i0 += 32) {
            const int here = min(32, pieces - i0);
            float own_m = -INFINITY, own_l = 0.0f;
            if (lane < here) {
                const float *part = piece(i0 + lane);
                own_m = __ldcg(part + p.most_rows * kDim + r);
                own_l = __ldcg(part + p.most_rows * (kDim + 1) + r);
            }
            float weight = 0.0f;
            for (int k = 0; k < here; k += kBatch * kSide) {
                float4 x[kBatch];
#pragma unroll
                for (int n = 0; n < kBatch; ++n) {
                    const int i = k + n * kSide + lane / kLanes;
                    x[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i < here)
                        x[n] = __ldcg(reinterpret_cast<const float4 *>(
                            piece(i0 + i) + r * kDim + lane % kLanes * 4));
                }
                if (k == 0) {  // the weights of these 32 pieces
                    float top = own_m;
#pragma unroll
                    for (int s = 16; s > 0; s >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(kFull, top, s));
                    top = fmaxf(top, m);
                    const float base = top == -INFINITY ? 0.0f : top;
                    const float f = exp2_fast(m - base);
                    l *= f;
                    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
                    weight = exp2_fast(own_m - base);
                    l = fmaf(weight, own_l, l);
                    m = top;
                }
#pragma unroll
                for (int n = 0; n < kBatch; ++n) {
                    const float w =
                        __shfl_sync(kFull, weight, min(31, k + n * kSide + lane / kLanes));
                    o.x = fmaf(w, x[n].x, o.x);
                    o.y = fmaf(w, x[n].y, o.y);
                    o.z = fmaf(w, x[n].z, o.z);
                    o.w = fmaf(w, x[n].w, o.w);
                }
            }
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(kFull, l, s);
        if constexpr (kSide == 2) {
            o.x += __shfl_xor_sync(kFull, o.x, 16);
            o.y += __shfl_xor_sync(kFull, o.y, 16);
            o.z += __shfl_xor_sync(kFull, o.z, 16);
            o.w += __shfl_xor_sync(kFull, o.w, 16);
        }
        const float f = l == 0.0f ? 0.0f : 1.0f / l;
        const int t = token_of(p, r);
        const long long row =
            (long long)(head.z + t) * p.q_heads + kv_head * p.group + r - t * p.group;
        if (lane < kLanes)
            *reinterpret_cast<uint2 *>(reinterpret_cast<T *>(p.out) + row * kDim + lane * 4) =
                make_uint2(pack(o.x * f, o.y * f, T()), pack(o.z * f, o.w * f, T()));
        if (lane == 0 && p.lse != nullptr) p.lse[row] = (m + log2f(l)) * kLn2;
    }
}

template <typename T, int kDim>
kda_status launch_join(const Params &p, int grid, void *stream) {
    void (*join)(const Params) = join_kernel<T, kDim>;
    const int blocks = min(kJoinRows, (p.most_rows + kWarps - 1) / kWarps);
    return kda_cache::launch(join, dim3(grid - 1, blocks), dim3(kThreads), 0, 1, stream, p);
}

// ------------------------------------------------------------------- host --

// Allows a kernel its shared memory, once per device (`done` is the kernel's).
bool allow_shared(const void *kernel, int bytes, bool (&done)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev >= 0 && dev < 64 && done[dev]) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess)
        return false;
    if (dev >= 0 && dev < 64) done[dev] = true;
    return true;
}

template <typename T, int kDim, int kMT, int kMW, int kCtas>
kda_status launch_attend(Params &p, int sms, void *stream) {
    using L = Layout<kDim, kMT, kMW, kCtas>;
    const int grid = min(kCtas * sms, kMaxCtas);
    p.by_grid = kda_cache::make_divider(grid);
    void (*kernel)(const Params) = attend_kernel<T, kDim, kMT, kMW, kCtas>;
    static bool allowed[64];
    if (!allow_shared(reinterpret_cast<const void *>(kernel), L::kBytes, allowed))
        return KDA_ERR_CUDA;
    kda_status st = kda_cache::launch(kernel, dim3(grid), dim3(kThreads), L::kBytes, 1, stream, p);
    if (st != KDA_OK || grid == 1) return st;
    return launch_join<T, kDim>(p, grid, stream);
}

// The driver's tensor-map encoder, looked up once through the runtime (the
// library links no driver library).
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// A cache as [block][head][token][channel], read in boxes of 64 channels of
// p.box tokens with the 128-byte swizzle.  False when it cannot be described.
template <typename T, int kDim>
bool cache_map(const Params &p, const char *base, CUtensorMap *map) {
    const EncodeTiledFn encode = encode_tiled();
    if (encode == nullptr) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)kDim, (cuuint64_t)p.rows.block_size,
                                (cuuint64_t)p.kv_heads, (cuuint64_t)p.rows.num_blocks};
    const cuuint64_t strides[3] = {(cuuint64_t)p.stride_token * 2, (cuuint64_t)p.stride_head * 2,
                                   (cuuint64_t)p.stride_block * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1}, step[4] = {1, 1, 1, 1};
    return encode(map,
                  sizeof(T) == 2 && __is_same(T, __nv_bfloat16) ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  4, const_cast<char *>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  kDim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                              : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int kDim, int kQRows, bool kSliding>
kda_status launch_tc(Params &p, const CUtensorMap &k_map, const CUtensorMap &v_map, int sms,
                     void *stream) {
    const int grid = min(tc::kCtasPerSm * sms, kMaxCtas);
    p.by_grid = kda_cache::make_divider(grid);
    using F = tc::Form<kDim, kQRows>;
    void (*kernel)(const Params, const CUtensorMap, const CUtensorMap) =
        tc::attend_tc_kernel<T, kDim, kQRows, kSliding>;
    static bool allowed[64];
    if (!allow_shared(reinterpret_cast<const void *>(kernel), F::kBytes, allowed))
        return KDA_ERR_CUDA;
    kda_status st = kda_cache::launch(kernel, dim3(grid), dim3(tc::kThreadCount), F::kBytes, 1,
                                      stream, p, k_map, v_map);
    if (st != KDA_OK || grid == 1) return st;
    return launch_join<T, kDim>(p, grid, stream);
}

template <typename T, int kDim>
kda_status launch_rows(Params &p, int sms, void *stream) {
    // Which kernel: measured on 96 rows of up to 2000 keys | 16 rows of up to
    // 30000 | 300 ragged rows of up to 1000 (us), 4 kv heads, the rows' lengths
    // spread evenly over an eighth of the longest to the longest.
    //   channels  query rows   16 rows a warp      tensor-core form     floor
    //   128       16           49 |  93 |  68      59 |  98 |  99       33 | 83 | 52
    //   128       32           56 |  98 |  74      63 | 100 | 102       34 | 83 | 53
    //   128       40           71 | 118 |  95      66 | 103 | 105       34 | 83 | 53
    //   128       64           79 | 125 | 100      74 | 106 | 109       35 | 83 | 55
    //   128       128         168 | 281 | 227     100 | 120 | 129       37 | 83 | 58
    //   64        32           35 |  57 |  49      53 |  70 |  89       17 | 41 | 27
    //   64        64           49 |  80 |  66      60 |  77 |  95       17 | 41 | 27
    //   64        96           77 | 121 | 102      65 |  84 |  99       18 | 42 | 28
    // (The lengths are on the device, so they are no part of the rule.)  The
    // tensor-core form reads the cache in boxes of p.box keys and 64 channels,
    // which have to be swizzled atoms of 8 rows; with 96 rows of 64 channels
    // 66 us in boxes of 8 keys, 65 of 16, and 76 for the other form.
    p.box = kTile;
    while (p.rows.block_size % p.box != 0) p.box /= 2;
    if (p.most_rows > (kDim == 128 ? 32 : 64) && p.box >= 8) {
        CUtensorMap k_map, v_map;  // (a cache they cannot describe goes the other way)
        // A sliding window is a kernel of its own: where one served both, what it
        // has to leave out cost calls without one too, 118 us for 300 rows of up
        // to 1000 keys and 64 query rows, 109 so, and 95 over the last 300 keys of
        // them, 92 so.
        if (cache_map<T, kDim>(p, p.key_cache, &k_map) &&
            cache_map<T, kDim>(p, p.value_cache, &v_map))
            return p.most_rows <= 64
                       ? (p.left_window > 0
                              ? launch_tc<T, kDim, 64, true>(p, k_map, v_map, sms, stream)
                              : launch_tc<T, kDim, 64, false>(p, k_map, v_map, sms, stream))
                       : (p.left_window > 0
                              ? launch_tc<T, kDim, 128, true>(p, k_map, v_map, sms, stream)
                              : launch_tc<T, kDim, 128, false>(p, k_map, v_map, sms, stream));
    }
    // With 64 channels and 32 or 64 rows three CTAs fit an SM: 35 and 49 us,
    // with two 40 and 54; with up to 16 rows two measured better (31 | 55 | 45
    // us against 34 | 64 | 52 at 8 rows).
    constexpr int kWide = kDim == 64 ? 3 : 2;
    if (p.most_rows <= 16) return launch_attend<T, kDim, 1, 1, 2>(p, sms, stream);
    if (p.most_rows <= 32) return launch_attend<T, kDim, 1, 2, kWide>(p, sms, stream);
    if (p.most_rows <= 64) return launch_attend<T, kDim, 1, 4, kWide>(p, sms, stream);
    return launch_attend<T, kDim, 2, 4, 2>(p, sms, stream);
}

kda_status check_attention(const kda_cache_config *c) {
    kda_status st = kda_cache::check_config(c);
    if (st != KDA_OK) return st;
    if (c->window < 1 || c->left_window < 0) return KDA_ERR_INVALID_ARG;
    if (c->window > KDA_MAX_WINDOW) return KDA_ERR_UNSUPPORTED;
    if (c->window * (c->q_heads / c->kv_heads) > KDA_MAX_QUERY_ROWS) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Floats of a partial slot, a multiple of 16 bytes.
long long slot_floats(const kda_cache_config *c) {
    const long long rows = c->window * (c->q_heads / c->kv_heads);
    return (rows * (c->head_dim + 2) + 3) / 4 * 4;
}

}  // namespace

extern "C" {

size_t kda_attention_workspace_bytes(const kda_cache_config *cfg, int32_t B) {
    if (check_attention(cfg) != KDA_OK || B < 0) return 0;
    return kMaxCtas * (sizeof(Cut) + 2 * (size_t)slot_floats(cfg) * sizeof(float));
}

kda_status kda_window_attention(const kda_cache_config *cfg, const void *q, const void *key_cache,
                                const void *value_cache, const int32_t *cu_seqlens, int32_t B,
                                int32_t num_tokens, const kda_align *align, void *workspace,
                                size_t workspace_bytes, void *out, float *lse,
                                int32_t *error_word, void *stream) {
    using kda_cache::aligned;
    kda_status st = check_attention(cfg);
    if (st != KDA_OK) return st;
    if (B < 0 || num_tokens < 0) return KDA_ERR_INVALID_ARG;
    if (B == 0 || num_tokens == 0) return KDA_OK;  // nothing to do; no pointer is inspected
    Params p;
    st = kda_cache::set_rows(cfg, align, cu_seqlens, B, num_tokens, error_word, p.rows);
    if (st != KDA_OK) return st;
    if (!q || !key_cache || !value_cache || !out || !workspace) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) ||
        !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4) ||
        !kda_cache::stride_ok(cfg->stride_q_t))
        return KDA_ERR_INVALID_ARG;
    if (!(cfg->scale == cfg->scale) || cfg->scale - cfg->scale != 0.0f) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < kda_attention_workspace_bytes(cfg, B)) return KDA_ERR_INVALID_ARG;
    const int sms = kda_cache::sm_count();
    if (sms <= 0) return KDA_ERR_CUDA;
    p.q = static_cast<const char *>(q);
    p.key_cache = static_cast<const char *>(key_cache);
    p.value_cache = static_cast<const char *>(value_cache);
    p.out = static_cast<char *>(out);
    p.lse = lse;
    p.cuts = static_cast<Cut *>(workspace);
    p.partials = reinterpret_cast<float *>(static_cast<char *>(workspace) + kMaxCtas * sizeof(Cut));
    p.stride_q = cfg->stride_q_t;
    p.stride_block = cfg->stride_block;
    p.stride_token = cfg->stride_token;
    p.stride_head = cfg->stride_head;
    p.q_heads = cfg->q_heads;
    p.kv_heads = cfg->kv_heads;
    p.group = cfg->q_heads / cfg->kv_heads;
    p.by_group = (65536 + p.group - 1) / p.group;
    p.by_heads = kda_cache::make_divider(p.kv_heads);
    p.window = cfg->window;
    p.left_window = cfg->left_window;
    p.most_rows = cfg->window * p.group;
    p.slot_size = slot_floats(cfg);
    p.scale_log2 = fabsf(cfg->scale) * kLog2e;
    if (p.scale_log2 == 0.0f) p.scale_log2 = 1.4e-45f;  // 0 times a masked -inf is NaN
    p.flip = cfg->scale < 0.0f ? 0x80008000u : 0u;
    if (cfg->dtype == KDA_DTYPE_BF16)
        return cfg->head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(p, sms, stream)
                                   : launch_rows<__nv_bfloat16, 128>(p, sms, stream);
    return cfg->head_dim == 64 ? launch_rows<__half, 64>(p, sms, stream)
                               : launch_rows<__half, 128>(p, sms, stream);
}

kda_status kda_window_attention_packed(const kda_attention_args *a) {
    if (a == nullptr) return KDA_ERR_INVALID_ARG;
    return kda_window_attention(&a->config, a->q, a->key_cache, a->value_cache, a->cu_seqlens,
                                a->B, a->num_tokens, &a->align, a->workspace, a->workspace_bytes, a->out,
                                a->lse, a->error_word, a->stream);
}

}  // extern "C"
