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
// Work split.  The unit is a tile of 64 keys of one (row, kv head); all tiles
// of the call, in row, head, key order, are cut into equal runs, one per CTA,
// two CTAs per SM.  Each CTA finds its run from the rows' lengths by itself.
// A run may cut a (row, head) segment: the pieces leave (m, l, O) in fp32 in
// the workspace, and a second, short kernel joins them in a fixed order.
//
// A CTA has 4 warps in groups of kMW.  A group's warps hold different query
// rows (16 * kMT each) of the same keys; the 4 / kMW groups take different
// keys of each tile.  Keys and values arrive by 16-byte cp.async in a ring of
// tiles, each warp loading its own 16 keys, so with kMW = 1 no warp waits for
// another inside a segment.  The products are mma.sync m16n8k16 on fragments
// that ldmatrix reads from XOR-swizzled rows.
#include "kda_async.cuh"
#include "kda_cache.cuh"

namespace {

using kda_cache::kFull;
using kda_cache::Row;
using kda_cache::Rows;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 64;             // keys of a tile
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 512;         // bound of the grid, for the workspace
constexpr float kLazy = 8.0f;         // log2 of the growth a stale maximum may have
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
    float *partials;         // [2 * grid][R_max * (D + 2)]
    Cut *cuts;               // [grid]
    long long stride_q, stride_block, stride_token, stride_head;  // elements
    int q_heads, kv_heads, group, window, left_window, most_rows;
    float scale_log2;
};

// ------------------------------------------------------------ instructions --

__device__ __forceinline__ float exp2_fast(float x) {  // within 2 ulp, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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

__device__ __forceinline__ uint32_t pack(float lo, float hi, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi, __half) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 unpack(uint32_t u, __nv_bfloat16) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

__device__ __forceinline__ float2 unpack(uint32_t u, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
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

// The tiles a row's keys span: [first, end).
__device__ __forceinline__ void row_tiles(const Params &p, const Row &row, int &first, int &end) {
    const int lo = p.left_window > 0 ? max(0, row.computed + 1 - p.left_window) : 0;
    first = lo / kTile;
    end = row.tokens > 0 ? (row.computed + row.tokens - 1) / kTile + 1 : first;
}

__device__ __forceinline__ int tile_count(const Params &p, int b, int &bits) {
    int first, end;
    const Row row = kda_cache::read_row(p.rows, b, p.window, bits);
    row_tiles(p, row, first, end);
    return end - first;
}

// Where a CTA's run stands: tile `tile` of kv head `head` of row `b`.
struct Cursor {
    Row row;
    int b, head, tile, first, end;

    __device__ __forceinline__ void set_row(const Params &p, int row_index) {
        b = row_index;
        int bits = 0;
        row = kda_cache::read_row(p.rows, b, p.window, bits);
        row_tiles(p, row, first, end);
        tile = first;
    }
    __device__ __forceinline__ void next_segment(const Params &p) {
        if (++head < p.kv_heads) {
            tile = first;
            return;
        }
        head = 0;
        do {
            if (b + 1 >= p.rows.B) return;  // past the last unit; never read
            set_row(p, b + 1);
        } while (end == first);
    }
};

struct Run {
    long long units, begin, end;  // of the call; this CTA's [begin, end)
    long long before_row;         // units before the starting row
    int row, ctas;                // CTAs with work
};

// First unit of CTA i's run, and the CTA whose run holds unit u.
__device__ __forceinline__ long long run_begin(long long units, int ctas, int i) {
    return units * i / ctas;
}

__device__ __forceinline__ int cta_of(long long units, int ctas, long long u) {
    return (int)(((u + 1) * ctas - 1) / units);
}

// Every CTA adds up the rows' tiles itself: thread i takes a run of rows, a
// scan over the threads gives the units before it, and the thread whose rows
// hold the CTA's first unit finds the row.
__device__ __forceinline__ Run plan(const Params &p) {
    __shared__ long long sums[kWarps];
    __shared__ long long found_before;
    __shared__ int found_row;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.rows.B + kThreads - 1) / kThreads;
    const int b0 = min(p.rows.B, tid * per), b1 = min(p.rows.B, b0 + per);
    long long mine = 0;
    int bits = 0;
    for (int b = b0; b < b1; ++b) mine += tile_count(p, b, bits);
    if (bits != 0 && blockIdx.x == 0) kda_cache::flag(p.rows.err, bits);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long other = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += other;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long before = upto - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    Run run;
    run.units = total * p.kv_heads;
    run.ctas = (int)min((long long)gridDim.x, run.units);
    run.begin = run.end = 0;
    if ((int)blockIdx.x >= run.ctas) return run;  // uniform over the CTA
    run.begin = run_begin(run.units, run.ctas, blockIdx.x);
    run.end = run_begin(run.units, run.ctas, blockIdx.x + 1);
    const long long at = run.begin / p.kv_heads;  // the first tile, counted over rows
    if (at >= before && at < before + mine) {
        int b = b0;
        for (;; ++b) {
            const int n = tile_count(p, b, bits);
            if (at < before + n) break;
            before += n;
        }
        found_row = b;
        found_before = before * p.kv_heads;
    }
    __syncthreads();
    run.row = found_row;
    run.before_row = found_before;
    return run;
}

// ---------------------------------------------------------------- layout --

template <int kDim, int kMT, int kMW>
struct Layout {
    static constexpr int kRows = 16 * kMT * kMW;       // query rows, padded
    static constexpr int kGroups = kWarps / kMW;
    static constexpr int kKeys = kTile / kGroups;      // keys of a group's step
    static constexpr int kRowBytes = kDim * 2;
    static constexpr int kHalfTile = kTile * kRowBytes;
    static constexpr int kStage = 2 * kHalfTile;       // keys, then values
    // the queries and, between segments, half of the channels of the sum
    // over the groups share one area
    static constexpr int kQuery = kRows * kRowBytes;
    static constexpr int kSum = kGroups > 1 ? kRows * kDim / 2 * 4 : 0;
    static constexpr int kShared = kQuery > kSum ? kQuery : kSum;
    static constexpr int kStats = kGroups * kRows * 8;
    static constexpr int kFixed = kShared + kStats;
    static constexpr int kBudget = 114000;             // two CTAs per SM
    static constexpr int kStages = (kBudget - kFixed) / kStage < 6 ? (kBudget - kFixed) / kStage : 6;
    static constexpr int kBytes = kFixed + kStages * kStage;
    static_assert(kStages >= 2, "the ring needs two tiles");
};

// Byte offset of 16-byte chunk c of row r in a swizzled tile.
template <int kDim>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    return (uint32_t)(r * kDim * 2 + ((c ^ (r & 7)) << 4));
}

// ---------------------------------------------------------------- kernel --

template <typename T, int kDim, int kMT, int kMW>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attend_kernel(const Params p) {
    using L = Layout<kDim, kMT, kMW>;
    constexpr int kNB = L::kKeys / 16;      // blocks of 16 keys in a group's step
    constexpr int kDT = kDim / 8;           // 8-channel tiles of O
    constexpr int kChunks = kDim / 8;       // 16-byte chunks of a cache row
    constexpr int kPerInstr = 32 / kChunks; // cache rows one cp.async of a warp covers
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint32_t there[kStages][kWarps];  // keys of each warp's 16 that are in the cache
    unsigned char *ring = smem;
    unsigned char *shared_area = smem + kStages * L::kStage;
    float *stat_m = reinterpret_cast<float *>(shared_area + L::kShared);
    float *stat_l = stat_m + L::kGroups * L::kRows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = warp / kMW, mwarp = warp % kMW;
    const int qr = lane >> 2, qc = lane & 3;  // row and column pair inside a fragment

    kda_cache::grid_dependents_launch();
    kda_cache::grid_dependency_wait();
    const Run run = plan(p);
    const int cta = blockIdx.x;
    if (cta >= run.ctas) {
        if (tid == 0) p.cuts[cta].pieces = 0;
        return;
    }

    // cursor of the tile to compute and of the tile to load
    Cursor at;
    at.head = 0;
    at.set_row(p, run.row);
    {
        const long long in_row = run.begin - run.before_row;
        const int n = at.end - at.first;
        at.head = (int)(in_row / n);
        at.tile = at.first + (int)(in_row % n);
    }
    Cursor ld = at;
    long long left = run.end - run.begin;       // tiles to compute
    long long to_load = left;

    if (tid == 0) {  // the join's work item: a segment first cut where this run begins
        Cut cut = {};
        const int n = at.end - at.first;
        const long long s = run.before_row + (long long)at.head * n;
        if (s < run.begin) {
            const int i0 = cta_of(run.units, run.ctas, s);
            if (i0 == cta - 1) {
                cut.pieces = cta_of(run.units, run.ctas, s + n - 1) - i0 + 1;
                cut.first_slot = 2 * i0 + (run_begin(run.units, run.ctas, i0) < s ? 1 : 0);
                cut.first_token = at.row.first;
                cut.tokens = at.row.tokens;
                cut.head = at.head;
            }
        }
        p.cuts[cta] = cut;
    }

    // Load one tile into ring slot `slot`: this warp's 16 keys and values.
    // Lane l looks up key l mod 16; the address goes to the loading lanes by
    // shuffle.  Keys past the row's end and in null blocks become zeros.
    auto load_tile = [&](int slot) {
        if (to_load > 0) {
            const int pos = ld.tile * kTile + 16 * warp + (lane & 15);
            int block = 0;
            long long off = 0;
            if (pos < ld.row.computed + ld.row.tokens) {
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

    for (int i = 0; i < kStages - 1; ++i) load_tile(i);

    int slot = 0;            // ring slot of the tile to compute
    int piece_first = 1;     // whether the segment is this run's first
    while (left > 0) {
        // ------------------------------------------------- a segment's piece
        const int tiles = (int)min(left, (long long)(at.end - at.tile));
        const bool whole = at.tile == at.first && tiles == at.end - at.first;
        const int partial_slot = 2 * cta + (piece_first ? 0 : 1);
        const int rows = at.row.tokens * p.group;
        // queries to shared memory (rows past the last one: zeros)
        for (int i = tid; i < L::kRows * kChunks; i += kThreads) {
            const int r = i / kChunks, c = i % kChunks;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const int t = r / p.group, h = at.head * p.group + r % p.group;
                x = *reinterpret_cast<const uint4 *>(
                    reinterpret_cast<const T *>(p.q) + (at.row.first + t) * p.stride_q +
                    (long long)h * kDim + c * 8);
            }
            *reinterpret_cast<uint4 *>(shared_area + swizzled<kDim>(r, c)) = x;
        }
        __syncthreads();
        const uint32_t q_addr = kda::smem_u32(shared_area);
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
                hi[a][h] = at.row.computed + min(r / p.group, at.row.tokens - 1);
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
            load_tile(slot == 0 ? kStages - 1 : slot - 1);
            cp_async_wait<kStages - 1>();
            group_sync<kMW>(group);
            const uint32_t k_addr = kda::smem_u32(ring + slot * L::kStage) +
                                    group * L::kKeys * L::kRowBytes;
            const uint32_t v_addr = k_addr + L::kHalfTile;
            const int key0 = (at.tile + done) * kTile + group * L::kKeys;
            unsigned long long seen = 0;  // keys of the step that are in the cache
#pragma unroll
            for (int w = 0; w < kMW; ++w)
                seen |= (unsigned long long)there[slot][group * kMW + w] << (16 * w);

            float s[kMT][2 * kNB][4];
#pragma unroll
            for (int a = 0; a < kMT; ++a)
#pragma unroll
                for (int n = 0; n < 2 * kNB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[a][n][e] = 0.0f;
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
#pragma unroll
            for (int a = 0; a < kMT; ++a)
#pragma unroll
                for (int n = 0; n < 2 * kNB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[a][n][e] *= p.scale_log2;

            // a step that some row does not see whole: at the window's own
            // keys, at a sliding window's start, at null blocks
            constexpr unsigned long long kAll = kNB == 4 ? ~0ull : (1ull << (16 * kNB % 64)) - 1;
            const bool edge =
                key0 + L::kKeys - 1 > at.row.computed || seen != kAll ||
                (p.left_window > 0 && key0 <= at.row.computed + at.row.tokens - 1 - p.left_window);
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
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 2));
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
                    const float base = m[a][h] == -INFINITY ? 0.0f : m[a][h];
#pragma unroll
                    for (int n = 0; n < 2 * kNB; ++n) {
                        s[a][n][2 * h] = exp2_fast(s[a][n][2 * h] - base);
                        s[a][n][2 * h + 1] = exp2_fast(s[a][n][2 * h + 1] - base);
                        l[a][h] += s[a][n][2 * h] + s[a][n][2 * h + 1];
                    }
                }

            // A value that is not finite must not reach the rows that do not
            // see its key (0 * inf is NaN in the product): where rows see
            // different keys, such values are added by hand to the rows that
            // do and zeroed for the product.
            if (edge) {
                unsigned long long odd = 0;
                for (int i = lane; i < L::kKeys * kChunks; i += 32) {
                    uint4 x;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                 : "r"(v_addr + swizzled<kDim>(i / kChunks, i % kChunks)));
                    if (not_finite(x.x, T()) || not_finite(x.y, T()) || not_finite(x.z, T()) ||
                        not_finite(x.w, T()))
                        odd |= 1ull << (i / kChunks);
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
                                    if (see0) {
                                        o[a][d][0] = fmaf(p0, x.x, o[a][d][0]);
                                        o[a][d][1] = fmaf(p0, x.y, o[a][d][1]);
                                    }
                                    if (see1) {
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
            group_sync<kMW>(group);  // the slot may be loaded again
            slot = slot + 1 == kStages ? 0 : slot + 1;
        }

        // ------------------------------------------- the groups' sums joined
#pragma unroll
        for (int a = 0; a < kMT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[a][h] += __shfl_xor_sync(kFull, l[a][h], 1);
                l[a][h] += __shfl_xor_sync(kFull, l[a][h], 2);
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
            __syncthreads();
#pragma unroll
            for (int a = 0; a < kMT; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (mwarp * kMT + a) * 16 + qr + 8 * h;
                    float all = -INFINITY, sum = 0.0f;
#pragma unroll
                    for (int g = 0; g < L::kGroups; ++g)
                        all = fmaxf(all, stat_m[g * L::kRows + r]);
                    const float base = all == -INFINITY ? 0.0f : all;
#pragma unroll
                    for (int g = 0; g < L::kGroups; ++g)
                        sum += stat_l[g * L::kRows + r] *
                               exp2_fast(stat_m[g * L::kRows + r] - base);
                    const float f = exp2_fast(m[a][h] - base);
                    m[a][h] = all;
                    l[a][h] = sum;
#pragma unroll
                    for (int d = 0; d < kDT; ++d) {
                        o[a][d][2 * h] *= f;
                        o[a][d][2 * h + 1] *= f;
                    }
                }
            // group after group adds its half of the channels; the last
            // group keeps the sum
            float2 *sum = reinterpret_cast<float2 *>(shared_area);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int g = 0; g < L::kGroups; ++g) {
                    if (group == g) {
#pragma unroll
                        for (int a = 0; a < kMT; ++a)
#pragma unroll
                            for (int d = 0; d < kDT / 2; ++d)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float *x = &o[a][half * (kDT / 2) + d][2 * h];
                                    float2 *y = sum + ((((mwarp * kMT + a) * (kDT / 2) + d) * 2 + h) *
                                                           32 +
                                                       lane);
                                    if (g > 0) {
                                        const float2 z = *y;
                                        x[0] += z.x;
                                        x[1] += z.y;
                                    }
                                    if (g + 1 < L::kGroups) *y = make_float2(x[0], x[1]);
                                }
                    }
                    __syncthreads();
                }
        } else {
            __syncthreads();  // every warp is done with the queries
        }

        // ---------------------------------------------------------- results
        if (group == L::kGroups - 1) {
#pragma unroll
            for (int a = 0; a < kMT; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (mwarp * kMT + a) * 16 + qr + 8 * h;
                    if (r >= rows) continue;
                    if (whole) {
                        const long long row = (long long)(at.row.first + r / p.group) * p.q_heads +
                                              at.head * p.group + r % p.group;
                        const float f = l[a][h] == 0.0f ? 0.0f : 1.0f / l[a][h];
                        uint32_t *dst = reinterpret_cast<uint32_t *>(p.out) + row * (kDim / 2) + qc;
#pragma unroll
                        for (int d = 0; d < kDT; ++d)
                            dst[4 * d] = pack(o[a][d][2 * h] * f, o[a][d][2 * h + 1] * f, T());
                        if (p.lse != nullptr && qc == 0)
                            p.lse[row] = (m[a][h] + log2f(l[a][h])) * kLn2;
                    } else {
                        float *part =
                            p.partials + (long long)partial_slot * p.most_rows * (kDim + 2);
                        float2 *dst = reinterpret_cast<float2 *>(part + r * kDim) + qc;
#pragma unroll
                        for (int d = 0; d < kDT; ++d)
                            dst[4 * d] = make_float2(o[a][d][2 * h], o[a][d][2 * h + 1]);
                        if (qc == 0) {
                            part[p.most_rows * kDim + r] = m[a][h];
                            part[p.most_rows * (kDim + 1) + r] = l[a][h];
                        }
                    }
                }
        }
        left -= tiles;
        piece_first = 0;
        if (left > 0) at.next_segment(p);
    }
    cp_async_wait<0>();
}

// Joins the pieces of the segments that runs cut: block (i, y) takes the
// segment first cut at the start of CTA i's run and its query rows y, y +
// gridDim.y, ...; a warp adds every fourth piece, then the warps' sums are
// added in order.
template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads) join_kernel(const Params p) {
    constexpr int kVec = kDim / 32;
    __shared__ float sum[kWarps][kDim];
    __shared__ float sum_l[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    kda_cache::grid_dependents_launch();
    kda_cache::grid_dependency_wait();
    const int cta = blockIdx.x + 1;
    const Cut cut = p.cuts[cta];
    if (cut.pieces == 0) return;
    const int rows = cut.tokens * p.group;
    const long long slot_size = (long long)p.most_rows * (kDim + 2);
    const float *first = p.partials + cut.first_slot * slot_size;
    const float *others = p.partials + 2 * (cta - 1) * slot_size;  // piece i > 0 at 2 i slots on
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float m = -INFINITY;
        for (int i = lane; i < cut.pieces; i += 32) {
            const float *part = i == 0 ? first : others + 2 * i * slot_size;
            m = fmaxf(m, __ldcg(part + p.most_rows * kDim + r));
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, x));
        const float base = m == -INFINITY ? 0.0f : m;
        float l = 0.0f, o[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) o[e] = 0.0f;
#pragma unroll 4
        for (int i = warp; i < cut.pieces; i += kWarps) {
            const float *part = i == 0 ? first : others + 2 * i * slot_size;
            const float f = exp2_fast(__ldcg(part + p.most_rows * kDim + r) - base);
            l = fmaf(f, __ldcg(part + p.most_rows * (kDim + 1) + r), l);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                o[e] = fmaf(f, __ldcg(part + r * kDim + lane * kVec + e), o[e]);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum[warp][lane * kVec + e] = o[e];
        if (lane == 0) sum_l[warp] = l;
        __syncthreads();
        float total = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += sum_l[w];
        const float f = total == 0.0f ? 0.0f : 1.0f / total;
        const long long row = (long long)(cut.first_token + r / p.group) * p.q_heads +
                              cut.head * p.group + r % p.group;
        if (tid < kDim / 2) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                x += sum[w][2 * tid];
                y += sum[w][2 * tid + 1];
            }
            reinterpret_cast<uint32_t *>(p.out)[row * (kDim / 2) + tid] = pack(x * f, y * f, T());
        }
        if (tid == 0 && p.lse != nullptr) p.lse[row] = (m + log2f(total)) * kLn2;
        __syncthreads();
    }
}

// ------------------------------------------------------------------- host --

template <typename T, int kDim, int kMT, int kMW>
kda_status launch_attend(const Params &p, int grid, void *stream) {
    using L = Layout<kDim, kMT, kMW>;
    void (*kernel)(const Params) = attend_kernel<T, kDim, kMT, kMW>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
        cudaSuccess)
        return KDA_ERR_CUDA;
    kda_status st = kda_cache::launch(kernel, dim3(grid), dim3(kThreads), L::kBytes, 1, stream, p);
    if (st != KDA_OK || grid == 1) return st;
    void (*join)(const Params) = join_kernel<T, kDim>;
    return kda_cache::launch(join, dim3(grid - 1, min(p.most_rows, 16)), dim3(kThreads), 0, 1,
                             stream, p);
}

template <typename T, int kDim>
kda_status launch_rows(const Params &p, int grid, void *stream) {
    if (p.most_rows <= 16) return launch_attend<T, kDim, 1, 1>(p, grid, stream);
    if (p.most_rows <= 32) return launch_attend<T, kDim, 2, 1>(p, grid, stream);
    if (p.most_rows <= 64) return launch_attend<T, kDim, 2, 2>(p, grid, stream);
    return launch_attend<T, kDim, 2, 4>(p, grid, stream);
}

kda_status check_attention(const kda_cache_config *c) {
    kda_status st = kda_cache::check_config(c);
    if (st != KDA_OK) return st;
    if (c->window < 1 || c->left_window < 0) return KDA_ERR_INVALID_ARG;
    if (c->window > KDA_MAX_WINDOW) return KDA_ERR_UNSUPPORTED;
    if (c->window * (c->q_heads / c->kv_heads) > KDA_MAX_QUERY_ROWS) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

size_t partial_bytes(const kda_cache_config *c) {
    return (size_t)2 * kMaxCtas * (size_t)(c->window * (c->q_heads / c->kv_heads)) *
           (size_t)(c->head_dim + 2) * 4u;
}

}  // namespace

extern "C" {

size_t kda_attention_workspace_bytes(const kda_cache_config *cfg, int32_t B) {
    if (check_attention(cfg) != KDA_OK || B < 0) return 0;
    return kMaxCtas * sizeof(Cut) + partial_bytes(cfg);
}

kda_status kda_window_attention(const kda_cache_config *cfg, const void *q, const void *key_cache,
                                const void *value_cache, const int32_t *cu_seqlens, int32_t B,
                                const kda_align *align, void *workspace, size_t workspace_bytes,
                                void *out, float *lse, int32_t *error_word, void *stream) {
    using kda_cache::aligned;
    kda_status st = check_attention(cfg);
    if (st != KDA_OK) return st;
    if (B < 0) return KDA_ERR_INVALID_ARG;
    if (B == 0) return KDA_OK;  // nothing to do; no pointer is inspected
    Params p;
    st = kda_cache::set_rows(cfg, align, cu_seqlens, B, error_word, p.rows);
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
    p.window = cfg->window;
    p.left_window = cfg->left_window;
    p.most_rows = cfg->window * p.group;
    p.scale_log2 = cfg->scale * kLog2e;
    const int grid = kCtasPerSm * sms < kMaxCtas ? kCtasPerSm * sms : kMaxCtas;
    if (cfg->dtype == KDA_DTYPE_BF16)
        return cfg->head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(p, grid, stream)
                                   : launch_rows<__nv_bfloat16, 128>(p, grid, stream);
    return cfg->head_dim == 64 ? launch_rows<__half, 64>(p, grid, stream)
                               : launch_rows<__half, 128>(p, grid, stream);
}

}  // extern "C"
