// Attention weight of cached keys, summed over the queries of the newest tokens: weight_j += sum_i exp(s_ij - lse_i).
//
// The lse is known, so that the softmax needs no pass of its own, and V is not read: D + 4 bytes per key and
// KV head, 2 D flop and an exponential per query row on it.  From some 100 rows on the exponentials and the
// products bound it, below that, in theory, HBM.  Calls of up to 32 rows a KV head are bsattn_weigh_step.cu's.
//
// Keys lie on the tensor cores' 128 rows and queries on their columns: S^T = K' Q^T with K' = bf16(code), exact,
// and Q as it is.  A thread has one key, so that the sum over the queries stays in its registers: weight = sum_r
// 2^(S_r c - lse_r log2(e)), c = ks softmax_scale log2(e).  The sum is fp32 within a block of 128 rows, and
// compensated from block to block: thousands of rows cost no more accuracy than one block does.
//
// Measured: 2048 tokens on 33792 keys, 8 heads, G = 4, int8, D = 128: 469 us, 1.17 PFLOP/s, where the products would take
// 281 and the exponentials 232; 64 tokens on 61440 keys, 24 heads, e4m3: 91 us, 2.2 TB/s.  There neither more units
// on their way (3 instead of 2: 93 us) nor query blocks that stay from unit to unit (102, where it was 102) made a
// difference; copies of a page instead of 16 keys did (95, 90), and fewer instructions for widening (102, 95).
//
// A unit is 256 keys of a (sequence, KV head): two tiles, one for each of two groups of 128 threads, whose blocks of
// query rows are loaded once for both.  Units are handed out along a line on which each counts its blocks and
// kUnitCost; every CTA numbers the line for itself (lengths are on the device).  A unit is not split: its weights
// have one writer, and their sums one order.
//
// Roles (896 threads, one CTA per SM, all of TMEM):
//   warp 0        issues the MMAs
//   warp 1        owns the TMEM allocation; finds the CTA's units
//   warp 2        fetches the codes of keys: bulk copies into raw tiles
//   warp 3        query blocks (TMA) and their lse
//   warps 4-7, 8-11, 12-15, 16-19   first halves of group 0 and 1, second halves: sums
//   warps 20-27   widen the codes (128-byte swizzle)
// Of few rows (kFew) a group has one half, and 16 warps widen.
// TMEM: S^T of group g and buffer i: [256 g + 128 i, 256 g + 128 i + 128).
#include "kv_codes.cuh"
#include "prefill_plan.cuh"

namespace bsattn {

namespace {

constexpr int kThreads = 896;
constexpr uint32_t kTmemCols = 512;
// 72 registers per thread at launch: 128 * 72 + 4 * 128 * 80 + 2 * 128 * 56 = 64512 = 896 * 72.
constexpr int kLaunchRegs = 72;
constexpr uint32_t kCtrlRegs = 72, kGroupRegs = 80, kWidenRegs = 56;
static_assert(128 * kCtrlRegs + 512 * kGroupRegs + 256 * kWidenRegs <= (uint32_t)kThreads * kLaunchRegs &&
                  128 * kCtrlRegs + 256 * kGroupRegs + 512 * kWidenRegs <= (uint32_t)kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr int kSums = 4;                    // units whose half sums wait to be joined
constexpr uint32_t kSub = kTile * 64 * 2;   // 128 rows x 64 bf16: one 128-byte swizzle span
constexpr int kUnitKeys = 2 * kTile;
constexpr int kUnitCost = 2;                // blocks that a unit's own work is worth (1, 2 and 4 measured alike)
constexpr int kSeqChunk = 2048;             // sequences whose places fit shared memory at a time
constexpr int kUnits = 2;                   // units found ahead
// Mean query rows of a KV head up to which bsattn_weigh_step.cu is the faster one.  32 sequences of 4096 keys, 8 heads,
// D = 128, us a call there and here: 4 rows 44, 80, 16 rows 49, 80, 32 rows 60, 80; D = 64: 33, 62, 40, 62, 50, 62.
// The mean says nothing of a chunk among single tokens: 127 tokens and a chunk of 400, 4096 keys each, 8 heads x 4 (mean
// 16 rows), take 691 us there, 396 here, and 149 as two calls, each with its own kernel.
constexpr int kStepRows = 32;

// Rows of a query block: tokens of all of a KV head's query heads.
struct Blocks {
    int tokens;              // of a block
    int cols;                // columns of the products: rows, up to a multiple of 32
};

struct Unit {
    int32_t b, h;            // b < 0: no more
    int32_t key0, n;         // first key, keys of the sequence
    int32_t first, m;        // the sequence's queries
    int32_t q0, q1;          // blocks that some of the keys are met by
};

// kFew: blocks of up to 64 rows.  Codes and their widening are what the kernel waits for: two units' codes on their
// way, and the next unit's first tile widened ahead.  Else more blocks of queries are, and the widened tiles are the two
// of a unit alone.  16 sequences of 4096 keys, 8 heads, 64 rows, us a call with this and without: D = 128, e4m3 44, 56;
// D = 64, int8 35, 48.
template <int D, bool kFew>
struct Cfg {
    static constexpr int kTiles = kFew ? 3 : 2, kBlocks = kFew ? 2 : 3, kRaws = kFew ? (D == 128 ? 2 : 4) : 1;
    static constexpr int kHalves = kFew ? 1 : 2, kGroupWarps = 8 * kHalves, kWidenWarps = 24 - kGroupWarps;
    static constexpr uint32_t kTileBytes = kTile * D * 2, kRawBytes = kTile * D;
    static constexpr uint32_t kBlockBytes = kFew ? kTileBytes / 2 : kTileBytes;
    static constexpr uint32_t kBlockSub = kFew ? kSub / 2 : kSub;    // 64 columns of a block
    static constexpr uint32_t kQ = 0, kK = kQ + kBlocks * kBlockBytes;
    static constexpr uint32_t kRaw = kK + kTiles * kTileBytes;       // [raws][2 groups]
    static constexpr uint32_t kScale = kRaw + kRaws * 2 * kRawBytes; // key scales of the raw tiles
    static constexpr uint32_t kLse = kScale + kRaws * 1024;          // -lse log2(e) of the blocks' rows
    static constexpr uint32_t kRow = kLse + kBlocks * 512;           // cache rows of the raw tiles' 16-key groups, -1: none
    static constexpr uint32_t kOdd = kRow + kRaws * 64;              // keys that have a NaN code, of kSums units
    static constexpr uint32_t kSum = kOdd + kSums * 32;                  // sums of the groups' second halves
    static constexpr uint32_t kUnit = kSum + kSums * 1024;
    static constexpr uint32_t kBar = kUnit + kUnits * (uint32_t)sizeof(Unit);
    // K' tiles full and empty, query blocks full and empty, S full and empty (2 group + buffer), raw units full and
    // empty, half sums there (2 of a unit: per group), units full and empty
    static constexpr int bKF = 0, bKE = bKF + kTiles, bQF = bKE + kTiles, bQE = bQF + kBlocks, bSF = bQE + kBlocks, bSE = bSF + 4,
                         bRF = bSE + 4, bRE = bRF + kRaws, bHF = bRE + kRaws, bUF = bHF + 2 * kSums, bUE = bUF + kUnits,
                         bDrain = bUE + kUnits, kNumBars = bDrain + 1;
    static constexpr uint32_t kMisc = kBar + kNumBars * 8;           // [0] tmem base, [1] abort
    static constexpr uint32_t kAlloc = kMisc + 8;
    static_assert(kUnits < kSums, "sums and odd keys of the units under way");
    static_assert(kAlloc <= 227u * 1024u, "shared memory");
};

// Where the CTA's piece of the line begins.
struct Start {
    int32_t b, h, u, pieces;
    long long begin, line;
    Chunk c;                 // of sequence b
};

// Blocks that meet a key of j0 .. j1 (below n): a range.
struct Range {
    int q0, q1;
};

__device__ __forceinline__ Range blocks_of(const ChunkParams &p, const Blocks &w, const Chunk &c, int j0, int j1) {
    const int nb = (c.m + w.tokens - 1) / w.tokens, pos = c.n - c.m;
    Range r = {0, nb};
    if (p.kind == BSATTN_MASK_CAUSAL || p.kind == BSATTN_MASK_SLIDING_WINDOW || (p.kind == BSATTN_MASK_PREFIX && j0 >= p.prefix_len))
        r.q0 = min(max(j0 - pos, 0) / w.tokens, nb);
    if (p.kind == BSATTN_MASK_SLIDING_WINDOW && j0 >= p.sink_tokens) {
        const long long t = (long long)j1 + p.window_left - pos;     // tokens below t meet the last key
        r.q1 = t <= 0 ? 0 : (int)min((t + w.tokens - 1) / w.tokens, (long long)nb);
    }
    r.q1 = max(r.q1, r.q0);
    return r;
}

__device__ __forceinline__ Range unit_blocks(const ChunkParams &p, const Blocks &w, const Chunk &c, int u) {
    return blocks_of(p, w, c, u * kUnitKeys, min(u * kUnitKeys, c.n - kUnitKeys) + kUnitKeys - 1);   // below 2^31
}

__device__ __forceinline__ int unit_count(const Chunk &c) { return c.m > 0 && c.n > 0 ? (c.n - 1) / kUnitKeys + 1 : 0; }

// Places of a unit in the line.  Of few blocks each counts, whether the unit's keys meet it or not.
__device__ __forceinline__ bool plain_places(const Blocks &w, const Chunk &c) { return c.m <= 2 * w.tokens; }

__device__ __forceinline__ int unit_places(const ChunkParams &p, const Blocks &w, const Chunk &c, int u) {
    if (plain_places(w, c)) return kUnitCost + (c.m + w.tokens - 1) / w.tokens;
    const Range r = unit_blocks(p, w, c, u);
    return kUnitCost + r.q1 - r.q0;
}

// Places of one head's units of a sequence, by a warp: a lane counts every 32nd unit.
__device__ __forceinline__ long long pass_places(const ChunkParams &p, const Blocks &w, const Chunk &c, int lane) {
    if (plain_places(w, c)) return (long long)unit_count(c) * unit_places(p, w, c, 0);
    long long sum = 0;
    for (int u = lane; u < unit_count(c); u += 32) sum += unit_places(p, w, c, u);
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
}

// The first unit of a sequence (st.c) that begins at or behind place `from`; the sequence begins at `begin`, each head
// has `places`.  A whole warp; fills h, u, begin.
__device__ __forceinline__ void first_unit(const ChunkParams &p, const Blocks &w, long long from, long long begin, long long places,
                                           int lane, Start &st) {
    const Chunk &c = st.c;
    st.h = (int)line_div(from - begin, places);
    st.begin = begin + st.h * places;
    st.u = 0;
    if (plain_places(w, c)) {
        const int x = unit_places(p, w, c, 0);
        st.u = min((int)line_div(from - st.begin + x - 1, x), unit_count(c));
        st.begin += (long long)st.u * x;
        return;
    }
    while (st.u < unit_count(c)) {
        const long long x = st.u + lane < unit_count(c) ? unit_places(p, w, c, st.u + lane) : 0;
        long long s = x;
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, st.u + lane < unit_count(c) && st.begin + s - x >= from);
        if (hit) {
            const int k = __ffs(hit) - 1;
            st.begin += __shfl_sync(0xffffffffu, s - x, k);
            st.u += k;
            return;
        }
        st.begin += __shfl_sync(0xffffffffu, s, 31);
        st.u = min(st.u + 32, unit_count(c));
    }
}

// Numbers the line and finds where the CTA's piece begins; all threads.
__device__ __forceinline__ void find_piece(const ChunkParams &p, const Blocks &w, Start *st, long long *pass) {
    const int tid = (int)threadIdx.x, lane = tid % 32, warp = tid / 32;
    long long *warps = pass + kSeqChunk;
    // of a chunk of sequences: each one's places before it (of all heads), and those of all
    auto number = [&](int b0, bool check, long long before) -> long long {
        const int n = min(kSeqChunk, p.B - b0);
        __syncthreads();
        // a thread per sequence; a warp for those whose units differ
        for (int i0 = warp * 32; i0 < n; i0 += kThreads) {
            Chunk c = {};
            if (i0 + lane < n) c = chunk_of(p, b0 + i0 + lane, check);
            const bool plain = plain_places(w, c);
            if (i0 + lane < n && plain) pass[i0 + lane] = (long long)unit_count(c) * unit_places(p, w, c, 0) * p.c.H;
            for (uint32_t left = __ballot_sync(0xffffffffu, !plain); left; left &= left - 1) {
                const int x = __ffs(left) - 1;
                Chunk y;
                y.first = __shfl_sync(0xffffffffu, c.first, x);
                y.m = __shfl_sync(0xffffffffu, c.m, x);
                y.n = __shfl_sync(0xffffffffu, c.n, x);
                const long long places = pass_places(p, w, y, lane);
                if (lane == 0) pass[i0 + x] = places * p.c.H;
            }
        }
        __syncthreads();
        // a thread sums consecutive sequences
        const int per = (n + kThreads - 1) / kThreads, lo = min(tid * per, n), hi = min(lo + per, n);
        long long s = 0;
        for (int i = lo; i < hi; ++i) s += pass[i];
        const long long own = s;
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) warps[warp] = s;
        __syncthreads();
        long long all = 0, at = before + s - own;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) at += warps[i];
            all += warps[i];
        }
        for (int i = lo; i < hi; ++i) {
            const long long x = pass[i];
            pass[i] = at;
            at += x;
        }
        __syncthreads();
        return before + all;
    };
    long long line = 0;
    for (int b0 = 0; b0 < p.B; b0 += kSeqChunk) line = number(b0, blockIdx.x == 0, line);
    const int pieces = (int)max(1ll, min((long long)gridDim.x, line_div(line, kUnitCost))), piece = (int)blockIdx.x;
    if (tid == 0) st->b = p.B, st->pieces = pieces, st->line = line;
    if (piece >= pieces || line == 0) return;
    const long long from = line_div(line * piece, pieces);
    long long at = 0;
    for (int b0 = 0; b0 < p.B; b0 += kSeqChunk) {
        const long long end = p.B > kSeqChunk ? number(b0, false, at) : line;
        const int n = min(kSeqChunk, p.B - b0);
        if (from >= at && from < end) {
            // the last sequence that begins at or before `from`
            int i = 0, hi = n - 1;
            while (i < hi) {
                const int mid = (i + hi + 1) / 2;
                if (pass[mid] <= from) i = mid;
                else hi = mid - 1;
            }
            if (warp == 0) {
                const Chunk c = chunk_of(p, b0 + i, false);
                const long long places = pass_places(p, w, c, lane);
                if (places > 0) {
                    Start x = {};
                    x.c = c;
                    first_unit(p, w, from, pass[i], places, lane, x);
                    if (lane == 0) st->b = b0 + i, st->h = x.h, st->u = x.u, st->begin = x.begin, st->c = c;
                }
            }
        }
        at = end;
    }
}

// The same by one warp, without a barrier, of up to 32 kLaneSeqs sequences.
constexpr int kLaneSeqs = 4;

__device__ __forceinline__ Start find_piece_warp(const ChunkParams &p, const Blocks &w, int lane) {
    Chunk c[kLaneSeqs];
    long long pass[kLaneSeqs], before[kLaneSeqs], line = 0;
#pragma unroll
    for (int k = 0; k < kLaneSeqs; ++k) {
        c[k] = Chunk{};
        if (32 * k + lane < p.B) c[k] = chunk_of(p, 32 * k + lane, blockIdx.x == 0);
    }
#pragma unroll
    for (int k = 0; k < kLaneSeqs; ++k) {
        if (32 * k >= p.B) break;
        const bool plain = plain_places(w, c[k]);
        pass[k] = plain ? (long long)unit_count(c[k]) * unit_places(p, w, c[k], 0) : 0;
        for (uint32_t left = __ballot_sync(0xffffffffu, !plain); left; left &= left - 1) {
            const int x = __ffs(left) - 1;
            Chunk y;
            y.first = __shfl_sync(0xffffffffu, c[k].first, x);
            y.m = __shfl_sync(0xffffffffu, c[k].m, x);
            y.n = __shfl_sync(0xffffffffu, c[k].n, x);
            const long long places = pass_places(p, w, y, lane);
            if (lane == x) pass[k] = places;
        }
        long long s = pass[k] * p.c.H;
        const long long own = s;
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        before[k] = line + s - own;
        line += __shfl_sync(0xffffffffu, s, 31);
    }
    Start st = {};
    st.line = line;
    st.pieces = (int)max(1ll, min((long long)gridDim.x, line_div(line, kUnitCost)));
    st.b = p.B;
    if ((int)blockIdx.x >= st.pieces) return st;
    const long long from = line_div(line * (int)blockIdx.x, st.pieces);
#pragma unroll
    for (int k = 0; k < kLaneSeqs; ++k) {
        if (32 * k >= p.B) break;
        const uint32_t hit = __ballot_sync(0xffffffffu, from >= before[k] && from < before[k] + pass[k] * p.c.H);
        if (!hit) continue;
        const int x = __ffs(hit) - 1;
        st.b = 32 * k + x;
        st.c.first = __shfl_sync(0xffffffffu, c[k].first, x);
        st.c.m = __shfl_sync(0xffffffffu, c[k].m, x);
        st.c.n = __shfl_sync(0xffffffffu, c[k].n, x);
        first_unit(p, w, from, __shfl_sync(0xffffffffu, before[k], x), __shfl_sync(0xffffffffu, pass[k], x), lane, st);
    }
    return st;
}

template <class C>
__device__ __forceinline__ bool next_unit(const Waiter &wait, const uint8_t *smem, uint32_t &count, Unit &x) {
    const int slot = (int)(count % kUnits);
    if (!__all_sync(0xffffffffu, wait(C::bUF + slot, count / kUnits))) return false;
    x = reinterpret_cast<const Unit *>(smem + C::kUnit)[slot];
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(wait.bar(C::bUE + slot));
    ++count;
    return x.b >= 0;
}

// Finds the units that begin in the CTA's piece.
template <class C>
__device__ __forceinline__ void unit_role(const ChunkParams &p, const Blocks &w, const Waiter &wait, uint8_t *smem, const Start &st) {
    uint32_t count = 0;
    auto emit = [&](const Unit &x) -> bool {
        const int slot = (int)(count % kUnits);
        if (!wait(C::bUE + slot, (count / kUnits) ^ 1u)) return false;
        reinterpret_cast<Unit *>(smem + C::kUnit)[slot] = x;
        mbar_arrive(wait.bar(C::bUF + slot));
        ++count;
        return true;
    };
    int b = st.b, h = st.h, u = st.u;
    if (b < p.B) {
        const long long to = line_div(st.line * ((long long)blockIdx.x + 1), st.pieces);
        long long begin = st.begin;
        Chunk c = st.c;
        int units = unit_count(c);
        while (begin < to) {
            if (u >= units) {
                u = 0;
                if (units == 0 || ++h >= p.c.H) {
                    h = 0;
                    if (++b >= p.B) break;
                    c = chunk_of(p, b, false);
                    units = unit_count(c);
                }
                continue;
            }
            const Range r = unit_blocks(p, w, c, u);
            // where weights are added to, keys that no query meets need nothing
            if (r.q1 > r.q0 || !p.accumulate) {
                Unit x;
                x.b = b, x.h = h, x.key0 = u * kUnitKeys, x.n = c.n;
                x.first = c.first, x.m = c.m, x.q0 = r.q0, x.q1 = r.q1;
                if (!emit(x)) return;
            }
            begin += unit_places(p, w, c, u);
            ++u;
        }
    }
    Unit stop = {};
    stop.b = -1;
    emit(stop);
}

// The sum over a block's columns from .. to - 1 once more, where it was not a number: a query whose lse is -inf gives no
// weight even so.  A function of its own, called on a vote of the warp (64 tokens on 61376 keys, 24 heads: 90.3 -> 90.9 us,
// 2048 on 31744: 461 -> 468): the loop that sums has no register to spare, a test there makes these 104 and 538, and this
// code written into it 94 and 468.
__device__ __noinline__ float sum_again(uint32_t at, const float *nl, float c, int from, int to, int cols) {
    float sum = 0.f;
#pragma unroll 1
    for (int col = 0; col < cols; col += 4) {
        uint32_t v[4];
        tmem_ld4(at + (uint32_t)col, v);
        tmem_wait_ld();
        reg_fence(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float n = nl[col + i];
            if (n != -INFINITY && col + i >= from && col + i < to) sum += ex2_approx(fmaf(__uint_as_float(v[i]), c, n));
        }
    }
    return sum;
}

// One half of a group: 128 threads, a key each, every other block (two buffers of S: one of either half's).  Four
// warps a scheduler hide the exponentials' and loads' latencies that two do not.
template <int D, bool kFew>
__device__ __forceinline__ void group_role(const ChunkParams &p, const Blocks &w, const Waiter &wait, uint32_t tmem, int g, int half,
                                           uint32_t warp, uint32_t lane, uint8_t *smem) {
    using C = Cfg<D, kFew>;
    const uint32_t quarter = warp & 3u;
    const int key = (int)(quarter * 32 + lane) + g * kTile;
    const uint32_t s_addr = tmem + ((quarter * 32u) << 16) + (uint32_t)g * 256u;
    uint32_t units = 0, ut = 0, it = 0;          // units, those with blocks, blocks so far
    Unit x;
    while (next_unit<C>(wait, smem, units, x)) {
        const int j = x.key0 + key;
        int row = -1;
        float c = 0.f;
        // tokens that meet the key: lo <= t < hi
        const int pos = x.n - x.m;
        int lo = 0, hi = 0;
        bool ok = true;
        if (x.q1 > x.q0) {
            const uint32_t raw = ut % C::kRaws;
            ok = __all_sync(0xffffffffu, wait(C::bRF + (int)raw, ut / C::kRaws));
            if (!ok) break;
            row = reinterpret_cast<const int *>(smem + C::kRow + raw * 64u)[key >> 4];
            row = j < x.n && row >= 0 ? row + (key & 15) : -1;
            c = reinterpret_cast<const float *>(smem + C::kScale + raw * 1024u)[key] * p.scale_log2;
            __syncwarp();
            if (lane == 0) mbar_arrive(wait.bar(C::bRE + (int)raw));
        } else if (j < x.n) {
            row = (int)cache_row(p.c, p.table + (long long)x.b * p.table_stride, x.h, j);
        }
        if (row >= 0) {
            hi = x.m;
            if (p.kind == BSATTN_MASK_CAUSAL || p.kind == BSATTN_MASK_SLIDING_WINDOW || (p.kind == BSATTN_MASK_PREFIX && j >= p.prefix_len))
                lo = max(j - pos, 0);
            if (p.kind == BSATTN_MASK_SLIDING_WINDOW && j >= p.sink_tokens)
                hi = (int)min(max((long long)j + p.window_left - pos, 0ll), (long long)x.m);
        }
        float sum = 0.f, lost = 0.f;             // compensated
        bool first = true;
        for (int q = x.q0; q < x.q1; ++q, ++it) {
            const uint32_t buf = it & 1u, blk = it % C::kBlocks;
            if (C::kHalves == 2 && (int)buf != half) continue;
            ok = __all_sync(0xffffffffu, wait(C::bSF + 2 * g + (int)buf, it >> 1) && wait(C::bQF + (int)blk, it / C::kBlocks));
            if (!ok) break;
            tc_fence_after();
            if (first && ((reinterpret_cast<const uint16_t *>(smem + C::kOdd)[16 * (ut % kSums) + 8 * g + 2 * quarter + (lane >> 4)] >> (lane & 15u)) & 1u))
                c = __uint_as_float(0x7fc00000u);
            first = false;
            // of the block: columns that meet the key; of none behind the sequence's last token
            const int t0 = q * w.tokens, tokens = min(w.tokens, x.m - t0);
            const int from = min(max(lo - t0, 0), tokens) * p.G, to = min(max(hi - t0, 0), tokens) * p.G;
            const bool masked = __any_sync(0xffffffffu, from > 0 || to < w.tokens * p.G);
            const float4 *nl = reinterpret_cast<const float4 *>(smem + C::kLse + blk * 512u);
            const uint32_t at = s_addr + buf * 128u;
            float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
            auto chunk = [&](int cc, uint32_t (&v)[16]) {
                float y[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 n = nl[4 * cc + i];
                    ffma2(y[4 * i], y[4 * i + 1], __uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), c, c, n.x, n.y);
                    ffma2(y[4 * i + 2], y[4 * i + 3], __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]), c, c, n.z, n.w);
                }
                if (masked) {
                    const int f = from - 16 * cc, t = to - 16 * cc;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < f || i >= t) y[i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = ex2_approx(y[i]);
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    fadd2(a0, a1, a0, a1, y[i], y[i + 1]);
                    fadd2(b0, b1, b0, b1, y[i + 2], y[i + 3]);
                }
            };
            uint32_t va[16], vb[16];
            const int chunks = w.cols / 16;     // even
            tmem_ld16(at, va);
#pragma unroll 1
            for (int cc = 0; cc < chunks; cc += 2) {
                tmem_wait_ld();
                reg_fence(va);
                tmem_ld16(at + 16u * (cc + 1), vb);
                chunk(cc, va);
                tmem_wait_ld();
                reg_fence(vb);
                if (cc + 2 < chunks) tmem_ld16(at + 16u * (cc + 2), va);
                chunk(cc + 1, vb);
            }
            float block = (a0 + b0) + (a1 + b1);
            if (__builtin_expect(__any_sync(0xffffffffu, block != block), 0))
                block = sum_again(at, reinterpret_cast<const float *>(nl), c, from, to, w.cols);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(wait.bar(C::bSE + 2 * g + (int)buf));
                mbar_arrive(wait.bar(C::bQE + (int)blk));
            }
            const float add = block - lost, next = sum + add;
            lost = (next - sum) - add;
            sum = next;
        }
        if (!ok) break;
        if (x.q1 > x.q0) {
            if constexpr (C::kHalves == 2) {
                // the second half's sum goes to the first, which has the weight written; it is at most kUnits units
                // ahead
                const uint32_t at = ut % kSums, full = C::bHF + 2 * at + (uint32_t)g;
                float *sums = reinterpret_cast<float *>(smem + C::kSum + at * 1024u);
                if (half == 1) {
                    sums[key] = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(wait.bar((int)full));
                } else {
                    if (!__all_sync(0xffffffffu, wait((int)full, ut / kSums))) break;
                    sum += sums[key];
                }
            }
            ++ut;
        }
        if (row >= 0 && half == 0) {
            if (!p.accumulate) p.weights[row] = sum;
            else if (hi > lo) atomicAdd(p.weights + row, sum);
        }
    }
}

// Fetches the codes and scales of a unit's two tiles: a copy per page or tile, none for keys past the last or on a
// page that is none.
template <int D, bool kFew>
__device__ __forceinline__ void fetch_role(const ChunkParams &p, const Waiter &wait, int lane, uint32_t base, uint8_t *smem) {
    using C = Cfg<D, kFew>;
    uint32_t units = 0, it = 0;
    bool ok = true;
    const int shift = min(p.c.page_shift, 7);    // keys of a copy
    Unit x;
    while (ok && next_unit<C>(wait, smem, units, x)) {
        const int32_t *table = p.table + (long long)x.b * p.table_stride;
        const int key = x.key0 + (lane << shift);
        long long row = -1;
        if (lane < kUnitKeys >> shift && key < x.n) {
            row = cache_row(p.c, table, x.h, key);
            if (row < 0 && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
        }
        if (x.q1 == x.q0) continue;              // no query meets them
        const uint32_t on = __ballot_sync(0xffffffffu, row >= 0), raw = it % C::kRaws;
        if (!(ok = __all_sync(0xffffffffu, wait(C::bRE + (int)raw, (it / C::kRaws) ^ 1u)))) break;
        const int whole = __shfl_sync(0xffffffffu, (int)row, (16 * lane & (kUnitKeys - 1)) >> shift);
        if (lane < 16) reinterpret_cast<int *>(smem + C::kRow + raw * 64u)[lane] = whole < 0 ? -1 : whole + (16 * lane & ((1 << shift) - 1));
        __syncwarp();
        const uint32_t full = wait.bar(C::bRF + (int)raw), lead = row >= 0 ? 1u : 0u;
        mbar_arrive_expect_tx_lead(lane == 0 ? 1u : 0u, full, ((uint32_t)__popc(on) * (D + 4u)) << shift);
        __syncwarp();
        bulk_g2s_lead(lead, base + C::kRaw + raw * 2u * C::kRawBytes + ((uint32_t)lane * D << shift), p.c.k + row * D, (uint32_t)D << shift, full);
        bulk_g2s_lead(lead, base + C::kScale + raw * 1024u + ((uint32_t)lane * 4u << shift), p.c.ks + row, 4u << shift, full);
        ++it;
    }
    // nothing may be on its way into a tile when the CTA ends
    for (uint32_t s = 0; s < (uint32_t)C::kRaws; ++s)
        if (it > s) mbar_wait_drain(wait.bar(C::bRF + (int)s), ((it - 1 - s) / C::kRaws) & 1u);
}

// Widens the codes of tiles, eight warps each, 16 keys a warp.  Lane: 16 codes of a row, two swizzle pieces; D / 16
// lanes to a row.  What no copy has filled is left: such keys are masked.
template <int D, bool kFew, bool kInt8>
__device__ __forceinline__ void widen_role(const Waiter &wait, int widener, int lane, uint8_t *smem) {
    using C = Cfg<D, kFew>;
    constexpr int kRowLanes = D / 16, kAtOnce = 32 / kRowLanes, kSteps = 16 / kAtOnce;
    constexpr uint32_t kEach = 2 * 8 / C::kWidenWarps;    // tiles of a unit that a warp works on
    const int warp = widener & 7, col = lane % kRowLanes, sub_row = lane / kRowLanes;
    // Eight lanes store 128 bytes at a time; where they share a row, half of them begin with their second
    // piece: every bank once.
    const bool swap = D == 128 && col >= 4;
    const int first = 2 * (col & 3) + (swap ? 1 : 0), second = first ^ 1;
    const uint8_t *raw = smem + C::kRaw + (warp * 16 + sub_row) * D + col * 16;
    uint8_t *dst = smem + C::kK + (uint32_t)(col >> 2) * kSub + (uint32_t)(warp * 16 + sub_row) * 128u;
    uint32_t units = 0, it = 0;
    Unit x;
    while (next_unit<C>(wait, smem, units, x)) {
        if (x.q1 == x.q0) continue;
        const uint32_t rs = it % C::kRaws;
        bool ok = wait(C::bRF + (int)rs, it / C::kRaws);
#pragma unroll 1
        for (uint32_t n = 0; n < kEach; ++n) {
            const uint32_t g = kEach == 2 ? n : (uint32_t)widener >> 3, tile = 2 * it + g, stage = tile % C::kTiles;
            const uint8_t *from = raw + (rs * 2u + g) * C::kRawBytes;
            uint4 v[kSteps];
            if (!__all_sync(0xffffffffu, ok)) return;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) v[i] = *reinterpret_cast<const uint4 *>(from + i * kAtOnce * D);
            if (!__all_sync(0xffffffffu, wait(C::bKE + (int)stage, (tile / C::kTiles) ^ 1u))) return;
            uint8_t *to = dst + stage * C::kTileBytes;
            uint32_t odd = 0;                        // rows that have a NaN code
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const uint32_t y[4] = {swap ? v[i].z : v[i].x, swap ? v[i].w : v[i].y, swap ? v[i].x : v[i].z, swap ? v[i].y : v[i].w};
                const int r7 = (i * kAtOnce + sub_row) & 7;
                if (!kInt8) {
                    uint32_t nan = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) nan |= (y[q] & 0x7f7f7f7fu) + 0x01010101u;
                    const uint32_t b = __ballot_sync(0xffffffffu, (nan & 0x80808080u) != 0u);
                    if (b) {
#pragma unroll
                        for (int q = 0; q < kAtOnce; ++q)
                            if ((b >> (q * kRowLanes)) & ((1u << kRowLanes) - 1u)) odd |= 1u << (i * kAtOnce + q);
                    }
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        o[2 * k] = codes_to_bf16x2<kInt8, false>(y[2 * q + k]);
                        o[2 * k + 1] = codes_to_bf16x2<kInt8, true>(y[2 * q + k]);
                    }
                    *reinterpret_cast<uint4 *>(to + i * kAtOnce * 128 + (((q ? second : first) ^ r7) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (lane == 0) reinterpret_cast<uint16_t *>(smem + C::kOdd)[16 * (it % kSums) + 8 * g + warp] = (uint16_t)odd;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(wait.bar(C::bKF + (int)stage));
        }
        if (lane == 0) mbar_arrive(wait.bar(C::bRE + (int)rs));
        ++it;
    }
}

template <int D, bool kFew, bool kInt8>
__global__ void __launch_bounds__(kThreads, 1)
    bsattn_weigh_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ Blocks w, const __grid_constant__ CUtensorMap tq) {
    using C = Cfg<D, kFew>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {  // the swizzle counts from 1024-byte boundaries
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, BSATTN_FLAG_TIMEOUT);
        return;
    }
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    Start *st = reinterpret_cast<Start *>(smem + C::kLse);   // read before the first lse is written
    const uint32_t warp = warp_id(), lane = lane_id();
    Waiter wait;
    wait.bars = base + C::kBar;
    wait.abort = reinterpret_cast<volatile int *>(misc + 1);
    wait.err = p.err;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kTiles; ++s) {
            mbar_init(wait.bar(C::bKF + s), 8);      // one arrival per widening warp
            mbar_init(wait.bar(C::bKE + s), 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(wait.bar(C::bSF + s), 1);
            mbar_init(wait.bar(C::bSE + s), 4);      // one per warp of the group's half
        }
        for (int s = 0; s < C::kBlocks; ++s) {
            mbar_init(wait.bar(C::bQF + s), 1);
            mbar_init(wait.bar(C::bQE + s), 9);      // the products' completion, one per warp that reads the block's lse
        }
        for (int s = 0; s < C::kRaws; ++s) {
            mbar_init(wait.bar(C::bRF + s), 1);
            mbar_init(wait.bar(C::bRE + s), 24);     // widening and group warps
        }
        for (int s = 0; s < 2 * kSums; ++s) mbar_init(wait.bar(C::bHF + s), 4);
        for (int s = 0; s < kUnits; ++s) {
            mbar_init(wait.bar(C::bUF + s), 1);
            mbar_init(wait.bar(C::bUE + s), 27);     // issuing, fetching, query, group and widening warps
        }
        mbar_init(wait.bar(C::bDrain), 1);
        misc[1] = 0;
        fence_barrier_init();
    }
    // rows of a block that no copy fills stay 0
    for (uint32_t i = threadIdx.x; i < C::kBlocks * C::kBlockBytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(smem + C::kQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc(base + C::kMisc, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    grid_launch_dependents();
    grid_dependency_wait();
    const bool alone = p.B <= 32 * kLaneSeqs;    // one warp numbers the line, while the others take their places
    if (!alone) {
        find_piece(p, w, st, reinterpret_cast<long long *>(smem + C::kK));
        __syncthreads();
    }
    if (warp == 0) {
        // ---------------------------------------------------- MMA issuer --
        // The whole warp runs in step; lane 0 issues.
        const uint32_t lead = lane == 0 ? 1u : 0u;
        const uint32_t idesc = idesc_bf16_f32(128, w.cols, false);
        const uint64_t desc_q = smem_desc_sw128(base + C::kQ, 16, 1024);
        const uint64_t desc_k = smem_desc_sw128(base + C::kK, 16, 1024);
        constexpr uint64_t kTileUnits = C::kTileBytes >> 4, kBlockUnits = C::kBlockBytes >> 4;
        uint32_t units = 0, kt = 0, it = 0;      // units; tiles, blocks so far
        bool ok = true;
        auto ready = [&](int b, uint32_t phase) -> bool {
            ok = ok && wait(b, phase);
            return ok;
        };
        Unit x;
        while (ok && next_unit<C>(wait, smem, units, x)) {
            if (x.q1 == x.q0) continue;
            for (int q = x.q0; ok && q < x.q1; ++q, ++it) {
                const uint32_t buf = it & 1u, blk = it % C::kBlocks;
                if (!ready(C::bQF + (int)blk, it / C::kBlocks)) break;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint32_t tile = kt + (uint32_t)g, stage = tile % C::kTiles;
                    if (q == x.q0 && !ready(C::bKF + (int)stage, tile / C::kTiles)) break;
                    if (!ready(C::bSE + 2 * g + (int)buf, (it >> 1) ^ 1u)) break;
                    tc_fence_after();
                    const uint64_t kd = desc_k + (uint64_t)stage * kTileUnits, qd = desc_q + (uint64_t)blk * kBlockUnits;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t in = (uint64_t)((kk & 3) * 2);
                        mma_ss_lead(lead, tmem + g * 256 + buf * 128, kd + (uint64_t)(kk >> 2) * (kSub >> 4) + in,
                                    qd + (uint64_t)(kk >> 2) * (C::kBlockSub >> 4) + in, idesc, kk > 0 ? 1u : 0u);
                    }
                    mma_commit_lead(lead, wait.bar(C::bSF + 2 * g + (int)buf));
                    if (q == x.q1 - 1) mma_commit_lead(lead, wait.bar(C::bKE + (int)stage));
                }
                if (!ok) break;
                mma_commit_lead(lead, wait.bar(C::bQE + (int)blk));
            }
            kt += 2;
        }
        // Wait until every tcgen05 operation issued above has completed.
        mma_commit_lead(lead, wait.bar(C::bDrain));
        mbar_wait_drain(wait.bar(C::bDrain), 0);
    } else if (warp == 1) {
        const Start from = alone ? find_piece_warp(p, w, (int)lane) : *st;
        if (lane == 0) unit_role<C>(p, w, wait, smem, from);
        __syncwarp();
    } else if (warp == 2) {
        fetch_role<D, kFew>(p, wait, (int)lane, base, smem);
    } else if (warp == 3) {
        // ------------------------------------------------- query blocks --
        if (lane == 0 && p.total > 0) tma_prefetch_desc(&tq);   // of no rows there is no map
        const uint32_t bytes = (uint32_t)(p.G * w.tokens) * D * 2u;
        uint32_t units = 0, it = 0;
        bool ok = true;
        // lse of the lane's four rows of a block, loaded while the block before waits for its place
        int at[4], tok[4];
        float nl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 32 * i + (int)lane;
            tok[i] = r / p.G;
            at[i] = tok[i] * p.Hq + r - tok[i] * p.G;
        }
        Unit x = {};
        auto load = [&](int q) {
            const float *lse = p.lse + (long long)(x.first + q * w.tokens) * p.Hq + x.h * p.G;
            const int tokens = min(w.tokens, x.m - q * w.tokens);
#pragma unroll
            for (int i = 0; i < 4; ++i) nl[i] = tok[i] < tokens ? __ldg(lse + at[i]) : INFINITY;
        };
        while (ok && next_unit<C>(wait, smem, units, x)) {
            if (x.q0 < x.q1) load(x.q0);
            for (int q = x.q0; q < x.q1; ++q, ++it) {
                const uint32_t blk = it % C::kBlocks;
                if (!(ok = __all_sync(0xffffffffu, wait(C::bQE + (int)blk, (it / C::kBlocks) ^ 1u)))) break;
                const uint32_t full = wait.bar(C::bQF + (int)blk), lead = lane == 0 ? 1u : 0u;
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d_lead(lead, base + C::kQ + blk * C::kBlockBytes + c * C::kBlockSub, &tq, full, c * 64, x.h * p.G,
                                     x.first + q * w.tokens);
#pragma unroll
                for (int i = 0; i < 4; ++i)     // -inf: a query without keys
                    reinterpret_cast<float *>(smem + C::kLse + blk * 512u)[32 * i + lane] = nl[i] == -INFINITY ? -INFINITY : nl[i] * -1.44269504088896340736f;
                __syncwarp();
                mbar_arrive_expect_tx_lead(lead, full, bytes);
                if (q + 1 < x.q1) load(q + 1);
            }
        }
        // nothing may be on its way into shared memory when the CTA ends
        for (uint32_t s = 0; s < (uint32_t)C::kBlocks; ++s)
            if (it > s) mbar_wait_drain(wait.bar(C::bQF + (int)s), ((it - 1 - s) / C::kBlocks) & 1u);
    } else if (warp < 4 + C::kGroupWarps) {
        regs_claim<kGroupRegs>();
        group_role<D, kFew>(p, w, wait, tmem, (int)(warp >> 2 & 1u) ^ 1, (int)(warp - 4) >> 3, warp, lane, smem);
    } else {
        regs_release<kWidenRegs>();
        widen_role<D, kFew, kInt8>(wait, (int)warp - 4 - C::kGroupWarps, (int)lane, smem);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool kFew, bool kInt8>
cudaError_t launch(const ChunkParams &p, const Blocks &w, cudaStream_t stream) {
    using C = Cfg<D, kFew>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set_for_device[dev]) {
        // the register split inside the kernel assumes exactly kLaunchRegs per thread at launch
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, bsattn_weigh_kernel<D, kFew, kInt8>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(bsattn_weigh_kernel<D, kFew, kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kAlloc);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    const int sms = current_device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    CUtensorMap tq = {};
    if (p.total > 0 && !encode_query_rows(&tq, p.q, p.total, p.Hq, D, p.q_stride, w.tokens, p.G)) return cudaErrorInvalidValue;
    void *args[] = {const_cast<ChunkParams *>(&p), const_cast<Blocks *>(&w), &tq};
    return launch_dependent(reinterpret_cast<const void *>(bsattn_weigh_kernel<D, kFew, kInt8>), dim3((unsigned)sms), kThreads,
                            C::kAlloc, args, stream);
}

template <int D, bool kFew>
cudaError_t launch_of(const ChunkParams &p, const Blocks &w, cudaStream_t stream) {
    return p.c.int8 ? launch<D, kFew, true>(p, w, stream) : launch<D, kFew, false>(p, w, stream);
}

}  // namespace

cudaError_t launch_weigh(const ChunkParams &p, cudaStream_t stream) {
    // Rows of a block: what the sequences have on the average, so that a decoding step's products are 32
    // columns wide.
    const long long mean = ((long long)p.total + p.B - 1) / p.B;
    const long long rows = (mean > 0 ? mean : 1) * p.G;
    if (rows <= kStepRows) return launch_weigh_step(p, (int)rows, stream);
    Blocks w;
    w.tokens = (int)(mean < kTile / p.G ? (mean > 0 ? mean : 1) : kTile / p.G);
    w.cols = (w.tokens * p.G + 31) & ~31;
    if (p.c.D == 128) return w.cols <= 64 ? launch_of<128, true>(p, w, stream) : launch_of<128, false>(p, w, stream);
    return w.cols <= 64 ? launch_of<64, true>(p, w, stream) : launch_of<64, false>(p, w, stream);
}

}  // namespace bsattn
