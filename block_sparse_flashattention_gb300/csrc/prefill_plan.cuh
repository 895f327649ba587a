// How the work of a bsattn_prefill call is numbered and where its parts lie in the workspace; shared by
// its two attention kernels (bsattn_prefill.cu, bsattn_prefill_rows.cu).
#pragma once

#include "chunk_common.cuh"
#include "decode_plan.cuh"

namespace bsattn {

constexpr int kPrefillCtas = 160;
// Places of the line that starting and ending a segment costs.  Prompts of 100 to 4096 tokens, 16 heads, D = 64, us a
// call: 225 with 1, 217 with 2, 223 with 4; 16 sequences with 1 to 512 new tokens: 245, 244, 247.
constexpr int kSegCost = 2;
// Places of a piece: each makes parts for the join, but where the line is short CTAs are free.  5 sequences of 10 to 243
// keys with 7 or 8 new tokens, 3 heads x 6, us a call: 18.7 with 1, 20.1 with 2, 29.1 with 4; 2 of 6 keys, 20 heads: 12.9,
// 11.4, 11.4.
constexpr int kLeastPiece = 2;
constexpr int kDescs = 2;                   // segments found ahead
constexpr float kNoKey = -0x1p100f;         // reference before the first key

// Flags of a tile: some r is not 1; some values are not numbers.
constexpr uint32_t kRest = 1u, kOdd = 2u;

// What goes with a tile: r of its keys, the keys that count, E (biased; 0: no value), flags, and the keys whose
// values are not numbers (NaN or infinite scales, NaN codes).  V' of those is 0, since a NaN times the
// weight 0 of a query that does not meet the key would be NaN; a query that does is told by its mask.
struct TileHead {
    float r[kTile];
    uint32_t keep[4];
    int32_t exp;
    uint32_t flags;
    int32_t pad[2];
    uint32_t odd[4];
};
static_assert(sizeof(TileHead) % 16 == 0, "copied in pieces of 16 bytes");

// A sequence as the plan kernel leaves it.
struct SeqPlan {
    int32_t first, m, n;     // as in Chunk
    int32_t tile0;           // its first tile in the workspace
    int32_t sinks, near;     // tiles that some query meets: below sinks, and from near to end
    int32_t end;
    int32_t block0, blocks;  // its row blocks (of every head)
    int32_t pass;            // places of all of a head's blocks in the line
    long long base;          // first place
};

struct PlanTotals {
    long long places;
    int32_t tiles;
    int32_t pieces;          // of the line; at most as many as the layout has room for
};

// A segment, or the part of it that lies in one piece of the line.
struct SegDesc {
    int32_t b, h;            // b < 0: no more
    int32_t token, tokens;   // first packed row, rows' tokens
    int32_t pos, n;          // position of the first token, keys of the sequence
    int32_t sinks, near;     // tiles visited: 0 .. sinks - 1, then near, near + 1, ...
    int32_t count[2];        // how many of them slot t meets
    int32_t k0, k1;          // those of this piece
    int32_t tile0;           // where the sequence's tiles lie in the workspace, one after the other:
    int32_t seq_sinks, seq_near;  // those below seq_sinks, and from seq_near on
    int32_t part;            // -1: the rows go to the output
    int32_t pad;
};

// A segment that is cut: its rows and how many parts there are.
struct CutInfo {
    int32_t token, tokens, h, parts;
};

struct Layout {
    int few;                 // rows of a segment, 0: two slots of 128 (see segment_rows)
    int tokens, step;        // of a slot: floor(128 / G); of a segment
    int pieces, ctas;
    long long tiles;         // of a head that the workspace has room for
    long long blocks;
    size_t seq, block_place, totals, cuts, part_o, part_l, k, v, head, total;
};

// Which kernel takes a call: with few query rows a KV head (per sequence, on the average) the one that
// widens codes in shared memory, for segments of up to 16, 32, 64 or 128 rows; else (0) the one that has them
// widened into the workspace first.  8 heads, e4m3, us a call there and here:
//   rows                                   16        32        64        96       128
//   D = 128, 16 sequences of 4096 keys   71, 172   78, 172  102, 176  142, 176  148, 178
//   D = 128, 64 of 1000                  86, 178  101, 180  140, 182  201, 184  207, 186
//   D = 64, 16 of 4096                   57, 122   63, 124   85, 129  124, 129  127, 131
//   D = 64, 64 of 1000                   75, 131   88, 131  120, 133  179, 135  183, 138
// Above 64 rows a segment's own cost counts: there, only where a CTA gets two at most.
// The mean says nothing of a chunk among single tokens: 255 tokens and a chunk of 2048, 4096 keys each, int8 (mean 36
// rows), take 1417 there and 2309 here, as two calls 737 + 135; 31 tokens and a chunk of 1024, 16384 keys each (mean
// 132), 1269 here, as two calls 351 + 264.
constexpr int kFewRows = 128, kFewSegs = 2 * kPrefillCtas;
inline int segment_rows(int total, int B, int H, int G) {
    const long long mean = ((long long)total * G + B - 1) / B;
    const int most = (long long)B * H <= kFewSegs ? kFewRows : kFewRows / 2;
    for (int rows = 16; rows <= most; rows *= 2)
        if (mean <= rows && G <= rows) return rows;
    return 0;
}

// Widened bytes that the CTAs work on at a time: of 129 MB of L2, less what else passes through.  2048 tokens on
// 63488 keys, 8 heads x 4, us a call: 1736 with 64 MB, 1760 with 128, 1768 without phases; 4096 tokens in a window of
// 4096, 32 heads: 341, 336, 332.
constexpr long long kPhaseBytes = 64ll << 20;
constexpr int kPhaseVisits = 16;

inline Layout make_layout(int total, int B, int H, int G, int D, long long keys, int ctas) {
    Layout w = {};
    w.tokens = kTile / G;
    w.few = segment_rows(total, B, H, G);
    w.step = w.few ? w.few / G : 2 * w.tokens;
    w.ctas = ctas;
    w.tiles = w.few ? 0 : keys / kTile + B;   // the other kernel widens in shared memory
    w.blocks = (long long)total / w.step + B;
    const long long bytes = w.tiles * H * kTile * D * 4;
    const long long phases = (bytes + kPhaseBytes - 1) / kPhaseBytes;
    w.pieces = ctas * (int)(phases < 1 ? 1 : phases > 64 ? 64 : phases);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255u) & ~(size_t)255u;
        return here;
    };
    w.seq = take((size_t)B * sizeof(SeqPlan));
    w.block_place = take((size_t)w.blocks * 4u);
    w.totals = take(sizeof(PlanTotals));
    w.cuts = take((size_t)w.pieces * sizeof(CutInfo));
    w.part_l = take((size_t)w.pieces * 2 * 256 * 4);
    w.part_o = take((size_t)w.pieces * 2 * 256 * D * 4);
    w.head = take((size_t)w.tiles * H * sizeof(TileHead));
    w.k = take((size_t)w.tiles * H * kTile * D * 2);
    w.v = take((size_t)w.tiles * H * kTile * D * 2);
    w.total = at;
    return w;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^d of an integer d, 0 below 2^-126.
__device__ __forceinline__ float pow2(int d) { return d < -126 ? 0.f : __uint_as_float((uint32_t)(127 + min(d, 127)) << 23); }

// Tiles that queries at positions i0 .. i1 of a sequence of n keys visit: 0 .. sinks - 1 and near .. end - 1.
struct Visit {
    int sinks, near, end;
    __device__ __forceinline__ int count() const { return sinks + end - near; }
};

__device__ __forceinline__ Visit visit(const ChunkParams &p, int n, int i0, int i1) {
    Visit v;
    const int ha = met(p, i1, n).ha;
    v.end = (ha + kTile - 1) / kTile;
    v.sinks = v.near = 0;
    if (p.kind == BSATTN_MASK_SLIDING_WINDOW) {
        v.near = min(met(p, i0, n).la / kTile, v.end);
        v.sinks = min((int)(((long long)p.sink_tokens + kTile - 1) / kTile), v.near);
    }
    return v;
}

__device__ __forceinline__ uint32_t span_bits(int lo, int hi) {
    lo = lo < 0 ? 0 : lo;
    hi = hi > 32 ? 32 : hi;
    if (hi <= lo) return 0u;
    return (hi >= 32 ? 0xffffffffu : ((1u << hi) - 1u)) & ~((1u << lo) - 1u);
}

// Waiting for one of the CTA's barriers; false where the CTA gives up.
struct Waiter {
    uint32_t bars;
    volatile int *abort;
    int *err;
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
    __device__ __forceinline__ bool operator()(int i, uint32_t phase) const {
        return mbar_wait(bar(i), phase & 1u, abort, err, BSATTN_FLAG_TIMEOUT);
    }
};

// Reads the next segment's descriptor (the whole warp), and gives its place back.
template <class C>
__device__ __forceinline__ bool next_desc(const Waiter &wait, const uint8_t *smem, uint32_t &count, SegDesc &d) {
    const int slot = (int)(count % kDescs);
    if (!__all_sync(0xffffffffu, wait(C::bUF + slot, count / kDescs))) return false;
    d = reinterpret_cast<const SegDesc *>(smem + C::kDesc)[slot];
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(wait.bar(C::bUE + slot));
    ++count;
    return d.b >= 0;
}

// Finds the segments of the CTA's pieces and writes their descriptors.
template <class C>
__device__ __forceinline__ void schedule_role(const ChunkParams &p, const Layout &w, const Waiter &wait, uint8_t *smem) {
    const SeqPlan *seq = reinterpret_cast<const SeqPlan *>(p.ws + w.seq);
    const int32_t *place = reinterpret_cast<const int32_t *>(p.ws + w.block_place);
    CutInfo *cuts = reinterpret_cast<CutInfo *>(p.ws + w.cuts);
    const PlanTotals totals = *reinterpret_cast<const PlanTotals *>(p.ws + w.totals);
    const long long line = totals.places;
    const int step = w.step, pieces = totals.pieces;
    uint32_t count = 0;
    bool ok = true;
    for (int piece = blockIdx.x; piece < w.pieces; piece += w.ctas) cuts[piece] = CutInfo{};   // also of pieces not come to
    auto emit = [&](const SegDesc &d) -> bool {
        const int slot = (int)(count % kDescs);
        if (!(ok = wait(C::bUE + slot, (count / kDescs) ^ 1u))) return false;
        reinterpret_cast<SegDesc *>(smem + C::kDesc)[slot] = d;
        mbar_arrive(wait.bar(C::bUF + slot));
        ++count;
        return true;
    };
    for (int piece = blockIdx.x; ok && piece < pieces; piece += w.ctas) {
        const long long from = line_div(line * piece, pieces), to = line_div(line * (piece + 1), pieces);
        CutInfo cut = {};
        if (from < to) {
            int b = 0, hi = p.B - 1;             // the last sequence that begins at or before `from`
            while (b < hi) {
                const int mid = (b + hi + 1) / 2;
                if (seq[mid].base <= from) b = mid;
                else hi = mid - 1;
            }
            SeqPlan s = seq[b];
            int h = s.pass > 0 ? (int)line_div(from - s.base, s.pass) : 0;
            int r = 0;
            if (s.pass > 0) {
                const int off = (int)(from - s.base - (long long)h * s.pass);
                int top = s.blocks - 1;
                while (r < top) {
                    const int mid = (r + top + 1) / 2;
                    if (place[s.block0 + mid] <= off) r = mid;
                    else top = mid - 1;
                }
            }
            while (ok) {
                if (r >= s.blocks) {
                    r = 0;
                    if (++h >= p.c.H || s.blocks == 0) {
                        h = 0;
                        if (++b >= p.B) break;
                        s = seq[b];
                        continue;
                    }
                }
                const long long begin = s.base + (long long)h * s.pass + place[s.block0 + r];
                if (begin >= to) break;
                SegDesc d = {};
                d.b = b, d.h = h, d.n = s.n;
                d.token = s.first + r * step, d.tokens = min(step, s.m - r * step);
                d.pos = s.n - s.m + r * step;
                d.part = -1;
                int tiles = 0;
                if (s.n > 0) {
                    const Visit v = visit(p, s.n, d.pos, d.pos + d.tokens - 1);
                    d.sinks = v.sinks, d.near = v.near;
                    tiles = v.count();
                    // slot 0 meets no tile past its own last position
                    const int mine = (met(p, d.pos + min(w.tokens, d.tokens) - 1, s.n).ha + kTile - 1) / kTile;
                    d.count[0] = v.sinks + max(mine - v.near, 0);
                    d.count[1] = d.tokens > w.tokens ? tiles : 0;
                    d.tile0 = s.tile0, d.seq_sinks = s.sinks, d.seq_near = s.near;
                }
                const long long first = begin + kSegCost;   // place of its first tile
                d.k0 = (int)max(from - first, 0ll);
                d.k1 = (int)min(to - first, (long long)tiles);
                if (tiles == 0 ? begin >= from : d.k1 > d.k0) {
                    if (tiles == 0) d.k0 = d.k1 = 0;
                    else if (d.k0 > 0 || d.k1 < tiles) {
                        d.part = 2 * piece + (d.k0 > 0 ? 0 : 1);
                        if (d.k0 == 0) {
                            // the piece that holds the last tile: place x is in piece ((x + 1) pieces - 1) / line
                            const int last = (int)line_div((first + tiles) * pieces - 1, line);
                            cut.token = d.token, cut.tokens = d.tokens, cut.h = h, cut.parts = last - piece + 1;
                        }
                    }
                    if (!emit(d)) break;
                }
                ++r;
            }
        }
        cuts[piece] = cut;
    }
    if (!ok) return;
    SegDesc stop = {};
    stop.b = -1;
    emit(stop);
}

cudaError_t launch_prefill_rows(const ChunkParams &p, const Layout &w, cudaStream_t stream);

}  // namespace bsattn
