// How a decode call's work is numbered and where its parts lie in the workspace; shared
// by the decode kernels (bsattn_decode.cu, bsattn_decode_rows.cu) and the prefix kernel
// (bsattn_prefix.cu).
#pragma once

#include "bsattn_internal.h"

namespace bsattn {

constexpr int kMaxCtas = 320;      // CTAs whose parts the workspace has room for
constexpr int kStreamWarps = 8;    // warps of a streaming CTA, each a worker of its own
// Query rows a streaming worker holds.  Up to there it beats the other kernel that could take
// the rows (us a call, e4m3, D = 128): against the block kernel 24 : 39 (16 sequences of 8192
// keys, 2 heads, G = 16), 36 : 60 (4 heads, G = 8); a prefix of 32768 keys, 8 heads, in the
// streaming line against the prefix kernel 20 : 33 (2 rows a head), 26 : 34 (16 rows).
constexpr int kStreamRows = 16;
constexpr int kBlockRows = 256;    // query rows of a segment in the prefix kernel

// How the keys of a shared prefix are met.  kEach: they are the first keys of every
// sequence's own segment, read (from L2) once per sequence: no kernel and no parts more
// than without a prefix.  kInLine: up to 16 query rows a KV head, as segments of the
// streaming kernel's line.  kOwnKernel: in the prefix kernel.
enum PrefixMode { kNoPrefix = 0, kInLine = 1, kOwnKernel = 2, kEach = 3 };

// Cache bytes that all sequences together may read of the prefix under kEach.  Measured
// (own keys of 100 tokens, us a call, kEach against the prefix kernel; int8 within 1.5 us):
//                                            17 MB        41 MB        68 MB        135 MB
//   32 sequences, 8 heads, G = 1, D = 128     11.3 : 14.9  14.4 : 15.5  17.8 : 16.2  26.5 : 19.4
//   G = 4                                     12.1 : 15.8  15.4 : 16.5  18.8 : 17.4  27.4 : 22.6
//   G = 16                                    19.3 : 21.7  22.5 : 28.1  26.0 : 29.7  34.9 : 30.3
//   64 sequences, 4 heads, G = 8, D = 64      12.6 : 14.5  16.3 : 16.0  20.3 : 20.3  29.2 : 21.0
//   128 sequences, 8 heads, G = 4, D = 128    19.1 : 29.8  21.6 : 30.0  25.3 : 30.3  33.8 : 30.6
constexpr long long kEachBytes = 76ll << 20;

// What the prefix kernel pays for a segment, in tiles: query rows, the first tiles' latency,
// the part.  512 rows of 8 heads, 32768 keys: CTAs with tiles of two segments took 178000
// cycles of 1.95 GHz, those with as many of one 157000.  A call with own keys (e4m3, int8):
// 120, 128 us without this weight, 111, 125 with it.
constexpr int kPreCost = 3;

// Quotient of numbers that mostly fit 32 bits, where a division costs a tenth.
__host__ __device__ inline long long line_div(long long a, long long b) {
    if ((((unsigned long long)a | (unsigned long long)b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
    return a / b;
}

// Segments: of the prefix, one per KV head (kInLine) or (KV head, block of 256 query
// rows); of the sequences' own keys, (sequence, KV head).  A line of keys is cut over
// workers (warps or CTAs), and part `segment + worker` holds what a worker computed of a
// segment: from one part of the line to the next either the segment or the worker
// advances, so no two parts share a number.
struct Plan {
    int mode;
    int direct;                            // a segment of the line holds all of its rows' keys
    int streaming;                         // G <= 16: bsattn_decode.cu, else bsattn_decode_rows.cu
    int row_blocks, pre_segs;              // prefix kernel: blocks per head, segments
    int rows_p;                            // rows a prefix part has room for
    int sp, ss;                            // prefix and own segments of the decode kernel's line
    int pre_cuts;                          // CTAs of the prefix kernel
    int pre_cost;                          // tiles that a segment costs it besides its own
    size_t rec, pre_o, pre_l, suf_o, suf_l, total;  // byte offsets: records, parts, size

    // The prefix kernel's line: of each segment pre_cost places, then its nt tiles.  First
    // tile, counted over all segments, of CTA `cta`'s piece.
    __host__ __device__ long long pre_first(int cta, int nt) const {
        const long long place = line_div((long long)pre_segs * (nt + pre_cost) * cta, pre_cuts);
        const long long seg = line_div(place, nt + pre_cost);
        const long long off = place - seg * (nt + pre_cost) - pre_cost;
        return seg * nt + (off > 0 ? off : 0);
    }
    // The CTA whose piece holds tile `off` of segment `seg`.
    __host__ __device__ int pre_owner(int seg, int off, int nt) const {
        const long long place = (long long)seg * (nt + pre_cost) + pre_cost + off;
        return (int)line_div((place + 1) * pre_cuts - 1, (long long)pre_segs * (nt + pre_cost));
    }
};

// sms: SMs of the device (0: only the workspace's layout is wanted).
inline Plan make_plan(int B, int H, int G, int D, int prefix_len, int sms) {
    Plan w = {};
    const int rows = B * G;
    w.streaming = G <= kStreamRows ? 1 : 0;
    const bool each = w.streaming && (long long)B * H * prefix_len * 2 * (D + 4) <= kEachBytes;
    w.mode = prefix_len <= 0 ? kNoPrefix : each ? kEach : rows <= kStreamRows ? kInLine : kOwnKernel;
    w.direct = w.mode == kNoPrefix || w.mode == kEach;
    w.row_blocks = w.mode == kOwnKernel ? (rows + kBlockRows - 1) / kBlockRows : 0;
    w.pre_segs = H * w.row_blocks;
    // the prefix kernel's parts hold both slots of 128 rows
    w.rows_p = w.mode == kOwnKernel ? kBlockRows : rows;
    w.sp = w.mode == kInLine ? H : 0;
    w.ss = B * H;
    const long long tiles = (long long)w.pre_segs * ((prefix_len + kTile - 1) / kTile);
    const int most = sms < kMaxCtas ? sms : kMaxCtas;
    w.pre_cuts = (int)(tiles < most ? tiles : most);
    // every piece keeps tiles of its own
    w.pre_cost = w.pre_cuts > 0 && tiles / w.pre_cuts > 2 * kPreCost ? kPreCost : 0;
    const size_t workers = w.streaming ? kMaxCtas * kStreamWarps : kMaxCtas;
    const size_t np = w.mode == kOwnKernel ? (size_t)(w.pre_segs + kMaxCtas) * w.rows_p
                    : w.mode == kInLine    ? ((size_t)w.sp + workers) * w.rows_p : 0;
    const size_t ns = (w.ss + workers) * G;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255u) & ~(size_t)255u;
        return here;
    };
    w.rec = take((size_t)(w.sp + w.ss) * sizeof(int2));
    w.pre_o = take(np * D * 4u);
    w.pre_l = take(np * 4u);
    w.suf_o = take(ns * D * 4u);
    w.suf_l = take(ns * 4u);
    w.total = at;
    return w;
}

cudaError_t launch_prefix(const DecodeParams &p, const Plan &w, cudaStream_t stream);
cudaError_t launch_decode_rows(const DecodeParams &p, const Plan &w, int sms, cudaStream_t stream);

}  // namespace bsattn
