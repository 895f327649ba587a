// Attention of chunks of few new tokens over a paged 8-bit K/V cache: up to 128 query rows of a KV head
// share each key, which is widened in shared memory on its way (more rows: bsattn_prefill.cu, whose line of
// work and parts this kernel shares).
//
// With few rows HBM bounds it: 2 (D + 4) bytes per key and KV head.  So the keys lie on the tensor cores' 128
// rows and the queries on their columns, of which there are 16 to 128:
//   S^T = K' Q'^T,  O^T += V'^T P^T,
//   K' = fp16(code), V' = fp16(code), exact, no scale in either; Q' = fp16(q 2^-e) with the row's largest
//   binary exponent e (exact for every element down to 2^-14 of the largest).
// A thread has one key of the tile: its scales are two registers, z_r = S_r c_r ks (c_r = softmax_scale
// log2(e) 2^e of row r) and p_r = 2^(z_r - m_r + 7); p_r vs 2^-E is rounded to fp16 (11 bits) for V'^T P^T,
// and the thread sums p_r of its keys by itself, in fp32.  Only at a segment's end are sums joined over the
// threads.  The reference m_r (per query row, kept by all) and E (2^2 above the largest binary exponent of a value
// scale so far, rounded up to a multiple of 4) are moved only when some weight could pass 2^14 or some scale passes E: the threads
// vote on every tile, and the maxima over the keys, which cost a pass of their own, are taken then.
//
// Up to 64 rows two groups of threads take the tiles in turn, each with sums of its own, joined at the end: while
// one group's weights are formed, the other's products run.  With more, each group has 64 of the rows.
//
// Measured (us a call, cold L2): 8 sequences of 100 to 4096 keys with drafts of 4 tokens, 8 heads x 4, e4m3, D = 128: 28
// (35 MB: 5.3 at the copy's rate), of which the join 5.5; 16 sequences of 4096 keys, 8 heads (142 MB: 21): 16 rows 71,
// 32 78, 64 102, 128 148.  Before a CTA's first product lie 6000 cycles for its piece of the line, 1300 for query rows,
// 3000 to 5000 for the first codes; then a tile takes some 3000, of which HBM's latency behind a ring of two is the
// largest part.  Copies of a page in place of 16 keys made no difference.
//
// Roles (640 threads, one CTA per SM):
//   warp 0        issues the MMAs
//   warp 1        owns the TMEM allocation; finds the segments of the CTA's piece of the line
//   warps 2, 3    fetch the codes of keys, of values: bulk copies of 16 keys into a ring of raw tiles
//   warps 4-7, 8-11   group 0, group 1: query rows, weights, output
//   warps 12-15   widen the codes of keys (128-byte swizzle, a tile's rows K-major)
//   warps 16-19   the same for values, as they lie (MN-major)
// TMEM: S^T of group g [64 g, 64 g + 64), O^T of group g [128 + 64 g, 192 + 64 g).
#include "kv_codes.cuh"
#include "prefill_plan.cuh"

namespace bsattn {

namespace {

constexpr int kThreads = 640;
constexpr uint32_t kTmemCols = 256;
// 96 registers per thread at launch: 128 * 80 + 2 * 128 * 144 + 2 * 128 * 56 = 61440 = 640 * 96.
constexpr int kLaunchRegs = 96;
constexpr uint32_t kCtrlRegs = 80, kGroupRegs = 144, kWidenRegs = 56;
static_assert(128 * kCtrlRegs + 256 * kGroupRegs + 256 * kWidenRegs <= (uint32_t)kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr uint32_t kSub = kTile * 64 * 2;   // 128 rows x 64 fp16: one 128-byte swizzle span
constexpr float kLift = 7.f, kReach = 7.f;
constexpr int kRoom = 2;                    // binary exponents of value scales up to which E stays

// kRows: query rows of a segment at most.
template <int D, int kRows>
struct Cfg {
    static constexpr int kCols = kRows < 64 ? kRows : 64;            // of a group
    static constexpr uint32_t kTileBytes = kTile * D * 2, kRawBytes = kTile * D;
    static constexpr uint32_t kQ = 0, kK = kQ + kTileBytes, kV = kK + kTileBytes, kP = kV + 2 * kTileBytes;
    static constexpr uint32_t kRaw = kP + 2 * kSub;                  // K0, K1, V0, V1
    static constexpr uint32_t kStat = kRaw + 4 * kRawBytes;          // see Stat
    static constexpr uint32_t kStatBytes = 128 * 4 * 2 + 2 * 64 * 4 * 2 + 64 * 4 + 128 + 2 * 16 + 2 * 8 + 8 + 16 + 16;
    static constexpr uint32_t kDesc = (kStat + kStatBytes + 15u) & ~15u;
    static constexpr uint32_t kBar = kDesc + kDescs * (uint32_t)sizeof(SegDesc);
    // K' full and empty, V' stages full and empty, query rows there, per group: S ready, P ready, O complete;
    // raw K / V stages full and empty (2 v + stage); descriptor full and empty
    static constexpr int bKF = 0, bKE = 1, bVF = 2, bVE = 4, bQF = 6, bSR = 7, bPR = 9, bOD = 11, bRF = 13, bRE = 17, bUF = 21,
                         bUE = bUF + kDescs, bDrain = bUE + kDescs, kNumBars = bDrain + 1;
    static constexpr uint32_t kMisc = kBar + kNumBars * 8;           // [0] tmem base, [1] abort
    static constexpr uint32_t kAlloc = kMisc + 16;
    static_assert(kAlloc <= 227u * 1024u, "shared memory");
};

// Numbers of the segment's rows, in shared memory.
struct Stat {
    float c[128];            // c_r, 0 of rows that are none
    int32_t out[128];        // row of the output or the parts, -1: none
    float nm[2][64];         // 7 - m_r of the groups' rows, -inf of rows that are none
    float alpha[2][64];      // what sums are multiplied by when m moves; at the end what O is
    float zero[64];
    uint8_t bad[128];        // the row meets a value that is not a number
    uint32_t odd[2][4];      // keys of the V' stages that have a NaN code
    int32_t exp[2], any[2];
    uint32_t groups[2];      // 16-key groups of the raw V tiles that are there
    int32_t b, h, r;         // where the CTA's piece of the line begins
    int32_t pieces;
    long long begin, line;   // place at which that segment begins; places in all
};
static_assert(sizeof(Stat) <= Cfg<64, 16>::kStatBytes, "stat area");

// Threads of a group, or of both, meet; whether `x` holds for one of them.
__device__ __forceinline__ bool any_of(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\tbarrier.cta.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(x ? 1u : 0u)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ bool any_of_both(bool x) { return any_of(1, 256, x); }
__device__ __forceinline__ bool any_of_group(int g, bool x) { return any_of(2 + g, 128, x); }
__device__ __forceinline__ void group_sync(int g) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + g) : "memory"); }

// Largest of a float over the warp, NaN left out.
__device__ __forceinline__ float warp_max(float x) {
    const int b = x == x ? __float_as_int(x) : (int)0xff800000;
    const int y = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
    return __int_as_float(y ^ ((y >> 31) & 0x7fffffff));
}

// Of 2 n sums of each of two lanes, `d` apart, either keeps the n of its own rows.
template <int n, int kCols>
__device__ __forceinline__ void fold(float (&l)[kCols], uint32_t lane, int d) {
    const bool upper = (lane & (uint32_t)d) != 0;
#pragma unroll
    for (int x = 0; x < n; ++x) {
        const float other = __shfl_xor_sync(0xffffffffu, upper ? l[x] : l[n + x], d);
        l[x] = (upper ? l[n + x] : l[x]) + other;
    }
}

// Key tile k of a segment's visiting list.
__device__ __forceinline__ int tile_of(const SegDesc &d, int k) { return k < d.sinks ? k : k - d.sinks + d.near; }

// The line of work of this kernel is numbered by every CTA for itself (lengths are on the device): places of
// one head's pass over a sequence's segments.
// Places that starting and ending a segment costs.  Drafts of 4 tokens, 8 sequences, us a call: 29.3 with 1, 28.3 with 2,
// 28.1 with 3, 29.5 with 4; 64 sequences of 1000 keys, 8 heads, 64 rows, e4m3: 150, 148, 140, 138.
constexpr int kRowsCost = 3;

__device__ __forceinline__ int segment_tiles(const ChunkParams &p, const Layout &w, const Chunk &c, int r) {
    if (c.n <= 0) return 0;
    return visit(p, c.n, c.n - c.m + r * w.step, c.n - c.m + min((r + 1) * w.step, c.m) - 1).count();
}

__device__ __forceinline__ long long pass_places(const ChunkParams &p, const Layout &w, const Chunk &c) {
    long long sum = 0;
    for (int r = 0; r * (long long)w.step < c.m; ++r) sum += kRowsCost + segment_tiles(p, w, c, r);
    return sum;
}

// Numbers the line and finds where the CTA's piece begins; all threads.
template <class C>
__device__ __forceinline__ void find_piece(const ChunkParams &p, const Layout &w, uint8_t *smem) {
    Stat *st = reinterpret_cast<Stat *>(smem + C::kStat);
    long long *warps = reinterpret_cast<long long *>(smem + C::kK);   // no tile is there yet
    const int tid = (int)threadIdx.x, lane = tid % 32, warp = tid / 32;
    auto scan = [&](long long x, long long &all) -> long long {       // sum over the threads before this one
        long long s = x;
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        __syncthreads();
        if (lane == 31) warps[warp] = s;
        __syncthreads();
        long long before = 0;
        all = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += warps[i];
            all += warps[i];
        }
        return before + s - x;
    };
    Chunk c = {};
    long long line = 0, pass = 0, before = 0, all;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        c = Chunk{};
        if (b0 + tid < p.B) c = chunk_of(p, b0 + tid, blockIdx.x == 0);
        pass = pass_places(p, w, c);
        before = line + scan(pass * p.c.H, all);
        line += all;
    }
    const int pieces = (int)max(1ll, min((long long)w.ctas, line_div(line, kLeastPiece))), piece = (int)blockIdx.x;
    const long long from = line_div(line * piece, pieces);
    if (tid == 0) st->pieces = pieces, st->line = line, st->b = p.B;
    __syncthreads();
    if (piece >= pieces || from >= line) return;
    // more sequences than threads: once more from the first
    long long sum = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        if (p.B > kThreads) {
            c = Chunk{};
            if (b0 + tid < p.B) c = chunk_of(p, b0 + tid, false);
            pass = pass_places(p, w, c);
            before = sum + scan(pass * p.c.H, all);
            sum += all;
        }
        if (from >= before && from < before + pass * p.c.H) {
            const int h = (int)line_div(from - before, pass);
            long long at = before + h * pass;
            int r = 0;
            for (int len; at + (len = kRowsCost + segment_tiles(p, w, c, r)) <= from; ++r) at += len;
            st->b = b0 + tid, st->h = h, st->r = r, st->begin = at;
        }
    }
}

// The same by one warp, without a barrier, of up to 32 kLaneSeqs sequences.
struct Start {
    int b, h, r, pieces;
    long long begin, line;
    Chunk c;                 // of sequence b
};
constexpr int kLaneSeqs = 4;

__device__ __forceinline__ Start find_piece_warp(const ChunkParams &p, const Layout &w, int lane) {
    Chunk c[kLaneSeqs];
    long long pass[kLaneSeqs], before[kLaneSeqs];
    Start st = {};
#pragma unroll
    for (int k = 0; k < kLaneSeqs; ++k) {
        c[k] = Chunk{};
        if (32 * k + lane < p.B) c[k] = chunk_of(p, 32 * k + lane, blockIdx.x == 0);
    }
#pragma unroll
    for (int k = 0; k < kLaneSeqs; ++k) {
        if (32 * k >= p.B) break;
        pass[k] = pass_places(p, w, c[k]);
        long long s = pass[k] * p.c.H;
        const long long own = s;
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        before[k] = st.line + s - own;
        st.line += __shfl_sync(0xffffffffu, s, 31);
    }
    st.pieces = (int)max(1ll, min((long long)w.ctas, line_div(st.line, kLeastPiece)));
    st.b = p.B;
    const long long from = line_div(st.line * (int)blockIdx.x, st.pieces);
    if ((int)blockIdx.x >= st.pieces) return st;
#pragma unroll
    for (int k = 0; k < kLaneSeqs; ++k) {
        if (32 * k >= p.B) break;
        const bool here = from >= before[k] && from < before[k] + pass[k] * p.c.H;
        const uint32_t hit = __ballot_sync(0xffffffffu, here);
        if (!hit) continue;
        if (here) {
            st.h = (int)line_div(from - before[k], pass[k]);
            st.begin = before[k] + st.h * pass[k];
            for (int len; st.begin + (len = kRowsCost + segment_tiles(p, w, c[k], st.r)) <= from; ++st.r) st.begin += len;
        }
        const int x = __ffs(hit) - 1;
        st.b = 32 * k + x;
        st.h = __shfl_sync(0xffffffffu, st.h, x);
        st.r = __shfl_sync(0xffffffffu, st.r, x);
        st.begin = __shfl_sync(0xffffffffu, st.begin, x);
        st.c.first = __shfl_sync(0xffffffffu, c[k].first, x);
        st.c.m = __shfl_sync(0xffffffffu, c[k].m, x);
        st.c.n = __shfl_sync(0xffffffffu, c[k].n, x);
    }
    return st;
}

// Finds the segments of the CTA's piece and writes their descriptors.
template <class C>
__device__ __forceinline__ void segment_role(const ChunkParams &p, const Layout &w, const Waiter &wait, uint8_t *smem, const Start &st) {
    CutInfo *cut = reinterpret_cast<CutInfo *>(p.ws + w.cuts) + blockIdx.x;
    *cut = CutInfo{};
    uint32_t count = 0;
    auto emit = [&](const SegDesc &d) -> bool {
        const int slot = (int)(count % kDescs);
        if (!wait(C::bUE + slot, (count / kDescs) ^ 1u)) return false;
        reinterpret_cast<SegDesc *>(smem + C::kDesc)[slot] = d;
        mbar_arrive(wait.bar(C::bUF + slot));
        ++count;
        return true;
    };
    const long long line = st.line;
    const int pieces = st.pieces, piece = (int)blockIdx.x;
    int b = st.b, h = st.h, r = st.r;
    if (b < p.B) {
        const long long from = line_div(line * piece, pieces), to = line_div(line * (piece + 1), pieces);
        long long begin = st.begin;
        Chunk s = st.c;
        while (begin < to) {
            if (r * (long long)w.step >= s.m) {
                r = 0;
                if (s.m == 0 || ++h >= p.c.H) {
                    h = 0;
                    if (++b >= p.B) break;
                    s = chunk_of(p, b, false);
                }
                continue;
            }
            SegDesc d = {};
            d.b = b, d.h = h, d.n = s.n;
            d.token = s.first + r * w.step, d.tokens = min(w.step, s.m - r * w.step);
            d.pos = s.n - s.m + r * w.step;
            d.part = -1;
            int tiles = 0;
            if (s.n > 0) {
                const Visit v = visit(p, s.n, d.pos, d.pos + d.tokens - 1);
                d.sinks = v.sinks, d.near = v.near;
                tiles = v.count();
            }
            const long long first = begin + kRowsCost;   // place of its first tile
            d.k0 = (int)max(from - first, 0ll);
            d.k1 = (int)min(to - first, (long long)tiles);
            if (tiles == 0 ? begin >= from : d.k1 > d.k0) {
                if (tiles == 0) d.k0 = d.k1 = 0;
                else if (d.k0 > 0 || d.k1 < tiles) {
                    d.part = 2 * piece + (d.k0 > 0 ? 0 : 1);
                    if (d.k0 == 0) {
                        // the piece that holds the last tile: place x is in piece ((x + 1) pieces - 1) / line
                        const int last = (int)line_div((first + tiles) * pieces - 1, line);
                        CutInfo x;
                        x.token = d.token, x.tokens = d.tokens, x.h = h, x.parts = last - piece + 1;
                        *cut = x;
                    }
                }
                if (!emit(d)) return;
            }
            begin = first + tiles;
            ++r;
        }
    }
    SegDesc stop = {};
    stop.b = -1;
    emit(stop);
}

// One group: 128 threads, one key of a tile each.
template <int D, int kRows, bool kInt8>
__device__ __forceinline__ void group_role(const ChunkParams &p, const Layout &w, const Waiter &wait, uint32_t tmem, int g,
                                           uint32_t warp, uint32_t lane, uint8_t *smem) {
    using C = Cfg<D, kRows>;
    constexpr int kCols = C::kCols, kChunks = kCols / 16;
    Stat *st = reinterpret_cast<Stat *>(smem + C::kStat);
    const uint32_t quarter = warp & 3u;
    const int key = (int)(quarter * 32 + lane), sw = (int)warp - 4;
    const uint32_t s_addr = tmem + ((quarter * 32u) << 16) + (uint32_t)g * 64u, o_addr = s_addr + 128u;
    uint8_t *pbuf = smem + C::kP + (uint32_t)g * kSub;
    float *red = reinterpret_cast<float *>(pbuf);     // [4][64] while no weights are in the buffer, then 4 exponents, sums
    auto sums = [&](int of) -> float * { return reinterpret_cast<float *>(smem + C::kP + (uint32_t)of * kSub) + 5 * 64; };
    uint32_t descs = 0, sc = 0, od = 0, tile0 = 0;
    SegDesc d;
    while (true) {
        const bool got = next_desc<C>(wait, smem, descs, d);
        if (any_of_both(!got)) break;
        const int rows = d.tokens * p.G;
        const bool turns = kRows <= 64 || rows <= 64;
        const int row0 = turns ? 0 : 64 * g, cols = turns ? rows : min(max(rows - row0, 0), kCols);
        const int chunks = (cols + 15) / 16;
        // ---- query rows: fp16 of q 2^-e (K-major, swizzled), D / 8 lanes to a row, the rows dealt out to all warps
        constexpr int kOwn = kRows / 8;
        if (kOwn * sw < ((rows + 15) & ~15)) {
            constexpr int kRowLanes = D / 8, kAtOnce = 32 / kRowLanes < kOwn ? 32 / kRowLanes : kOwn, kSteps = kOwn / kAtOnce;
            const int piece = (int)lane % kRowLanes, sub = (int)lane / kRowLanes;
            uint4 x[kSteps];
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int r = kOwn * sw + i * kAtOnce + min(sub, kAtOnce - 1), tok = r / p.G;
                x[i] = make_uint4(0, 0, 0, 0);
                if (r < rows)
                    x[i] = __ldg(reinterpret_cast<const uint4 *>(p.q + (long long)(d.token + tok) * p.q_stride +
                                                                 (long long)(d.h * p.G + r - tok * p.G) * D) + piece);
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int r = kOwn * sw + i * kAtOnce + min(sub, kAtOnce - 1);
                uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, a = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) a = __vmaxu2(a, y[k] & 0x7fff7fffu);
                a = max(a & 0xffffu, a >> 16);
#pragma unroll
                for (int s = 1; s < kRowLanes; s <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
                // zero rows and rows that are not finite stay as they are
                const int e = a == 0 || a >= 0x7f80u ? 127 : min(max((int)(a >> 7), 1), 253);
                const float f = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[k] = pack_f16x2(__uint_as_float(y[k] << 16) * f, __uint_as_float(y[k] & 0xffff0000u) * f);
                const uint32_t at = C::kQ + (uint32_t)(piece >> 3) * kSub + (uint32_t)r * 128u + ((((uint32_t)piece & 7u) ^ ((uint32_t)r & 7u)) << 4);
                *reinterpret_cast<uint4 *>(smem + at) = make_uint4(y[0], y[1], y[2], y[3]);
                if (piece == 0) {
                    const int tok = r / p.G;
                    st->c[r] = r < rows ? p.scale_log2 * __uint_as_float((uint32_t)e << 23) : 0.f;
                    st->out[r] = r >= rows ? -1 : d.part >= 0 ? d.part * 2 * kTile + r : (d.token + tok) * p.Hq + d.h * p.G + r - tok * p.G;
                }
            }
        }
        if (key < kCols) {
            st->nm[g][key] = key < cols ? kLift - kNoKey : -INFINITY;
            st->bad[64 * g + key] = 0;
        }
        fence_proxy_async_smem();
        any_of_both(false);
        if (lane == 0) mbar_arrive(wait.bar(C::bQF));
        // ---- the group's tiles
        float l[kCols];
#pragma unroll
        for (int x = 0; x < kCols; ++x) l[x] = 0.f;
        int exp_run = 0;
        bool ok = true, begun = false;
        const int step = turns ? 2 : 1, k_first = turns ? d.k0 + g : d.k0;
        const int32_t *table = p.table + (long long)d.b * p.table_stride;
        // scales of the thread's key in the next tile; row -1: no such key
        long long row_next = -1;
        float ks_next = 0.f, vs_next = 0.f;
        auto look = [&](int k) {
            const int j = tile_of(d, k) * kTile + key;
            row_next = k < d.k1 && j < d.n ? cache_row(p.c, table, d.h, j) : -1;
            if (row_next >= 0) ks_next = __ldg(p.c.ks + row_next), vs_next = __ldg(p.c.vs + row_next);
        };
        look(k_first);
        for (int k = k_first; k < d.k1; k += step) {
            const uint32_t it = tile0 + (uint32_t)(k - d.k0), stage = it & 1u;
            const bool there = row_next >= 0;
            const float ks = there ? ks_next : 0.f;
            float vs = there ? vs_next : 0.f;
            const int j = tile_of(d, k) * kTile + key;
            look(k + step);
            // rows that meet the key: lo <= r < hi
            int lo = 0, hi = 0;
            if (there) {
                hi = rows;
                if (p.kind == BSATTN_MASK_CAUSAL || p.kind == BSATTN_MASK_SLIDING_WINDOW || (p.kind == BSATTN_MASK_PREFIX && j >= p.prefix_len))
                    lo = min(max(j - d.pos, 0), d.tokens) * p.G;
                if (p.kind == BSATTN_MASK_SLIDING_WINDOW && j >= p.sink_tokens)
                    hi = (int)min(max((long long)j + p.window_left - d.pos, 0ll), (long long)d.tokens) * p.G;
            }
            lo -= row0, hi -= row0;
            const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < cols);
            const uint32_t vb = __float_as_uint(vs) & 0x7fffffffu;
            const int vexp = vb < 0x7f800000u && vb > 1u << 23 ? (int)(vb >> 23) : 0;
            ok = __all_sync(0xffffffffu, wait(C::bSR + g, sc) && (kInt8 || wait(C::bVF + (int)stage, it >> 1)));
            ++sc;
            tc_fence_after();
            if (there && (vb >= 0x7f800000u || (!kInt8 && ok && ((st->odd[stage][quarter] >> lane) & 1u)))) {
                vs = 0.f;
                for (int r = max(lo, 0); r < min(hi, cols); ++r) st->bad[64 * g + r] = 1;
            }
            // scores of columns 16 c .. less m, in units of log2: 7 for the largest (nm zero: the scores)
            auto scores = [&](int c, const float *nm, float (&y)[16]) {
                uint32_t v[16];
                tmem_ld16(s_addr + 16u * c, v);
                tmem_wait_ld();
                reg_fence(v);
                const float4 *cr = reinterpret_cast<const float4 *>(st->c + row0 + 16 * c), *less = reinterpret_cast<const float4 *>(nm + 16 * c);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float4 f = cr[x], n = less[x];
                    float *z = y + 4 * x;
                    fmul2(z[0], z[1], __uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1]), f.x, f.y);
                    fmul2(z[2], z[3], __uint_as_float(v[4 * x + 2]), __uint_as_float(v[4 * x + 3]), f.z, f.w);
                    ffma2(z[0], z[1], z[0], z[1], ks, ks, n.x, n.y);
                    ffma2(z[2], z[3], z[2], z[3], ks, ks, n.z, n.w);
                }
                if (masked) {
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        if (16 * c + x < lo || 16 * c + x >= hi) y[x] = -INFINITY;
                }
            };
            // Does m, or E, have to move?  All threads of the group decide as one.
            bool move = !begun;
            if (begun) {
                float top = -INFINITY;
                if (ok) {
#pragma unroll 1
                    for (int c = 0; c < chunks; ++c) {
                        float y[16];
                        scores(c, st->nm[g], y);
#pragma unroll
                        for (int x = 0; x < 16; x += 2) top = fmax3(top, y[x], y[x + 1]);
                    }
                }
                move = any_of_group(g, !ok || top > kLift + kReach || vexp > exp_run);
            }
            if (move) {
                if (any_of_group(g, !ok)) {
                    ok = false;
                    break;
                }
                int *rexp = reinterpret_cast<int *>(red + 256);
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    float y[16];
                    scores(c, st->zero, y);
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const float m = warp_max(y[x]);
                        if (lane == 0) red[quarter * 64 + 16 * c + x] = m;
                    }
                }
                const int we = __reduce_max_sync(0xffffffffu, vexp);
                if (lane == 0) rexp[quarter] = we;
                group_sync(g);
                if (key < kCols) {
                    float alpha = 1.f;
                    if (key < cols) {
                        const float old = kLift - st->nm[g][key];
                        const float m = fmaxf(old, fmaxf(fmaxf(red[key], red[64 + key]), fmaxf(red[128 + key], red[192 + key])));
                        alpha = ex2_approx(old - m);
                        st->nm[g][key] = kLift - m;
                    }
                    st->alpha[g][key] = alpha;
                }
                // with room for a scale or two that are larger
                const int e = min(((max(max(max(rexp[0], rexp[1]), max(rexp[2], rexp[3])), 8) + 3) & ~3) + kRoom, 252);
                const float drop = pow2(exp_run - max(exp_run, e));
                exp_run = max(exp_run, e);
                group_sync(g);
                if (begun) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        if (kChunks > 1 && c >= chunks) break;
                        // S of this tile was issued after the group's previous V P: O is up to date
                        uint32_t v[16];
                        tmem_ld16(o_addr + 16u * c, v);
                        tmem_wait_ld();
                        reg_fence(v);
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const float f = st->alpha[g][16 * c + x];
                            l[16 * c + x] *= f;
                            v[x] = __float_as_uint(__uint_as_float(v[x]) * (f * drop));
                        }
                        tmem_st16(o_addr + 16u * c, v);
                    }
                    tmem_wait_st();
                }
            }
            begun = true;
            const float wv = vs * pow2(127 - exp_run);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (kChunks > 1 && c >= chunks) break;
                float y[16];
                scores(c, st->nm[g], y);
                uint32_t pk[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int i = 16 * c + 2 * x;
                    float p0 = ex2_approx(y[2 * x]), p1 = ex2_approx(y[2 * x + 1]);
                    fadd2(l[i], l[i + 1], l[i], l[i + 1], p0, p1);
                    fmul2(p0, p1, p0, p1, wv, wv);
                    pk[x] = pack_f16x2(p0, p1);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    *reinterpret_cast<uint4 *>(pbuf + key * 128 + (((2 * c + x) ^ (key & 7)) << 4)) =
                        make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(wait.bar(C::bPR + g));
        }
        tile0 += (uint32_t)(d.k1 - d.k0);
        if (ok && begun) {
            ok = wait(C::bOD + g, od);
            ++od;
            tc_fence_after();
        }
        // ---- sums over the keys: each exchange halves the rows that a lane has sums of
        if constexpr (kCols == 64) fold<32>(l, lane, 16), fold<16>(l, lane, 8), fold<8>(l, lane, 4), fold<4>(l, lane, 2), fold<2>(l, lane, 1);
        else if constexpr (kCols == 32) fold<16>(l, lane, 16), fold<8>(l, lane, 8), fold<4>(l, lane, 4), fold<2>(l, lane, 2), fold<1>(l, lane, 1);
        else fold<8>(l, lane, 16), fold<4>(l, lane, 8), fold<2>(l, lane, 4), fold<1>(l, lane, 2), l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
        if constexpr (kCols == 64) {
            red[quarter * 64 + 2 * lane] = l[0];
            red[quarter * 64 + 2 * lane + 1] = l[1];
        } else {
            red[quarter * 64 + lane * kCols / 32] = l[0];
        }
        group_sync(g);
        if (key < kCols) sums(g)[key] = (red[key] + red[64 + key]) + (red[128 + key] + red[192 + key]);
        if (key == 0) st->exp[g] = exp_run, st->any[g] = begun ? 1 : 0;
        if (any_of_both(!ok)) break;
        // ---- a row's weight of either group's O, its LSE
        {
            const int r = g * kTile + key;      // of 256 threads, the first 128 have a row each
            if (r < (turns ? kCols : 128)) {
                const int g0 = turns ? 0 : r / 64, c = turns ? r : r % 64;
                const float m0 = kLift - st->nm[g0][c], l0 = sums(g0)[c];
                const float m1 = turns ? kLift - st->nm[1][c] : kNoKey, l1 = turns ? sums(1)[c] : 0.f;
                const float m = fmaxf(m0, m1), f0 = ex2_approx(m0 - m), f1 = ex2_approx(m1 - m);
                const float sum = l0 * f0 + l1 * f1;
                const bool empty = sum == 0.f;       // NaN is not empty
                const bool bad = st->bad[64 * g0 + c] || (turns && st->bad[64 + c]);
                const float inv = empty ? 0.f : bad ? __uint_as_float(0x7fc00000u) : 1.f / sum;
                st->alpha[g0][c] = f0 * inv;
                if (turns) st->alpha[1][c] = f1 * inv;
                const int out = r < rows ? st->out[r] : -1;
                if (out >= 0) {
                    if (d.part >= 0) reinterpret_cast<float *>(p.ws + w.part_l)[out] = empty ? -INFINITY : m - kLift + lg2_approx(sum);
                    else p.lse[out] = empty ? -INFINITY : (m - kLift) * 0.69314718055994530942f + logf(sum);
                }
            }
        }
        // Either group is about to read what the other has waited for.
        tc_fence_before();
        any_of_both(false);
        tc_fence_after();
        // ---- output: lanes are columns of V, a warp writes 32 of them of one row at a time
        {
            const bool f32 = d.part >= 0 || p.out_f32;
            uint8_t *out = d.part >= 0 ? p.ws + w.part_o : static_cast<uint8_t *>(p.out);
            const bool any0 = st->any[turns ? 0 : g] != 0, any1 = turns && st->any[1] != 0;
            const float u0 = pow2(st->exp[turns ? 0 : g] - 127), u1 = pow2(st->exp[1] - 127);
            const uint32_t o0 = tmem + ((quarter * 32u) << 16) + 128u + (turns ? 0 : (uint32_t)g * 64u), o1 = o0 + 64u;
            // chunks of 16 rows: each group's own, or, in turns, every other
            const int c0 = turns ? g : 0, dc = turns ? 2 : 1;
#pragma unroll 1
            for (int c = c0; 16 * c < cols; c += dc) {
                float v[16];
                uint32_t x0[16], x1[16];
                tmem_ld16(o0 + 16u * c, x0);
                if (any1) tmem_ld16(o1 + 16u * c, x1);
                tmem_wait_ld();
                reg_fence(x0);
                if (any1) reg_fence(x1);
                const float *f0 = st->alpha[turns ? 0 : g] + 16 * c, *f1 = st->alpha[1] + 16 * c;
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    v[x] = any0 ? __uint_as_float(x0[x]) * f0[x] * u0 : 0.f * f0[x];
                    if (any1) v[x] += __uint_as_float(x1[x]) * f1[x] * u1;
                }
                if (key < D) {
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const int at = row0 + 16 * c + x < rows ? st->out[row0 + 16 * c + x] : -1;
                        if (at < 0) continue;
                        if (f32) reinterpret_cast<float *>(out)[(long long)at * D + key] = v[x];
                        else reinterpret_cast<uint16_t *>(out)[(long long)at * D + key] = (uint16_t)pack_bf16x2(v[x], 0.f);
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
    }
}

// Fetches the codes of K or V tiles, a warp each: a copy per 16 keys (no page is smaller), none for keys
// past the sequence's last or on a page that is none.
template <int D, int kRows>
__device__ __forceinline__ void fetch_role(const ChunkParams &p, const Waiter &wait, bool values, int lane, uint32_t base, uint8_t *smem) {
    using C = Cfg<D, kRows>;
    const int v = values ? 2 : 0;
    const uint8_t *codes = values ? p.c.v : p.c.k;
    uint32_t *groups = reinterpret_cast<Stat *>(smem + C::kStat)->groups;
    uint32_t descs = 0, it = 0;
    bool ok = true;
    SegDesc d;
    while (ok && next_desc<C>(wait, smem, descs, d)) {
        const int32_t *table = p.table + (long long)d.b * p.table_stride;
        for (int k = d.k0; k < d.k1; ++k, ++it) {
            const int key = tile_of(d, k) * kTile + 16 * lane, stage = (int)(it & 1u);
            long long row = -1;
            if (lane < 8 && key < d.n) {
                row = cache_row(p.c, table, d.h, key);
                if (row < 0 && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
            }
            const uint32_t on = __ballot_sync(0xffffffffu, row >= 0);
            ok = __all_sync(0xffffffffu, wait(C::bRE + v + stage, (it >> 1) ^ 1u));
            if (!ok) break;
            if (values && lane == 0) groups[stage] = on;
            mbar_arrive_expect_tx_lead(lane == 0 ? 1u : 0u, wait.bar(C::bRF + v + stage), (uint32_t)__popc(on) * 16u * D);
            __syncwarp();
            bulk_g2s_lead(row >= 0 ? 1u : 0u, base + C::kRaw + (uint32_t)(v + stage) * C::kRawBytes + (uint32_t)lane * 16u * D,
                          codes + row * D, 16u * D, wait.bar(C::bRF + v + stage));
        }
    }
    // nothing may be on its way into a tile when the CTA ends
    for (uint32_t s = 0; s < 2; ++s)
        if (it > s) mbar_wait_drain(wait.bar(C::bRF + v + (int)s), ((it - 1 - s) >> 1) & 1u);
}

// Widens the codes of K tiles (four warps, 32 keys each) or V tiles (four more).  Lane: 16 codes of a row, two
// swizzle pieces of fp16; D / 16 lanes to a row.  Rows of V that are no key, or have a NaN code, become 0:
// a weight of 0 must leave nothing of them.
template <int D, int kRows, bool kInt8>
__device__ __forceinline__ void widen_role(const Waiter &wait, bool values, int warp, int lane, uint8_t *smem) {
    using C = Cfg<D, kRows>;
    constexpr int kRowLanes = D / 16, kAtOnce = 32 / kRowLanes, kSteps = 32 / kAtOnce;
    const int v = values ? 2 : 0, col = lane % kRowLanes, sub_row = lane / kRowLanes;
    Stat *st = reinterpret_cast<Stat *>(smem + C::kStat);
    const uint32_t *groups = st->groups;
    // Eight lanes store 128 bytes at a time; where they share a row, half of them begin with their second
    // piece: every bank once.
    const bool swap = D == 128 && col >= 4;
    const int first = 2 * (col & 3) + (swap ? 1 : 0), second = first ^ 1;
    const uint32_t dst = (values ? C::kV : C::kK) + (uint32_t)(col >> 2) * kSub + (uint32_t)(warp * 32 + sub_row) * 128u;
    uint32_t descs = 0, it = 0;
    SegDesc d;
    while (next_desc<C>(wait, smem, descs, d)) {
        for (int k = d.k0; k < d.k1; ++k, ++it) {
            const uint32_t stage = it & 1u;
            const bool ok = values ? wait(C::bVE + (int)stage, (it >> 1) ^ 1u) : wait(C::bKE, it ^ 1u);
            if (!__all_sync(0xffffffffu, ok && wait(C::bRF + v + (int)stage, it >> 1))) return;
            const uint8_t *raw = smem + C::kRaw + (uint32_t)(v + (int)stage) * C::kRawBytes + (warp * 32 + sub_row) * D + col * 16;
            uint8_t *tile = smem + dst + (values ? stage * C::kTileBytes : 0u);
            const uint32_t on = values ? groups[stage] >> (2 * warp) : 3u;
            const int left = d.n - tile_of(d, k) * kTile - warp * 32;
            uint32_t odd = 0;                        // rows that have a NaN code
#pragma unroll 2
            for (int i = 0; i < kSteps; ++i) {
                const int r = i * kAtOnce + sub_row;
                uint4 x = *reinterpret_cast<const uint4 *>(raw + i * kAtOnce * D);
                if (values) {
                    bool none = r >= left || !((on >> (r >> 4)) & 1u);
                    if (!kInt8) {
                        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
                        uint32_t nan = 0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) nan |= ((y[q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        const uint32_t b = __ballot_sync(0xffffffffu, nan != 0u);
                        // one bit per row of the step
#pragma unroll
                        for (int q = 0; q < kAtOnce; ++q)
                            if ((b >> (q * kRowLanes)) & ((1u << kRowLanes) - 1u)) odd |= 1u << (i * kAtOnce + q);
                        none |= ((odd >> r) & 1u) != 0u;
                    }
                    if (none) x = make_uint4(0, 0, 0, 0);
                }
                const uint32_t y[4] = {swap ? x.z : x.x, swap ? x.w : x.y, swap ? x.x : x.z, swap ? x.y : x.w};
                const int r7 = r & 7;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t o[4];
                    codes_to_f16x2<kInt8>(y[2 * q], o[0], o[1]);
                    codes_to_f16x2<kInt8>(y[2 * q + 1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(tile + i * kAtOnce * 128 + (((q ? second : first) ^ r7) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (!kInt8 && values && lane == 0) st->odd[stage][warp] = odd;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(wait.bar(values ? C::bVF + (int)stage : C::bKF));
                mbar_arrive(wait.bar(C::bRE + v + (int)stage));
            }
        }
    }
}

template <int D, int kRows, bool kInt8>
__global__ void __launch_bounds__(kThreads, 1)
    bsattn_prefill_rows_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ Layout w) {
    using C = Cfg<D, kRows>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {  // the swizzle counts from 1024-byte boundaries
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, BSATTN_FLAG_TIMEOUT);
        return;
    }
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    const uint32_t warp = warp_id(), lane = lane_id();
    Waiter wait;
    wait.bars = base + C::kBar;
    wait.abort = reinterpret_cast<volatile int *>(misc + 1);
    wait.err = p.err;
    if (threadIdx.x == 0) {
        mbar_init(wait.bar(C::bKF), 4);          // one arrival per widening warp
        mbar_init(wait.bar(C::bKE), 1);
        mbar_init(wait.bar(C::bQF), 8);          // one per warp of the groups
        for (int s = 0; s < 2; ++s) {
            mbar_init(wait.bar(C::bVF + s), 4);
            mbar_init(wait.bar(C::bVE + s), 1);
            mbar_init(wait.bar(C::bSR + s), 1);
            mbar_init(wait.bar(C::bPR + s), 4);
            mbar_init(wait.bar(C::bOD + s), 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(wait.bar(C::bRF + s), 1);  // the fetching warp's arrival and the bytes
            mbar_init(wait.bar(C::bRE + s), 4);
        }
        for (int s = 0; s < kDescs; ++s) {
            mbar_init(wait.bar(C::bUF + s), 1);
            mbar_init(wait.bar(C::bUE + s), 19); // issuing, fetching, group and widening warps
        }
        mbar_init(wait.bar(C::bDrain), 1);
        misc[1] = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (threadIdx.x < 64) reinterpret_cast<Stat *>(smem + C::kStat)->zero[threadIdx.x] = 0.f;
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
        find_piece<C>(p, w, smem);
        __syncthreads();
    }
    if (warp == 0) {
        regs_release<kCtrlRegs>();
        // ---------------------------------------------------- MMA issuer --
        // The whole warp runs in step; lane 0 issues.
        const uint32_t lead = lane == 0 ? 1u : 0u;
        // kind::f16, fp16 A and B, fp32 D; M = 128; N below
        constexpr uint32_t idesc_s = (1u << 4) | (static_cast<uint32_t>(128 >> 4) << 24);
        constexpr uint32_t idesc_o = idesc_s | (1u << 15) | (1u << 16);   // A and B MN-major
        const uint64_t desc_q = smem_desc_sw128(base + C::kQ, 16, 1024);
        const uint64_t desc_k = smem_desc_sw128(base + C::kK, 16, 1024);
        const uint64_t desc_v = smem_desc_sw128(base + C::kV, kSub, 1024);
        const uint64_t desc_p = smem_desc_sw128(base + C::kP, kSub, 1024);
        constexpr uint64_t kTileUnits = C::kTileBytes >> 4, kSubUnits = kSub >> 4;
        uint32_t descs = 0, tile0 = 0, segs = 0, pc[2] = {0, 0};
        bool ok = true;
        auto ready = [&](int b, uint32_t phase) -> bool {
            ok = ok && wait(b, phase);
            return ok;
        };
        SegDesc d;
        while (ok && next_desc<C>(wait, smem, descs, d)) {
            const int rows = d.tokens * p.G, n = d.k1 - d.k0;
            const bool turns = kRows <= 64 || rows <= 64;
            const uint32_t cols[2] = {(uint32_t)(min(rows, 64) + 15) & ~15u, (uint32_t)((turns ? rows : rows - 64) + 15) & ~15u};
            auto score = [&](int g) {
                const uint64_t qd = desc_q + (turns ? 0u : (uint64_t)g * (64 * 128 >> 4));
                const uint32_t idesc = idesc_s | ((cols[g] >> 3) << 17);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = (uint64_t)((kk >> 2) * kSubUnits + (kk & 3) * 2);
                    mma_ss_lead(lead, tmem + g * 64, desc_k + off, qd + off, idesc, kk > 0 ? 1u : 0u);
                }
                mma_commit_lead(lead, wait.bar(C::bSR + g));
            };
            auto output = [&](int g, uint32_t it, bool first) -> bool {
                if (!ready(C::bVF + (int)(it & 1u), it >> 1) || !ready(C::bPR + g, pc[g])) return false;
                ++pc[g];
                tc_fence_after();
                const uint64_t vd = desc_v + (uint64_t)(it & 1u) * kTileUnits, pd = desc_p + (uint64_t)g * kSubUnits;
                const uint32_t idesc = idesc_o | ((cols[g] >> 3) << 17);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    mma_ss_lead(lead, tmem + 128 + g * 64, vd + (uint64_t)(kk * (2048 >> 4)),
                                pd + (uint64_t)(kk * (2048 >> 4)), idesc, kk > 0 || !first ? 1u : 0u);
                return true;
            };
            if (!ready(C::bQF, segs)) break;
            ++segs;
            tc_fence_after();
            for (int k = 0; ok && k < n; ++k) {
                const uint32_t it = tile0 + (uint32_t)k;
                if (!ready(C::bKF, it)) break;
                tc_fence_after();
                if (turns) {
                    const int g = k & 1;
                    if (k >= 2) {
                        if (!output(g, it - 2, k < 4)) break;
                        mma_commit_lead(lead, wait.bar(C::bVE + (int)(it & 1u)));
                    }
                    score(g);
                } else {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (k > 0 && !output(g, it - 1, k == 1)) break;
                        score(g);
                    }
                    if (!ok) break;
                    if (k > 0) mma_commit_lead(lead, wait.bar(C::bVE + (int)((it - 1) & 1u)));
                }
                mma_commit_lead(lead, wait.bar(C::bKE));
            }
            if (!ok) break;
            const uint32_t last = tile0 + (uint32_t)n - 1;
            if (turns) {
                for (int k = max(n - 2, 0); k < n; ++k) {
                    const uint32_t it = tile0 + (uint32_t)k;
                    if (!output(k & 1, it, k < 2)) break;
                    mma_commit_lead(lead, wait.bar(C::bVE + (int)(it & 1u)));
                    mma_commit_lead(lead, wait.bar(C::bOD + (k & 1)));
                }
            } else if (n > 0) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (!output(g, last, n == 1)) break;
                    mma_commit_lead(lead, wait.bar(C::bOD + g));
                }
                if (ok) mma_commit_lead(lead, wait.bar(C::bVE + (int)(last & 1u)));
            }
            tile0 += (uint32_t)n;
        }
        // Wait until every tcgen05 operation issued above has completed.
        mma_commit_lead(lead, wait.bar(C::bDrain));
        mbar_wait_drain(wait.bar(C::bDrain), 0);
    } else if (warp < 4) {
        regs_release<kCtrlRegs>();
        if (warp == 1) {
            Start from;
            if (alone) {
                from = find_piece_warp(p, w, (int)lane);
            } else {
                const Stat *st = reinterpret_cast<const Stat *>(smem + C::kStat);
                from.b = st->b, from.h = st->h, from.r = st->r, from.pieces = st->pieces, from.begin = st->begin, from.line = st->line;
                if (from.b < p.B) from.c = chunk_of(p, from.b, false);
            }
            if (lane == 0) segment_role<C>(p, w, wait, smem, from);
            __syncwarp();
        } else {
            fetch_role<D, kRows>(p, wait, warp == 3, (int)lane, base, smem);
        }
    } else if (warp < 12) {
        regs_claim<kGroupRegs>();
        group_role<D, kRows, kInt8>(p, w, wait, tmem, warp >= 8 ? 1 : 0, warp, lane, smem);
    } else {
        regs_release<kWidenRegs>();
        widen_role<D, kRows, kInt8>(wait, warp >= 16, (int)(warp & 3u), (int)lane, smem);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, int kRows, bool kInt8>
cudaError_t launch(const ChunkParams &p, const Layout &w, cudaStream_t stream) {
    using C = Cfg<D, kRows>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set_for_device[dev]) {
        // the register split inside the kernel assumes exactly kLaunchRegs per thread at launch
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, bsattn_prefill_rows_kernel<D, kRows, kInt8>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(bsattn_prefill_rows_kernel<D, kRows, kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kAlloc);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    void *args[] = {const_cast<ChunkParams *>(&p), const_cast<Layout *>(&w)};
    return launch_dependent(reinterpret_cast<const void *>(bsattn_prefill_rows_kernel<D, kRows, kInt8>), dim3((unsigned)w.ctas), kThreads,
                            C::kAlloc, args, stream);
}

template <int D, bool kInt8>
cudaError_t launch_of(const ChunkParams &p, const Layout &w, cudaStream_t stream) {
    switch (w.few) {
    case 16: return launch<D, 16, kInt8>(p, w, stream);
    case 32: return launch<D, 32, kInt8>(p, w, stream);
    case 64: return launch<D, 64, kInt8>(p, w, stream);
    default: return launch<D, 128, kInt8>(p, w, stream);
    }
}

}  // namespace

cudaError_t launch_prefill_rows(const ChunkParams &p, const Layout &w, cudaStream_t stream) {
    if (p.c.D == 128) return p.c.int8 ? launch_of<128, true>(p, w, stream) : launch_of<128, false>(p, w, stream);
    return p.c.int8 ? launch_of<64, true>(p, w, stream) : launch_of<64, false>(p, w, stream);
}

}  // namespace bsattn
