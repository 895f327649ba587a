// Attention of chunks of new tokens over a paged 8-bit K/V cache: four launches.
//
// Of a KV head's queries, (token, query head) pairs are rows of one attention over the
// sequence's keys: 4 D flop per row and key, so that from some hundred rows on the products bound
// it.  The codes are widened once per call, into the workspace, and the attention reads tiles that
// lie there as its shared memory wants them (bulk copies, no tensor map):
//   K' = bf16(code 2^e), exact: e the binary exponent of the key's scale; what is left of the
//        scale, r in [1, 2), multiplies the key's scores in fp32, and only in tiles where some
//        r != 1 (int8; the scales that e4m3 rows are given are powers of two);
//   V' = fp16(code vs 2^(6 - E)), E (a multiple of 4) the largest binary exponent of the tile's value
//        scales vs: exact where vs is a power of two (e4m3), else rounded to 11 bits (a value 2^28 below
//        the tile's largest may count as 0).
// With z_j the scores in units of log2: p_j = 2^(z_j - m + 7) is rounded to fp16 (11 bits) for P V',
// l sums it in fp32; out = O 2^(E - 6) / l, lse = ln 2 (m - 7 + log2 l).  The reference m is moved
// only when some weight could pass 2^15 (the output is then rescaled), and O is rescaled to
// another E only where it is larger or more than 2^8 smaller, then no further than O stays below 2^100.
//
// Work.  A segment is (sequence, KV head, block of 2 x floor(128 / G) tokens): two 128-row
// tiles ("slots") that share each K/V tile.  It visits the key tiles that its rows meet: all up to
// its last position, or the sink tiles and those from the window's first on.  A plan kernel numbers
// the tiles of all segments along one line (each segment also counts kSegCost places for what
// starting and ending one costs), which is cut into equal pieces, so many per CTA that the keys
// of those which the CTAs work on at a time fit L2.  What a piece
// computes of a segment that it does not hold whole goes to the workspace (fp32 output and LSE);
// the last launch joins these parts in a fixed order.
//
// Measured (us a call, cold L2; of it the plan 8, widening 27 to 83, the join 13 to 48; products at 1955 TFLOP/s in
// brackets): 2048 tokens on 63488 keys, 8 heads x 4, int8, D = 128: 1720 (1072), 1.22 PFLOP/s; 4096 tokens, window of 4096
// behind 512 sinks, 32 heads, e4m3: 340 (158); prompts of 100 to 4096 tokens, 16 heads, e4m3, D = 64: 218 (53); 16
// sequences with 1 to 512 new tokens, 8 heads x 4, int8: 245 (75).  Within a segment the chain of one tile's softmax
// bounds it, 3600 cycles of which 2048 are the products'; short segments add some 10000 cycles each for their
// description, query rows, output and the slots' unequal tiles.
//
// Roles of the attention kernel (384 threads, one CTA per SM, all of TMEM):
//   warp 0      copies: query tiles (TMA), K and V tiles with their scales (bulk)
//   warp 1      issues the MMAs: S_t = Q_t K'^T into TMEM, O_t += P_t V' with P in TMEM
//   warp 2      owns the TMEM allocation
//   warp 3      finds the segments of the CTA's pieces, one ahead of the others
//   warps 4-7, 8-11   slot 0, slot 1: softmax, O rescale, output
// TMEM: S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D,256+2D); P_t over S_t.
#include "prefill_plan.cuh"
#include "kv_codes.cuh"

namespace bsattn {

namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
// 168 registers per thread at launch: 128 * 120 + 2 * 128 * 192 = 64512 = 384 * 168.
constexpr int kLaunchRegs = 168;
constexpr uint32_t kCtrlRegs = 120, kSoftmaxRegs = 192;
static_assert(128 * kCtrlRegs + 2 * 128 * kSoftmaxRegs <= (uint32_t)kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr uint32_t kSub = kTile * 64 * 2;   // 128 rows x 64 elements: one 128-byte swizzle span
constexpr int kPlanThreads = 1024, kWidenThreads = 256, kJoinThreads = 256;

// Binary exponents (biased) that go into K' (what lies outside stays in r), and those that E is taken from
// (2^(E - 6) and its inverse are then normal numbers).
constexpr int kLeastKey = 27, kMostKey = 227, kLeastValue = 7, kMostValue = 254, kLeastExp = (kLeastValue + 3) & ~3;
constexpr float kLift = 7.f, kReach = 8.f;
// Binary exponent below which O stays where another E moves it up: 2^24 tiles of 2^38 each may still be added.
constexpr int kMostO = 100;

// ------------------------------------------------------------------- plan --

// Sum over the block's threads before this one; *all: over all of them.
__device__ __forceinline__ long long block_scan(long long x, long long *all, long long *warps) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    long long s = x;
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    long long before = 0, sum = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += warps[w];
        sum += warps[w];
    }
    *all = sum;
    return before + s - x;
}

__global__ void __launch_bounds__(kPlanThreads) bsattn_prefill_plan_kernel(const __grid_constant__ ChunkParams p,
                                                                           const __grid_constant__ Layout w) {
    __shared__ long long warps[kPlanThreads / 32];
    grid_launch_dependents();
    grid_dependency_wait();
    SeqPlan *seq = reinterpret_cast<SeqPlan *>(p.ws + w.seq);
    int32_t *place = reinterpret_cast<int32_t *>(p.ws + w.block_place);
    const int step = w.step, tid = threadIdx.x, lane = tid % 32;
    long long tiles = 0, blocks = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        SeqPlan s = {};
        if (b < p.B) {
            const Chunk c = chunk_of(p, b, true);
            s.first = c.first, s.m = c.m, s.n = c.n;
            s.blocks = (c.m + step - 1) / step;
            if (c.m > 0 && c.n > 0) {
                const Visit v = visit(p, c.n, c.n - c.m, c.n - 1);
                s.sinks = v.sinks, s.near = v.near, s.end = v.end;
            }
        }
        long long sum;
        s.tile0 = (int)min(tiles + block_scan(s.sinks + s.end - s.near, &sum, warps), (long long)INT32_MAX);
        if (s.m > 0 && (long long)s.tile0 + s.sinks + s.end - s.near > w.tiles) {
            // no room for its keys
            if (p.err) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
            s.m = s.blocks = s.sinks = s.near = s.end = 0;
        }
        tiles += sum;
        const long long block0 = blocks + block_scan(s.blocks, &sum, warps);
        s.block0 = (int)min(block0, (long long)INT32_MAX);
        if (s.blocks > 0 && block0 + s.blocks > w.blocks) {
            // offsets that decrease in between: more rows than there are
            if (p.err) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
            s.m = s.blocks = s.sinks = s.near = s.end = 0;
        }
        blocks += sum;
        if (b < p.B) seq[b] = s;
    }
    __syncthreads();
    // places of the row blocks within a head's pass over them: a warp per sequence
    for (int b = tid / 32; b < p.B; b += kPlanThreads / 32) {
        const SeqPlan s = seq[b];
        long long sum = 0;
        for (int r0 = 0; r0 < s.blocks; r0 += 32) {
            const int r = r0 + lane;
            int x = 0;
            if (r < s.blocks) {
                x = kSegCost;
                if (s.n > 0) x += visit(p, s.n, s.n - s.m + r * step, s.n - s.m + min((r + 1) * step, s.m) - 1).count();
            }
            int y = x;
            for (int d = 1; d < 32; d <<= 1) {
                const int z = __shfl_up_sync(0xffffffffu, y, d);
                if (lane >= d) y += z;
            }
            if (r < s.blocks) place[s.block0 + r] = (int)min(sum + y - x, (long long)INT32_MAX);
            sum += __shfl_sync(0xffffffffu, y, 31);
        }
        if (lane == 0 && sum > INT32_MAX) {
            // a head's pass is numbered in 32 bits
            if (p.err) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
            seq[b].m = seq[b].blocks = 0;
            sum = 0;
        }
        if (lane == 0) seq[b].pass = (int)sum;
    }
    __syncthreads();
    long long places = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        long long sum;
        const long long before = block_scan(b < p.B ? (long long)seq[b].pass * p.c.H : 0, &sum, warps);
        if (b < p.B) seq[b].base = places + before;
        places += sum;
    }
    if (tid == 0) {
        PlanTotals t = {};
        t.places = places;
        t.tiles = (int)min(tiles, w.tiles);
        // Phases only where tiles are visited so often that reading them again from HBM would bound the call: a
        // prompt's chunk of 2048 tokens x 4 heads behind 61440 (32 visits a tile) takes 1716 us with phases of 64 MB, 1778
        // with one; 16 ragged chunks (4 visits) 269 and 240, a window of 4096 (9 visits) 366 and 329 us: each phase has
        // parts to be joined.
        const long long phases = places < kPhaseVisits * t.tiles * p.c.H ? 1 : (t.tiles * (long long)p.c.H * (kTile * 4 * p.c.D) + kPhaseBytes - 1) / kPhaseBytes;
        t.pieces = (int)max(1ll, min(min((long long)w.pieces, w.ctas * max(phases, 1ll)), places / kLeastPiece));
        *reinterpret_cast<PlanTotals *>(p.ws + w.totals) = t;
    }
}

// ------------------------------------------------------------------ widen --

// One tile of one head per turn: rows of K and V in pieces of 16 codes, D / 16 lanes to a row.
template <int D, bool kInt8>
__global__ void __launch_bounds__(kWidenThreads) bsattn_prefill_widen_kernel(const __grid_constant__ ChunkParams p,
                                                                             const __grid_constant__ Layout w) {
    constexpr int kRowLanes = D / 16, kRows = kWidenThreads / kRowLanes, kSteps = kTile / kRows;
    __shared__ int s_row[kTile];                 // cache row of each key, -1: none
    __shared__ float s_k[kTile];                 // 2^e
    __shared__ float s_v[kTile];                 // vs 2^(6 - E)
    __shared__ int s_top[4];
    __shared__ uint32_t s_keep[4], s_rest[4], s_odd[4];
    __shared__ int s_nan[kTile];                 // the key's value is not a number
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const SeqPlan *seq = reinterpret_cast<const SeqPlan *>(p.ws + w.seq);
    grid_launch_dependents();
    grid_dependency_wait();
    const long long items = (long long)reinterpret_cast<const PlanTotals *>(p.ws + w.totals)->tiles * p.c.H;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int slot = (int)(it / p.c.H), h = (int)(it - (long long)slot * p.c.H);
        // the last sequence whose tiles begin at or before this one
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (seq[mid].tile0 <= slot) lo = mid;
            else hi = mid - 1;
        }
        const SeqPlan s = seq[lo];
        int tile = slot - s.tile0;
        if (tile >= s.sinks) tile += s.near - s.sinks;
        if (tile >= s.end) continue;             // a sequence that has no room
        __syncthreads();
        float ks = 1.f, vs = 1.f;
        int f = 0;
        if (tid < kTile) {
            const int j = tile * kTile + tid;
            const long long row = j < s.n ? cache_row(p.c, p.table + (long long)lo * p.table_stride, h, j) : -1;
            if (j < s.n && row < 0 && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
            if (row >= 0) ks = p.c.ks[row], vs = p.c.vs[row];
            s_row[tid] = (int)row;
            const uint32_t kb = __float_as_uint(ks) & 0x7fffffffu, vb = __float_as_uint(vs) & 0x7fffffffu;
            const int e = kb < 0x7f800000u ? min(max((int)(kb >> 23), kLeastKey), kMostKey) : 127;
            s_k[tid] = pow2(e - 127);
            ks *= pow2(127 - e);
            const bool number = vb < 0x7f800000u;
            // rows of zeros have the smallest scale; they, NaN and infinity do not count for E
            f = row >= 0 && number && vb > 1u << 23 ? min(max((int)(vb >> 23), kLeastValue), kMostValue) : 0;
            s_nan[tid] = number ? 0 : 1;
            const int top = __reduce_max_sync(0xffffffffu, max(f, kLeastValue));
            if (lane == 0) s_top[warp] = top;
            const uint32_t keep = __ballot_sync(0xffffffffu, row >= 0);
            if (lane == 0) s_keep[warp] = keep;
        }
        __syncthreads();
        const int exp = (max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3])) + 3) & ~3;   // kLeastExp: maybe no value at all
        if (tid < kTile) s_v[tid] = vs * pow2(133 - exp);
        const long long at = (long long)h * w.tiles + slot;
        TileHead *head = reinterpret_cast<TileHead *>(p.ws + w.head) + at;
        const int piece = tid % kRowLanes, sub = tid / kRowLanes;
        uint4 x[2][kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const long long row = s_row[i * kRows + sub];
            x[0][i] = x[1][i] = make_uint4(0, 0, 0, 0);
            if (row >= 0) {
                x[0][i] = __ldg(reinterpret_cast<const uint4 *>(p.c.k + row * D) + piece);
                x[1][i] = __ldg(reinterpret_cast<const uint4 *>(p.c.v + row * D) + piece);
            }
        }
        if (!kInt8) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const uint32_t y[4] = {x[1][i].x, x[1][i].y, x[1][i].z, x[1][i].w};
                uint32_t nan = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) nan |= ((y[q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                if (nan) s_nan[i * kRows + sub] = 1;
            }
        }
        __syncthreads();
        bool none = false;                       // no value that is not 0
        if (exp <= kLeastExp) {
            uint32_t some = 0;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int r = i * kRows + sub;
                if (s_v[r] != 0.f && s_nan[r] == 0) some |= (x[1][i].x | x[1][i].y | x[1][i].z | x[1][i].w) & (kInt8 ? 0xffffffffu : 0x7f7f7f7fu);
            }
            none = !__syncthreads_or(some != 0u);
        }
        if (tid < kTile) {
            const bool odd = s_nan[tid] != 0;
            head->r[tid] = ks;
            const uint32_t rest = __any_sync(0xffffffffu, ks != 1.f) ? kRest : 0u;
            const uint32_t odds = __ballot_sync(0xffffffffu, odd);
            if (lane == 0) s_rest[warp] = rest | (odds ? kOdd : 0u), s_odd[warp] = odds;
        }
        __syncthreads();
        if (tid == 0) {
            *reinterpret_cast<uint4 *>(head->keep) = make_uint4(s_keep[0], s_keep[1], s_keep[2], s_keep[3]);
            *reinterpret_cast<uint4 *>(head->odd) = make_uint4(s_odd[0], s_odd[1], s_odd[2], s_odd[3]);
            head->exp = none ? 0 : exp;
            head->flags = s_rest[0] | s_rest[1] | s_rest[2] | s_rest[3];
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = i * kRows + sub;
            const bool nan = s_nan[r] != 0;
            const float kf = s_k[r], vf = nan ? 0.f : s_v[r];
            if (nan) x[1][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int values = 0; values < 2; ++values) {
                const uint32_t y[4] = {x[values][i].x, x[values][i].y, x[values][i].z, x[values][i].w};
                uint32_t o[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t c2[2];
                    codes_to_f16x2<kInt8>(y[q], c2[0], c2[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float a, c;
                        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
                            : "=f"(a), "=f"(c)
                            : "r"(c2[k]));
                        const float f32 = values ? vf : kf;
                        o[2 * q + k] = values ? pack_f16x2(a * f32, c * f32) : pack_bf16x2(a * f32, c * f32);
                    }
                }
                uint8_t *dst = p.ws + (values ? w.v : w.k) + at * (kTile * D * 2) + (size_t)(piece >> 2) * kSub + r * 128;
                const int c0 = 2 * (piece & 3);
                *reinterpret_cast<uint4 *>(dst + ((c0 ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4 *>(dst + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

// -------------------------------------------------------------- attention --

template <int D>
struct Cfg {
    static constexpr uint32_t kTileBytes = kTile * D * 2;
    static constexpr uint32_t kQ = 0, kK = kQ + 2 * kTileBytes, kV = kK + 2 * kTileBytes;
    static constexpr uint32_t kHead = kV + 2 * kTileBytes;
    static constexpr uint32_t kDesc = kHead + 2 * (uint32_t)sizeof(TileHead);
    static constexpr uint32_t kBar = kDesc + kDescs * (uint32_t)sizeof(SegDesc);
    // K / V stage full and empty, per slot: query tile full and empty, S ready, two halves of P
    // ready, O complete; descriptor full and empty
    static constexpr int bKF = 0, bKE = 2, bVF = 4, bVE = 6, bQF = 8, bQE = 10, bSR = 12, bPR = 14, bOD = 18, bUF = 20,
                         bUE = bUF + kDescs, bDrain = bUE + kDescs, kNumBars = bDrain + 1;
    static constexpr uint32_t kMisc = kBar + kNumBars * 8;                     // [0] tmem base, [1] abort
    static constexpr uint32_t kBytes = kMisc + 16;
    static constexpr uint32_t kAlloc = kBytes + 1024;                          // slack for 1024-byte alignment
    static_assert(kAlloc <= 227u * 1024u, "shared memory");
};

// 32 bytes; `whole`: the address is a multiple of 32.
__device__ __forceinline__ void store32(uint8_t *dst, const uint32_t *v, bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// One slot: warps 4-7 (t = 0) or 8-11 (t = 1), one row per thread.
template <int D, bool kInt8>
__device__ __forceinline__ void softmax_role(const ChunkParams &p, const Layout &w, const Waiter &wait, uint32_t tmem,
                                             int t, uint32_t warp, uint32_t lane, uint8_t *smem) {
    using C = Cfg<D>;
    const uint32_t quarter = warp & 3u;
    const int row = (int)(quarter * 32 + lane), token_of = row / p.G, head_of = row - token_of * p.G;
    const uint32_t lane_addr = tmem + ((quarter * 32u) << 16);
    const uint32_t s_col = (uint32_t)t * 128u, o_col = 256u + (uint32_t)t * D;
    const float sl2 = p.scale_log2;
    uint32_t descs = 0, sc = 0, od = 0, tile0 = 0;   // descriptors; phases of S and O; tiles of earlier segments
    bool ok = true;
    SegDesc d;
    while (ok && next_desc<C>(wait, smem, descs, d)) {
        const int tok = t * w.tokens + token_of;     // of the segment
        const bool row_ok = token_of < w.tokens && tok < d.tokens;
        const int end = min(d.k1, d.count[t]);
        // keys that the row meets: below hb, or from la to ha - 1
        const Met own = d.n > 0 ? met(p, d.pos + min(tok, d.tokens - 1), d.n) : Met{0, 0, 0};
        // what every row of the slot meets: the first row's end, the last one's window
        const int slot_first = d.pos + min(t * w.tokens, d.tokens - 1), slot_last = d.pos + min((t + 1) * w.tokens, d.tokens) - 1;
        const Met low = met(p, slot_first, d.n), high = met(p, slot_last, d.n);
        float m_run = kNoKey, l_run = 0.f;
        int exp_run = 0;
        bool nan = false;                            // the row meets a value that is not a number
        for (int k = d.k0; k < end; ++k) {
            const uint32_t it = tile0 + (uint32_t)(k - d.k0), st = it & 1u;
            // S first: a slot that left tiles out may be more than a phase ahead of the V stages, of which S
            // says that they have come to this tile
            ok = wait(C::bSR + t, sc) && wait(C::bVF + (int)st, it >> 1);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            ++sc;
            tc_fence_after();
            const TileHead *head = reinterpret_cast<const TileHead *>(smem + C::kHead) + st;
            const int4 info = *reinterpret_cast<const int4 *>(&head->exp);
            const uint4 kw = *reinterpret_cast<const uint4 *>(head->keep);
            const int j0 = (k < d.sinks ? k : k - d.sinks + d.near) * kTile;
            const bool rest = ((uint32_t)info.y & kRest) != 0;
            // a tile that every row of the slot meets whole needs no mask
            const bool masked = (kw.x & kw.y & kw.z & kw.w) != 0xffffffffu || j0 + kTile > low.ha ||
                                (high.la > j0 && high.hb < j0 + kTile);
            const bool plain = !rest && !masked;
            // columns of 32 g .. that the row meets
            auto meets = [&](int g) -> uint32_t {
                const int c = j0 + 32 * g;
                return span_bits(own.la - c, own.ha - c) | span_bits(0, own.hb - c);
            };
            float top = -INFINITY, s[kInt8 ? 128 : 1], hm[4];
            // 32 scores of columns 32 g .. times r, -inf where the row does not meet the key
            auto scores = [&](int g, float (&y)[32]) {
                uint32_t v[32];
                tmem_ld32(lane_addr + s_col + 32u * g, v);
                tmem_wait_ld();
                reg_fence(v);
                if (rest) {
                    const float4 *r = reinterpret_cast<const float4 *>(head->r) + 8 * g;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const float4 f = r[x];
                        fmul2(y[4 * x], y[4 * x + 1], __uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1]), f.x, f.y);
                        fmul2(y[4 * x + 2], y[4 * x + 3], __uint_as_float(v[4 * x + 2]), __uint_as_float(v[4 * x + 3]), f.z, f.w);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) y[x] = __uint_as_float(v[x]);
                }
                if (masked) {
                    const uint32_t bits = (g == 0 ? kw.x : g == 1 ? kw.y : g == 2 ? kw.z : kw.w) & meets(g);
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (!((bits >> x) & 1u)) y[x] = -INFINITY;
                }
            };
            if constexpr (kInt8) {
                // Almost every tile's scores take factors: they stay in registers between the passes.
                {
                    uint32_t v0[32], v1[32], v2[32], v3[32];
                    tmem_ld32_max(lane_addr + s_col + 0, v0, hm[0]);
                    tmem_ld32_max(lane_addr + s_col + 32, v1, hm[1]);
                    tmem_ld32_max(lane_addr + s_col + 64, v2, hm[2]);
                    tmem_ld32_max(lane_addr + s_col + 96, v3, hm[3]);
                    tmem_wait_ld();
                    reg_fence(v0), reg_fence(v1), reg_fence(v2), reg_fence(v3);
#pragma unroll
                    for (int x = 0; x < 4; ++x) reg_fence(hm[x]);
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        s[x] = __uint_as_float(v0[x]);
                        s[32 + x] = __uint_as_float(v1[x]);
                        s[64 + x] = __uint_as_float(v2[x]);
                        s[96 + x] = __uint_as_float(v3[x]);
                    }
                }
                auto group_max = [&](int g) {
                    float a = fmax3(s[32 * g], s[32 * g + 1], s[32 * g + 2]);
#pragma unroll
                    for (int x = 3; x < 31; x += 2) a = fmax3(a, s[32 * g + x], s[32 * g + x + 1]);
                    hm[g] = fmaxf(a, s[32 * g + 31]);
                };
                if (rest) {
                    const float4 *r = reinterpret_cast<const float4 *>(head->r);
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        const float4 f = r[x];
                        fmul2(s[4 * x], s[4 * x + 1], s[4 * x], s[4 * x + 1], f.x, f.y);
                        fmul2(s[4 * x + 2], s[4 * x + 3], s[4 * x + 2], s[4 * x + 3], f.z, f.w);
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) group_max(g);
                }
                if (masked) {
                    const uint32_t keep[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint32_t bits = keep[g] & meets(g);
                        if (bits == 0xffffffffu) continue;
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (!((bits >> x) & 1u)) s[32 * g + x] = -INFINITY;
                        group_max(g);
                    }
                }
                top = fmax3(hm[0], hm[1], fmaxf(hm[2], hm[3]));
            } else {
                // First pass, the maximum: the load's own reduction where scores need no factor and no mask.  The loops of
                // the passes are small (the roles share the instruction caches).
                if (plain) {
                    float hm[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t v[32];
                        tmem_ld32_max(lane_addr + s_col + 32u * g, v, hm[g]);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < 4; ++g) reg_fence(hm[g]);
                    top = fmax3(hm[0], hm[1], fmaxf(hm[2], hm[3]));
                } else {
#pragma unroll 1
                    for (int g = 0; g < 4; ++g) {
                        float y[32];
                        scores(g, y);
                        float t0 = fmax3(y[0], y[1], y[2]), t1 = fmax3(y[3], y[4], y[5]);
#pragma unroll
                        for (int x = 6; x < 30; x += 4) {
                            t0 = fmax3(t0, y[x], y[x + 1]);
                            t1 = fmax3(t1, y[x + 2], y[x + 3]);
                        }
                        top = fmaxf(top, fmax3(t0, fmaxf(y[30], y[31]), t1));
                    }
                }
            }
            const float m_new = fmaxf(m_run, top * sl2);
            const bool begun = k > d.k0;
            const bool grew = !begun || __any_sync(0xffffffffu, m_new - m_run > kReach);
            float alpha = 1.f;
            if (grew) {
                alpha = ex2_approx(m_run - m_new);
                m_run = m_new;
            }
            // The tile's E (a tile without values: O's) against that of O: a little smaller, and the weights make up for it
            // (unit), else O moves.  Down only as far as O stays below 2^kMostO: where that is not all the way, the
            // tile's values are so far below what O holds that their weights' lost bits are too.
            const int exp = info.x != 0 ? info.x : exp_run;
            float f = alpha, unit = 1.f;
            bool rescale = begun && grew, scaled = false;   // the same for the whole warp
            if (!begun) exp_run = exp;
            if (__builtin_expect(__any_sync(0xffffffffu, exp_run != exp), 0)) {
                const int below = exp_run - exp;
                if (__any_sync(0xffffffffu, below < 0 || below > 8)) {
                    int room = below;
                    if (__any_sync(0xffffffffu, below > 8)) {
                        // S of this tile was issued after the slot's previous P V: O is up to date
                        float top_o = 0.f;
#pragma unroll 1
                        for (int c = 0; c < D / 8; ++c) {
                            uint32_t v[8];
                            tmem_ld8(lane_addr + o_col + 8u * c, v);
                            tmem_wait_ld();
                            reg_fence(v);
#pragma unroll
                            for (int x = 0; x < 8; ++x) top_o = fmaxf(top_o, fabsf(__uint_as_float(v[x])));
                        }
                        top_o *= alpha;
                        // below 2^-27 it counts as 0 beside what weighs most
                        if (!(top_o < 0x1p-27f)) room = max(127 + kMostO - (int)(__float_as_uint(top_o) >> 23), 0);
                    }
                    const int shift = below > 8 ? min(below, room) : min(below, 0);
                    exp_run -= shift;
                    f *= pow2(shift);
                    rescale |= __any_sync(0xffffffffu, shift != 0);
                }
                unit = pow2(exp - exp_run);
                scaled = __any_sync(0xffffffffu, unit != 1.f);
            }
            const float nm = kLift - m_run;
            float la0 = 0.f, la1 = 0.f, lb0 = 0.f, lb1 = 0.f;
            auto rescale_output = [&] {
                if (!rescale) return;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(lane_addr + o_col + c * 32, v);
                    tmem_wait_ld();
                    reg_fence(v);
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * f);
                    tmem_st32(lane_addr + o_col + c * 32, v);
                }
            };
            if (__builtin_expect(((uint32_t)info.y & kOdd) != 0, 0)) {
#pragma unroll 1
                for (int g = 0; g < 4; ++g) nan |= (head->odd[g] & meets(g)) != 0u;
            }
            // Second pass: 32 columns at a time, P over scores that have been read; 64 keys are handed over at a time.
            auto hand_over = [&](int half) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(wait.bar(C::bPR + 2 * t + half));
            };
            auto part = [&](int g, float (&y)[32]) {
#pragma unroll
                for (int x = 0; x < 16; ++x) ffma2(y[2 * x], y[2 * x + 1], y[2 * x], y[2 * x + 1], sl2, sl2, nm, nm);
                uint32_t pk[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    float p0 = ex2_approx(y[2 * x]), p1 = ex2_approx(y[2 * x + 1]);
                    if (x & 1) fadd2(lb0, lb1, lb0, lb1, p0, p1);
                    else fadd2(la0, la1, la0, la1, p0, p1);
                    pk[x] = pack_f16x2(p0, p1);
                }
                if (__builtin_expect(scaled, 0)) {   // by powers of two
                    const uint32_t u2 = pack_f16x2(unit, unit);
#pragma unroll
                    for (int x = 0; x < 16; ++x) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(pk[x]) : "r"(u2));
                }
                tmem_st16(lane_addr + s_col + 16u * g, pk);
            };
            if constexpr (kInt8) {
                auto half = [&](int c) {
                    uint32_t pk[32];
                    if (__builtin_expect(!scaled, 1)) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            float x0, x1;
                            ffma2(x0, x1, s[c * 64 + 2 * x], s[c * 64 + 2 * x + 1], sl2, sl2, nm, nm);
                            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                            if (x & 1) fadd2(lb0, lb1, lb0, lb1, p0, p1);
                            else fadd2(la0, la1, la0, la1, p0, p1);
                            pk[x] = pack_f16x2(p0, p1);
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            const float p0 = ex2_approx(fmaf(s[c * 64 + 2 * x], sl2, nm)), p1 = ex2_approx(fmaf(s[c * 64 + 2 * x + 1], sl2, nm));
                            la0 += p0, la1 += p1;
                            pk[x] = pack_f16x2(p0 * unit, p1 * unit);
                        }
                    }
                    tmem_st32(lane_addr + s_col + c * 32, pk);
                };
                half(0);
                rescale_output();
                hand_over(0);
                half(1);
                hand_over(1);
            } else {
                rescale_output();
                if (plain) {
                    auto plain_part = [&](int g, uint32_t (&v)[32]) {
                        float y[32];
#pragma unroll
                        for (int x = 0; x < 32; ++x) y[x] = __uint_as_float(v[x]);
                        part(g, y);
                    };
                    uint32_t va[32], vb[32];
                    tmem_ld32(lane_addr + s_col, va);
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        tmem_wait_ld();
                        reg_fence(va);
                        tmem_ld32(lane_addr + s_col + 64u * i + 32u, vb);
                        plain_part(2 * i, va);
                        tmem_wait_ld();
                        reg_fence(vb);
                        if (i == 0) tmem_ld32(lane_addr + s_col + 64u, va);
                        plain_part(2 * i + 1, vb);
                        hand_over(i);
                    }
                } else {
#pragma unroll 1
                    for (int g = 0; g < 4; ++g) {
                        float y[32];
                        scores(g, y);
                        part(g, y);
                        if (g & 1) hand_over(g >> 1);
                    }
                }
            }
            l_run = l_run * alpha + ((la0 + lb0) + (la1 + lb1));
        }
        if (!ok) break;
        tile0 += (uint32_t)(d.k1 - d.k0);
        const bool any = end > d.k0;
        if (any) {
            ok = wait(C::bOD + t, od);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            ++od;
            tc_fence_after();
        }
        const bool empty = !any || l_run == 0.f;     // NaN is not empty
        const float inv = empty ? 0.f : nan ? __uint_as_float(0x7fc00000u) : 1.f / l_run;
        const float scale = any ? pow2(exp_run - 127 - 6) : 0.f;
        // Each lane writes its row, whole sectors of 32 bytes at a time.
        const bool part = d.part >= 0;
        const long long out_row = part ? ((long long)d.part * 2 + t) * kTile + row
                                       : (long long)(d.token + tok) * p.Hq + d.h * p.G + head_of;
        const bool half_words = !part && !p.out_f32;
        uint8_t *dst = (part ? p.ws + w.part_o : static_cast<uint8_t *>(p.out)) + out_row * (D * (half_words ? 2 : 4));
        const bool sectors = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            if (any) {
                tmem_ld32(lane_addr + o_col + c * 32, v);
                tmem_wait_ld();
                reg_fence(v);
            }
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = empty ? 0u : __float_as_uint(__uint_as_float(v[x]) * inv * scale);
            if (row_ok && half_words) {
#pragma unroll
                for (int x = 0; x < 16; ++x) v[x] = pack_bf16x2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1]));
                store32(dst + c * 64, v, sectors);
                store32(dst + c * 64 + 32, v + 8, sectors);
            } else if (row_ok) {
#pragma unroll
                for (int x = 0; x < 4; ++x) store32(dst + c * 128 + 32 * x, v + 8 * x, sectors);
            }
            __syncwarp();
        }
        if (row_ok) {
            const float lse2 = empty ? -INFINITY : m_run - kLift + lg2_approx(l_run);
            if (part) reinterpret_cast<float *>(p.ws + w.part_l)[out_row] = lse2;
            else p.lse[out_row] = empty ? -INFINITY : (m_run - kLift) * 0.69314718055994530942f + logf(l_run);
        }
        tc_fence_before();
    }
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(kThreads, 1)
    bsattn_prefill_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ Layout w,
                          const __grid_constant__ CUtensorMap tq) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    const uint32_t warp = warp_id(), lane = lane_id();
    Waiter wait;
    wait.bars = base + C::kBar;
    wait.abort = reinterpret_cast<volatile int *>(misc + 1);
    wait.err = p.err;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(wait.bar(C::bKF + s), 1);
            mbar_init(wait.bar(C::bKE + s), 1);
            mbar_init(wait.bar(C::bVF + s), 1);
            mbar_init(wait.bar(C::bVE + s), 1);
            mbar_init(wait.bar(C::bQF + s), 1);
            mbar_init(wait.bar(C::bQE + s), 1);
            mbar_init(wait.bar(C::bSR + s), 1);
            mbar_init(wait.bar(C::bPR + 2 * s), 4);
            mbar_init(wait.bar(C::bPR + 2 * s + 1), 4);
            mbar_init(wait.bar(C::bOD + s), 1);
        }
        for (int s = 0; s < kDescs; ++s) {
            mbar_init(wait.bar(C::bUF + s), 1);
            mbar_init(wait.bar(C::bUE + s), 10);   // copying warp, issuing warp, eight softmax warps
        }
        mbar_init(wait.bar(C::bDrain), 1);
        misc[1] = 0;
        fence_barrier_init();
    }
    // rows of a query tile that no token fills stay 0
    for (uint32_t i = threadIdx.x; i < 2 * C::kTileBytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(smem + C::kQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 2) {
        tmem_alloc(base + C::kMisc, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    grid_launch_dependents();
    grid_dependency_wait();
    if (warp == 0) {
        regs_release<kCtrlRegs>();
        // ------------------------------------------------------- copies --
        const uint32_t lead = lane == 0 ? 1u : 0u;
        if (lane == 0) tma_prefetch_desc(&tq);
        uint32_t descs = 0, kc = 0, vc = 0, qc[2] = {0, 0};
        const uint32_t q_bytes = (uint32_t)(p.G * w.tokens) * D * 2u;
        bool ok = true;
        SegDesc d;
        while (ok && next_desc<C>(wait, smem, descs, d)) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!ok || min(d.k1, d.count[t]) <= d.k0) continue;
                if (!(ok = __all_sync(0xffffffffu, wait(C::bQE + t, qc[t] ^ 1u)))) break;
                mbar_arrive_expect_tx_lead(lead, wait.bar(C::bQF + t), q_bytes);
                __syncwarp();
                for (int x = 0; x < D / 64; ++x)
                    tma_load_3d_lead(lead, base + C::kQ + t * C::kTileBytes + x * kSub, &tq, wait.bar(C::bQF + t), x * 64,
                                     d.h * p.G, d.token + t * w.tokens);
                ++qc[t];
            }
            for (int k = d.k0; ok && k < d.k1; ++k) {
                const int tile = k < d.sinks ? k : k - d.sinks + d.near;
                const int slot = d.tile0 + (tile < d.seq_sinks ? tile : tile - d.seq_near + d.seq_sinks);
                const long long at = (long long)d.h * w.tiles + slot;
                const int ks = (int)(kc & 1u), vs = (int)(vc & 1u);
                if (!(ok = __all_sync(0xffffffffu, wait(C::bKE + ks, (kc >> 1) ^ 1u)))) break;
                mbar_arrive_expect_tx_lead(lead, wait.bar(C::bKF + ks), C::kTileBytes);
                bulk_g2s_lead(lead, base + C::kK + ks * C::kTileBytes, p.ws + w.k + at * C::kTileBytes, C::kTileBytes,
                              wait.bar(C::bKF + ks));
                ++kc;
                if (!(ok = __all_sync(0xffffffffu, wait(C::bVE + vs, (vc >> 1) ^ 1u)))) break;
                mbar_arrive_expect_tx_lead(lead, wait.bar(C::bVF + vs), C::kTileBytes + (uint32_t)sizeof(TileHead));
                bulk_g2s_lead(lead, base + C::kHead + vs * (uint32_t)sizeof(TileHead),
                              p.ws + w.head + at * (long long)sizeof(TileHead), (uint32_t)sizeof(TileHead), wait.bar(C::bVF + vs));
                bulk_g2s_lead(lead, base + C::kV + vs * C::kTileBytes, p.ws + w.v + at * C::kTileBytes, C::kTileBytes,
                              wait.bar(C::bVF + vs));
                ++vc;
            }
        }
        // nothing may be on its way into shared memory when the CTA ends
        for (uint32_t s = 0; s < 2; ++s) {
            if (kc > s) mbar_wait_drain(wait.bar(C::bKF + (int)s), ((kc - 1 - s) >> 1) & 1u);
            if (vc > s) mbar_wait_drain(wait.bar(C::bVF + (int)s), ((vc - 1 - s) >> 1) & 1u);
            if (qc[s] > 0) mbar_wait_drain(wait.bar(C::bQF + (int)s), (qc[s] - 1) & 1u);
        }
    } else if (warp == 1) {
        regs_release<kCtrlRegs>();
        // ---------------------------------------------------- MMA issuer --
        // The whole warp runs in step; lane 0 issues.
        const uint32_t lead = lane == 0 ? 1u : 0u;
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, true) & ~((1u << 7) | (1u << 10));   // fp16 A and B
        const uint64_t desc_q = smem_desc_sw128(base + C::kQ, 16, 1024);
        const uint64_t desc_k = smem_desc_sw128(base + C::kK, 16, 1024);
        const uint64_t desc_v = smem_desc_sw128(base + C::kV, kSub, 1024);
        constexpr uint64_t kTileUnits = C::kTileBytes >> 4, kSubUnits = kSub >> 4;
        uint32_t descs = 0, tile0 = 0, qc[2] = {0, 0}, pc[2] = {0, 0};
        bool ok = true;
        auto ready = [&](int b, uint32_t phase) -> bool {
            ok = ok && wait(b, phase);
            return ok;
        };
        auto score = [&](int t, uint32_t it) {
            const uint64_t qd = desc_q + (uint64_t)t * kTileUnits, kd = desc_k + (uint64_t)(it & 1u) * kTileUnits;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (uint64_t)((kk >> 2) * kSubUnits + (kk & 3) * 2);
                mma_ss_lead(lead, tmem + t * 128, qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit_lead(lead, wait.bar(C::bSR + t));
        };
        auto output = [&](int t, uint32_t it, bool first) -> bool {
            if (!ready(C::bVF + (int)(it & 1u), it >> 1)) return false;
            const uint64_t vd = desc_v + (uint64_t)(it & 1u) * kTileUnits;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!ready(C::bPR + 2 * t + half, pc[t])) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                    mma_ts_lead(lead, tmem + 256 + t * D, tmem + t * 128 + kk * 8, vd + (uint64_t)(kk * (2048 >> 4)), idesc_pv,
                                kk > 0 || !first ? 1u : 0u);
            }
            ++pc[t];
            return true;
        };
        SegDesc d;
        while (ok && next_desc<C>(wait, smem, descs, d)) {
            const int end[2] = {min(d.k1, d.count[0]), min(d.k1, d.count[1])};
            for (int t = 0; t < 2; ++t)
                if (end[t] > d.k0) {
                    ready(C::bQF + t, qc[t]);
                    ++qc[t];
                }
            if (!ok) break;
            tc_fence_after();
            for (int k = d.k0; ok && k <= d.k1; ++k) {
                const uint32_t it = tile0 + (uint32_t)(k - d.k0);
                if (k < d.k1) {
                    if (!ready(C::bKF + (int)(it & 1u), it >> 1)) break;
                    tc_fence_after();
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (k > d.k0 && k - 1 < end[t]) {
                        if (!output(t, it - 1, k - 1 == d.k0)) break;
                        if (k == end[t]) mma_commit_lead(lead, wait.bar(C::bOD + t));
                    }
                    if (k < end[t]) {
                        score(t, it);
                        if (k == end[t] - 1) mma_commit_lead(lead, wait.bar(C::bQE + t));
                    }
                }
                if (!ok) break;
                if (k > d.k0) mma_commit_lead(lead, wait.bar(C::bVE + (int)((it - 1) & 1u)));
                if (k < d.k1) mma_commit_lead(lead, wait.bar(C::bKE + (int)(it & 1u)));
            }
            tile0 += (uint32_t)(d.k1 - d.k0);
        }
        // Wait until every tcgen05 operation issued above has completed.
        mma_commit_lead(lead, wait.bar(C::bDrain));
        mbar_wait_drain(wait.bar(C::bDrain), 0);
    } else if (warp < 4) {
        regs_release<kCtrlRegs>();
        if (warp == 3 && lane == 0) schedule_role<C>(p, w, wait, smem);
        __syncwarp();
    } else {
        regs_claim<kSoftmaxRegs>();
        softmax_role<D, kInt8>(p, w, wait, tmem, warp >= 8 ? 1 : 0, warp, lane, smem);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------- join --

// Blocks x, x + gridDim.x, ..: the segment that begins in that piece and ends in a later one; its rows are dealt out to the
// warps of the blocks (x, 0), (x, 1), ..  kAhead parts are on their way at a time, whatever their weights: of few rows, where the join is a fifth of the call,
// 4 (drafts of 4 tokens 29.0 -> 27.9 us); of many, whose parts are mostly two, 1 (a window of 4096 tokens 338; 4: 346).
template <int D, int kAhead>
__global__ void __launch_bounds__(kJoinThreads) bsattn_prefill_join_kernel(const __grid_constant__ ChunkParams p,
                                                                           const __grid_constant__ Layout w) {
    constexpr int kWarps = kJoinThreads / 32;
    grid_launch_dependents();
    const int lane = (int)(threadIdx.x % 32), rows = w.few ? w.few : 2 * kTile;
    const float *part_l = reinterpret_cast<const float *>(p.ws + w.part_l);
    const float *part_o = reinterpret_cast<const float *>(p.ws + w.part_o);
    grid_dependency_wait();
    for (int piece = blockIdx.x; piece < w.pieces; piece += gridDim.x) {
        const CutInfo cut = reinterpret_cast<const CutInfo *>(p.ws + w.cuts)[piece];
        if (cut.parts == 0) continue;
        for (int r = (int)(blockIdx.y * kWarps + threadIdx.x / 32); r < rows; r += (int)gridDim.y * kWarps) {
            const int t = r / kTile, row = r % kTile, token_of = row / p.G, tok = t * w.tokens + token_of;
            if (token_of >= w.tokens || tok >= cut.tokens) continue;
            auto at = [&](int x) -> long long { return ((long long)(x == 0 ? 2 * piece + 1 : 2 * (piece + x)) * 2 + t) * kTile + row; };
            float m = -INFINITY, sum = 0.f, o[D / 32] = {};
            for (int x0 = 0; x0 < cut.parts; x0 += 32) {
                const float l = x0 + lane < cut.parts ? part_l[at(x0 + lane)] : -INFINITY;
                float top = l;
                for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float m_new = fmaxf(m, top);
                const float f = l == -INFINITY ? 0.f : ex2_approx(l - m_new), drop = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
                m = m_new;
                sum *= drop;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) o[c] *= drop;
                const int n = min(32, cut.parts - x0);
#pragma unroll 1
                for (int y0 = 0; y0 < n; y0 += kAhead) {
                    float v[kAhead][D / 32];
#pragma unroll
                    for (int y = 0; y < kAhead; ++y) {
                        const float *from = part_o + at(x0 + min(y0 + y, n - 1)) * D + lane * (D / 32);
                        if constexpr (D == 128) {
                            const float4 u = *reinterpret_cast<const float4 *>(from);
                            v[y][0] = u.x, v[y][1] = u.y, v[y][2] = u.z, v[y][3] = u.w;
                        } else {
                            const float2 u = *reinterpret_cast<const float2 *>(from);
                            v[y][0] = u.x, v[y][1] = u.y;
                        }
                    }
#pragma unroll
                    for (int y = 0; y < kAhead; ++y) {
                        const float fx = __shfl_sync(0xffffffffu, f, (y0 + y) & 31);
                        if (y0 + y >= n || fx == 0.f) continue;  // no key, or next to nothing
                        sum += fx;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) o[c] += fx * v[y][c];
                    }
                }
            }
            const bool empty = sum == 0.f;
            const float inv = empty ? 0.f : 1.f / sum;
            const long long out = (long long)(cut.token + tok) * p.Hq + cut.h * p.G + row - token_of * p.G;
            if (p.out_f32) {
                float *dst = static_cast<float *>(p.out) + out * D + lane * (D / 32);
#pragma unroll
                for (int c = 0; c < D / 32; c += 2) reinterpret_cast<float2 *>(dst)[c / 2] = make_float2(o[c] * inv, o[c + 1] * inv);
            } else {
                uint32_t *dst = static_cast<uint32_t *>(p.out) + (out * D + lane * (D / 32)) / 2;
#pragma unroll
                for (int c = 0; c < D / 32; c += 2) dst[c / 2] = pack_bf16x2(o[c] * inv, o[c + 1] * inv);
            }
            if (lane == 0) p.lse[out] = empty ? -INFINITY : m * 0.69314718055994530942f + logf(sum);
        }
    }
}

template <int D, bool kInt8>
cudaError_t launch(const ChunkParams &p, cudaStream_t stream) {
    using C = Cfg<D>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set_for_device[dev]) {
        // the register split inside the kernel assumes exactly kLaunchRegs per thread at launch
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, bsattn_prefill_kernel<D, kInt8>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(bsattn_prefill_kernel<D, kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kAlloc);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    const int sms = current_device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const Layout w = make_layout(p.total, p.B, p.c.H, p.G, D, p.keys, sms < kPrefillCtas ? sms : kPrefillCtas);
    CUtensorMap tq = {};
    if (p.total > 0 && !w.few && !encode_query_rows(&tq, p.q, p.total, p.Hq, D, p.q_stride, w.tokens, p.G)) return cudaErrorInvalidValue;
    void *args[] = {const_cast<ChunkParams *>(&p), const_cast<Layout *>(&w), &tq};
    const auto join = w.few ? reinterpret_cast<const void *>(bsattn_prefill_join_kernel<D, 4>) : reinterpret_cast<const void *>(bsattn_prefill_join_kernel<D, 1>);
    if (w.few) {
        e = launch_prefill_rows(p, w, stream);
        return e != cudaSuccess || p.total == 0 ? e : launch_dependent(join, dim3((unsigned)w.pieces, (unsigned)(w.few * 32 / kJoinThreads)), kJoinThreads, 0, args, stream);
    }
    e = launch_dependent(reinterpret_cast<const void *>(bsattn_prefill_plan_kernel), dim3(1), kPlanThreads, 0, args, stream);
    if (e != cudaSuccess || p.total == 0) return e;
    const long long items = w.tiles * p.c.H;
    const unsigned blocks = (unsigned)(items < sms * 8ll ? items : sms * 8ll);
    e = launch_dependent(reinterpret_cast<const void *>(bsattn_prefill_widen_kernel<D, kInt8>), dim3(blocks), kWidenThreads, 0, args, stream);
    if (e != cudaSuccess) return e;
    e = launch_dependent(reinterpret_cast<const void *>(bsattn_prefill_kernel<D, kInt8>), dim3((unsigned)w.ctas), kThreads, C::kAlloc, args, stream);
    if (e != cudaSuccess) return e;
    return launch_dependent(join, dim3((unsigned)(w.pieces < 1024 ? w.pieces : 1024), 8), kJoinThreads, 0, args, stream);
}

}  // namespace

cudaError_t launch_dependent(const void *kernel, dim3 grid, int threads, size_t smem, void **args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

// Of `total` query tokens or fewer: those for which another kernel is built may need a little more.
size_t prefill_workspace_bytes(int total, int B, int H, int G, int D, long long keys) {
    size_t most = make_layout(total, B, H, G, D, keys, kPrefillCtas).total;
    for (long long rows = 16; rows <= kFewRows; rows *= 2) {
        const long long last = rows * B / G;     // the most tokens of a mean of so many rows
        if (last >= total) break;
        const size_t less = make_layout((int)last, B, H, G, D, keys, kPrefillCtas).total;
        if (less > most) most = less;
    }
    return most;
}

cudaError_t launch_prefill(const ChunkParams &p, cudaStream_t stream) {
    if (p.c.D == 128) return p.c.int8 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
    return p.c.int8 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace bsattn
