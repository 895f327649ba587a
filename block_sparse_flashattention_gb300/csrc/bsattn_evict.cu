// Eviction from a paged 8-bit K/V cache by weight: per sequence and KV head the `sinks` first
// and the `recent` newest keys stay, and of the others those of largest weight, `keep` in all
// (equal weights: the lower positions).  What stays is moved, in order, to the places 0, 1, ... of
// the sequence's row of out_table.
//
// Two kernels.  bsattn_evict_select_kernel, a CTA per (sequence, head), finds the weight w* of
// the last key that stays by a radix selection (weights as ordered 32-bit integers, four digits of
// 8 bits, the highest first, a histogram of the digit among the keys that agree so far), then
// writes the positions of all keys above w* and of the first ones equal to it: every warp
// counts its piece of the positions, a scan over the warps gives each its place in the list.
// bsattn_evict_move_kernel moves rows.  To other pages every row is independent; within
// its own pages row i comes from position kept[i] >= i, so one CTA per (sequence, head)
// goes through the rows in ascending blocks, each read whole before it is written.
#include "bsattn_internal.h"
#include "sm100_ptx.cuh"

namespace bsattn {

namespace {

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kMoveThreads = 256, kMoveWarps = kMoveThreads / 32;
constexpr uint32_t kForced = 0xffffffffu;

// Weights as integers in the same order: NaN above all, -0 equal to 0.  kForced is none of them
// (the largest is NaN's 0xffc00000), nor is 0, a key on a page outside the cache.
__device__ __forceinline__ uint32_t ordered(float w) {
    if (w != w) return 0xffc00000u;
    const uint32_t x = __float_as_uint(w + 0.f);
    return x & 0x80000000u ? ~x : x | 0x80000000u;
}

struct Evicted {
    int n, m;   // keys before and after; m = 0: nothing to be done
};

__device__ __forceinline__ Evicted sequence(const EvictParams &p, int b, bool check) {
    Evicted s;
    s.n = max(__ldg(p.seqlens + b), 0);
    s.m = min(s.n, p.keep);
    if (s.n > (p.table_cols << p.c.page_shift)) {
        if (check && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
        s.n = s.m = 0;
    }
    return s;
}

__device__ __forceinline__ long long row_at(const CacheView &c, const int32_t *table_row, int h, int j) {
    const int page = __ldg(table_row + (j >> c.page_shift));
    if (page < 0 || page >= c.num_pages) return -1;
    return (((long long)page * c.H + h) << c.page_shift) + (j & ((1 << c.page_shift) - 1));
}

__global__ void __launch_bounds__(kSelectThreads) bsattn_evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ uint32_t hist[256], s_digit, s_left;
    __shared__ int above[kSelectWarps], equal[kSelectWarps];
    const int b = blockIdx.x / p.c.H, h = blockIdx.x - b * p.c.H, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const Evicted s = sequence(p, b, h == 0 && tid == 0);
    if (h == 0 && tid == 0) p.lens[b] = s.m;
    const int32_t *table = p.table + (long long)b * p.table_stride;
    int32_t *kept = p.kept + ((long long)b * p.c.H + h) * p.keep;
    for (int i = s.m + tid; i < p.keep; i += kSelectThreads) kept[i] = -1;
    if (s.n <= p.keep) {
        for (int i = tid; i < s.m; i += kSelectThreads) kept[i] = i;
        return;
    }
    auto key = [&](int j) -> uint32_t {
        if (j < p.sinks || j >= s.n - p.recent) return kForced;
        const long long row = row_at(p.c, table, h, j);
        return row < 0 ? 0u : ordered(p.weights[row]);
    };
    // the digits of w*: `left` keys are still to be found among those that agree with `prefix`
    uint32_t prefix = 0, left = (uint32_t)p.keep;
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < s.n; j += kSelectThreads) {
            const uint32_t k = key(j);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane: 8 digits, the highest first; `more`: keys of larger digits
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
            uint32_t more = sum;
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, more, d);
                if (lane >= d) more += x;
            }
            more -= sum;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (more < left && left <= more + c[i]) {
                    s_digit = 255u - 8u * lane - i;
                    s_left = left - more;
                }
                more += c[i];
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        left = s_left;
        __syncthreads();
    }
    // warps' pieces of the positions
    const int per = ((s.n + kSelectWarps - 1) / kSelectWarps + 31) & ~31;
    const int lo = min(s.n, warp * per), hi = min(s.n, lo + per);
    int na = 0, ne = 0;
    for (int j0 = lo; j0 < hi; j0 += 32) {
        const uint32_t k = j0 + lane < hi ? key(j0 + lane) : 0u;
        const bool in = j0 + lane < hi;
        na += __popc(__ballot_sync(0xffffffffu, in && k > prefix));
        ne += __popc(__ballot_sync(0xffffffffu, in && k == prefix));
    }
    if (lane == 0) above[warp] = na, equal[warp] = ne;
    __syncthreads();
    int out = 0, before = 0;   // places taken, equal keys, both before this warp's piece
    for (int w = 0; w < warp; ++w) {
        out += above[w] + min(equal[w], max((int)left - before, 0));
        before += equal[w];
    }
    for (int j0 = lo; j0 < hi; j0 += 32) {
        const bool in = j0 + lane < hi;
        const uint32_t k = in ? key(j0 + lane) : 0u;
        const uint32_t eq = __ballot_sync(0xffffffffu, in && k == prefix), below = (1u << lane) - 1u;
        const bool stays = in && (k > prefix || (k == prefix && before + __popc(eq & below) < (int)left));
        const uint32_t st = __ballot_sync(0xffffffffu, stays);
        if (stays) kept[out + __popc(st & below)] = j0 + lane;
        out += __popc(st);
        before += __popc(eq);
    }
}

// One row: codes of K and V (16 bytes a lane), scales and weight.  D / 16 lanes to a row.
struct Moved {
    uint4 k, v;
    float ks, vs, w;
};

template <int D>
__device__ __forceinline__ Moved load_row(const EvictParams &p, long long row, int piece) {
    Moved x = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), 0.f, 0.f, 0.f};
    if (row < 0) return x;
    x.k = reinterpret_cast<const uint4 *>(p.c.k + row * D)[piece];
    x.v = reinterpret_cast<const uint4 *>(p.c.v + row * D)[piece];
    if (piece == 0) x.ks = p.c.ks[row], x.vs = p.c.vs[row], x.w = p.weights[row];
    return x;
}

template <int D>
__device__ __forceinline__ void store_row(const EvictParams &p, long long row, int piece, const Moved &x) {
    if (row < 0) return;
    reinterpret_cast<uint4 *>(p.c.k + row * D)[piece] = x.k;
    reinterpret_cast<uint4 *>(p.c.v + row * D)[piece] = x.v;
    if (piece == 0) p.c.ks[row] = x.ks, p.c.vs[row] = x.vs, p.weights[row] = x.w;
}

template <int D, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads) bsattn_evict_move_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kLanes = D / 16, kRows = kMoveThreads / kLanes;
    const int b = blockIdx.x / p.c.H, h = blockIdx.x - b * p.c.H, tid = threadIdx.x;
    const Evicted s = sequence(p, b, false);
    const int32_t *table = p.table + (long long)b * p.table_stride, *out = p.out_table + (long long)b * p.out_stride;
    const int32_t *kept = p.kept + ((long long)b * p.c.H + h) * p.keep;
    const int piece = tid % kLanes;
    for (int i0 = blockIdx.y * kRows; i0 < s.m; i0 += gridDim.y * kRows) {
        const int i = i0 + tid / kLanes;
        const int from = i < s.m ? kept[i] : -1;
        const bool move = from >= 0 && !(kInPlace && from == i);
        Moved x;
        long long to = -1;
        if (move) {
            const long long row = row_at(p.c, table, h, from);
            to = row_at(p.c, out, h, i);
            if ((row < 0 || to < 0) && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
            x = load_row<D>(p, row, piece);
        }
        if (kInPlace) __syncthreads();
        if (move) store_row<D>(p, to, piece, x);
    }
    if (kInPlace)   // the places given up: their next keys' weights start at 0
        for (int j = s.m + tid; j < s.n; j += kMoveThreads) {
            const long long row = row_at(p.c, out, h, j);
            if (row >= 0) p.weights[row] = 0.f;
        }
}

template <int D>
void launch_move(const EvictParams &p, cudaStream_t stream) {
    constexpr int kRows = kMoveThreads / (D / 16);
    if (p.table == p.out_table)
        bsattn_evict_move_kernel<D, true><<<p.B * p.c.H, kMoveThreads, 0, stream>>>(p);
    else
        bsattn_evict_move_kernel<D, false><<<dim3(p.B * p.c.H, min((p.keep + kRows - 1) / kRows, 1024)), kMoveThreads, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t stream) {
    bsattn_evict_select_kernel<<<p.B * p.c.H, kSelectThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.c.D == 128) launch_move<128>(p, stream);
    else launch_move<64>(p, stream);
    return cudaGetLastError();
}

}  // namespace bsattn
