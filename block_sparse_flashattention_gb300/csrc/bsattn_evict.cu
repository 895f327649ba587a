// Eviction from a paged 8-bit K/V cache by weight: per sequence and KV head the `sinks` first
// and the `recent` newest keys stay, and of the others those of largest weight, `keep` in all
// (equal weights: the lower positions).  What stays is moved, in order, to the places 0, 1, ... of
// the sequence's row of out_table.
//
// Two kernels.  bsattn_evict_select_kernel, a cluster of 1 to 8 CTAs per (sequence, head), finds the weight w* of
// the last key that stays by a radix selection: weights as ordered 32-bit integers, three digits of 11, 11 and
// 10 bits, the highest first, a histogram of the digit among the keys that agree so far.  Each CTA reads its
// piece of the positions once and keeps it in shared memory; histograms are summed through distributed shared
// memory.  Then the positions of all keys above w* and of the first ones equal to it are written: every warp counts its
// piece, and the counts before it, of the CTA's warps and of the CTAs before, give it its place in the list.
// bsattn_evict_move_kernel moves rows to other pages, each independent of the others; bsattn_evict_close_kernel
// moves them within their pages, in waves.
//
// HBM bounds it: 4 bytes per key, and 2 (2 D + 12) per row that is moved.  int8, D = 128, us a call, to other pages /
// within the pages: a sequence of 131072 keys, 32 heads, keeping 32768 (536 MB of rows): 156 (select 50, move 93: 5.8
// TB/s), 193; 8 heads: 74, 134; 64 sequences of 4096, 8 heads, keeping 1024 (268 MB): 83, 89; 8 of 32768 keeping 8192:
// 85, 101.  With one CTA per (sequence, head) instead of clusters, the selection made it 625, 556, 83, 119, and the
// rows within the pages 1412, 1176, 97, 394.
#include "bsattn_internal.h"
#include "sm100_ptx.cuh"

namespace bsattn {

namespace {

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32, kBins = 2048;
constexpr int kMostKeys = 40960;             // of a CTA that shared memory holds; more are read again for every digit
constexpr int kMoveThreads = 256, kCloseThreads = 512, kCloseRows = 4;   // rows that a thread has on their way
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

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A word of another CTA of the cluster.
__device__ __forceinline__ uint32_t peer_word(const uint32_t *mine, uint32_t rank) {
    uint32_t at, x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}

__device__ __forceinline__ uint4 peer_words(const uint32_t *mine, uint32_t rank) {
    uint32_t at;
    uint4 x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
    return x;
}

// ranks: CTAs of a cluster; room: keys that `keys` holds.
__global__ void __launch_bounds__(kSelectThreads, 3) bsattn_evict_select_kernel(const __grid_constant__ EvictParams p, int ranks, int room) {
    extern __shared__ uint32_t keys[];
    __shared__ __align__(16) uint32_t hist[2][kBins];
    __shared__ uint32_t s_digit, s_left, s_warps[kSelectWarps], s_count[2];
    __shared__ int above[kSelectWarps], equal[kSelectWarps];
    const int rank = (int)blockIdx.x % ranks, seg = (int)blockIdx.x / ranks;
    const int b = seg / p.c.H, h = seg - b * p.c.H, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    grid_launch_dependents();
    grid_dependency_wait();
    const Evicted s = sequence(p, b, h == 0 && rank == 0 && tid == 0);
    if (h == 0 && rank == 0 && tid == 0) p.lens[b] = s.m;
    const int32_t *table = p.table + (long long)b * p.table_stride;
    int32_t *kept = p.kept + ((long long)b * p.c.H + h) * p.keep;
    // Positions are counted without sign: a step past the last of them stays below 2^32, not below 2^31.
    const unsigned all = rank * kSelectThreads + tid, step = ranks * kSelectThreads;
    for (unsigned i = s.m + all; i < (unsigned)p.keep; i += step) kept[i] = -1;
    if (s.n <= p.keep) {
        for (unsigned i = all; i < (unsigned)s.m; i += step) kept[i] = (int)i;
        return;
    }
    // the CTA's positions first .. first + n - 1
    const int per = ((s.n + ranks - 1) / ranks + 31) & ~31;
    const int first = (int)min((long long)rank * per, (long long)s.n), n = min(per, s.n - first);
    auto kept_anyway = [&](int j) -> bool { return j < p.sinks || j >= s.n - p.recent; };
    auto load = [&](int i) -> uint32_t {
        const int j = first + i;
        if (kept_anyway(j)) return kForced;
        const long long row = row_at(p.c, table, h, j);
        return row < 0 ? 0u : ordered(p.weights[row]);
    };
    const int held = min(n, room);
    for (int i0 = tid; i0 < held; i0 += 8 * kSelectThreads) {
        long long row[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) row[k] = i0 + k * kSelectThreads < held ? row_at(p.c, table, h, first + i0 + k * kSelectThreads) : -1;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = row[k] >= 0 ? __ldg(p.weights + row[k]) : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kSelectThreads;
            if (i < held) keys[i] = kept_anyway(first + i) ? kForced : row[k] < 0 ? 0u : ordered(x[k]);
        }
    }
    auto key = [&](int i) -> uint32_t { return i < held ? keys[i] : load(i); };
    for (int i = tid; i < kBins; i += kSelectThreads) hist[0][i] = 0;
    __syncthreads();
    // the digits of w*: `left` keys are still to be found among those that agree with it so far
    uint32_t star = 0, left = (uint32_t)p.keep;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        uint32_t *mine = hist[pass & 1];
#pragma unroll 4
        for (unsigned i = tid; i < (unsigned)n; i += kSelectThreads) {
            const uint32_t k = key((int)i);
            if (pass == 0 || ((k ^ star) >> (shift + bits)) == 0u) atomicAdd(&mine[(k >> shift) & ((1u << bits) - 1u)], 1u);
        }
        if (ranks > 1) cluster_sync();
        else __syncthreads();
        // a thread: four digits, the highest first; `more`: keys of larger ones
        constexpr int kOwn = 4;
        static_assert(kOwn * kSelectThreads == kBins, "digits of a thread");
        const int top = kBins - kOwn * (tid + 1);
        uint4 x[8];
        x[0] = *reinterpret_cast<const uint4 *>(mine + top);
        if (ranks > 1) {
#pragma unroll
            for (int r = 0; r < 8; ++r) x[r] = r < ranks ? peer_words(mine + top, (uint32_t)r) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 1; r < 8; ++r) x[0].x += x[r].x, x[0].y += x[r].y, x[0].z += x[r].z, x[0].w += x[r].w;
        }
        const uint32_t c[kOwn] = {x[0].w, x[0].z, x[0].y, x[0].x}, sum = (c[0] + c[1]) + (c[2] + c[3]);
        uint32_t more = sum;
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, more, d);
            if (lane >= d) more += y;
        }
        if (lane == 31) s_warps[warp] = more;
        // the other histogram, read in the pass before the last barrier, is free
        for (int i = tid; i < kBins; i += kSelectThreads) hist[(pass & 1) ^ 1][i] = 0;
        __syncthreads();
        more -= sum;
        for (int w = 0; w < warp; ++w) more += s_warps[w];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (more < left && left <= more + c[i]) {
                s_digit = (uint32_t)(kBins - 1 - kOwn * tid - i);
                s_left = left - more;
            }
            more += c[i];
        }
        __syncthreads();
        star |= s_digit << shift;
        left = s_left;
        __syncthreads();
    }
    // warps' pieces of the positions
    const int piece = ((n + kSelectWarps - 1) / kSelectWarps + 31) & ~31;
    const int lo = min(n, warp * piece), hi = min(n, lo + piece);
    int na = 0, ne = 0;
#pragma unroll 4
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const bool in = i0 + lane < hi;
        const uint32_t k = in ? key(i0 + lane) : 0u;
        na += __popc(__ballot_sync(0xffffffffu, in && k > star));
        ne += __popc(__ballot_sync(0xffffffffu, in && k == star));
    }
    if (lane == 0) above[warp] = na, equal[warp] = ne;
    __syncthreads();
    if (tid == 0) {
        uint32_t a = 0, e = 0;
        for (int w = 0; w < kSelectWarps; ++w) a += (uint32_t)above[w], e += (uint32_t)equal[w];
        s_count[0] = a, s_count[1] = e;
    }
    if (ranks > 1) cluster_sync();
    // keys above w*, equal ones, before this warp's piece; the first `left` equal ones stay
    int out = 0, before = 0;
    for (int r = 0; r < rank; ++r) {
        out += (int)peer_word(&s_count[0], (uint32_t)r);
        before += (int)peer_word(&s_count[1], (uint32_t)r);
    }
    for (int w = 0; w < warp; ++w) out += above[w], before += equal[w];
    out += min(before, (int)left);
#pragma unroll 4
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const bool in = i0 + lane < hi;
        const uint32_t k = in ? key(i0 + lane) : 0u;
        const uint32_t eq = __ballot_sync(0xffffffffu, in && k == star), below = (1u << lane) - 1u;
        const bool stays = in && (k > star || (k == star && before + __popc(eq & below) < (int)left));
        const uint32_t st = __ballot_sync(0xffffffffu, stays);
        if (stays) kept[out + __popc(st & below)] = first + i0 + lane;
        out += __popc(st);
        before += __popc(eq);
    }
    if (ranks > 1) cluster_sync();   // no CTA ends while another reads its counts
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

// What goes from position `from` to place i.
__device__ __forceinline__ void places(const EvictParams &p, const int32_t *table, const int32_t *out, int h, int from, int i,
                                       long long &row, long long &to) {
    row = row_at(p.c, table, h, from);
    to = row_at(p.c, out, h, i);
    if ((row < 0 || to < 0) && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) bsattn_evict_move_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kLanes = D / 16, kRows = kMoveThreads / kLanes;
    const int b = blockIdx.x / p.c.H, h = blockIdx.x - b * p.c.H, tid = threadIdx.x;
    const int32_t *table = p.table + (long long)b * p.table_stride, *out = p.out_table + (long long)b * p.out_stride;
    const int32_t *kept = p.kept + ((long long)b * p.c.H + h) * p.keep;
    const int piece = tid % kLanes;
    grid_launch_dependents();
    grid_dependency_wait();
    const Evicted s = sequence(p, b, false);
    for (unsigned i = blockIdx.y * kRows + tid / kLanes; i < (unsigned)s.m; i += gridDim.y * kRows) {
        const int from = kept[i];
        if (from < 0) continue;
        long long row, to;
        places(p, table, out, h, from, (int)i, row, to);
        store_row<D>(p, to, piece, load_row<D>(p, row, piece));
    }
}

// Within the pages: a cluster's CTAs read a wave of rows, meet, and write it.  Row i comes from kept[i] >= i, so what
// a wave writes lies before all that later waves read.  512 threads of 4 rows each: with 2 rows the first of the cases
// above is 221 us, with 256 threads of 8 rows 210.
template <int D>
__global__ void __launch_bounds__(kCloseThreads) bsattn_evict_close_kernel(const __grid_constant__ EvictParams p, int ranks) {
    constexpr int kLanes = D / 16, kRows = kCloseThreads / kLanes;
    const int seg = blockIdx.x / ranks, rank = blockIdx.x - seg * ranks;
    const int b = seg / p.c.H, h = seg - b * p.c.H, tid = threadIdx.x;
    const int32_t *table = p.table + (long long)b * p.table_stride;
    const int32_t *kept = p.kept + ((long long)b * p.c.H + h) * p.keep;
    const int piece = tid % kLanes;
    grid_launch_dependents();
    grid_dependency_wait();
    const Evicted s = sequence(p, b, false);
    const auto meet = [&] {
        if (ranks > 1) cluster_sync();
        else __syncthreads();
    };
    for (unsigned i0 = 0; i0 < (unsigned)s.m; i0 += ranks * kRows * kCloseRows) {
        Moved x[kCloseRows];
        long long to[kCloseRows];
        int from[kCloseRows];
        const unsigned i1 = i0 + rank * kRows * kCloseRows + tid / kLanes;
#pragma unroll
        for (int u = 0; u < kCloseRows; ++u) from[u] = i1 + u * kRows < (unsigned)s.m ? kept[i1 + u * kRows] : -1;
#pragma unroll
        for (int u = 0; u < kCloseRows; ++u) {
            const int i = (int)(i1 + u * kRows);
            to[u] = -1;
            if (from[u] < 0 || from[u] == i) continue;
            long long row;
            places(p, table, table, h, from[u], i, row, to[u]);
            x[u] = load_row<D>(p, row, piece);
        }
        meet();
#pragma unroll
        for (int u = 0; u < kCloseRows; ++u) store_row<D>(p, to[u], piece, x[u]);
    }
    // Rows that do not move are the first ones (kept ascends): of each page that has any, its own first one is.
    if (p.err) {
        for (unsigned i = (unsigned)(rank * kCloseThreads + tid) << p.c.page_shift; i < (unsigned)s.m;
             i += (unsigned)(ranks * kCloseThreads) << p.c.page_shift)
            if (kept[i] == (int)i && row_at(p.c, table, h, (int)i) < 0) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
    }
    // the places given up: their next keys' weights start at 0
    for (unsigned j = s.m + rank * kCloseThreads + tid; j < (unsigned)s.n; j += ranks * kCloseThreads) {
        const long long row = row_at(p.c, table, h, (int)j);
        if (row >= 0) p.weights[row] = 0.f;
    }
}

cudaError_t launch_ex(const void *kernel, dim3 grid, int threads, size_t smem, int cluster, void **args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cfg.stream = stream;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <int D>
cudaError_t launch_move(const EvictParams &p, int sms, cudaStream_t stream) {
    constexpr int kRows = kMoveThreads / (D / 16);
    void *args[] = {const_cast<EvictParams *>(&p)};
    const unsigned segs = (unsigned)(p.B * p.c.H);
    if (p.table == p.out_table) {
        int close_ranks = 1;
        while (close_ranks < 8 && (long long)segs * close_ranks <= sms && p.keep / close_ranks > 2 * (kCloseThreads / (D / 16)) * kCloseRows) close_ranks *= 2;
        void *close_args[] = {const_cast<EvictParams *>(&p), &close_ranks};
        return launch_ex(reinterpret_cast<const void *>(bsattn_evict_close_kernel<D>), dim3(segs * close_ranks), kCloseThreads, 0,
                         close_ranks, close_args, stream);
    }
    const long long room = min((long long)p.keep, (long long)p.table_cols << p.c.page_shift);
    const unsigned blocks = (unsigned)min((room + kRows - 1) / kRows, 1024ll);
    return launch_ex(reinterpret_cast<const void *>(bsattn_evict_move_kernel<D>), dim3(segs, blocks), kMoveThreads, 0, 1, args, stream);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t stream) {
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(bsattn_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    const int sms = current_device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Clusters while they fill no more than two CTAs per SM and leave each CTA some thousand of the keys that
    // the table has room for.
    const long long segs = (long long)p.B * p.c.H, most = (long long)p.table_cols << p.c.page_shift;
    int ranks = 1;
    while (ranks < 8 && segs * ranks <= sms && most / ranks > 4096) ranks *= 2;
    int room = (int)min((most + ranks - 1) / ranks + 32, (long long)kMostKeys);
    void *args[] = {const_cast<EvictParams *>(&p), &ranks, &room};
    if (segs * ranks > INT32_MAX) return cudaErrorInvalidValue;
    e = launch_ex(reinterpret_cast<const void *>(bsattn_evict_select_kernel), dim3((unsigned)(segs * ranks)), kSelectThreads,
                  (size_t)room * 4, ranks, args, stream);
    if (e != cudaSuccess) return e;
    return p.c.D == 128 ? launch_move<128>(p, sms, stream) : launch_move<64>(p, sms, stream);
}

}  // namespace bsattn
