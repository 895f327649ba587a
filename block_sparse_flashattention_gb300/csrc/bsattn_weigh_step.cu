// Attention weight of cached keys (bsattn_weigh.cu has the mathematics) where a KV head has few query rows in the mean:
// decoding steps, drafts of a few tokens.
//
// HBM bounds it: D + 8 bytes per key and KV head, against 2 D flop per row.  So every warp streams keys through a ring
// of its own: a lane copies the pieces of codes that it feeds to mma.sync itself, and widens them on the way into the
// products.  No warp waits for another.  A 16-byte piece of a key's codes is four k-steps of a lane's row of A; query
// rows are put into B in the same order of dimensions.
//
// Keys lie on the products' 16 rows, queries on 8 kCols columns: S = K' Q'^T with K' = fp16(code), exact, and
// Q' = fp16(q 2^a), which keeps all bits of what is 2^-29 of a row's largest or more.  A unit is 16 keys of a
// (sequence, KV head), all on one page.  Units form a line on which each counts its blocks of query rows; every warp
// takes an equal piece of it and finds it by itself (lengths are on the device).  A weight has one writer and one
// order of its sum: over a block's columns, compensated from block to block.
//
// Measured (us a call, cold L2): 64 sequences of 100 to 4096 keys, 8 heads x 4, int8, D = 128 (146 MB: 21.9 at the copy's
// rate): 34.5, of which 5 before the first codes are there; 2 sequences of 1024 keys, 4 heads: 5.2.  20 warps with rings
// of 3 (16 warps 37.4, 24 35.3; rings of 4 35.1): what a warp does for 16 keys bounds it, some 200 instructions, not
// HBM's latency.  With bf16 products, whose widening takes twice the instructions, and a page looked up for every unit
// it was 51.6 (16 warps, rings of 4; 37.5 with fp16 and 32 units looked up at a time).  Two and four column
// groups have fewer warps for the registers.
//
// Of a sliding window only the units that some query meets are on the line; the others' weights are zeroed by a
// second pass that is divided in the same way.
#include "chunk_common.cuh"
#include "decode_common.cuh"
#include "kv_codes.cuh"

namespace bsattn {

namespace {

constexpr int kKeys = 16;

// A warp's ring in shared memory: of each stage the lanes' pieces of codes, the scales, the unit.
template <int D, int kCols>
struct Ring {
    static constexpr int kWarps = kCols == 1 ? 20 : kCols == 2 ? 16 : 12;
    static constexpr int kVecs = D / 64, kStages = D == 128 ? 3 : 5;
    static constexpr uint32_t kCodes = 0, kScales = kStages * 1024u * kVecs, kUnits = kScales + kStages * 64u,
                              kBytes = kUnits + kStages * 32u, kAlloc = kWarps * kBytes;
    static_assert(kAlloc <= 227u * 1024u && kBytes % 16 == 0, "shared memory");
};

// The sequence's units of 16 keys: 0 .. sinks - 1 and near .. end - 1 have keys that a query meets.
struct Units {
    int sinks, near, end;
    __device__ __forceinline__ int met() const { return sinks + end - near; }
    __device__ __forceinline__ int unmet() const { return near - sinks; }
};

__device__ __forceinline__ Units units_of(const ChunkParams &p, const Chunk &c) {
    Units u = {0, 0, 0};
    if (c.m <= 0) return u;
    u.end = (c.n + kKeys - 1) / kKeys;
    if (p.kind == BSATTN_MASK_SLIDING_WINDOW) {
        u.near = max(c.n - c.m + 1 - p.window_left, 0) / kKeys;
        u.sinks = (int)min(((long long)min(p.sink_tokens, c.n) + kKeys - 1) / kKeys, (long long)u.near);
    }
    return u;
}

// A walk along the units of one warp's piece of the line.
template <bool kMet>
struct Walk {
    const ChunkParams &p;
    int tokens;              // of a block of query rows
    long long begin, to;     // places
    int b, h, u, count, cost;
    Chunk c;
    Units s;

    // places of one head's units; what a unit costs
    __device__ __forceinline__ long long measure(const Chunk &x) {
        s = units_of(p, x);
        count = kMet ? s.met() : s.unmet();
        cost = kMet ? (x.m + tokens - 1) / tokens : 1;
        return (long long)count * cost;
    }

    // A whole warp: its piece of the line.
    __device__ __forceinline__ Walk(const ChunkParams &p_, int tokens_, int piece, int pieces, int lane, bool check)
        : p(p_), tokens(tokens_) {
        long long line = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < p.B; b0 += 32)
            if (b0 + lane < p.B) line += measure(chunk_of(p, b0 + lane, check));
        for (int d = 16; d; d >>= 1) line += __shfl_xor_sync(0xffffffffu, line, d);
        line *= p.c.H;
        b = p.B, h = u = count = cost = 0, begin = to = 0;
        pieces = (int)min((long long)pieces, line);
        if (piece >= pieces) return;
        const long long from = line_div(line * piece, pieces);
        to = line_div(line * (piece + 1), pieces);
        long long before = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            Chunk x = {};
            if (b0 + lane < p.B) x = chunk_of(p, b0 + lane, false);
            const long long own = measure(x) * p.c.H;
            long long sum = own;
            for (int d = 1; d < 32; d <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += y;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, from >= before + sum - own && from < before + sum);
            if (hit) {
                const int k = __ffs(hit) - 1;
                b = b0 + k;
                begin = __shfl_sync(0xffffffffu, before + sum - own, k);
                c.first = __shfl_sync(0xffffffffu, x.first, k);
                c.m = __shfl_sync(0xffffffffu, x.m, k);
                c.n = __shfl_sync(0xffffffffu, x.n, k);
                const long long places = measure(c);
                h = (int)line_div(from - begin, places);
                begin += h * places;
                u = (int)line_div(from - begin + cost - 1, cost);
                begin += (long long)u * cost;
                return;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
    }

    // To the next unit that there is.
    __device__ __forceinline__ bool here() {
        while (begin < to && b < p.B) {
            if (u < count) return true;
            u = 0;
            if (count == 0 || ++h >= p.c.H) {
                h = 0;
                if (++b >= p.B) return false;
                c = chunk_of(p, b, false);
                measure(c);
            }
        }
        return false;
    }

    __device__ __forceinline__ int unit(int i) const {
        if (!kMet) return s.sinks + i;
        return i < s.sinks ? i : i - s.sinks + s.near;
    }
};

struct __align__(16) Unit {
    int b, h, j;             // its first key; b < 0: none
    int row;                 // of its first key, -1: it has no page
    Chunk c;
    int pad;
};
static_assert(sizeof(Unit) == 32, "ring");

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x, float f) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(x & 0xffff0000u) * f), "f"(__uint_as_float(x << 16) * f));
    return r;
}

template <int D, int kCols, bool kInt8>
struct Warp {
    using R = Ring<D, kCols>;
    static constexpr int kVecs = D / 64, kSteps = D / 16;
    const ChunkParams &p;
    uint8_t *ring;
    const int tokens, lane, g, t;
    uint32_t q[kSteps][kCols][2];
    float nl[kCols][2];      // -lse log2(e) of the lane's columns, -inf: none
    float back[kCols][2];    // of their products: scale 2^e
    int qb, qh, qi;          // which block of query rows these are

    __device__ __forceinline__ Warp(const ChunkParams &p_, uint8_t *ring_, int tokens_, int lane_)
        : p(p_), ring(ring_), tokens(tokens_), lane(lane_), g(lane_ >> 2), t(lane_ & 3), qb(-1), qh(0), qi(0), row(-1), batch(0), i(0), from(0) {}

    // Up to 32 units of one (sequence, KV head) are looked up at a time, one by each lane.
    int row, batch, i, from;

    __device__ __forceinline__ Unit next(Walk<true> &w) {
        Unit x = {};
        x.b = -1;
        if (i == batch) {
            i = batch = 0;
            if (!w.here()) return x;
            batch = (int)min((long long)min(w.count - w.u, 32), line_div(w.to - w.begin + w.cost - 1, w.cost));
            from = w.u;
            if (lane < batch) row = (int)cache_row(p.c, p.table + (long long)w.b * p.table_stride, w.h, w.unit(from + lane) * kKeys);
            w.u += batch, w.begin += (long long)batch * w.cost;
        }
        x.b = w.b, x.h = w.h, x.c = w.c;
        x.j = w.unit(from + i) * kKeys;
        x.row = __shfl_sync(0xffffffffu, row, i);
        ++i;
        return x;
    }

    // Fetches a unit's codes and scales: a lane its own pieces, of keys g and g + 8 the pieces t and t + 4.  Keys
    // behind the sequence's last are read too (they are on its page) and have no weight.
    __device__ __forceinline__ void load(const Unit &x, int stage) const {
        if (lane == 0) reinterpret_cast<Unit *>(ring + R::kUnits)[stage] = x;
        if (x.b >= 0 && x.row >= 0) {
            const uint8_t *from = p.c.k + ((long long)x.row + g) * D + 16 * t;
            const uint32_t to = smem_u32(ring) + R::kCodes + (uint32_t)stage * 1024u * kVecs + 16u * lane;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < kVecs; ++i) copy_async(to + 512u * (r * kVecs + i), from + 8 * r * D + 64 * i);
            if (lane < 4) copy_async(smem_u32(ring) + R::kScales + (uint32_t)stage * 64u + 16u * lane, p.c.ks + x.row + 4 * lane);
        }
        copy_commit();
    }

    __device__ __forceinline__ void load_rows(const Unit &x, int block) {
        if (x.b == qb && x.h == qh && block == qi) return;
        qb = x.b, qh = x.h, qi = block;
        const int t0 = block * tokens, rows = min(tokens, x.c.m - t0) * p.G;
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
            const int r = 8 * n + g, tok = r / p.G;
            const uint16_t *from = p.q + (x.c.first + t0 + tok) * p.q_stride + (long long)(x.h * p.G + r - tok * p.G) * D + 16 * t;
            uint32_t y[kVecs][8];
            uint32_t top = 0;                    // largest magnitude
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                if (r < rows) {
                    lo = __ldg(reinterpret_cast<const uint4 *>(from + 64 * i));
                    hi = __ldg(reinterpret_cast<const uint4 *>(from + 64 * i) + 1);
                }
                y[i][0] = lo.x, y[i][1] = lo.y, y[i][2] = lo.z, y[i][3] = lo.w;
                y[i][4] = hi.x, y[i][5] = hi.y, y[i][6] = hi.z, y[i][7] = hi.w;
#pragma unroll
                for (int k = 0; k < 8; ++k) top = max(top, max(y[i][k] & 0x7fffu, y[i][k] >> 16 & 0x7fffu));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // fp16(q 2^(141 - e)) < 2^15: what is 2^-29 of the row's largest is still exact
            const int e = top >= 0x7f80u ? 141 : min(max((int)(top >> 7), 16), 253);
            const float f = __uint_as_float((uint32_t)(254 - e) << 23) * 0x1p14f;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) q[4 * i + k / 2][n][k % 2] = bf16x2_to_f16x2(y[i][k], f);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                back[n][i] = p.scale_log2 * __uint_as_float((uint32_t)(__shfl_sync(0xffffffffu, e, 8 * t + 4 * i) << 23)) * 0x1p-14f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = 8 * n + 2 * t + i, at = c / p.G;
                float l = INFINITY;
                if (c < rows) l = __ldg(p.lse + (long long)(x.c.first + t0 + at) * p.Hq + x.h * p.G + c - at * p.G);
                nl[n][i] = l == -INFINITY ? -INFINITY : l * -1.44269504088896340736f;   // -inf: a query without keys
            }
        }
    }

    // The unit's weights.
    __device__ __forceinline__ void run(int stage) {
        const Unit x = reinterpret_cast<const Unit *>(ring + R::kUnits)[stage];
        if (x.row < 0) {
            if (lane == 0 && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
            return;
        }
        const uint4 *codes = reinterpret_cast<const uint4 *>(ring + R::kCodes + stage * 1024 * kVecs) + lane;
        const float *scales = reinterpret_cast<const float *>(ring + R::kScales + stage * 64);
        const float c[2] = {scales[g], scales[g + 8]};
        const int pos = x.c.n - x.c.m, last = x.j + kKeys - 1;
        // all tokens meet all of the unit's keys
        bool whole = p.kind == BSATTN_MASK_NONE ? last < x.c.n : last <= pos;
        if (p.kind == BSATTN_MASK_SLIDING_WINDOW) whole = whole && (last < p.sink_tokens || (long long)x.j + p.window_left >= x.c.n);
        // tokens that meet the lane's keys: lo <= token < hi
        int lo[2] = {0, 0}, hi[2] = {x.c.m, x.c.m};
        if (!whole) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int j = x.j + g + 8 * r;
                if (j >= x.c.n) hi[r] = 0;
                if (p.kind == BSATTN_MASK_CAUSAL || p.kind == BSATTN_MASK_SLIDING_WINDOW || (p.kind == BSATTN_MASK_PREFIX && j >= p.prefix_len))
                    lo[r] = max(j - pos, 0);
                if (p.kind == BSATTN_MASK_SLIDING_WINDOW && j >= p.sink_tokens)
                    hi[r] = (int)min(max((long long)j + p.window_left - pos, 0ll), (long long)hi[r]);
            }
        }
        float sum[2] = {0.f, 0.f}, lost[2] = {0.f, 0.f};   // compensated
#pragma unroll 1
        for (int t0 = 0, block = 0; t0 < x.c.m; t0 += tokens, ++block) {
            load_rows(x, block);
            float s[kCols][4];
#pragma unroll
            for (int n = 0; n < kCols; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const uint4 v0 = codes[32 * i], v1 = codes[32 * (kVecs + i)];
                const uint32_t y[2][4] = {{v0.x, v0.y, v0.z, v0.w}, {v1.x, v1.y, v1.z, v1.w}};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4];
                    codes_to_f16x2<kInt8>(y[0][k], a[0], a[2]);
                    codes_to_f16x2<kInt8>(y[1][k], a[1], a[3]);
#pragma unroll
                    for (int n = 0; n < kCols; ++n) mma_f16(s[n], a[0], a[1], a[2], a[3], q[4 * i + k][n][0], q[4 * i + k][n][1]);
                }
            }
            float add[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < kCols; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float &z = s[n][2 * r + i];
                        z = ex2_approx(fmaf(z * back[n][i], c[r], nl[n][i]));
                        if (nl[n][i] == -INFINITY) z = 0.f;
                    }
            if (!whole) {
                const int left = min(tokens, x.c.m - t0);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int from = min(max(lo[r] - t0, 0), left) * p.G, to = min(max(hi[r] - t0, 0), left) * p.G;
#pragma unroll
                    for (int n = 0; n < kCols; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int col = 8 * n + 2 * t + i;
                            if (col < from || col >= to) s[n][2 * r + i] = 0.f;
                        }
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int n = 0; n < kCols; ++n) add[r] += s[n][2 * r] + s[n][2 * r + 1];
                const float less = add[r] - lost[r], all = sum[r] + less;
                lost[r] = (all - sum[r]) - less;
                sum[r] = all;
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
        }
        const float w = t == 0 ? sum[0] : sum[1];
        const int j = x.j + g + 8 * t;
        if (t < 2 && j < x.c.n) {
            float *at = p.weights + x.row + g + 8 * t;
            if (!p.accumulate) *at = w;
            else if (t == 0 ? hi[0] > lo[0] : hi[1] > lo[1]) atomicAdd(at, w);
        }
    }
};

template <int D, int kCols, bool kInt8>
__global__ void __launch_bounds__(Ring<D, kCols>::kWarps * 32, 1) bsattn_weigh_step_kernel(const __grid_constant__ ChunkParams p, int tokens) {
    using R = Ring<D, kCols>;
    extern __shared__ __align__(16) uint8_t smem[];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = (int)threadIdx.x % 32, piece = (int)(threadIdx.x / 32 * gridDim.x + blockIdx.x);   // few pieces: all SMs
    const int pieces = (int)gridDim.x * R::kWarps;
    {
        Warp<D, kCols, kInt8> warp(p, smem + threadIdx.x / 32 * R::kBytes, tokens, lane);
        Walk<true> walk(p, tokens, piece, pieces, lane, piece == 0);
        const Unit first = warp.next(walk);
        warp.load(first, 0);
        for (int i = 1; i < R::kStages - 1; ++i) warp.load(warp.next(walk), i);
        if (first.b >= 0) warp.load_rows(first, 0);   // on their way with the first codes
        for (int stage = 0;; stage = stage + 1 < R::kStages ? stage + 1 : 0) {
            copy_wait<R::kStages - 2>();
            __syncwarp();                        // all lanes' copies are there, and all are done with the stage before
            if (reinterpret_cast<const Unit *>(warp.ring + R::kUnits)[stage].b < 0) break;
            warp.load(warp.next(walk), stage > 0 ? stage - 1 : R::kStages - 1);
            warp.run(stage);
        }
        copy_wait<0>();
    }
    if (p.kind != BSATTN_MASK_SLIDING_WINDOW || p.accumulate) return;
    Walk<false> walk(p, tokens, piece, pieces, lane, false);
    while (walk.here()) {                        // a unit per lane
        const int n = (int)min((long long)min(walk.count - walk.u, 32), walk.to - walk.begin);
        if (lane < n) {
            const long long row = cache_row(p.c, p.table + (long long)walk.b * p.table_stride, walk.h, walk.unit(walk.u + lane) * kKeys);
            if (row >= 0) {
#pragma unroll
                for (int i = 0; i < kKeys; ++i) p.weights[row + i] = 0.f;
            } else if (p.err) {
                atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
            }
        }
        walk.u += n, walk.begin += n;
    }
}

template <int D, int kCols, bool kInt8>
cudaError_t launch(const ChunkParams &p, cudaStream_t stream) {
    using R = Ring<D, kCols>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(bsattn_weigh_step_kernel<D, kCols, kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)R::kAlloc);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    const int sms = current_device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    int tokens = 8 * kCols / p.G;
    void *args[] = {const_cast<ChunkParams *>(&p), &tokens};
    return launch_dependent(reinterpret_cast<const void *>(bsattn_weigh_step_kernel<D, kCols, kInt8>), dim3((unsigned)sms), R::kWarps * 32,
                            R::kAlloc, args, stream);
}

template <int D, int kCols>
cudaError_t launch_of(const ChunkParams &p, cudaStream_t stream) {
    return p.c.int8 ? launch<D, kCols, true>(p, stream) : launch<D, kCols, false>(p, stream);
}

}  // namespace

cudaError_t launch_weigh_step(const ChunkParams &p, int rows, cudaStream_t stream) {
    if (p.c.D == 128) return rows <= 8 ? launch_of<128, 1>(p, stream) : rows <= 16 ? launch_of<128, 2>(p, stream) : launch_of<128, 4>(p, stream);
    return rows <= 8 ? launch_of<64, 1>(p, stream) : rows <= 16 ? launch_of<64, 2>(p, stream) : launch_of<64, 4>(p, stream);
}

}  // namespace bsattn
