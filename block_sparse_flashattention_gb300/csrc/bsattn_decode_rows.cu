// Attention of one query token per sequence over a paged 8-bit K/V cache with 17 to 128
// query heads per KV head (fewer: bsattn_decode.cu, whose mathematics and fragments this
// kernel shares).
//
// With several tiles of 16 query rows the keys are better shared than streamed per warp:
// a CTA keeps a ring of 128-key tiles in shared memory (TMA: codes by rows with the
// 128-byte or 64-byte swizzle, scales as plain copies), and its eight computing warps
// divide into R row tiles x 8 / R groups of 16 keys, which join at the segment's end.  All
// tiles of all (sequence, KV head) segments form one line, cut into equal pieces, one per
// CTA, one CTA per SM; parts of segments that span CTAs are joined by the kernel in
// bsattn_decode.cu.  With the swizzled rows none of the 16-byte shared-memory loads meets
// a bank twice (the 8-byte loads of V at D = 64 do, two ways).
//
// Bound by the issue of mma.sync and of the widening before it, not by HBM (us a call in a
// graph over the same memory, e4m3, D = 128): 16 sequences of 8192 keys, 2 heads, G = 17 or 32: 39 us, 1.8 TB/s, G = 128: 104 us;
// 2 sequences of 65536 keys, 8 heads, G = 32: 103 us, 2.7 TB/s, G = 128: 314 us, 219 TFLOP/s.
//
// 288 threads: warp 8 looks up lists and pages, 32 at a time, and keeps the ring full;
// warps 0-7 compute.
#include "bsattn_internal.h"
#include "decode_common.cuh"
#include "kv_codes.cuh"

namespace bsattn {

namespace {

constexpr int kConsumers = 8;                    // computing warps
constexpr int kThreads = (kConsumers + 1) * 32;

// TileMsg flags: a segment's first / last tile in this CTA, its whole line lies here.
constexpr uint32_t kFirst = 1u, kLast = 2u, kComplete = 4u;

// What the producer tells the computing warps about a stage.
struct TileMsg {
    int32_t seg;      // -1: no further tiles
    int32_t lim;      // keys of the tile that count
    uint32_t groups;  // bit i: the page of keys 16 i .. 16 i + 15 is loaded
    uint32_t flags;
};

template <int D>
struct Cfg {
    // 4 x 33 KB or 8 x 17 KB in flight per SM; what HBM needs at 6.7 TB/s and ~1 us is 44 KB
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr uint32_t kCodes = 128u * D;                 // K or V codes of a tile
    static constexpr uint32_t kStageBytes = 2u * kCodes;
    static constexpr uint32_t kScales = kStages * kStageBytes;   // per stage 128 K scales, 128 V scales
    static constexpr uint32_t kRed = kScales + kStages * 1024u;  // join: 8 warps x (D / 2) x 32 lanes fp32
    static constexpr uint32_t kStat = kRed + kConsumers * (D / 2) * 128u;  // [8 x 16 rows] (m, u, l, -)
    static constexpr uint32_t kMsg = kStat + kConsumers * 16u * 16u;
    static constexpr uint32_t kBar = kMsg + kStages * (uint32_t)sizeof(TileMsg);
    static constexpr uint32_t kMisc = kBar + (2u * kStages + 1u) * 8u;  // abort flag, start, scan
    static constexpr uint32_t kBytes = kMisc + 128u;
    static constexpr uint32_t kAlloc = kBytes + 1024u;           // slack for 1024-byte alignment
    static_assert(kAlloc <= 227u * 1024u, "shared memory");
};

struct Misc {
    int32_t abort, start_seg;
    long long start_off;
    long long warp_sum[kConsumers + 1];
};
static_assert(sizeof(Misc) <= 128, "misc area");

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a));
    return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 x;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a));
    return x;
}

// Byte offset in a swizzled tile of D-byte rows: 16-byte piece `c` of row `r`.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    if constexpr (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
    else return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// The computing warps.
template <int D, bool kInt8>
struct Consumer {
    using C = Cfg<D>;
    static constexpr int kSteps = D / 16;   // k-steps of Q K^T, row tiles of V^T
    static constexpr int kCols = 2;         // groups of 8 query rows
    const DecodeParams &p;
    const Plan &w;
    uint8_t *smem;
    uint32_t base;
    int warp, lane, g, t;
    uint32_t q[kSteps][4];
    float qs[kCols];                         // c_r of rows g, g + 8
    float m[kCols], u[kCols], l[kCols];
    float o[kSteps][kCols][4];
    int row_tile, key_group, key_groups;
    uint32_t sync_phase;

    __device__ __forceinline__ uint32_t bar(int i) const { return base + C::kBar + 8u * (uint32_t)i; }

    // All computing warps meet.
    __device__ __forceinline__ bool meet(volatile int *abort) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(2 * C::kStages));
        const bool ok = mbar_wait(bar(2 * C::kStages), sync_phase, abort, p.err, BSATTN_FLAG_TIMEOUT);
        sync_phase ^= 1u;
        return __all_sync(0xffffffffu, ok);
    }

    __device__ __forceinline__ void begin(const Seg &s) {
        const int tiles = (s.rows + 15) / 16;
        const int R = tiles <= 2 ? 2 : tiles <= 4 ? 4 : 8;
        row_tile = warp % R;
        key_group = warp / R;
        key_groups = kConsumers / R;
#pragma unroll
        for (int hf = 0; hf < kCols; ++hf) {
            const int r = row_tile * 16 + g + 8 * hf;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.q + (long long)s.b * p.q_stride + (long long)(s.h * p.G + min(r, s.rows - 1)) * D + t * (D / 4));
            uint32_t x[D / 8], a = 0;        // D / 4 bf16 elements of the row
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 y = r < s.rows ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                x[4 * i] = y.x;
                x[4 * i + 1] = y.y;
                x[4 * i + 2] = y.z;
                x[4 * i + 3] = y.w;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) a = __vmaxu2(a, x[i] & 0x7fff7fffu);
            a = max(a & 0xffffu, a >> 16);
            a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
            float f;
            row_scale(a, p.scale_log2, f, qs[hf]);
            // k-step i / 2: elements 4 s, 4 s + 1 are a0 (a1 for row g + 8), 4 s + 2, 4 s + 3 are a2 (a3)
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                q[i / 2][2 * (i & 1) + hf] =
                    pack_f16x2(__uint_as_float(x[i] << 16) * f, __uint_as_float(x[i] & 0xffff0000u) * f);
            m[hf] = u[hf] = kNoKey;
            l[hf] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int n = 0; n < kCols; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[i][n][x] = 0.f;
    }

    // 16 keys of a stage (group c), the first nv of which count (all of them: kFull).
    template <bool kFull>
    __device__ __forceinline__ void keys16(uint32_t sk, uint32_t ssc, int c, int nv) {
        const uint32_t sv = sk + C::kCodes;
        float s[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
            const int r = 16 * c + 8 * nb + g;
            uint32_t x[D / 16];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint4 y = lds128(sk + piece_at<D>(r, (D / 64) * t + i));
                x[4 * i] = y.x;
                x[4 * i + 1] = y.y;
                x[4 * i + 2] = y.z;
                x[4 * i + 3] = y.w;
            }
            // two accumulators: half the length of the dependent chain
            float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t b0, b1;
                codes_to_f16x2<kInt8>(x[i], b0, b1);
                mma_f16(acc[i & 1], q[i][0], q[i][1], q[i][2], q[i][3], b0, b1);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nb][i] = acc[0][i] + acc[1][i];
        }
        // V: D / 8 codes of keys 2t, 2t + 1, 2t + 8, 2t + 9
        uint32_t v[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 2 * t + (i & 1) + 8 * (i >> 1), r = 16 * c + j;
            if constexpr (D == 128) {
                const uint4 y = lds128(sv + piece_at<D>(r, g));
                v[i][0] = y.x;
                v[i][1] = y.y;
                v[i][2] = y.z;
                v[i][3] = y.w;
            } else {
                const uint2 y = lds64(sv + piece_at<D>(r, g >> 1) + 8u * (g & 1));
                v[i][0] = y.x;
                v[i][1] = y.y;
            }
            if (!kFull && j >= nv) {  // what lies behind the last key may be NaN codes
#pragma unroll
                for (int x = 0; x < D / 32; ++x) v[i][x] = 0u;
            }
        }
        // x = z - m and y = z + log2 vs - u + 7 of this lane's keys 2t, 2t + 1, 2t + 8, 2t + 9
        float sc[kCols][4], lv[4], x[kCols][4], y[kCols][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
            const uint2 kb = lds64(ssc + 4u * (16 * c + 8 * nb + 2 * t));
            const uint2 vb = lds64(ssc + 512u + 4u * (16 * c + 8 * nb + 2 * t));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool on = kFull || 8 * nb + 2 * t + e < nv;
                lv[2 * nb + e] = lg2_approx(__uint_as_float(e ? vb.y : vb.x));
                if (!on) lv[2 * nb + e] = -INFINITY;
#pragma unroll
                for (int hf = 0; hf < kCols; ++hf) {
                    sc[hf][2 * nb + e] = s[nb][2 * hf + e] * __uint_as_float(e ? kb.y : kb.x);
                    if (!on) sc[hf][2 * nb + e] = -INFINITY;
                }
            }
        }
        float top[kCols];
        auto relative = [&](int hf) {
            const float mu = m[hf] - u[hf] + 7.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[hf][i] = fmaf(sc[hf][i], qs[hf], -m[hf]);
                y[hf][i] = x[hf][i] + (lv[i] + mu);
            }
            top[hf] = fmaxf(fmax3(x[hf][0], x[hf][1], x[hf][2]), x[hf][3]);
            top[hf] = fmaxf(top[hf], fmaxf(fmax3(y[hf][0], y[hf][1], y[hf][2]), y[hf][3]) - 7.f);
        };
        bool grow = false;
#pragma unroll
        for (int hf = 0; hf < kCols; ++hf) {
            relative(hf);
            grow |= top[hf] > 8.f;
        }
        // The references move only when some key is 2^8 above them: l and O stay finite
        // (weights reach 2^15 in fp16), and the quotient is the same.
        if (__any_sync(0xffffffffu, grow)) {
            float ao[kCols];
#pragma unroll
            for (int hf = 0; hf < kCols; ++hf) {
                float a = -INFINITY, b = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float z = sc[hf][i] * qs[hf];
                    a = fmaxf(a, z);
                    b = fmaxf(b, z + lv[i]);
                }
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 1));
                a = fmaxf(m[hf], fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2)));
                b = fmaxf(u[hf], fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 2)));
                l[hf] *= ex2_approx(m[hf] - a);
                ao[hf] = ex2_approx(u[hf] - b);
                m[hf] = a;
                u[hf] = b;
                relative(hf);
            }
            // O's columns are query rows 2t, 2t + 1 (and 8 above)
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
                const float a0 = __shfl_sync(0xffffffffu, ao[n], 8 * t);
                const float a1 = __shfl_sync(0xffffffffu, ao[n], 8 * t + 4);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    o[i][n][0] *= a0;
                    o[i][n][1] *= a1;
                    o[i][n][2] *= a0;
                    o[i][n][3] *= a1;
                }
            }
        }
        uint32_t pb[kCols][2];
#pragma unroll
        for (int hf = 0; hf < kCols; ++hf) {
            l[hf] += (ex2_approx(x[hf][0]) + ex2_approx(x[hf][1])) + (ex2_approx(x[hf][2]) + ex2_approx(x[hf][3]));
            pb[hf][0] = pack_f16x2(ex2_approx(y[hf][0]), ex2_approx(y[hf][1]));
            pb[hf][1] = pack_f16x2(ex2_approx(y[hf][2]), ex2_approx(y[hf][3]));
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            // bytes d, d + 1 of both keys of a pair side by side, then bytes d + 2, d + 3
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const uint32_t sel = hi ? 0x7362u : 0x5140u;
                uint32_t a0, a1, a2, a3;
                codes_to_f16x2<kInt8>(__byte_perm(v[0][w], v[1][w], sel), a0, a1);
                codes_to_f16x2<kInt8>(__byte_perm(v[2][w], v[3][w], sel), a2, a3);
#pragma unroll
                for (int n = 0; n < kCols; ++n) mma_f16(o[2 * w + hi][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
        }
    }

    // Joins the key groups of each row tile and writes the rows: every warp leaves its
    // sums and references in shared memory, all meet, and the warps of a row tile share
    // out its columns; they meet again before the next segment's sums are left there.
    __device__ __forceinline__ bool finish(const Seg &s, int seg, bool complete, volatile int *abort) {
        float4 *stat = reinterpret_cast<float4 *>(smem + C::kStat);
        float *red = reinterpret_cast<float *>(smem + C::kRed);
        constexpr int kRegs = kSteps * kCols * 4;
#pragma unroll
        for (int hf = 0; hf < kCols; ++hf) {
            l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
            l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
            if (t == 0)
                stat[(row_tile * 16 + g + 8 * hf) * key_groups + key_group] = make_float4(m[hf], u[hf], l[hf], 0.f);
        }
        {
            float *x = red + warp * kRegs * 32 + lane;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int n = 0; n < kCols; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[((i * kCols + n) * 4 + e) * 32] = o[i][n][e];
        }
        if (!meet(abort)) return false;
        const int R = kConsumers / key_groups;
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * t + e;  // a row of this lane's columns
                const float4 *st = stat + (row_tile * 16 + r) * key_groups;
                float bm = kNoKey, bu = kNoKey, ll = 0.f;
                for (int k = 0; k < key_groups; ++k) {
                    bm = fmaxf(bm, st[k].x);
                    bu = fmaxf(bu, st[k].y);
                }
                for (int k = 0; k < key_groups; ++k) ll += st[k].z * ex2_approx(st[k].x - bm);
                const bool empty = ll == 0.f;
                // no key with a value scale above 0: O is 0, whatever the quotient of the references
                const float2 inv = empty || bu == kNoKey ? make_float2(0.f, 0.f) : quotient(bu - bm - 7.f, ll);
                const float lse2 = empty ? -INFINITY : bm + lg2_approx(ll);
                if (row_tile * 16 + r < s.rows) {
                    const RowOut at = row_out(s, seg, complete, row_tile * 16 + r);
                    for (int i = key_group; i < kSteps; i += key_groups) {
                        float y0 = 0.f, y1 = 0.f;
                        for (int k = 0; k < key_groups; ++k) {
                            const float f = ex2_approx(st[k].y - bu);
                            const float *x = red + (k * R + row_tile) * kRegs * 32 + ((i * kCols + n) * 4 + e) * 32 + lane;
                            y0 = fmaf(f, x[0], y0);
                            y1 = fmaf(f, x[64], y1);
                        }
                        store_pair(at, g * (D / 8) + 2 * i, y0 * inv.x * inv.y, y1 * inv.x * inv.y);
                    }
                    if (key_group == 0 && g == 0) store_lse(p, w, at, lse2);
                }
            }
        return meet(abort);
    }

    __device__ __forceinline__ RowOut row_out(const Seg &s, int seg, bool complete, int r) const {
        if (complete && w.direct) return RowOut{0, (long long)s.b * p.Hq + s.h * p.G + r};
        return RowOut{2, ((long long)seg + blockIdx.x) * p.G + r};
    }

    __device__ __forceinline__ void store_pair(const RowOut &at, int d, float x, float y) const {
        if (at.kind == 0 && !p.out_f32) {
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + at.row * D + d) = pack_bf16x2(x, y);
        } else {
            float *o = at.kind == 0 ? static_cast<float *>(p.out)
                                    : reinterpret_cast<float *>(p.ws + w.suf_o);
            *reinterpret_cast<float2 *>(o + at.row * D + d) = make_float2(x, y);
        }
    }

    __device__ __forceinline__ void run(volatile int *abort) {
        Seg s = {};
        for (uint32_t it = 0;; ++it) {
            const uint32_t st = it % C::kStages;
            const bool ok = mbar_wait(bar(st), (it / C::kStages) & 1u, abort, p.err, BSATTN_FLAG_TIMEOUT);
            if (!__all_sync(0xffffffffu, ok)) return;
            const TileMsg msg = reinterpret_cast<const TileMsg *>(smem + C::kMsg)[st];
            if (msg.seg < 0) return;
            if (msg.flags & kFirst) {
                s = segment(p, w, msg.seg);
                begin(s);
            }
            const uint32_t sk = base + st * C::kStageBytes, ssc = base + C::kScales + st * 1024u;
            for (int c = key_group; c < 8; c += key_groups) {
                const int nv = min(16, msg.lim - 16 * c);
                if (nv <= 0 || !((msg.groups >> c) & 1u)) continue;
                if (nv == 16) keys16<true>(sk, ssc, c, nv);
                else keys16<false>(sk, ssc, c, nv);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kStages + st));
            if (msg.flags & kLast) {
                if (!finish(s, msg.seg, (msg.flags & kComplete) != 0, abort)) return;
            }
        }
    }
};

template <int D, bool kInt8>
__global__ void __launch_bounds__(kThreads, 1)
    bsattn_decode_rows_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ Plan w,
                         const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    Misc *misc = reinterpret_cast<Misc *>(smem + C::kMisc);
    volatile int *abort = &misc->abort;
    auto bar = [&](int i) -> uint32_t { return base + C::kBar + 8u * (uint32_t)i; };
    const int warp = (int)warp_id(), lane = (int)lane_id(), tid = threadIdx.x;
    grid_launch_dependents();  // the joining kernel may take its place; it waits for this grid
    // Beside the prefix kernel (which has waited) this one needs nothing that it writes.
    if (w.mode != kOwnKernel) grid_dependency_wait();
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar(s), 1);
            mbar_init(bar(C::kStages + s), kConsumers);
        }
        mbar_init(bar(2 * C::kStages), kConsumers);
        misc->abort = 0;
        misc->start_seg = w.ss;
        fence_barrier_init();
        fence_proxy_async_smem();
    }

    // Where this CTA's piece of the line of tiles begins.  Each thread sums the tiles of a
    // run of sequences (or, with lists, of (sequence, head) pairs); CTA c also writes the
    // records of every gridDim-th of them: the CTAs its segments' parts lie in.
    const int units = p.has_lists ? p.B * p.c.H : p.B, per = (units + kThreads - 1) / kThreads;
    const int u0 = min(units, tid * per), u1 = min(units, u0 + per);
    auto unit_tiles = [&](int x, bool check) -> int {
        if (!p.has_lists) return (seq_keys(p, x, check) + kTile - 1) / kTile;
        const int b = x / p.c.H, h = x - b * p.c.H;
        int n;
        const ListRow r = list_row(p, b, h, n, check);
        return r.full + r.mask;
    };
    const int reps = p.has_lists ? 1 : p.c.H;  // segments of a unit, of equal length
    long long sum = 0;
    for (int x = u0; x < u1; ++x) sum += (long long)unit_tiles(x, x % (int)gridDim.x == (int)blockIdx.x) * reps;
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) misc->warp_sum[warp] = incl;
    __syncthreads();
    long long at = incl - sum, total = 0;
    for (int i = 0; i <= kConsumers; ++i) {
        if (i < warp) at += misc->warp_sum[i];
        total += misc->warp_sum[i];
    }
    // no CTA's piece is empty while a later one's is not: a segment's parts are consecutive
    const long long cuts = min((long long)gridDim.x, total), cta = blockIdx.x;
    const long long lo = cta < cuts ? total * cta / cuts : 0, hi = cta < cuts ? total * (cta + 1) / cuts : 0;
    auto owner = [&](long long tile) -> int {
        const unsigned long long a = (unsigned long long)(tile + 1) * (unsigned long long)cuts - 1u;
        if (a <= 0xffffffffu) return (int)((unsigned)a / (unsigned)total);   // 64-bit division costs 10 times as much
        return (int)(a / (unsigned long long)total);
    };
    int2 *rec = reinterpret_cast<int2 *>(p.ws + w.rec);
    for (int x = u0; x < u1; ++x) {
        const bool mine = x % (int)gridDim.x == (int)blockIdx.x;
        const int n = unit_tiles(x, false);
        const long long end = at + (long long)n * reps;
        if (lo < hi && lo >= at && lo < end) {
            misc->start_seg = x * reps + (int)((lo - at) / n);
            misc->start_off = (lo - at) % n;
        }
        if (mine)
            for (int r = 0; r < reps; ++r) {
                const long long a = at + (long long)r * n;
                rec[x * reps + r] = n ? make_int2(owner(a), owner(a + n - 1)) : make_int2(0, -1);
            }
        at = end;
    }
    __syncthreads();
    if (lo >= hi) {
        if (w.mode == kOwnKernel) grid_dependency_wait();
        return;
    }

    if (warp == kConsumers) {
        // ------------------------------------------------------- producer --
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        const int ps_shift = p.c.page_shift, ps = 1 << ps_shift;
        const int ppt = kTile >> ps_shift, batch = 32 / ppt;   // pages per tile, tiles looked up at once
        const int mine = lane / ppt, sub = lane - mine * ppt;
        const uint32_t page_bytes = (uint32_t)ps * (2u * D + 8u);
        TileMsg *msgs = reinterpret_cast<TileMsg *>(smem + C::kMsg);
        uint32_t it = 0;
        bool ok = true;
        // A window of 32 segments, one per lane; x counts tiles from the window's first.
        int seg0 = misc->start_seg;
        long long x = misc->start_off, pos = lo;
        // (the segments end where the line does, unless a length is changed while the kernel runs)
        while (ok && pos < hi && seg0 < w.ss) {
            const int ws = seg0 + lane;
            int n = 0, nt = 0;
            ListRow r = {};
            if (ws < w.ss) {
                const int b = ws / p.c.H;
                n = seq_keys(p, b, false);
                nt = (n + kTile - 1) / kTile;
                if (p.has_lists) {
                    r = list_row(p, b, ws - b * p.c.H, n, false);
                    nt = r.full + r.mask;
                }
            }
            int incl = nt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            const int in_window = __shfl_sync(0xffffffffu, incl, 31);
            const int end = (int)min((long long)in_window, x + (hi - pos));
            for (int x0 = (int)x; ok && x0 < end; x0 += batch) {
                // lane: page `sub` of tile x0 + mine; the segment is the first whose end lies behind it
                const int xt = min(x0 + mine, end - 1);
                int at = 0;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    if (__shfl_sync(0xffffffffu, incl, at + d - 1) <= xt) at += d;
                const int seg = seg0 + at;
                const int sn = __shfl_sync(0xffffffffu, n, at), snt = __shfl_sync(0xffffffffu, nt, at);
                const int start = __shfl_sync(0xffffffffu, incl, at) - snt, i = xt - start;
                const int full = __shfl_sync(0xffffffffu, r.full, at), nn = __shfl_sync(0xffffffffu, r.nn, at);
                const long long list_at = __shfl_sync(0xffffffffu, r.at, at);
                const Seg s = segment(p, w, seg);
                int tile = i, lim = kTile, page = -1;
                if (p.has_lists) {
                    const bool masked = i >= full;
                    tile = __ldg((masked ? p.mask_idx + (i - full) : p.full_idx + i) + list_at);
                    if (tile < 0 || tile >= nn) {
                        if (sub == 0) raise(p, BSATTN_FLAG_BAD_INDEX);
                        tile = -1;
                    } else if (masked && p.vl) {
                        lim = min(kTile, __ldg(p.vl + (long long)s.b * p.list_n + tile));
                    }
                }
                lim = tile < 0 || tile * (long long)kTile >= sn ? 0 : min(lim, sn - tile * kTile);
                if ((sub << ps_shift) < lim) {
                    const int32_t *table = p.table + (long long)s.b * p.table_stride;
                    page = __ldg(table + ((tile * kTile) >> ps_shift) + sub);
                    if (page < 0 || page >= p.c.num_pages) {
                        raise(p, BSATTN_FLAG_BAD_INDEX);
                        page = -1;
                    }
                }
                // the CTA's piece begins at x (of this window) and ends hi - pos tiles behind it
                uint32_t fl = xt == max(start, (int)x) ? kFirst : 0u;
                if (i == snt - 1 || xt + 1 == x + (hi - pos)) fl |= kLast;
                if (start >= (int)x && i == snt - 1) fl |= kComplete;
                for (int j = 0; j < batch && x0 + j < end; ++j, ++it) {
                    const uint32_t st = it % C::kStages;
                    ok = mbar_wait(bar(C::kStages + st), ((it / C::kStages) & 1u) ^ 1u, abort, p.err,
                                   BSATTN_FLAG_TIMEOUT);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const bool load = mine == j && page >= 0;
                    const uint32_t loads = __ballot_sync(0xffffffffu, load);
                    const uint32_t groups = __reduce_or_sync(
                        0xffffffffu, load ? ((1u << (ps >> 4)) - 1u) << (sub * (ps >> 4)) : 0u);
                    if (mine == j && sub == 0) {
                        msgs[st] = TileMsg{seg, lim, groups, fl};
                        if (loads) mbar_arrive_expect_tx(bar(st), (uint32_t)__popc(loads) * page_bytes);
                        else mbar_arrive(bar(st));
                    }
                    __syncwarp();
                    if (load) {
                        const int row = ((page * p.c.H + s.h) << ps_shift), in = sub << ps_shift;
                        const uint32_t dst = base + st * C::kStageBytes + (uint32_t)in * D;
                        const uint32_t sc = base + C::kScales + st * 1024u + 4u * (uint32_t)in;
                        tma_load_2d(dst, &tk, bar(st), 0, row);
                        tma_load_2d(dst + C::kCodes, &tv, bar(st), 0, row);
                        bulk_g2s_lead(1u, sc, p.c.ks + row, 4u * (uint32_t)ps, bar(st));
                        bulk_g2s_lead(1u, sc + 512u, p.c.vs + row, 4u * (uint32_t)ps, bar(st));
                    }
                }
            }
            pos += end - x;
            x = 0;
            seg0 += 32;
        }
        if (ok) {
            const uint32_t st = it % C::kStages;
            ok = mbar_wait(bar(C::kStages + st), ((it / C::kStages) & 1u) ^ 1u, abort, p.err, BSATTN_FLAG_TIMEOUT);
            if (__all_sync(0xffffffffu, ok)) {
                if (lane == 0) {
                    msgs[st] = TileMsg{-1, 0, 0u, 0u};
                    mbar_arrive(bar(st));
                }
                ++it;
            }
        }
        // no copy into this CTA's shared memory may be in flight when it ends
        for (uint32_t s = 0; s < (uint32_t)C::kStages; ++s)
            if (it > s) mbar_wait_drain(bar((int)((it - 1 - s) % C::kStages)), ((it - 1 - s) / C::kStages) & 1u);
        // Launched beside the prefix kernel: this grid must not end before that one, since
        // the join waits for this grid alone.
        if (w.mode == kOwnKernel) grid_dependency_wait();
    } else {
        Consumer<D, kInt8> c{p, w, smem, base, warp, lane, lane >> 2, lane & 3};
        c.sync_phase = 0u;
        c.run(abort);
    }
}

template <int D, bool kInt8>
cudaError_t launch(const DecodeParams &p, const Plan &w, int sms, cudaStream_t stream) {
    using C = Cfg<D>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(bsattn_decode_rows_kernel<D, kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)C::kAlloc);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    CUtensorMap tk, tv;
    const long long rows = ((long long)(p.c.num_pages > 0 ? p.c.num_pages : 1) * p.c.H) << p.c.page_shift;
    if (!encode_code_rows(&tk, p.c.k, rows, D, 1 << p.c.page_shift) ||
        !encode_code_rows(&tv, p.c.v, rows, D, 1 << p.c.page_shift))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.stream = stream;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(sms < kMaxCtas ? sms : kMaxCtas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kAlloc;
    return cudaLaunchKernelEx(&cfg, bsattn_decode_rows_kernel<D, kInt8>, p, w, tk, tv);
}

}  // namespace

cudaError_t launch_decode_rows(const DecodeParams &p, const Plan &w, int sms, cudaStream_t stream) {
    if (p.c.D == 128) return p.c.int8 ? launch<128, true>(p, w, sms, stream) : launch<128, false>(p, w, sms, stream);
    return p.c.int8 ? launch<64, true>(p, w, sms, stream) : launch<64, false>(p, w, sms, stream);
}

}  // namespace bsattn
