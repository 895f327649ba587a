// Attention of one query token per sequence over a paged 8-bit K/V cache, alone or
// behind a prefix that every sequence of the batch shares: up to 16 query heads per KV
// head (more: bsattn_decode_rows.cu), and the kernel that joins parts.
//
// For one KV head, query rows r (the head's G queries of one sequence; for the prefix
// the queries of every sequence) meet keys j:
//   z_rj = c_r ks_j (q'_r . kcode_j),  c_r = softmax_scale log2(e) 2^e_r, q' = q 2^-e_r,
//   l_r = sum_j 2^(z_rj - m_r),  O_r = sum_j 2^(z_rj + log2 vs_j - u_r) vcode_j,
//   out_r = O_r 2^(u_r - m_r) / l_r,  lse_r = ln 2 (m_r + log2 l_r),
// with running references m_r and u_r.  Both products run on the tensor cores in fp16
// with fp32 accumulation: codes (e4m3 or int8) are exact in fp16, and so is q' for every
// element that matters (2^e_r is the row's largest binary exponent, so q' keeps all 8
// bits of a bf16 element down to 2^-14 of the largest).  The weight of a key carries
// its value scale in the exponent, with a reference u_r of its own: what is rounded to
// fp16 (11 bits) is a number relative to the largest contribution, whatever the scales
// are, and 2^7 of headroom keeps full precision down to 2^-21 of that.
//
// Bound by HBM: 2 (D + 4) bytes per key and KV head, 4 D flop per query on it.  Measured
// (D = 128, each call on other memory than the one before): 131072 keys x 32 heads (e4m3)
// 177 us, 6.2 TB/s of 6.7; 64 sequences of 100 .. 4096 keys x 8 heads, 4 queries a head (int8)
// 57.5 us, 4.9 TB/s: 5 us until the first codes
// arrive (the look-up of the pieces 2, of the pages 1), 6 to 8 us from the first warp that is
// done to the last (the SMs do not reach HBM equally fast, and pieces handed out as warps come
// free cost more than they save), 3 us for the join.  2 sequences of 1024 keys x 4 heads:
// 8.6 to 9.7 us, the latencies of the two launches.  Times beside the rules below are of calls
// in a graph over the same memory, which for small ones lies in L2.
//
// Work split.  Every warp is a worker of its own.  A segment is one (sequence, KV head),
// or one KV head of the prefix while at most 16 query rows a head meet it (more take
// bsattn_prefix.cu); its keys are groups of 16.  The groups of all segments form one
// line, where a segment also counts kSegCost groups for what it costs to start and end
// one, and the line is cut evenly over the warps of the device: every warp streams the
// same number of bytes whatever the lengths.  A warp holds the query rows and the sums in
// registers and keeps a ring of its own in shared memory full with asynchronous copies;
// nothing in its loop waits for another warp.  A segment within one warp's piece is finished
// there; the parts of the others (fp32 output and LSE) go to the workspace, and a second
// kernel, a programmatic dependent of the first, joins them.
//
// Fragments without a transpose.  In S = Q K^T (m16n8k16) the contraction index may be
// permuted alike on both sides, so lane 4g + t takes the D / 4 consecutive codes d =
// (D / 4) t .. of key g, four per k-step.  In O^T = V^T P^T the rows d may be permuted
// freely, so the lane takes D / 8 consecutive codes of each of its four keys and
// interleaves the bytes of two keys before they are widened.  P leaves the first product
// in the layout the second wants.  16-byte pieces lie at piece ^ (row mod 8) (D = 64:
// piece ^ (row / 2 mod 4)): no 16-byte load meets a bank twice (the 8-byte loads of V at
// D = 64 do, two ways).
#include "bsattn_internal.h"
#include "decode_common.cuh"
#include "kv_codes.cuh"

namespace bsattn {

namespace {

// Groups of 16 keys that starting and ending a segment costs: 128 sequences of 1 .. 400 keys,
// 8 heads: 25.5 us a call with 0, 20.5 with 2, 21.0 with 4.
constexpr int kSegCost = 2;
constexpr int kMinPiece = 2;  // places that make a worker of their own worth its part in the join (1, 4, 8 measured
                              // slower on short calls)

// 16 bytes from global to shared memory, past L1; counted by the thread's copy groups.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Loads that stay where they are written (the query rows go out before the look-ups).
__device__ __forceinline__ uint4 ld_row16(const uint16_t *p) {
    uint4 x;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
    return x;
}

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

// Byte offset of 16-byte piece `c` of row `r` in a group's codes.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    if constexpr (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
    else return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// A warp's ring: per stage the codes of 16 keys (K, then V) and their scales (K, then V).
template <int D, int kCols>
struct Ring {
    static constexpr int kWarps = kCols == 1 ? kStreamWarps : 12;      // per CTA
    static constexpr int kCtas = kCols == 1 ? 2 : 1;                   // per SM
    static constexpr uint32_t kCodes = 16u * D;
    static constexpr uint32_t kStage = 2u * kCodes + 128u;
    // ~200 KB in flight per SM (HBM needs 44 KB at 6.7 TB/s and ~1 us).  131072 keys x 32 heads
    // with 5, 6, 7, 8 warps a CTA (4, 4, 3, 3 stages): 184, 176, 184, 173 us.
    static constexpr int kStages = (int)(101376u * (2 / kCtas) / (kWarps * kStage));
    static constexpr uint32_t kBytes = kWarps * kStages * kStage;
};

// The segment that a warp works on; in shared memory, where looking groups up and finishing
// find it, since the loop over groups needs every register.
struct SegKeys {
    Seg s;
    ListRow lists;
    int n, lead;   // keys, groups of the shared prefix before them
};

// One warp's state: kCols groups of 8 query rows.
template <int D, bool kInt8, int kCols>
struct Worker {
    static constexpr int kSteps = D / 16;        // k-steps of Q K^T, row tiles of V^T
    const DecodeParams &p;
    int lane, g, t;
    uint32_t q[kSteps][2 * kCols];
    float qs[kCols];                             // c_r of rows g, g + 8
    float m[kCols], u[kCols], l[kCols];
    float o[kSteps][kCols][4];
    uint32_t ring;                               // shared address of the warp's ring

    using R = Ring<D, kCols>;

    // The segment's query rows, as they lie: D / 4 bf16 elements of rows g, g + 8.
    struct RawRows {
        uint4 x[kCols][D / 32];
    };
    __device__ __forceinline__ void load_rows(const Seg &s, RawRows &raw) const {
#pragma unroll
        for (int hf = 0; hf < kCols; ++hf) {
            const int r = g + 8 * hf;
            const int b = s.prefix ? r / p.G : s.b, gi = s.prefix ? r - b * p.G : r;
            const uint16_t *row = p.q + (long long)b * p.q_stride + (long long)(s.h * p.G + gi) * D + t * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                raw.x[hf][i] = make_uint4(0, 0, 0, 0);
                if (r < s.rows) raw.x[hf][i] = ld_row16(row + 8 * i);
            }
        }
    }

    __device__ __forceinline__ void begin(const RawRows &raw) {
#pragma unroll
        for (int hf = 0; hf < kCols; ++hf) {
            uint32_t x[D / 8], a = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                x[4 * i] = raw.x[hf][i].x;
                x[4 * i + 1] = raw.x[hf][i].y;
                x[4 * i + 2] = raw.x[hf][i].z;
                x[4 * i + 3] = raw.x[hf][i].w;
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
                q[i / 2][kCols * (i & 1) + hf] =
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

    // Starts the copies of the group whose first key is row `row` of the cache.
    __device__ __forceinline__ void fetch(uint32_t stage, int row) {
        constexpr int kPieces = D / 16, kRowsPerStep = 32 / kPieces;
        const int r0 = lane / kPieces, c = lane % kPieces;
        const long long at = (long long)row * D + lane * 16;
#pragma unroll
        for (int i = 0; i < 16 / kRowsPerStep; ++i) {
            const uint32_t dst = stage + piece_at<D>(r0 + i * kRowsPerStep, c);
            copy16(dst, p.c.k + at + i * 512);
            copy16(dst + R::kCodes, p.c.v + at + i * 512);
        }
        if (lane < 8)
            copy16(stage + 2 * R::kCodes + lane * 16, (lane < 4 ? p.c.ks : p.c.vs) + row + (lane & 3) * 4);
    }

    __device__ __forceinline__ void mma_q(float (&c)[4], int i, uint32_t b0, uint32_t b1) const {
        if constexpr (kCols == 2) mma_f16(c, q[i][0], q[i][1], q[i][2], q[i][3], b0, b1);
        else mma_f16(c, q[i][0], 0u, q[i][1], 0u, b0, b1);
    }

    // The group in `stage`, the first nv keys of which count (all 16: kFull).
    template <bool kFull>
    __device__ __forceinline__ void keys16(uint32_t stage, int nv) {
        float s[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
            uint32_t kx[D / 16];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint4 y = lds128(stage + piece_at<D>(8 * nb + g, (D / 64) * t + i));
                kx[4 * i] = y.x;
                kx[4 * i + 1] = y.y;
                kx[4 * i + 2] = y.z;
                kx[4 * i + 3] = y.w;
            }
            // two accumulators: half the length of the dependent chain
            float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t b0, b1;
                codes_to_f16x2<kInt8>(kx[i], b0, b1);
                mma_q(acc[i & 1], i, b0, b1);
            }
#pragma unroll
            for (int i = 0; i < 2 * kCols; ++i) s[nb][i] = acc[0][i] + acc[1][i];
        }
        // x = z - m and y = z + log2 vs - u + 7 of this lane's keys 2t, 2t + 1, 2t + 8, 2t + 9
        float sc[kCols][4], lv[4], x[kCols][4], y[kCols][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
            const uint2 kb = lds64(stage + 2 * R::kCodes + 4u * (8 * nb + 2 * t));
            const uint2 vb = lds64(stage + 2 * R::kCodes + 64u + 4u * (8 * nb + 2 * t));
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
        // V: D / 8 codes of keys 2t, 2t + 1, 2t + 8, 2t + 9
        uint32_t vx[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 2 * t + (i & 1) + 8 * (i >> 1);
            if constexpr (D == 128) {
                const uint4 y = lds128(stage + R::kCodes + piece_at<D>(r, g));
                vx[i][0] = y.x;
                vx[i][1] = y.y;
                vx[i][2] = y.z;
                vx[i][3] = y.w;
            } else {
                const uint2 y = lds64(stage + R::kCodes + piece_at<D>(r, g >> 1) + 8u * (g & 1));
                vx[i][0] = y.x;
                vx[i][1] = y.y;
            }
            if (!kFull && r >= nv) {  // what lies behind the last key may be NaN codes
#pragma unroll
                for (int w = 0; w < D / 32; ++w) vx[i][w] = 0u;
            }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            // bytes d, d + 1 of both keys of a pair side by side, then bytes d + 2, d + 3
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const uint32_t sel = hi ? 0x7362u : 0x5140u;
                uint32_t a0, a1, a2, a3;
                codes_to_f16x2<kInt8>(__byte_perm(vx[0][w], vx[1][w], sel), a0, a1);
                codes_to_f16x2<kInt8>(__byte_perm(vx[2][w], vx[3][w], sel), a2, a3);
#pragma unroll
                for (int n = 0; n < kCols; ++n) mma_f16(o[2 * w + hi][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
        }
    }

    // Starts a segment of n keys, behind `lead` groups of the shared prefix, and works on
    // its groups t0 .. t1.
    __device__ __forceinline__ void groups(const SegKeys *seg_keys, int t0, int t1) {
        const Seg &s = seg_keys->s;
        // cache row of group i's first key (-1: nothing to read) and how many of its keys count, one group per lane
        auto look_up = [&](int i, int &row, int &nv) {
            row = -1;
            nv = 0;
            if (i >= t1) return;
            const ListRow &lr = seg_keys->lists;
            const int lead = seg_keys->lead, n = seg_keys->n;
            const bool own = !s.prefix && i >= lead;   // not a group of the shared prefix
            const int32_t *table = own ? p.table + (long long)s.b * p.table_stride : p.prefix_table;
            int keys = own ? n : p.prefix_len, lim = 16;
            if (own) i -= lead;
            int key = i * 16;
            if (p.has_lists && own) {
                const int e = i >> 3;
                const bool masked = e >= lr.full;
                const int tile = __ldg((masked ? p.mask_idx + (e - lr.full) : p.full_idx + e) + lr.at);
                if (tile < 0 || tile >= lr.nn) {
                    if ((i & 7) == 0 || i + lead == t0) raise(p, BSATTN_FLAG_BAD_INDEX);
                    return;
                }
                if (tile >= (n + kTile - 1) / kTile) return;
                key = tile * kTile + (i & 7) * 16;
                if (masked && p.vl) lim = __ldg(p.vl + (long long)s.b * p.list_n + tile) - (i & 7) * 16;
            }
            nv = min(min(lim, 16), keys - key);
            if (nv <= 0) return;
            const int page = __ldg(table + (key >> p.c.page_shift));
            if (page < 0 || page >= p.c.num_pages) {
                raise(p, BSATTN_FLAG_BAD_INDEX);
                return;
            }
            row = ((page * p.c.H + s.h) << p.c.page_shift) + (key & ((1 << p.c.page_shift) - 1));
        };
        int row0, nv0, row1 = -1, nv1 = 0;
        RawRows raw;
        load_rows(s, raw);
        look_up(t0 + lane, row0, nv0);
        // kStages - 1 groups are on their way while one is worked on; a group without keys
        // takes its turn as an empty copy group
        constexpr int kLead = R::kStages - 1;
#pragma unroll
        for (int k = 0; k < kLead; ++k) {
            const int row = __shfl_sync(0xffffffffu, row0, k);
            if (row >= 0) fetch(ring + k * R::kStage, row);
            copy_commit();
        }
        begin(raw);
        uint32_t cur = ring, ahead = ring + kLead * R::kStage;
        constexpr uint32_t kWrap = R::kStages * R::kStage;
        for (int i = t0; i < t1; ++i) {
            const int j = (i - t0) & 31;
            if (j == 0) look_up(i + 32 + lane, row1, nv1);
            const int far = __shfl_sync(0xffffffffu, j + kLead < 32 ? row0 : row1, (j + kLead) & 31);
            if (far >= 0) fetch(ahead, far);   // the stage that every lane left in the round before
            copy_commit();
            const int row = __shfl_sync(0xffffffffu, row0, j), nv = __shfl_sync(0xffffffffu, nv0, j);
            copy_wait<kLead>();
            __syncwarp();
            if (row >= 0) {
                if (nv == 16) keys16<true>(cur, nv);
                else keys16<false>(cur, nv);
            }
            __syncwarp();
            cur = cur + R::kStage == ring + kWrap ? ring : cur + R::kStage;
            ahead = ahead + R::kStage == ring + kWrap ? ring : ahead + R::kStage;
            if (j == 31) {
                row0 = row1;
                nv0 = nv1;
            }
        }
        copy_wait<0>();  // only empty groups are left
        __syncwarp();
    }

    // Writes the rows of a segment (or of the part of it that this worker has).
    __device__ __forceinline__ void finish(const Plan &w, const SegKeys *seg_keys, int seg, int worker, bool complete) {
        const Seg &s = seg_keys->s;
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
            const bool empty = l[n] == 0.f;
            // no key with a value scale above 0: O is 0, whatever the quotient of the references
            const float2 own_inv = empty || u[n] == kNoKey ? make_float2(0.f, 0.f) : quotient(u[n] - m[n] - 7.f, l[n]);
            const float own_lse = empty ? -INFINITY : m[n] + lg2_approx(l[n]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float inv = __shfl_sync(0xffffffffu, own_inv.x, 8 * t + 4 * e);
                const float rest = __shfl_sync(0xffffffffu, own_inv.y, 8 * t + 4 * e);
                const float lse2 = __shfl_sync(0xffffffffu, own_lse, 8 * t + 4 * e);
                const int r = 8 * n + 2 * t + e;
                if (r >= s.rows) continue;
                float y[D / 8];                  // elements (D / 8) g ..
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    y[2 * i] = o[i][n][e] * inv * rest;
                    y[2 * i + 1] = o[i][n][2 + e] * inv * rest;
                }
                RowOut at;
                if (!s.prefix && complete && w.direct) at = RowOut{0, (long long)s.b * p.Hq + s.h * p.G + r};
                else if (s.prefix) at = RowOut{1, ((long long)seg + worker) * w.rows_p + r};
                else at = RowOut{2, ((long long)(seg - w.sp) + worker) * p.G + r};
                if (at.kind == 0 && !p.out_f32) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at.row * D + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
                        dst[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                            pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
                } else {
                    float *dst = at.kind == 0 ? static_cast<float *>(p.out)
                                              : reinterpret_cast<float *>(p.ws + (at.kind == 1 ? w.pre_o : w.suf_o));
                    dst += at.row * D + g * (D / 8);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        reinterpret_cast<float4 *>(dst)[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                }
                if (g == 0) store_lse(p, w, at, lse2);
            }
        }
    }
};

// One group of columns takes two CTAs of 8 warps per SM at 128 registers a thread; two
// groups take 12 warps at 168.
template <int D, bool kInt8, int kCols>
__global__ void __launch_bounds__(Ring<D, kCols>::kWarps * 32, Ring<D, kCols>::kCtas)
    bsattn_decode_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ Plan w) {
    using R = Ring<D, kCols>;
    constexpr int kW = R::kWarps, kThreads = kW * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long warp_sum[kW], run_at[kThreads], piece[kW][2], start_at[kW], line[2];
    __shared__ int start_seg[kW];
    __shared__ SegKeys seg_keys[kW];
    const int warp = (int)warp_id(), lane = (int)lane_id(), tid = threadIdx.x;
    grid_launch_dependents();  // the joining kernel may take its place; it waits for this grid
    // Beside the prefix kernel (which has waited) this one needs nothing that it writes.
    if (w.mode != kOwnKernel) grid_dependency_wait();

    // Where each worker's piece of the line begins.  Each thread sums the cost of a run
    // of sequences (or, with lists, of (sequence, head) pairs); CTA c also checks every
    // gridDim-th of them and writes the records of those without keys.  The record of any
    // other segment, the workers its parts lie with, is written by the first of these.
    // Each warp then looks for the run, and in it the segment, that its piece begins in.
    const int g_pre = w.sp ? (p.prefix_len + 15) / 16 : 0, lead = w.mode == kEach ? (p.prefix_len + 15) / 16 : 0;
    const long long line_pre = (long long)w.sp * (g_pre + kSegCost);
    const int units = p.has_lists ? p.B * p.c.H : p.B, per = (units + kThreads - 1) / kThreads;
    const int u0 = min(units, tid * per), u1 = min(units, u0 + per);
    auto unit_groups = [&](int x, bool check) -> int {
        if (!p.has_lists) return lead + (seq_keys(p, x, check) + 15) / 16;
        const int b = x / p.c.H, h = x - b * p.c.H;
        int n;
        const ListRow r = list_row(p, b, h, n, check);
        return lead + 8 * (r.full + r.mask);
    };
    const int reps = p.has_lists ? 1 : p.c.H;  // segments of a unit, of equal length
    long long sum = 0;
    for (int x = u0; x < u1; ++x) {
        const int n = unit_groups(x, x % (int)gridDim.x == (int)blockIdx.x);
        sum += n ? (long long)(n + kSegCost) * reps : 0;
    }
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long at = line_pre + incl - sum, total = line_pre;
    for (int i = 0; i < kW; ++i) {
        if (i < warp) at += warp_sum[i];
        total += warp_sum[i];
    }
    run_at[tid] = at;
    int2 *rec = reinterpret_cast<int2 *>(p.ws + w.rec);
    for (int x = u0; x < u1; ++x)
        if (x % (int)gridDim.x == (int)blockIdx.x && unit_groups(x, false) == 0)
            for (int r = 0; r < reps; ++r) rec[w.sp + x * reps + r] = make_int2(0, -1);
    __syncthreads();
    // pieces of kMinPiece places or a few less: a segment's parts lie with consecutive workers
    const long long cuts = min((long long)gridDim.x * kW, (total + kMinPiece - 1) / kMinPiece);
    if (const long long worker = (long long)blockIdx.x * kW + warp; worker < cuts) {
        const long long lo = line_div(total * worker, cuts);
        int seg;
        long long begin;   // where it begins
        if (lo < line_pre) {
            seg = (int)line_div(lo, g_pre + kSegCost);
            begin = (long long)seg * (g_pre + kSegCost);
        } else {
            int run = -1;   // the last run that begins at or before lo
#pragma unroll
            for (int i = 0; i < kThreads; i += 32) run += __popc(__ballot_sync(0xffffffffu, run_at[i + lane] <= lo));
            begin = run_at[run];
            const int run_end = min(units, (run + 1) * per);
            for (int x0 = run * per;; x0 += 32) {   // 32 of its units at a time
                const int n = x0 + lane < run_end ? unit_groups(x0 + lane, false) : 0;
                const long long len = n ? (long long)(n + kSegCost) * reps : 0;
                long long end = len;
                if (per > 1) {
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const long long y = __shfl_up_sync(0xffffffffu, end, d);
                        if (lane >= d) end += y;
                    }
                }
                end += begin;
                const unsigned behind = __ballot_sync(0xffffffffu, end > lo);
                if (behind == 0u && x0 + 32 < run_end) {
                    begin = __shfl_sync(0xffffffffu, end, 31);
                    continue;
                }
                const int hit = behind ? __ffs(behind) - 1 : 31, un = __shfl_sync(0xffffffffu, n, hit) + kSegCost;
                begin = __shfl_sync(0xffffffffu, end - len, hit);
                const int k = (int)line_div(lo - begin, un);
                begin += (long long)k * un;
                seg = w.sp + (x0 + hit) * reps + k;
                break;
            }
        }
        if (lane == 0) {
            piece[warp][0] = lo;
            piece[warp][1] = line_div(total * (worker + 1), cuts);
            start_at[warp] = begin;
            start_seg[warp] = seg;
        }
    }
    if (tid == 0) line[0] = total, line[1] = cuts;
    __syncthreads();
    // what is needed between segments waits in shared memory: a segment's groups take every register
    auto owner = [&](long long place) -> int {
        const volatile long long *l = line;
        return (int)line_div((place + 1) * l[1] - 1, l[0]);
    };
    if ((int)blockIdx.x * kW + warp < line[1]) {
        const int worker = (int)blockIdx.x * kW + warp;
        const volatile long long *pc = piece[warp];
        int seg = start_seg[warp];
        // (the segments end where the line does, unless a length is changed while the kernel runs)
        for (long long begin = start_at[warp]; begin < pc[1] && seg < w.sp + w.ss; ++seg) {
            const Seg s = segment(p, w, seg);
            int n = p.prefix_len, g;
            ListRow lr = {};
            if (p.has_lists && !s.prefix) {
                lr = list_row(p, s.b, s.h, n, false);
                g = 8 * (lr.full + lr.mask);
            } else {
                if (!s.prefix) n = seq_keys(p, s.b, false);
                g = (n + 15) / 16;
            }
            if (!s.prefix) g += lead;
            if (g == 0) continue;
            const long long first = begin + kSegCost;
            const int t0 = (int)max(0ll, min((long long)g, pc[0] - first)), t1 = (int)max(0ll, min((long long)g, pc[1] - first));
            if (t0 < t1) {
                if (t0 == 0 && lane == 0) rec[seg] = make_int2(worker, t1 == g ? worker : owner(first + g - 1));
                Worker<D, kInt8, kCols> k{p, lane, lane >> 2, lane & 3};
                k.ring = smem_u32(smem) + (uint32_t)warp * R::kStages * R::kStage;
                __syncwarp();
                if (lane == 0) seg_keys[warp] = SegKeys{s, lr, n, lead};
                __syncwarp();
                k.groups(&seg_keys[warp], t0, t1);
                k.finish(w, &seg_keys[warp], seg, worker, t0 == 0 && t1 == g);
            }
            begin = first + g;
        }
    }
    // Launched beside the prefix kernel: this grid must not end before that one, since the
    // join waits for this grid alone.
    if (w.mode == kOwnKernel) grid_dependency_wait();
}

// Joins the parts of one output row: out = sum_i o_i 2^(L_i - L), L = log2 sum_i 2^L_i.
// One block per row, its warps share the parts; a row that the first kernel finished is
// left alone.  Few rows have many parts each: blocks have 16 warps while four such blocks
// per SM hold all rows, else 4 (us a call, 16 : 4 warps: 32 rows of 131072 keys 177 : 179.5,
// 512 rows behind a prefix of 8192 keys 28.6 : 29.7; 2048 rows of 100 .. 4096 keys 64 : 56).
template <int D, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) bsattn_decode_join_kernel(const __grid_constant__ DecodeParams p,
                                                                            const __grid_constant__ Plan w) {
    grid_launch_dependents();
    grid_dependency_wait();
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = (int)blockIdx.x;
    const int b = row / p.Hq, hq = row - b * p.Hq, h = hq / p.G, gi = hq - h * p.G;
    const int2 *rec = reinterpret_cast<const int2 *>(p.ws + w.rec);
    const int2 rs = rec[w.sp + b * p.c.H + h];
    // the prefix's parts of this row: np of them, pre_step rows apart
    int np = 0;
    long long pre_row = 0, pre_step = w.rows_p;
    const int r = b * p.G + gi;
    if (w.mode == kInLine) {
        const int2 rp = rec[h];
        np = rp.y - rp.x + 1;
        pre_row = (long long)(h + rp.x) * w.rows_p + r;
    } else if (w.mode == kOwnKernel) {
        const int blk = r / kBlockRows, sp = h * w.row_blocks + blk;
        const int nt = (p.prefix_len + kTile - 1) / kTile;
        const int c0 = w.pre_owner(sp, 0, nt), c1 = w.pre_owner(sp, nt - 1, nt);
        np = c1 - c0 + 1;
        pre_row = (long long)(sp + c0) * w.rows_p + (r - blk * kBlockRows);
        if (p.B * p.G - blk * kBlockRows <= kTile) {  // both slots hold parts of the row
            np *= 2;
            pre_step = kTile;
        }
    } else if (rs.x == rs.y) {
        return;
    }
    const int n = np + rs.y - rs.x + 1;
    const long long suf_row = (long long)(b * p.c.H + h + rs.x) * p.G + gi;
    const float *pre_o = reinterpret_cast<const float *>(p.ws + w.pre_o), *pre_l = reinterpret_cast<const float *>(p.ws + w.pre_l);
    const float *suf_o = reinterpret_cast<const float *>(p.ws + w.suf_o), *suf_l = reinterpret_cast<const float *>(p.ws + w.suf_l);
    auto at = [&](int i) -> long long { return i < np ? pre_row + i * pre_step : suf_row + (long long)(i - np) * p.G; };
    // A warp's parts in rounds of kRound, whose loads go out together; a NaN is carried by the weights.
    constexpr int kRound = 4;
    float o[E], l = 0.f, base = kNoKey;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int i0 = warp; i0 < n; i0 += kJoinWarps * kRound) {
        float x[kRound], y[kRound][E], top = base;
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
            const int i = i0 + k * kJoinWarps;
            x[k] = -INFINITY;
#pragma unroll
            for (int e = 0; e < E; ++e) y[k][e] = 0.f;
            if (i < n) {
                const long long at_i = at(i);
                const float *src = (i < np ? pre_o : suf_o) + at_i * D + lane * E;
                x[k] = (i < np ? pre_l : suf_l)[at_i];
                if constexpr (E == 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(src);
                    y[k][0] = f.x, y[k][1] = f.y, y[k][2] = f.z, y[k][3] = f.w;
                } else {
                    const float2 f = *reinterpret_cast<const float2 *>(src);
                    y[k][0] = f.x, y[k][1] = f.y;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kRound; ++k) top = fmaxf(top, x[k]);
        const float a = ex2_approx(base - top);
        base = top;
        l *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= a;
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
            const float f = ex2_approx(x[k] - base);
            l += f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(f, y[k][e], o[e]);
        }
    }
    __shared__ float so[kJoinWarps][D], sl[kJoinWarps], sb[kJoinWarps];
    if (n > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
        if (lane == 0) sl[warp] = l, sb[warp] = base;
        __syncthreads();
        if (warp > 0) return;
        float top = base;
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) top = fmaxf(top, sb[k]);
        float a = ex2_approx(base - top);
        l *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= a;
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) {
            a = ex2_approx(sb[k] - top);
            l = fmaf(sl[k], a, l);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(so[k][lane * E + e], a, o[e]);
        }
        base = top;
    } else if (warp > 0) {
        return;
    }
    const bool empty = l == 0.f;   // NaN is not empty
    const float inv = empty ? 0.f : 1.f / l;
    const long long dst = (long long)row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float y0 = o[e] * inv, y1 = o[e + 1] * inv;
        if (p.out_f32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + dst + e) = make_float2(y0, y1);
        else *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + dst + e) = pack_bf16x2(y0, y1);
    }
    if (lane == 0) p.lse[row] = empty ? -INFINITY : (base + lg2_approx(l)) * 0.69314718055994530942f;
}

template <int D, bool kInt8, int kCols>
cudaError_t launch(const DecodeParams &p, const Plan &w, int sms, cudaStream_t stream) {
    using R = Ring<D, kCols>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(bsattn_decode_kernel<D, kInt8, kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)R::kBytes);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.stream = stream;
    cfg.numAttrs = 1;
    const int most = kMaxCtas * kStreamWarps / R::kWarps;
    const int grid = sms * R::kCtas;
    cfg.gridDim = dim3((unsigned)(grid < most ? grid : most));
    cfg.blockDim = dim3(R::kWarps * 32);
    cfg.dynamicSmemBytes = R::kBytes;
    return cudaLaunchKernelEx(&cfg, bsattn_decode_kernel<D, kInt8, kCols>, p, w);
}

template <int D>
cudaError_t launch_d(const DecodeParams &p, const Plan &w, int sms, cudaStream_t stream) {
    cudaError_t e;
    if (!w.streaming) {
        e = launch_decode_rows(p, w, sms, stream);
    } else if (p.G <= 8 && (w.mode != kInLine || p.B * p.G <= 8)) {
        e = p.c.int8 ? launch<D, true, 1>(p, w, sms, stream) : launch<D, false, 1>(p, w, sms, stream);
    } else {
        e = p.c.int8 ? launch<D, true, 2>(p, w, sms, stream) : launch<D, false, 2>(p, w, sms, stream);
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3((unsigned)((long long)p.B * p.Hq));
    if ((long long)p.B * p.Hq <= 4ll * sms) {
        cfg.blockDim = dim3(16 * 32);
        return cudaLaunchKernelEx(&cfg, bsattn_decode_join_kernel<D, 16>, p, w);
    }
    cfg.blockDim = dim3(4 * 32);
    return cudaLaunchKernelEx(&cfg, bsattn_decode_join_kernel<D, 4>, p, w);
}

}  // namespace

size_t decode_workspace_bytes(int B, int H, int G, int D, int prefix_len) {
    return make_plan(B, H, G, D, prefix_len, 0).total;
}

cudaError_t launch_decode(const DecodeParams &p, cudaStream_t stream) {
    const int sms = current_device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const Plan w = make_plan(p.B, p.c.H, p.G, p.c.D, p.prefix_len, sms);
    if (w.mode == kOwnKernel) {
        const cudaError_t e = launch_prefix(p, w, stream);
        if (e != cudaSuccess) return e;
    }
    return p.c.D == 128 ? launch_d<128>(p, w, sms, stream) : launch_d<64>(p, w, sms, stream);
}

}  // namespace bsattn
