// The shared prefix of a decoding batch, when many query rows meet it: tcgen05 kernel.
//
// For one KV head, the queries of every sequence are rows of one attention over the
// prefix's keys, 4 D flop per row and key against 2 (D + 4) bytes per key: from about
// 150 rows on the products bound it, not HBM.  The 8-bit codes are widened once per 256
// rows, in shared memory:
//   K' = fp16(code) 2^(f - F + 6), exact: f the binary exponent of the key's scale, F the
//        largest in the tile; what is left of the scale, r in [1, 2), multiplies the
//        key's scores in fp32, and only where some key of 32 has r != 1 (int8; the scales
//        that e4m3 rows are given are powers of two).  Where f < F - 14 it is
//        K' = fp16(code) 2^6 and r times 2^(f - F) instead;
//   V' = fp16(code) fp16(vs 2^(6 - E)), E the largest binary exponent of a value scale
//        so far (O is rescaled when it grows): exact for power-of-two scales, otherwise
//        off by two roundings to 11 bits;
//   Q' = fp16(q 2^-e), e the row's largest binary exponent (as in bsattn_decode.cu).
// With t_j the scores in true units and c = softmax_scale log2(e) 2^e: p_j = 2^(c t_j - m + 7)
// is rounded to fp16 for P V', l sums it in fp32; out = O 2^(E - 6) / l, log2-LSE = m - 7 +
// log2 l.  The reference m is moved only when some weight could pass 2^15.
//
// A weight below 2^-32 of the largest is 0 in fp16, which is enough while the value scales lie
// within 2^13 of each other.  From the first tile on where they do not, the weights of P V'
// carry them as in bsattn_decode.cu: V' = fp16(code) fp16(vs 2^(6 - f)), p_j = 2^(c t_j + f - E -
// u + 7) with a reference u of their own, out = O 2^(u - m + E - 6) / l.  A call where every
// tile does so takes 1.5 to 1.8 (64 and 128 rows) or 2.4 to 2.7 times (512) as long; the limit
// leaves out a first token whose values are 2^8 smaller than the others', as models learn it.
//
// A segment is (KV head, 256 query rows): two 128-row tiles ("slots") that share each
// K/V tile.  With 128 rows or fewer both slots hold the same rows and take the key tiles
// in turn, each with sums of its own: the softmax of one slot always runs beside the
// products of the other.  The line of all segments' 128-key tiles is cut evenly over the
// SMs; each part (fp32 output and LSE per slot row) goes to the workspace for the join.
//
// Measured (8 heads, D = 128, 32768 prefix keys, own keys of one token; us a call in a
// graph, launches and join within): 512 rows a head e4m3 77, int8 94 (the products alone take 35 at 1958 TFLOP/s);
// 128 rows int8 46.  A 128-key tile of 256 rows takes 5000 to 5500 cycles, 2048 of them in the
// tensor pipe: each slot's chain of S, softmax (3000 to 3800 cycles, the schedulers shared
// with the widening warps) and P V bounds it.  The first S is there 15000 cycles after the
// start (page table, codes, cold instructions), 8000 when all of that is in L2.
//
// Roles (640 threads, one CTA per SM, all of TMEM):
//   warp 0        issues the MMAs: S_t = Q_t K'^T into TMEM, O_t += P_t V' with P in TMEM
//   warp 1        owns the TMEM allocation
//   warps 2, 3    fetch the codes of keys, of values: bulk copies into a raw tile each, on
//                 their way from when the tile before has been read
//   warps 4-7, 8-11   slot 0, slot 1: load the query rows, softmax, O rescale, part
//   warps 12-15   widen the codes of keys from the raw tile into the K stages (128-byte
//                 swizzle); the scales of the next tile wait in registers
//   warps 16-19   the same for values, as they lie (MN-major)
// TMEM: S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D,256+2D); P_t over S_t.
#include "bsattn_internal.h"
#include "decode_common.cuh"
#include "kv_codes.cuh"

namespace bsattn {

namespace {

constexpr int kThreads = 640;
constexpr uint32_t kTmemCols = 512;
// 96 registers per thread at launch; the control warpgroup's surplus and some of the
// widening ones' go to the softmax: 128 * 48 + 2 * 128 * 144 + 2 * 128 * 72 = 61440 =
// 640 * 96.  Int8 codes take more to widen, the e4m3 softmax keeps more loads in flight.
constexpr int kLaunchRegs = 96;
constexpr uint32_t kCtrlRegs = 48;
template <bool kInt8>
constexpr uint32_t kSoftmaxRegs = kInt8 ? 144 : 152;
template <bool kInt8>
constexpr uint32_t kWidenRegs = kInt8 ? 72 : 64;
static_assert(128 * kCtrlRegs + 256 * kSoftmaxRegs<true> + 256 * kWidenRegs<true> <= (uint32_t)kThreads * kLaunchRegs &&
                  128 * kCtrlRegs + 256 * kSoftmaxRegs<false> + 256 * kWidenRegs<false> <= (uint32_t)kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr uint32_t kSub = kTile * 64 * 2;  // 128 rows x 64 fp16: one 128-byte swizzle span
constexpr int kMsgs = 4;                   // tiles whose key scales and masks are kept

// The factors' exponents E and F are at least this (biased): 2^(6 - E) and its inverse are then
// normal numbers, also for the smallest scales, those of rows of zeros.
constexpr int kLeastExp = 7;

// Binary exponents by which a scale may lie below the largest and share its factor.  Keys:
// codes (multiples of 2^-9 in e4m3, of 1 in int8) times 2^(6 - 14) are exact in fp16.  Values:
// so far below E, and so much may E grow within a segment, before the weights carry the scales.
constexpr int kNearKeys = 14, kNearValues = 10, kGrowth = 3;

// log2 of the largest weight when the reference moves, and how far it may grow before it does again.
constexpr float kLift = 7.f, kReach = 8.f;

// 2^(e - 6) of a biased exponent e in [kLeastExp, 254].
__device__ __forceinline__ float scale_down(int e) { return __uint_as_float((uint32_t)(e - 6) << 23); }

struct KeyMsg {
    uint32_t keep[4];  // keys that count, one bit each
    int32_t exp;       // E (biased) of the value factors
    int32_t key_exp;   // F (biased) of the key factors
    uint8_t rest[4];   // whether some r of keys 32 q .. is not 1
    int32_t wide;      // value scales are far apart: the weights of P V' carry them
};
constexpr uint32_t kZeroRow = 255;  // in place of a key's E - f: its values count as 0

template <int D>
struct Cfg {
    static constexpr uint32_t kTileBytes = kTile * D * 2;
    static constexpr uint32_t kQ = 0, kK = kQ + 2 * kTileBytes, kV = kK + 2 * kTileBytes;
    static constexpr uint32_t kRaw = kV + 2 * kTileBytes;            // codes of a key and of a value tile
    static constexpr uint32_t kRawBytes = kTile * D;
    static constexpr uint32_t kScale = kRaw + 2 * kRawBytes;         // kMsgs x 128 rests r of key scales
    static constexpr uint32_t kMsg = kScale + kMsgs * 512u;
    static constexpr uint32_t kDown = kMsg + kMsgs * (uint32_t)sizeof(KeyMsg);  // kMsgs x 128 bytes: E - f, if wide
    static constexpr uint32_t kBar = kDown + kMsgs * 128u;
    // K / V stage full and empty, per slot: query rows there, S ready, two halves of P ready, O complete
    // (once a segment, also for a slot without tiles); raw K / V tile full and empty
    static constexpr int bKF = 0, bKE = 2, bVF = 4, bVE = 6, bQF = 8, bSR = 10, bPR = 12, bOD = 16, bDrain = 18,
                         bRF = 19, bRE = 21, kNumBars = 23;
    static constexpr uint32_t kMisc = kBar + kNumBars * 8;           // [0] tmem base, [1] abort
    static constexpr uint32_t kBytes = kMisc + 16;
    static constexpr uint32_t kAlloc = kBytes;
    static_assert(kAlloc <= 227u * 1024u, "shared memory");
};

// This CTA's pieces of the line, one segment at a time; every role walks them alike.
struct Walk {
    long long pos, end;
    int nt;
    int seg, off, n;  // segment, its first tile here, tiles here
    __device__ __forceinline__ bool next() {
        if (pos >= end) return false;
        seg = (int)line_div(pos, nt);
        off = (int)(pos - (long long)seg * nt);
        n = (int)min((long long)(nt - off), end - pos);
        pos += n;
        return true;
    }
};

// Instruction descriptor, kind::f16 with fp16 A and B, fp32 D (see idesc_bf16_f32).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// One slot: warps 4-7 (t = 0) or 8-11 (t = 1), one row per thread.
template <int D, bool kInt8>
__device__ __forceinline__ void softmax_role(const DecodeParams &p, const Plan &w, Walk walk, uint32_t tmem, int t,
                                             uint32_t warp, uint32_t lane, uint32_t base, uint8_t *smem,
                                             volatile int *abort) {
    using C = Cfg<D>;
    auto bar = [&](int i) -> uint32_t { return base + C::kBar + 8u * (uint32_t)i; };
    const uint32_t quarter = warp & 3u;
    const int r = (int)(quarter * 32 + lane);
    const uint32_t lane_addr = tmem + ((quarter * 32u) << 16);
    const uint32_t s_col = (uint32_t)t * 128u, o_col = 256u + (uint32_t)t * D;
    const int rows_total = p.B * p.G;
    uint32_t sc = 0, od = 0;   // phases of S ready and O complete
    uint32_t tile0 = 0;        // tiles of earlier segments (they number the K stages and messages)
    bool ok = true;
    while (ok && walk.next()) {
        const int h = walk.seg / w.row_blocks, row0 = (walk.seg - h * w.row_blocks) * kBlockRows;
        const int rows = min(kBlockRows, rows_total - row0);
        const bool split = rows <= kTile;
        const int row = split ? r : t * kTile + r;   // of the segment
        const bool row_ok = row < rows;
        // ---- the warp's query rows: fp16 of q 2^-e into the slot's tile (K-major, swizzled).
        // D / 8 lanes load a row together, eight steps' loads at a time.
        float c = 0.f;
        {
            constexpr int kRowLanes = D / 8, kRows = 32 / kRowLanes, kSteps = 32 / kRows;
            const int piece = (int)lane % kRowLanes, sub = (int)lane / kRowLanes;
            const int m = row0 + row, b = row_ok ? m / p.G : 0;
            const long long mine = row_ok ? (long long)b * p.q_stride + (long long)(h * p.G + m - b * p.G) * D : -1;
#pragma unroll 1
            for (int i0 = 0; i0 < kSteps; i0 += 8) {
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const long long at = __shfl_sync(0xffffffffu, mine, (i0 + i) * kRows + sub);
                    x[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4 *>(p.q + at) + piece) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, a = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) a = __vmaxu2(a, y[k] & 0x7fff7fffu);
                    a = max(a & 0xffffu, a >> 16);
#pragma unroll
                    for (int d = 1; d < kRowLanes; d <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
                    float f, back;
                    row_scale(a, p.scale_log2, f, back);
                    back = __shfl_sync(0xffffffffu, back, ((int)lane % kRows) * kRowLanes);
                    if ((int)lane / kRows == i0 + i) c = back;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[k] = pack_f16x2(__uint_as_float(y[k] << 16) * f, __uint_as_float(y[k] & 0xffff0000u) * f);
                    const uint32_t rr = quarter * 32u + (uint32_t)((i0 + i) * kRows + sub);
                    const uint32_t at = C::kQ + (uint32_t)t * C::kTileBytes + (uint32_t)(piece >> 3) * kSub + rr * 128u +
                                        ((((uint32_t)piece & 7u) ^ (rr & 7u)) << 4);
                    *reinterpret_cast<uint4 *>(smem + at) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::bQF + t));
        // ---- the slot's tiles
        float m_run = kNoKey, l_run = 0.f, u_run = kNoKey;   // u_run: m_run unless wide
        int exp_run = 0, done = 0;
        bool wide = false;
        for (int k = split ? t : 0; ok && k < walk.n; k += split ? 2 : 1) {
            ok = mbar_wait(bar(C::bSR + t), sc & 1u, abort, p.err, BSATTN_FLAG_TIMEOUT);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            ++sc;
            tc_fence_after();
            const uint32_t slot = (tile0 + (uint32_t)k) % kMsgs;
            const KeyMsg *msg = reinterpret_cast<const KeyMsg *>(smem + C::kMsg) + slot;
            const float4 *ks = reinterpret_cast<const float4 *>(smem + C::kScale + slot * 512u);
            const uint4 kw = *reinterpret_cast<const uint4 *>(msg->keep);
            const bool masked = (kw.x & kw.y & kw.z & kw.w) != 0xffffffffu;
            const int4 info = *reinterpret_cast<const int4 *>(&msg->exp);   // exp, key_exp, rest, wide
            const int exp_new = info.x;
            // what a score of S is worth in units of log2; above 0: a masked key's -inf stays -inf
            const float ct = fmaxf(c * scale_down(info.y), 0x1p-126f);
            // Int8 tiles take the general way, whose two passes are rolled: 512 rows by 32768 keys,
            // 8 heads, own keys of one token, 94 us a call against 102 with the passes unrolled
            // (the roles' loops share the instruction caches).  E4m3 tiles with power-of-two scales
            // take the short one, its second pass with loads ahead: 77 us against 95.
            wide = info.w != 0;
            const bool plain = !kInt8 && !masked && !wide && info.z == 0;
            // 32 scores of columns 32 q .. times r; -inf where a key does not count
            auto scores = [&](int q, float (&s)[32]) {
                uint32_t v[32];
                tmem_ld32(lane_addr + s_col + 32u * q, v);
                tmem_wait_ld();
                reg_fence(v);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float4 f = ks[8 * q + x];
                    fmul2(s[4 * x], s[4 * x + 1], __uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1]), f.x, f.y);
                    fmul2(s[4 * x + 2], s[4 * x + 3], __uint_as_float(v[4 * x + 2]), __uint_as_float(v[4 * x + 3]), f.z, f.w);
                }
                if (masked) {
                    const uint32_t keep = q == 0 ? kw.x : q == 1 ? kw.y : q == 2 ? kw.z : kw.w;
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (!((keep >> x) & 1u)) s[x] = -INFINITY;
                }
            };
            // The first pass, the maximum: the load's own reduction where scores need no factor and no mask.
            float m_new = m_run;
            if (plain) {
                float hm[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[32];
                    tmem_ld32_max(lane_addr + s_col + 32u * q, v, hm[q]);
                }
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 4; ++q) reg_fence(hm[q]);
                m_new = fmaxf(m_run, fmax3(hm[0], hm[1], fmaxf(hm[2], hm[3])) * ct);
            } else {
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    float s[32];
                    scores(q, s);
                    float g0 = fmax3(s[0], s[1], s[2]), g1 = fmax3(s[3], s[4], s[5]);
#pragma unroll
                    for (int x = 6; x < 30; x += 4) {
                        g0 = fmax3(g0, s[x], s[x + 1]);
                        g1 = fmax3(g1, s[x + 2], s[x + 3]);
                    }
                    m_new = fmaxf(m_new, fmax3(g0, fmaxf(s[30], s[31]), g1) * ct);
                }
            }
            const bool grew = done == 0 || __any_sync(0xffffffffu, m_new - m_run > kReach);
            // O is rescaled when m moves or E grew; if wide, when u moves
            float alpha = 1.f;
            if (grew) {
                alpha = ex2_approx(m_run - m_new);
                m_run = m_new;
            }
            float alpha_o = alpha * ex2_approx((float)(exp_run - exp_new));
            bool rescale = grew || exp_new != exp_run;
            const uint32_t *down = reinterpret_cast<const uint32_t *>(smem + C::kDown + slot * 128u);
            // 8 scores of columns 8 c .. in units of log2 and their keys' E - f, infinite for rows of zeros
            // (small loops: they are rare, and the usual ones share the instruction caches with them)
            auto wide_scores = [&](int c, float (&z)[8], float (&d)[8]) {
                uint32_t v[8];
                tmem_ld8(lane_addr + s_col + 8u * c, v);
                tmem_wait_ld();
                reg_fence(v);
                const uint32_t keep = (c < 8 ? c < 4 ? kw.x : kw.y : c < 12 ? kw.z : kw.w) >> (8 * (c & 3));
                const float *r = reinterpret_cast<const float *>(ks) + 8 * c;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    z[x] = (keep >> x) & 1u ? __uint_as_float(v[x]) * r[x] * ct : -INFINITY;
                    const uint32_t byte = (down[2 * c + (x >> 2)] >> (8 * (x & 3))) & 255u;
                    d[x] = byte == kZeroRow ? INFINITY : (float)byte;
                }
            };
            if (__builtin_expect(wide, 0)) {
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 16; ++c) {
                    float z[8], d[8];
                    wide_scores(c, z, d);
#pragma unroll
                    for (int x = 0; x < 8; ++x) top = fmaxf(top, z[x] - d[x]);
                }
                const float kept = u_run + (float)(exp_run - exp_new);   // O as it is, in units of E
                rescale = __any_sync(0xffffffffu, done == 0 || top - kept > kReach);
                u_run = rescale ? fmaxf(kept, top) : kept;
                alpha_o = ex2_approx(kept - u_run);
            } else {
                u_run = m_run;
            }
            if (done > 0 && rescale) {
                // S of this tile was issued after the slot's previous P V: O is up to date
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t v[32];
                    tmem_ld32(lane_addr + o_col + q * 32, v);
                    tmem_wait_ld();
                    reg_fence(v);
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * alpha_o);
                    tmem_st32(lane_addr + o_col + q * 32, v);
                }
            }
            exp_run = exp_new;
            const float nm = kLift - m_run;
            float la0 = 0.f, la1 = 0.f, lb0 = 0.f, lb1 = 0.f;
            // 32 columns at a time, P over scores that have been read; 64 keys are handed over at a time.
            auto hand_over = [&](int half) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::bPR + 2 * t + half));
            };
            auto part = [&](int q, float (&s)[32]) {
#pragma unroll
                for (int x = 0; x < 16; ++x) ffma2(s[2 * x], s[2 * x + 1], s[2 * x], s[2 * x + 1], ct, ct, nm, nm);
                uint32_t pk[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float p0 = ex2_approx(s[2 * x]), p1 = ex2_approx(s[2 * x + 1]);
                    if (x & 1) fadd2(lb0, lb1, lb0, lb1, p0, p1);
                    else fadd2(la0, la1, la0, la1, p0, p1);
                    pk[x] = pack_f16x2(p0, p1);
                }
                tmem_st16(lane_addr + s_col + 16u * q, pk);
            };
            auto plain_part = [&](int q, uint32_t (&v)[32]) {
                float s[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) s[x] = __uint_as_float(v[x]);
                part(q, s);
            };
            if (plain) {
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
            } else if (__builtin_expect(!wide, 1)) {
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    float s[32];
                    scores(q, s);
                    part(q, s);
                    if (q & 1) hand_over(q >> 1);
                }
            } else {
                const float nu = kLift - u_run;
#pragma unroll 1
                for (int c = 0; c < 16; ++c) {
                    float z[8], d[8];
                    uint32_t pk[4];
                    wide_scores(c, z, d);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        la0 += ex2_approx(z[2 * x] + nm);
                        la1 += ex2_approx(z[2 * x + 1] + nm);
                        pk[x] = pack_f16x2(ex2_approx(z[2 * x] + nu - d[2 * x]), ex2_approx(z[2 * x + 1] + nu - d[2 * x + 1]));
                    }
                    tmem_st4(lane_addr + s_col + 4u * c, pk);
                    if ((c & 7) == 7) hand_over(c >> 3);
                }
            }
            const float l_tile = (la0 + lb0) + (la1 + lb1);
            l_run = l_run * alpha + l_tile;
            ++done;
        }
        if (!ok) break;
        tile0 += (uint32_t)walk.n;
        // ---- the part: rows of 128-byte blocks go through the slot's query tile (no S of
        // this segment is outstanding), so that every store writes whole row pieces.  A slot
        // without tiles waits too: its warps would otherwise arrive for the next segment's
        // query rows before the issuing warp, or each other, are through with this one's.
        ok = mbar_wait(bar(C::bOD + t), od & 1u, abort, p.err, BSATTN_FLAG_TIMEOUT);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        ++od;
        tc_fence_after();
        const bool empty = done == 0 || l_run == 0.f;   // NaN is not empty
        // l and the values' scale one after the other: their quotient may be below fp32's range, the result not
        const float inv = empty ? 0.f : 1.f / l_run;
        const float unit = done == 0 ? 0.f : wide ? ex2_approx(u_run - m_run + (float)(exp_run - 127 - 6)) : scale_down(exp_run);
        const long long part_row = ((long long)walk.seg + blockIdx.x) * w.rows_p + t * kTile;
        float *po = reinterpret_cast<float *>(p.ws + w.pre_o) + part_row * D;
        uint4 *scr = reinterpret_cast<uint4 *>(smem + C::kQ + (uint32_t)t * C::kTileBytes + quarter * 4096u);
        const int first = (int)(quarter * 32u) + 8 * (int)(lane >> 3);   // rows this lane stores
        const int limit = split ? rows : rows - t * kTile;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
            uint32_t v[32];
            if (done > 0) {
                tmem_ld32(lane_addr + o_col + q * 32, v);
                tmem_wait_ld();
                reg_fence(v);
            } else {
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                scr[lane * 8u + ((uint32_t)i ^ (lane & 7u))] =
                    make_uint4(__float_as_uint(__uint_as_float(v[4 * i]) * inv * unit),
                               __float_as_uint(__uint_as_float(v[4 * i + 1]) * inv * unit),
                               __float_as_uint(__uint_as_float(v[4 * i + 2]) * inv * unit),
                               __float_as_uint(__uint_as_float(v[4 * i + 3]) * inv * unit));
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint4 x = scr[(lane >> 3) * 64u + (uint32_t)k * 8u + ((lane & 7u) ^ (uint32_t)k)];
                if (first + k < limit)
                    *reinterpret_cast<uint4 *>(po + (long long)(first + k) * D + q * 32 + 4 * (lane & 7u)) = x;
            }
            __syncwarp();
        }
        if (row_ok)
            reinterpret_cast<float *>(p.ws + w.pre_l)[part_row + r] = empty ? -INFINITY : m_run - kLift + lg2_approx(l_run);
        tc_fence_before();
    }
}

// Fetches the codes of K or V tiles, one warp each: a copy per 16 keys (no page is smaller),
// none for keys past the prefix or on a page that is none.
template <int D>
__device__ __forceinline__ void fetch_role(const DecodeParams &p, const Plan &w, Walk walk, bool values, int lane,
                                           uint32_t base, volatile int *abort) {
    using C = Cfg<D>;
    const uint32_t full = base + C::kBar + 8u * (uint32_t)(C::bRF + (values ? 1 : 0));
    const uint32_t empty = base + C::kBar + 8u * (uint32_t)(C::bRE + (values ? 1 : 0));
    const uint32_t raw = base + C::kRaw + (values ? C::kRawBytes : 0u);
    const uint8_t *codes = values ? p.c.v : p.c.k;
    uint32_t it = 0;
    bool ok = true;
    while (ok && walk.next()) {
        const int h = walk.seg / w.row_blocks;
        for (int k = 0; k < walk.n; ++k, ++it) {
            const int key = (walk.off + k) * kTile + 16 * lane;
            long long row = -1;
            if (lane < 8 && key < p.prefix_len) {
                const int page = __ldg(p.prefix_table + (key >> p.c.page_shift));
                if (page >= 0 && page < p.c.num_pages)
                    row = (((long long)page * p.c.H + h) << p.c.page_shift) + (key & ((1 << p.c.page_shift) - 1));
                else
                    raise(p, BSATTN_FLAG_BAD_INDEX);
            }
            const uint32_t on = __ballot_sync(0xffffffffu, row >= 0);
            ok = __all_sync(0xffffffffu, mbar_wait(empty, (it & 1u) ^ 1u, abort, p.err, BSATTN_FLAG_TIMEOUT));
            if (!ok) break;
            mbar_arrive_expect_tx_lead(lane == 0 ? 1u : 0u, full, (uint32_t)__popc(on) * 16u * D);
            __syncwarp();
            bulk_g2s_lead(row >= 0 ? 1u : 0u, raw + (uint32_t)lane * 16u * D, codes + row * D, 16u * D, full);
        }
    }
    // nothing may be on its way into the tile when the CTA ends
    if (it > 0) mbar_wait_drain(full, (it - 1u) & 1u);
}

// Widens the codes of K tiles (four warps, 32 keys each) or V tiles (four more); one code
// for both, so that the warps share the instruction caches.
//
// Lane: 16 codes of a row (two swizzle pieces of fp16), D / 16 lanes to a row.  A tile's
// scales are loaded while the tile before it is widened.  The codes come through a raw tile:
// loaded into registers instead, the lines on their way filled the load unit, and every
// softmax warp stood still for some 1000 cycles a tile.
template <int D, bool kInt8>
__device__ __forceinline__ void widen_role(const DecodeParams &p, const Plan &w, Walk walk, bool values, int warp,
                                           int lane, uint32_t base, uint8_t *smem, volatile int *abort) {
    using C = Cfg<D>;
    constexpr int kRowLanes = D / 16, kRows = 32 / kRowLanes, kSteps = 32 / kRows;   // rows of a step, steps
    auto bar = [&](int i) -> uint32_t { return base + C::kBar + 8u * (uint32_t)i; };
    const int col = lane % kRowLanes, sub_row = lane / kRowLanes;
    const int ps_shift = p.c.page_shift, n_keys = p.prefix_len;
    const float *scales = values ? p.c.vs : p.c.ks;
    // Cache row of this lane's keys 4 lane .. 4 lane + 3 of a tile (one page), or -1.
    auto look_up = [&](int tile, int h) -> int {
        const int key = tile * kTile + 4 * lane;
        if (key >= n_keys) return -1;
        const int page = __ldg(p.prefix_table + (key >> ps_shift));
        if (page < 0 || page >= p.c.num_pages) return -1;
        return ((page * p.c.H + h) << ps_shift) + (key & ((1 << ps_shift) - 1));
    };
    // What is loaded of a tile one tile ahead.
    int n;              // keys of the tile
    uint32_t keep;      // those of the warp's 32 keys that count
    float scale;        // of the warp's key `lane`
    uint4 ks4, vs4;     // scales of the tile's keys 4 lane ..
    auto load = [&](int row4, int tile) {
        n = min(kTile, n_keys - tile * kTile);
        const int row = __shfl_sync(0xffffffffu, row4, warp * 8 + (lane >> 2));
        const bool on = row >= 0 && warp * 32 + lane < n;
        keep = __ballot_sync(0xffffffffu, on);
        scale = on ? __ldg(scales + (long long)row + (lane & 3)) : 0.f;
        const bool on4 = row4 >= 0;
        ks4 = on4 && !values ? __ldg(reinterpret_cast<const uint4 *>(p.c.ks + row4)) : make_uint4(0, 0, 0, 0);
        vs4 = on4 ? __ldg(reinterpret_cast<const uint4 *>(p.c.vs + row4)) : make_uint4(0, 0, 0, 0);
        if (n < kTile) {   // behind the last key
            auto cut = [&](uint32_t &x, int i) {
                if (4 * lane + i >= n) x = 0u;
            };
            cut(ks4.x, 0), cut(ks4.y, 1), cut(ks4.z, 2), cut(ks4.w, 3);
            cut(vs4.x, 0), cut(vs4.y, 1), cut(vs4.z, 2), cut(vs4.w, 3);
        }
    };
    // Largest binary exponent (biased, at least kLeastExp) of a tile's scales; NaN and infinity do not count.
    auto largest_exp = [&](uint4 x) -> int {
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
        uint32_t top = (uint32_t)kLeastExp << 23;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (v[i] < 0x7f800000u) top = max(top, v[i]);
        return (int)(__reduce_max_sync(0xffffffffu, top) >> 23);
    };
    // A scale of 0, or the smallest, which rows of zeros have.
    auto zero_row = [](uint32_t bits) -> bool { return (bits & 0x7fffffffu) <= 1u << 23; };
    // E - f of this lane's four values, kZeroRow for rows of zeros; one byte each.
    auto far_bytes = [&](int exp) -> uint32_t {
        const uint32_t v[4] = {vs4.x, vs4.y, vs4.z, vs4.w};
        uint32_t out = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = max(exp - max((int)(v[i] >> 23 & 255u), kLeastExp), 0);
            out |= (zero_row(v[i]) ? kZeroRow : (uint32_t)d) << (8 * i);
        }
        return out;
    };
    // Whether one of the tile's values that are not rows of zeros lies more than 2^kNearValues below E.
    auto any_far = [&](int exp) -> bool {
        const uint32_t v[4] = {vs4.x, vs4.y, vs4.z, vs4.w}, least = (1u << 23) + 1u;
        const uint32_t near = (uint32_t)max(exp - kNearValues, 1) << 23;
        bool far = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) far |= v[i] - least < near - least;   // in [least, near)
        return __any_sync(0xffffffffu, far && near > least);
    };
    // `ahead` walks two tiles in front: its tile's page is being looked up while the scales of
    // the tile before it are loaded and the one before that is widened.
    Walk ahead = walk;
    int ak = 0;
    bool more2 = ahead.next();
    if (!more2) return;
    auto step = [&] {
        if (more2 && ++ak >= ahead.n) {
            ak = 0;
            more2 = ahead.next();
        }
    };
    auto look_ahead = [&]() -> int { return more2 ? look_up(ahead.off + ak, ahead.seg / w.row_blocks) : -1; };
    load(look_ahead(), ahead.off);
    step();
    bool more1 = more2;
    int tile1 = ahead.off + ak, row4 = look_ahead();
    const uint8_t *raw = smem + C::kRaw + (values ? C::kRawBytes : 0u) + (warp * 32 + sub_row) * D + col * 16;
    // Eight lanes store 128 bytes at a time; where they share a row, half of them begin with
    // their second piece: every bank once.
    const bool swap = D == 128 && col >= 4;
    const int first = 2 * (col & 3) + (swap ? 1 : 0), second = first ^ 1;
    const uint32_t dst = (values ? C::kV : C::kK) + (uint32_t)(col >> 2) * kSub + (uint32_t)(warp * 32 + sub_row) * 128u;
    uint32_t it = 0;
    while (walk.next()) {
        int exp_run = kLeastExp, exp_first = 0;   // E starts anew with a segment's sums
        bool wide = false;
        for (int k = 0; k < walk.n; ++k, ++it) {
            const uint32_t st = it & 1u, ph = (it >> 1) & 1u;
            exp_run = max(exp_run, largest_exp(vs4));
            if (exp_first <= kLeastExp) exp_first = exp_run;   // tiles of zeros do not count
            // what no tile had far below its E lies within 2^(kNearValues + kGrowth) of the present E
            wide = wide || exp_run - exp_first > kGrowth || any_far(exp_run);
            const int exp = values ? exp_run : largest_exp(ks4);
            step();
            const int row4_2 = look_ahead();
            // V: vs 2^(6 - E); K: the power of two in ks, times 2^(6 - F), but NaN where ks is: an
            // infinity, the power of two in a NaN, could give a score that drops the key.  A key
            // far below the largest keeps its own exponent, and the difference goes into r.
            const uint32_t bits = __float_as_uint(scale);
            const bool number = (bits & 0x7fffffffu) < 0x7f800000u;
            const int own = max((int)(bits >> 23 & 255u), kLeastExp);
            const int base_exp = (values ? wide && !zero_row(bits) : exp - own > kNearKeys) ? own : exp;
            const float f32 = (values ? scale : __uint_as_float(number ? bits & 0x7f800000u : 0x7fc00000u)) *
                              __uint_as_float((uint32_t)(260 - base_exp) << 23);
            const uint32_t factor = pack_f16x2(f32, f32);
            const int empty = values ? C::bVE : C::bKE, full = values ? C::bVF : C::bKF, v = values ? 1 : 0;
            if (!__all_sync(0xffffffffu,
                            mbar_wait(bar(empty + (int)st), ph ^ 1u, abort, p.err, BSATTN_FLAG_TIMEOUT) &&
                                mbar_wait(bar(C::bRF + v), it & 1u, abort, p.err, BSATTN_FLAG_TIMEOUT)))
                return;
            uint8_t *tile = smem + dst + st * C::kTileBytes;
            const bool whole = keep == 0xffffffffu;
            // two steps at a time: 94 us as above, 95 with all eight unrolled
#pragma unroll 2
            for (int i = 0; i < kSteps; ++i) {
                uint4 x = *reinterpret_cast<const uint4 *>(raw + i * kRows * D);
                // what lies in the tile where no key was copied is of an earlier one
                if (!whole && !((keep >> (i * kRows + sub_row)) & 1u)) x = make_uint4(0, 0, 0, 0);
                const uint32_t f = __shfl_sync(0xffffffffu, factor, i * kRows + sub_row);
                const uint32_t y[4] = {swap ? x.z : x.x, swap ? x.w : x.y, swap ? x.x : x.z, swap ? x.y : x.w};
                const int r7 = (i * kRows + sub_row) & 7;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t o[4];
                    codes_to_f16x2<kInt8>(y[2 * j], o[0], o[1]);
                    codes_to_f16x2<kInt8>(y[2 * j + 1], o[2], o[3]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[q]) : "r"(f));
                    *reinterpret_cast<uint4 *>(tile + i * kRows * 128 + (((j ? second : first) ^ r7) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (!values) {
                const int below = min(exp - base_exp, 126);
                reinterpret_cast<float *>(smem + C::kScale + (it % kMsgs) * 512u)[warp * 32 + lane] =
                    __uint_as_float((bits & 0x7fffffu) | (uint32_t)(127 - below) << 23);
                const bool rest = __any_sync(0xffffffffu, (bits & 0x7fffffu) != 0u || below > 0);
                if (wide && warp == 0)
                    reinterpret_cast<uint32_t *>(smem + C::kDown + (it % kMsgs) * 128u)[lane] = far_bytes(exp_run);
                if (lane == 0) {
                    KeyMsg *msg = reinterpret_cast<KeyMsg *>(smem + C::kMsg) + it % kMsgs;
                    msg->keep[warp] = keep;
                    msg->rest[warp] = rest ? 1 : 0;
                    if (warp == 0) {
                        msg->exp = exp_run;
                        msg->key_exp = exp;
                        msg->wide = wide ? 1 : 0;
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(full + (int)st));
                mbar_arrive(bar(C::bRE + v));
            }
            if (more1) load(row4, tile1);
            row4 = row4_2;
            more1 = more2;
            tile1 = ahead.off + ak;
        }
    }
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(kThreads, 1)
    bsattn_prefix_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ Plan w) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {  // the swizzle counts from 1024-byte boundaries
        if (threadIdx.x == 0) raise(p, BSATTN_FLAG_TIMEOUT);
        return;
    }
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::kMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(misc + 1);
    auto bar = [&](int i) -> uint32_t { return base + C::kBar + 8u * (uint32_t)i; };
    const uint32_t warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(C::bKF + s), 4);       // one arrival per widening warp
            mbar_init(bar(C::bKE + s), 1);
            mbar_init(bar(C::bVF + s), 4);
            mbar_init(bar(C::bVE + s), 1);
            mbar_init(bar(C::bQF + s), 4);       // one per softmax warp of the slot
            mbar_init(bar(C::bSR + s), 2);
            mbar_init(bar(C::bPR + 2 * s), 4);
            mbar_init(bar(C::bPR + 2 * s + 1), 4);
            mbar_init(bar(C::bOD + s), 1);
        }
        mbar_init(bar(C::bDrain), 1);
        for (int v = 0; v < 2; ++v) {
            mbar_init(bar(C::bRF + v), 1);       // the fetching warp's arrival and the bytes
            mbar_init(bar(C::bRE + v), 4);       // one per widening warp
        }
        misc[1] = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    Walk walk;
    walk.nt = (p.prefix_len + kTile - 1) / kTile;
    walk.pos = w.pre_first((int)blockIdx.x, walk.nt);
    walk.end = w.pre_first((int)blockIdx.x + 1, walk.nt);
    if (warp == 1) {
        tmem_alloc(base + C::kMisc, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    // Launched as a dependent of whatever preceded it on the stream; the decode kernel, which
    // does not wait for what this grid writes, may start once that has completed.
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0) {
        regs_release<kCtrlRegs>();
        // ---------------------------------------------------- MMA issuer --
        // The whole warp runs in step; lane 0 issues.
        const uint32_t lead = lane == 0 ? 1u : 0u;
        constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, false);
        constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, true);
        const uint64_t desc_q = smem_desc_sw128(base + C::kQ, 16, 1024);
        const uint64_t desc_k = smem_desc_sw128(base + C::kK, 16, 1024);
        const uint64_t desc_v = smem_desc_sw128(base + C::kV, kSub, 1024);
        constexpr uint64_t kTileUnits = C::kTileBytes >> 4, kSubUnits = kSub >> 4;
        uint32_t it = 0, seg = 0;          // tiles, segments so far
        uint32_t pc[2] = {0, 0};
        bool ok = true;
        auto wait = [&](int b, uint32_t phase) -> bool {
            ok = ok && mbar_wait(bar(b), phase, abort, p.err, BSATTN_FLAG_TIMEOUT);
            return ok;
        };
        auto score = [&](int t, uint32_t tile) {
            const uint64_t qd = desc_q + (uint64_t)t * kTileUnits, kd = desc_k + (uint64_t)(tile & 1u) * kTileUnits;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (uint64_t)((kk >> 2) * kSubUnits + (kk & 3) * 2);
                mma_ss_lead(lead, tmem + t * 128, qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit_lead(lead, bar(C::bSR + t));
            mbar_arrive_lead(lead, bar(C::bSR + t));
        };
        auto output = [&](int t, uint32_t tile, bool first) -> bool {
            if (!wait(C::bVF + (int)(tile & 1u), (tile >> 1) & 1u)) return false;
            const uint64_t vd = desc_v + (uint64_t)(tile & 1u) * kTileUnits;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!wait(C::bPR + 2 * t + half, pc[t] & 1u)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                    mma_ts_lead(lead, tmem + 256 + t * D, tmem + t * 128 + kk * 8, vd + (uint64_t)(kk * (2048 >> 4)),
                                idesc_pv, kk > 0 || !first ? 1u : 0u);
            }
            ++pc[t];
            return true;
        };
        while (ok && walk.next()) {
            const int h = walk.seg / w.row_blocks, row0 = (walk.seg - h * w.row_blocks) * kBlockRows;
            const bool split = p.B * p.G - row0 <= kTile;
            if (!wait(C::bQF, seg & 1u) || !wait(C::bQF + 1, seg & 1u)) break;
            tc_fence_after();
            // slot 1 has no tile and no O of its own to wait for
            mbar_arrive_lead(split && walk.n == 1 ? lead : 0u, bar(C::bOD + 1));
            for (int k = 0; ok && k < walk.n; ++k) {
                const uint32_t tile = it + (uint32_t)k;
                if (!wait(C::bKF + (int)(tile & 1u), (tile >> 1) & 1u)) break;
                tc_fence_after();
                if (split) {
                    const int t = k & 1;
                    if (k >= 2) {
                        if (!output(t, tile - 2, k < 4)) break;
                        mma_commit_lead(lead, bar(C::bVE + (int)(tile & 1u)));
                    }
                    score(t, tile);
                } else {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (k > 0 && !output(t, tile - 1, k == 1)) break;
                        score(t, tile);
                    }
                    if (!ok) break;
                    if (k > 0) mma_commit_lead(lead, bar(C::bVE + (int)((tile - 1) & 1u)));
                }
                mma_commit_lead(lead, bar(C::bKE + (int)(tile & 1u)));
            }
            if (!ok) break;
            const uint32_t last = it + (uint32_t)walk.n - 1;
            if (split) {
                if (walk.n >= 2) {
                    const int t = (walk.n - 2) & 1;
                    if (!output(t, last - 1, walk.n - 2 < 2)) break;
                    mma_commit_lead(lead, bar(C::bVE + (int)((last - 1) & 1u)));
                    mma_commit_lead(lead, bar(C::bOD + t));
                }
                const int t = (walk.n - 1) & 1;
                if (!output(t, last, walk.n - 1 < 2)) break;
                mma_commit_lead(lead, bar(C::bVE + (int)(last & 1u)));
                mma_commit_lead(lead, bar(C::bOD + t));
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!output(t, last, walk.n == 1)) break;
                    mma_commit_lead(lead, bar(C::bOD + t));
                }
                if (!ok) break;
                mma_commit_lead(lead, bar(C::bVE + (int)(last & 1u)));
            }
            it += (uint32_t)walk.n;
            ++seg;
        }
        // Wait until every tcgen05 operation issued above has completed.
        mma_commit_lead(lead, bar(C::bDrain));
        mbar_wait_drain(bar(C::bDrain), 0);
    } else if (warp < 4) {
        regs_release<kCtrlRegs>();
        if (warp >= 2) fetch_role<D>(p, w, walk, warp == 3, (int)lane, base, abort);
    } else if (warp < 12) {
        regs_claim<kSoftmaxRegs<kInt8>>();
        softmax_role<D, kInt8>(p, w, walk, tmem, warp >= 8 ? 1 : 0, warp, lane, base, smem, abort);
    } else {
        regs_release<kWidenRegs<kInt8>>();
        widen_role<D, kInt8>(p, w, walk, warp >= 16, (int)(warp & 3u), (int)lane, base, smem, abort);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool kInt8>
cudaError_t launch(const DecodeParams &p, const Plan &w, cudaStream_t stream) {
    using C = Cfg<D>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set_for_device[dev]) {
        // the register split inside the kernel assumes exactly kLaunchRegs per thread at launch
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, bsattn_prefix_kernel<D, kInt8>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(bsattn_prefix_kernel<D, kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)C::kAlloc);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3((unsigned)w.pre_cuts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kAlloc;
    return cudaLaunchKernelEx(&cfg, bsattn_prefix_kernel<D, kInt8>, p, w);
}

}  // namespace

cudaError_t launch_prefix(const DecodeParams &p, const Plan &w, cudaStream_t stream) {
    if (p.c.D == 128) return p.c.int8 ? launch<128, true>(p, w, stream) : launch<128, false>(p, w, stream);
    return p.c.int8 ? launch<64, true>(p, w, stream) : launch<64, false>(p, w, stream);
}

}  // namespace bsattn
