// Paged 8-bit K/V cache: quantising rows as they are written, and reading them back.
//
// A row is the D bf16 values of one token and head.  With a = max |x|:
//   e4m3  scale = 2^e, e = max(-126, ceil(log2(a / 448))).  a = 1.m 2^k and 448 =
//         1.75 2^8, so e = k - 8, one more where 1.m > 1.75: integer work on a's bits.
//         x / scale is exact, so the code is x rounded once.
//   int8  scale = a (1 / 127), code = rint(x (127 (1 / a))), each operation in fp32.
// The maximum is taken on the bit patterns without the sign (ordered like the
// magnitudes, infinities and NaNs above all numbers).
//
// Both kernels move bytes and compute little: 2 D bytes of bf16 against D + 4 bytes
// of codes and scale per row.  A warp takes 8 heads of one token: the row's position
// is found once, D / 8 lanes hold a row (16 bytes of bf16 or 8 of codes each), and all
// loads of the 8 K and 8 V rows go out before the first is used.
//
// Measured, each call on other memory than the one before, against 6.7 TB/s of a plain copy:
// 61440 tokens x 24 heads x 128 (int8) appended in 184 us, 6.2 TB/s; the same (e4m3) read in
// 168 us, 6.8 TB/s; 8 sequences of 100 .. 4096 tokens, 16 heads, appended in 39.6 us, 5.7 TB/s,
// read (D = 64, pages of 16) in 19.1 us.  One token each for 8 sequences: 3.3 us, the launch
// and three dependent loads (offsets, page, rows).
#include "bsattn_internal.h"
#include "kv_codes.cuh"
#include "sm100_ptx.cuh"

namespace bsattn {

namespace {

constexpr int kWarps = 8;           // warps per block
constexpr int kHeadsPerWarp = 8;    // rows of K and of V that one warp moves

// The sequence whose packed rows [cu[b], cu[b + 1]) hold row t, found by the whole
// warp: 32 offsets are compared at a time.  Offsets that do not ascend give some b
// in [0, B); the caller checks the range it finds.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int B, int t, int lane) {
    int lo = 0, n = B - 1;  // the answer is in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int i = lo + (lane + 1) * step;  // candidates for "starts at or before t"
        const bool in = i <= lo + n;
        const unsigned le = __ballot_sync(0xffffffffu, in && __ldg(cu + (in ? i : lo)) <= t);
        const int k = __popc(le);
        const int nlo = lo + k * step;
        n = min(step - 1, lo + n - nlo);
        lo = nlo;
    }
    return lo;
}

__device__ __forceinline__ uint4 ld_stream(const uint16_t *p) {
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p));
    return x;
}

// Codes of the 8 bf16 values in x, and the row's scale; kLanes lanes hold the row.
template <int kLanes, bool kInt8>
__device__ __forceinline__ uint2 quantise(uint4 x, float &scale) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
    const uint32_t a = max(m & 0xffffu, m >> 16);  // bf16 bits of max |x|
    float f;
    if constexpr (kInt8) {
        const float af = fmaxf(__uint_as_float(a << 16), 127.f * 0x1p-126f);
        scale = __fmul_rn(af, 1.f / 127.f);
        f = __fmul_rn(127.f, __frcp_rn(af));
    } else {
        const int e = max(-126, (int)(a >> 7) - 127 - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0));
        scale = __uint_as_float((uint32_t)(e + 127) << 23);
        f = __uint_as_float((uint32_t)(127 - e) << 23);
    }
    if (a >= 0x7f80u) {
        scale = __uint_as_float(0x7fc00000u);
        return make_uint2(0u, 0u);
    }
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            y[2 * j] = __fmul_rn(__uint_as_float(w[2 * i + j] << 16), f);
            y[2 * j + 1] = __fmul_rn(__uint_as_float(w[2 * i + j] & 0xffff0000u), f);
        }
        c[i] = kInt8 ? pack_int8(y) : pack_e4m3(y);
    }
    return make_uint2(c[0], c[1]);
}

struct SeqRows {
    int c0, c1, len;
};

template <int D, bool kInt8>
__global__ void __launch_bounds__(kWarps * 32) bsattn_kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = kHeadsPerWarp / kRows;
    grid_launch_dependents();  // a dependent waits for this grid's end, as this one for what came before
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int cap = p.table_cols << p.c.page_shift;  // tokens of a table row (checked < 2^31 below)
    if (p.err) {
        // every sequence is checked once, by one thread of the grid
        const long long nt = (long long)gridDim.x * kWarps * 32;
        for (long long b = (long long)blockIdx.x * kWarps * 32 + threadIdx.x; b < p.B; b += nt) {
            const int c0 = p.cu ? p.cu[b] : (int)b, c1 = p.cu ? p.cu[b + 1] : (int)b + 1, len = p.seqlens[b];
            const bool bad = c0 < 0 || c1 < c0 || c1 > p.total;
            if (bad || (len > 0 && (c1 - c0 > len || len > cap))) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
        }
    }
    const int chunks = (p.c.H + kHeadsPerWarp - 1) / kHeadsPerWarp;
    const long long t64 = gw / chunks;
    if (t64 >= p.total) return;
    const int t = (int)t64, h0 = (int)(gw - t64 * chunks) * kHeadsPerWarp;
    const int l = lane % kLanes, sub = lane / kLanes;
    uint4 x[2][kIters];
    const uint16_t *src[2] = {p.k + t * p.k_stride + l * 8, p.v + t * p.v_stride + l * 8};
#pragma unroll
    for (int i = 0; i < kIters; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int h = h0 + i * kRows + sub;
            x[s][i] = h < p.c.H ? ld_stream(src[s] + (long long)h * D) : make_uint4(0, 0, 0, 0);
        }
    const int b = p.cu ? find_sequence(p.cu, p.B, t, lane) : t;
    const int c0 = p.cu ? __ldg(p.cu + b) : b, c1 = p.cu ? __ldg(p.cu + b + 1) : b + 1;
    const int len = __ldg(p.seqlens + b);
    if (c0 < 0 || t < c0 || t >= c1 || c1 > p.total || len <= 0 || c1 - c0 > len || len > cap) return;
    const int pos = len - (c1 - t);
    const int page = __ldg(p.table + (long long)b * p.table_stride + (pos >> p.c.page_shift));
    if (page < 0 || page >= p.c.num_pages) {
        if (p.err && lane == 0) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
        return;
    }
    const int in_page = pos & ((1 << p.c.page_shift) - 1);
#pragma unroll
    for (int i = 0; i < kIters; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int h = h0 + i * kRows + sub;
            float scale;
            const uint2 c = quantise<kLanes, kInt8>(x[s][i], scale);
            if (h >= p.c.H) continue;
            const long long row = (((long long)page * p.c.H + h) << p.c.page_shift) + in_page;
            *reinterpret_cast<uint2 *>((s ? p.c.v : p.c.k) + row * D + l * 8) = c;
            if (l == 0) (s ? p.c.vs : p.c.ks)[row] = scale;
        }
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(kWarps * 32) bsattn_kv_read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = kHeadsPerWarp / kRows;
    grid_launch_dependents();  // a dependent waits for this grid's end, as this one for what came before
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long gw = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int cap = p.table_cols << p.c.page_shift;
    if (p.err) {
        const long long nt = (long long)gridDim.x * kWarps * 32;
        for (long long b = (long long)blockIdx.x * kWarps * 32 + threadIdx.x; b < p.B; b += nt) {
            const int c0 = p.cu[b], c1 = p.cu[b + 1];
            if (c0 < 0 || c1 < c0 || c1 > p.total || c1 - c0 > cap) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
        }
    }
    const int chunks = (p.c.H + kHeadsPerWarp - 1) / kHeadsPerWarp;
    const long long t64 = gw / chunks;
    if (t64 >= p.total) return;
    const int t = (int)t64, h0 = (int)(gw - t64 * chunks) * kHeadsPerWarp;
    const int l = lane % kLanes, sub = lane / kLanes;
    const int b = find_sequence(p.cu, p.B, t, lane);
    const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
    if (c0 < 0 || t < c0 || t >= c1 || c1 > p.total || c1 - c0 > cap) return;
    const int pos = t - c0;
    const int page = __ldg(p.table + (long long)b * p.table_stride + (pos >> p.c.page_shift));
    const bool ok = page >= 0 && page < p.c.num_pages;
    if (!ok && p.err && lane == 0) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
    const int in_page = pos & ((1 << p.c.page_shift) - 1);
    uint2 x[2][kIters];
    float sc[2][kIters];
#pragma unroll
    for (int i = 0; i < kIters; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int h = h0 + i * kRows + sub;
            const bool on = ok && h < p.c.H;
            const long long row = on ? (((long long)page * p.c.H + h) << p.c.page_shift) + in_page : 0;
            x[s][i] = on ? __ldcs(reinterpret_cast<const uint2 *>((s ? p.c.v : p.c.k) + row * D + l * 8))
                         : make_uint2(0, 0);
            sc[s][i] = on ? __ldg((s ? p.c.vs : p.c.ks) + row) : 0.f;
        }
#pragma unroll
    for (int i = 0; i < kIters; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int h = h0 + i * kRows + sub;
            if (h >= p.c.H) continue;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float y[4];
                if constexpr (kInt8) unpack_int8(j ? x[s][i].y : x[s][i].x, y);
                else unpack_e4m3(j ? x[s][i].y : x[s][i].x, y);
                w[2 * j] = pack_bf16x2(y[0] * sc[s][i], y[1] * sc[s][i]);
                w[2 * j + 1] = pack_bf16x2(y[2] * sc[s][i], y[3] * sc[s][i]);
            }
            uint16_t *dst = (s ? p.v : p.k) + ((long long)t * p.c.H + h) * D + l * 8;
            __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
        }
}

// One warp per token and 8 heads, and at least one block: with an error word the offsets
// are checked also where there is no row.
unsigned blocks_for(long long total, int H) {
    const long long warps = total * ((H + kHeadsPerWarp - 1) / kHeadsPerWarp);
    return (unsigned)(warps > 0 ? (warps + kWarps - 1) / kWarps : 1);
}

// Launches as a programmatic dependent of what precedes on the stream: the launch
// overlaps the end of the kernel before.
template <class P>
cudaError_t launch(void (*kernel)(P), const P &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(blocks_for(p.total, p.c.H));
    cfg.blockDim = dim3(kWarps * 32);
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream) {
    if (p.c.D == 128) return launch(p.c.int8 ? bsattn_kv_append_kernel<128, true> : bsattn_kv_append_kernel<128, false>, p, stream);
    return launch(p.c.int8 ? bsattn_kv_append_kernel<64, true> : bsattn_kv_append_kernel<64, false>, p, stream);
}

cudaError_t launch_read(const ReadParams &p, cudaStream_t stream) {
    if (p.c.D == 128) return launch(p.c.int8 ? bsattn_kv_read_kernel<128, true> : bsattn_kv_read_kernel<128, false>, p, stream);
    return launch(p.c.int8 ? bsattn_kv_read_kernel<64, true> : bsattn_kv_read_kernel<64, false>, p, stream);
}

}  // namespace bsattn
