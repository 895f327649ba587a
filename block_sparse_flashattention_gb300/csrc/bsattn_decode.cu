// Attention of one query token per sequence over a paged 8-bit K/V cache.
//
// One block per (sequence, query head); each of its warps walks the keys with a
// stride, a lane holding D / 32 elements of the row, with a running maximum and sum
// of its own; the warps' results are joined at the end.
#include "bsattn_internal.h"
#include "kv_codes.cuh"
#include "sm100_ptx.cuh"

namespace bsattn {

namespace {

constexpr int kWarps = 4;

// D / 32 consecutive codes of a row as fp32.
template <int D>
__device__ __forceinline__ void load_codes(const uint8_t *row, int lane, bool int8, float (&y)[D / 32]) {
    uint32_t x;
    if constexpr (D == 128) x = *reinterpret_cast<const uint32_t *>(row + lane * 4);
    else x = *reinterpret_cast<const uint16_t *>(row + lane * 2);
    float f[4];
    if (int8) unpack_int8(x, f);
    else unpack_e4m3(x, f);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) y[i] = f[i];
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) bsattn_decode_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int E = D / 32;
    const int hq = blockIdx.x, b = blockIdx.y, h = hq / p.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = __uint_as_float((uint32_t)p.q[b * p.q_stride + (long long)hq * D + lane * E + i] << 16);
        o[i] = 0.f;
    }
    const int ps = 1 << p.c.page_shift;
    auto visit = [&](const int32_t *table, int j) {
        const int page = __ldg(table + (j >> p.c.page_shift));
        if (page < 0 || page >= p.c.num_pages) {
            if (p.err && lane == 0) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
            return;
        }
        const long long row = (((long long)page * p.c.H + h) << p.c.page_shift) + (j & (ps - 1));
        float x[E];
        load_codes<D>(p.c.k + row * D, lane, p.c.int8, x);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= p.c.ks[row] * p.scale_log2;
        const float mn = fmaxf(m, s);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m - base), w = exp2f(s - base);
        m = mn;
        l = l * a + w;
        load_codes<D>(p.c.v + row * D, lane, p.c.int8, x);
        const float wv = w * p.c.vs[row];
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * a + wv * x[i];
    };
    for (int j = warp; j < p.prefix_len; j += kWarps) visit(p.prefix_table, j);
    const int cap = p.table_cols << p.c.page_shift;
    int n = max(p.seqlens[b], 0);
    if (n > cap) {
        n = cap;
        if (p.err && threadIdx.x == 0) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
    }
    const int32_t *table = p.table + (long long)b * p.table_stride;
    if (!p.has_lists) {
        for (int j = warp; j < n; j += kWarps) visit(table, j);
    } else {
        const int nn = p.lists_varlen ? (n + kTile - 1) / kTile : p.list_n;
        const long long cnt_at = p.lists_varlen ? (long long)h * p.B + b : (long long)b * p.c.H + h;
        long long idx_at = cnt_at * p.list_n;
        bool ok = true;
        if (p.lists_varlen) {
            const int off = p.cu_off[b];
            idx_at = (long long)h * p.total_n + off;
            ok = off >= 0 && (long long)off + nn <= p.total_n && !(p.vl && nn > p.list_n);
            if (!ok && p.err && threadIdx.x == 0) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
        }
        for (int list = 0; ok && list < 2; ++list) {
            int cnt = (list ? p.mask_cnt : p.full_cnt)[cnt_at];
            if (cnt < 0 || cnt > nn) {
                cnt = cnt < 0 ? 0 : nn;
                if (p.err && threadIdx.x == 0) atomicOr(p.err, BSATTN_FLAG_BAD_COUNT);
            }
            const int32_t *idx = (list ? p.mask_idx : p.full_idx) + idx_at;
            for (int i = 0; i < cnt; ++i) {
                const int t = idx[i];
                if (t < 0 || t >= nn) {
                    if (p.err && threadIdx.x == 0) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
                    continue;
                }
                int lim = min(kTile, n - t * kTile);
                if (list && p.vl) lim = min(lim, p.vl[(long long)b * p.list_n + t]);
                for (int j = warp; j < lim; j += kWarps) visit(table, t * kTile + j);
            }
        }
    }
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int i = 0; i < E; ++i) so[warp][lane * E + i] = o[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w]);
    const float base = mm == -INFINITY ? 0.f : mm;
    for (int w = 0; w < kWarps; ++w) ll += sl[w] * exp2f(sm[w] - base);
    const bool empty = ll == 0.f;
    const long long at = (long long)b * p.Hq + hq;
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += so[w][d] * exp2f(sm[w] - base);
        x = empty ? 0.f : x / ll;
        if (p.out_f32) static_cast<float *>(p.out)[at * D + d] = x;
        else static_cast<uint16_t *>(p.out)[at * D + d] = (uint16_t)pack_bf16x2(x, 0.f);
    }
    if (threadIdx.x == 0) p.lse[at] = empty ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994530942f;
}

}  // namespace

size_t decode_workspace_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_decode(const DecodeParams &p, cudaStream_t stream) {
    const dim3 g((unsigned)p.Hq, (unsigned)p.B);
    if (p.c.D == 128) bsattn_decode_kernel<128><<<g, kWarps * 32, 0, stream>>>(p);
    else bsattn_decode_kernel<64><<<g, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace bsattn
