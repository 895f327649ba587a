// Attention of a chunk of new tokens over a paged 8-bit K/V cache.
#include "chunk_common.cuh"
#include "kv_codes.cuh"

namespace bsattn {

namespace {

constexpr int kWarps = 4;

// One warp per query row, 32 keys at a time: each lane scores a key, then all lanes sum the
// values' columns.
template <int D, bool kInt8>
__global__ void __launch_bounds__(kWarps * 32) bsattn_prefill_kernel(const __grid_constant__ ChunkParams p) {
    __shared__ float sq[kWarps][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int t = blockIdx.x, hq = blockIdx.y * kWarps + warp;
    int b = -1;
    Chunk s = {};
    for (int x = 0; x < p.B; ++x) {
        s = chunk_of(p, x, t == 0 && hq == 0 && lane == 0);
        if (t >= s.first && t < s.first + s.m) { b = x; break; }
    }
    if (t == 0 && hq == 0)
        for (int x = max(b, 0); x < p.B; ++x) chunk_of(p, x, lane == 0);
    if (b < 0 || hq >= p.Hq) return;
    const int h = hq / p.G;
    for (int d = lane; d < D; d += 32)
        sq[warp][d] = __uint_as_float((uint32_t)p.q[(long long)t * p.q_stride + (long long)hq * D + d] << 16);
    __syncwarp();
    const Met r = s.n > 0 ? met(p, s.n - s.m + t - s.first, s.n) : Met{0, 0, 0};
    const int32_t *table = p.table + (long long)b * p.table_stride;
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int j0 = 0; j0 < r.ha; j0 += 32) {
        const int j = j0 + lane;
        const bool in = j < r.hb || (j >= r.la && j < r.ha);
        if (!__any_sync(0xffffffffu, in)) continue;
        const long long row = in ? cache_row(p.c, table, h, j) : -1;
        if (in && row < 0 && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
        float z = -INFINITY;
        if (row >= 0) {
            float acc = 0.f;
            for (int d = 0; d < D; d += 4) {
                float y[4];
                const uint32_t x = *reinterpret_cast<const uint32_t *>(p.c.k + row * D + d);
                if (kInt8) unpack_int8(x, y);
                else unpack_e4m3(x, y);
                for (int i = 0; i < 4; ++i) acc += sq[warp][d + i] * y[i];
            }
            z = acc * p.c.ks[row] * p.scale_log2;
        }
        float top = z;
        bool nan = z != z;
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float m_new = fmaxf(m, top);
        if (m_new == -INFINITY && !__any_sync(0xffffffffu, nan)) continue;
        const float ref = m_new == -INFINITY ? 0.f : m_new, alpha = exp2f(m - ref), w = row >= 0 ? exp2f(z - ref) : 0.f;
        float sum = w;
        for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l = l * alpha + sum;
        for (int c = 0; c < D / 32; ++c) o[c] *= alpha;
        m = m_new;
        const float wv = row >= 0 ? w * p.c.vs[row] : 0.f;
        for (int x = 0; x < 32; ++x) {
            const long long at = __shfl_sync(0xffffffffu, row, x);
            const float f = __shfl_sync(0xffffffffu, wv, x);
            if (at < 0) continue;
            for (int c = 0; c < D / 32; ++c) {
                float y[4];
                const uint32_t code = p.c.v[at * D + c * 32 + lane];
                if (kInt8) unpack_int8(code, y);
                else unpack_e4m3(code, y);
                o[c] += f * y[0];
            }
        }
    }
    const bool empty = l == 0.f;
    const long long at = (long long)t * p.Hq + hq;
    for (int c = 0; c < D / 32; ++c) {
        const float v = empty ? 0.f : o[c] / l;
        if (p.out_f32) static_cast<float *>(p.out)[at * D + c * 32 + lane] = v;
        else static_cast<uint16_t *>(p.out)[at * D + c * 32 + lane] = (uint16_t)pack_bf16x2(v, 0.f);
    }
    if (lane == 0) p.lse[at] = empty ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

template <int D, bool kInt8>
cudaError_t launch(const ChunkParams &p, cudaStream_t stream) {
    bsattn_prefill_kernel<D, kInt8><<<dim3(p.total > 0 ? p.total : 1, (p.Hq + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t prefill_workspace_bytes(int, int, int, int, int, long long) { return 256; }

cudaError_t launch_prefill(const ChunkParams &p, cudaStream_t stream) {
    if (p.c.D == 128) return p.c.int8 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
    return p.c.int8 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace bsattn
