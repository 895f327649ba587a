// Attention weight of cached keys, summed over the queries of the newest tokens.
#include "chunk_common.cuh"
#include "kv_codes.cuh"

namespace bsattn {

namespace {

constexpr int kThreads = 128, kRows = 32;

// One thread per key, 32 query rows at a time in shared memory.
template <int D, bool kInt8>
__global__ void __launch_bounds__(kThreads) bsattn_weigh_kernel(const __grid_constant__ ChunkParams p) {
    __shared__ float sq[kRows][D], sl[kRows];
    const int b = blockIdx.y, h = blockIdx.z;
    const Chunk s = chunk_of(p, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
    const int32_t *table = p.table + (long long)b * p.table_stride;
    const int rows = s.m * p.G;
    if (rows == 0) return;
    for (int j0 = blockIdx.x * kThreads; j0 < s.n; j0 += gridDim.x * kThreads) {
        const int j = j0 + threadIdx.x;
        const long long row = j < s.n ? cache_row(p.c, table, h, j) : -1;
        if (j < s.n && row < 0 && h == 0 && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_INDEX);
        float k[D], w = 0.f;
        for (int d = 0; d < D; d += 4) {
            float y[4] = {};
            if (row >= 0) {
                const uint32_t x = *reinterpret_cast<const uint32_t *>(p.c.k + row * D + d);
                if (kInt8) unpack_int8(x, y);
                else unpack_e4m3(x, y);
            }
            for (int i = 0; i < 4; ++i) k[d + i] = y[i];
        }
        const float f = row >= 0 ? p.c.ks[row] * p.scale_log2 : 0.f;
        for (int r0 = 0; r0 < rows; r0 += kRows) {
            __syncthreads();
            for (int x = threadIdx.x; x < kRows * D; x += kThreads) {
                const int r = r0 + x / D, t = s.first + r / p.G, hq = h * p.G + r % p.G;
                sq[x / D][x % D] = r < rows ? __uint_as_float((uint32_t)p.q[(long long)t * p.q_stride + (long long)hq * D + x % D] << 16) : 0.f;
                if (x % D == 0) {
                    const float lse = r < rows ? p.lse[(long long)t * p.Hq + hq] : -INFINITY;
                    sl[x / D] = lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
                }
            }
            __syncthreads();
            for (int r = 0; r < kRows && r0 + r < rows; ++r) {
                const Met e = met(p, s.n - s.m + (r0 + r) / p.G, s.n);
                if (!(j < e.hb || (j >= e.la && j < e.ha)) || row < 0) continue;
                float acc = 0.f;
                for (int d = 0; d < D; ++d) acc += sq[r][d] * k[d];
                w += exp2f(acc * f - sl[r]);
            }
        }
        if (row >= 0) p.weights[row] = p.accumulate ? p.weights[row] + w : w;
    }
}

template <int D, bool kInt8>
cudaError_t launch(const ChunkParams &p, cudaStream_t stream) {
    bsattn_weigh_kernel<D, kInt8><<<dim3(256, p.B, p.c.H), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weigh(const ChunkParams &p, cudaStream_t stream) {
    if (p.c.D == 128) return p.c.int8 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
    return p.c.int8 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace bsattn
