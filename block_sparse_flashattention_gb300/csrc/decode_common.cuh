// Device code that the decode kernels share: segments, lists, the fp16 MMA.
#pragma once

#include "decode_plan.cuh"
#include "sm100_ptx.cuh"

namespace bsattn {

// References before the first key: far below any score, yet finite, so that a difference
// with it is never NaN.
constexpr float kNoKey = -0x1p100f;

struct Seg {
    int prefix, h, b, rows;
};

__device__ __forceinline__ Seg segment(const DecodeParams &p, const Plan &w, int seg) {
    Seg s;
    if (seg < w.sp) {
        s.prefix = 1;
        s.h = seg;
        s.rows = p.B * p.G;
        s.b = 0;
    } else {
        s.prefix = 0;
        s.b = (seg - w.sp) / p.c.H;
        s.h = seg - w.sp - s.b * p.c.H;
        s.rows = p.G;
    }
    return s;
}

__device__ __forceinline__ void raise(const DecodeParams &p, int bit) {
    if (p.err) atomicOr(p.err, bit);
}

// Keys of sequence b's own part; `check`: flag a length past the page table.
__device__ __forceinline__ int seq_keys(const DecodeParams &p, int b, bool check) {
    const int n = max(__ldg(p.seqlens + b), 0), cap = p.table_cols << p.c.page_shift;
    if (n > cap && check) raise(p, BSATTN_FLAG_BAD_SEQLENS);
    return min(n, cap);
}

struct ListRow {
    int full, mask, nn;  // entries of the two lists, tiles an entry may name
    long long at;        // first index entry
};

// The lists of (sequence b, head h), and the sequence's keys n.  All loads go out at once.
__device__ __forceinline__ ListRow list_row(const DecodeParams &p, int b, int h, int &n, bool check) {
    ListRow r;
    const long long cnt_at = p.lists_varlen ? (long long)h * p.B + b : (long long)b * p.c.H + h;
    const int f = __ldg(p.full_cnt + cnt_at), m = __ldg(p.mask_cnt + cnt_at);
    const int off = p.lists_varlen ? __ldg(p.cu_off + b) : 0;
    n = seq_keys(p, b, check && h == 0);
    r.full = r.mask = 0;
    r.nn = p.lists_varlen ? (n + kTile - 1) / kTile : p.list_n;
    r.at = cnt_at * p.list_n;
    if (p.lists_varlen) {
        r.at = (long long)h * p.total_n + off;
        if (off < 0 || (long long)off + r.nn > p.total_n || (p.vl && r.nn > p.list_n)) {
            if (check) raise(p, BSATTN_FLAG_BAD_SEQLENS);
            return r;
        }
    }
    r.full = min(max(f, 0), r.nn);
    r.mask = min(max(m, 0), r.nn);
    if (check && (r.full != f || r.mask != m)) raise(p, BSATTN_FLAG_BAD_COUNT);
    return r;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^x / l as two factors: with the smallest value scales it may be below fp32's range, while
// what it multiplies is large enough for the product to be within.
__device__ __forceinline__ float2 quotient(float x, float l) {
    return make_float2(ex2_approx(fmaxf(x, -100.f)) / l, ex2_approx(fminf(x + 100.f, 0.f)));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Largest element of a query row as a power of two: rows are handed to the tensor cores
// as fp16(q 2^-e).  `a`: bf16 bits of the row's largest magnitude; zero rows and rows that
// are not finite stay as they are.
__device__ __forceinline__ void row_scale(uint32_t a, float scale_log2, float &to_fp16, float &back) {
    const int e = (a == 0 || a >= 0x7f80u) ? 127 : min(max((int)(a >> 7), 1), 253);
    to_fp16 = __uint_as_float((uint32_t)(254 - e) << 23);
    // above 0: a masked key's score, -inf, stays -inf
    back = fmaxf(scale_log2 * __uint_as_float((uint32_t)e << 23), 0x1p-126f);
}

// Where a finished row goes: the call's output, or a part in the workspace.
struct RowOut {
    int kind;        // 0 the output, 1 a prefix part, 2 a part of a sequence's own keys
    long long row;
};

__device__ __forceinline__ void store_lse(const DecodeParams &p, const Plan &w, const RowOut &at, float lse2) {
    if (at.kind == 0) p.lse[at.row] = lse2 * 0.69314718055994530942f;
    else reinterpret_cast<float *>(p.ws + (at.kind == 1 ? w.pre_l : w.suf_l))[at.row] = lse2;
}

}  // namespace bsattn
