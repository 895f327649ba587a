// Device code that the kernels for chunks of new tokens share (bsattn_prefill, bsattn_kv_weigh):
// a sequence's numbers and what a query may meet.
#pragma once

#include "bsattn_internal.h"
#include "sm100_ptx.cuh"

namespace bsattn {

// A sequence: its queries are the packed rows first .. first + m - 1, at the positions
// n - m .. n - 1 of its n keys.  m = 0: nothing is to be done (no token, or faulty numbers).
struct Chunk {
    int first, m, n;
};

// `check`: flag what is faulty: offsets that leave the packed rows or decrease, more new
// tokens than keys, more keys than the page table's row holds.  A sequence of length 0 or less
// has no key (n = 0): its queries, if it has any, meet nothing.
__device__ __forceinline__ Chunk chunk_of(const ChunkParams &p, int b, bool check) {
    Chunk s;
    int end;
    if (p.cu) {
        s.first = __ldg(p.cu + b);
        end = __ldg(p.cu + b + 1);
    } else {
        s.first = b;
        end = b + 1;
    }
    const int n = __ldg(p.seqlens + b);
    s.n = max(n, 0);
    s.m = 0;
    const bool rows_ok = s.first >= 0 && end >= s.first && end <= p.total;
    if (!rows_ok || (n > 0 && (end - s.first > n || n > (p.table_cols << p.c.page_shift)))) {
        if (check && p.err) atomicOr(p.err, BSATTN_FLAG_BAD_SEQLENS);
        return s;
    }
    s.m = end - s.first;
    return s;
}

// The keys that the query at position i of a sequence of n keys meets: j < hb or la <= j < ha.
struct Met {
    int hb, la, ha;
};

__device__ __forceinline__ Met met(const ChunkParams &p, int i, int n) {
    Met r = {0, 0, n};
    if (p.kind == BSATTN_MASK_CAUSAL) {
        r.ha = min(n, i + 1);
    } else if (p.kind == BSATTN_MASK_SLIDING_WINDOW) {
        r.ha = min(n, i + 1);
        r.la = i + 1 <= p.window_left ? 0 : i + 1 - p.window_left;
        r.hb = min(r.ha, p.sink_tokens);
    } else if (p.kind == BSATTN_MASK_PREFIX) {
        r.ha = min(n, max(p.prefix_len, i + 1));
    }
    return r;
}

// Cache row of position j of sequence b, head h (the first of its page's, plus j mod page), or -1.
__device__ __forceinline__ long long cache_row(const CacheView &c, const int32_t *table_row, int h, int j) {
    const int page = __ldg(table_row + (j >> c.page_shift));
    if (page < 0 || page >= c.num_pages) return -1;
    return (((long long)page * c.H + h) << c.page_shift) + (j & ((1 << c.page_shift) - 1));
}

// Codes 0 and 1 (or 2 and 3) of four as bf16, exact.  e4m3: under a sign-extended byte shifted by 4 its exponent and
// mantissa lie where bf16 has its lowest, the value times 2^-120.  int8, whose low 7 bits l and sign s make 128 + l (bits
// 0x4300 | l) less 128 or, where s, 256.
template <bool kInt8, bool kUpper>
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t x) {
    uint32_t r;
    if constexpr (kInt8) {
        const uint32_t y = __byte_perm(x, 0x43434343u, kUpper ? 0x4342 : 0x4140);
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y & 0xff7fff7fu), "r"(y & 0xff80ff80u));
    } else {
        uint32_t y;
        asm("prmt.b32 %0, %1, %1, %2;" : "=r"(y) : "r"(x), "n"(kUpper ? 0xb3a2 : 0x9180));   // 8 + i: the sign of byte i
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"((y << 4) & 0x87f087f0u), "r"(0x7b807b80u));   // 2^120
    }
    return r;
}

// 4, 16 consecutive 32-bit columns of this thread's TMEM lane -> registers.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

}  // namespace bsattn
