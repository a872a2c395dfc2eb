// fa_paged.cuh — pieces shared by the append to the paged e4m3 cache and the
// attention over it.
#pragma once

#include <cuda_fp16.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

// Exponents of a block's scale: 448 * 2^120 covers bf16's largest value, and
// 2^-100 keeps the reciprocal and sums of it far inside fp32.
constexpr int kScaleExpMin = -100;
constexpr int kScaleExpMax = 120;

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two e4m3 codes (the low and high byte of `pair`) as packed f16: exact.
__device__ __forceinline__ uint32_t decode_e4m3x2_f16(uint16_t pair) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(pair));
    return r;
}
__device__ __forceinline__ void decode_e4m3x4(uint32_t w, float (&x)[4]) {
    const uint32_t lo = decode_e4m3x2_f16(static_cast<uint16_t>(w & 0xffffu));
    const uint32_t hi = decode_e4m3x2_f16(static_cast<uint16_t>(w >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

// The tokens a sequence brings along: rows first .. first + n - 1 of the packed
// arrays; its cache holds `len` tokens, these being the last n.
struct NewTokens {
    int first, n, len;
};

// False where the offsets are not a valid partition, a sequence brings more
// than max_new tokens or more than its cache length, or its cache length
// passes max_len (at most what its page table holds).
__device__ __forceinline__ bool new_tokens(const int* cu, const int* lens, int b, int total, int max_new,
                                           int max_len, NewTokens& t) {
    const int c0 = cu[b], c1 = cu[b + 1], len = lens[b];
    const bool ok = 0 <= c0 && c0 <= c1 && c1 <= total && c1 - c0 <= max_new && len >= c1 - c0 &&
                    len <= max_len;
    t.first = ok ? c0 : 0;
    t.n = ok ? c1 - c0 : 0;
    t.len = ok ? len : 0;
    return ok;
}

// Host side (fa_paged.cu): checks a cache's description.
fa_status check_cache(const fa_paged_cache* cache);
inline int log2_exact(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

}  // namespace fa
