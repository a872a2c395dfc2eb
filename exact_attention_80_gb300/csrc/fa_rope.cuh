// fa_rope.cuh — the position rotation shared by fa_rope and fa_kv_append_fp8.
//
// A head's first `rot` columns are rot / 2 pairs; pair i of a token turns by
// the angle whose cosine and sine the table holds in row pos, columns i and
// rot / 2 + i (pos: the token's position on the axis that pair i belongs to):
//   y_a = x_a cos - x_b sin,   y_b = x_b cos + x_a sin.
// Pairs are columns (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved. The
// inverse (sin negated) is the gradient of the rotation, which is orthogonal.
// Products and sums are rounded one by one in fp32 (no fused multiply-add), so
// a value is the same wherever it is computed (here, in the append, or with
// elementwise fp32 operations); the append's block scales follow from it.
//
// A thread works on sixteen columns of a head, two 16-byte vectors: the pairs
// 8 v .. 8 v + 7 for v < rot / 16 (two vectors rot / 2 columns apart, or next
// to each other when interleaved), and two neighbouring vectors of the columns
// behind `rot`, which are copied. So the threads of a token read and write
// whole 128-byte lines at head dims from 64 up, and a thread keeps its eight
// cosines and sines for all the heads it walks.
#pragma once

#include <cuda_bf16.h>

#include "fa_internal.h"
#include "fa_launch.h"
#include "sm103_ptx.cuh"

namespace fa {

struct RopeParams {
    const float* table;     // fp32 [max_pos][rot]: cosines, then sines; null: no rotation
    const int* positions;   // int32 [axes][pos_stride], or null (the caller's own position)
    long long pos_stride;   // tokens per axis
    int rot, axes, max_pos, interleaved;
    int sec_end[FA_MAX_AXES];  // pairs below sec_end[a] (and not below sec_end[a - 1]) turn with axis a
    float sign;             // -1: inverse
};

// Columns of vector 0 and 1 of part v of a head.
__device__ __forceinline__ void rope_columns(const RopeParams& r, int v, int& c0, int& c1) {
    const bool pair = v < (r.rot >> 4);
    c0 = (pair && !r.interleaved) ? 8 * v : 16 * v;
    c1 = (pair && !r.interleaved) ? 8 * v + (r.rot >> 1) : 16 * v + 8;
}

// Where the positions of the axis that pair 8 v turns with begin.
__device__ __forceinline__ const int* rope_axis(const RopeParams& r, int v) {
    int a = 0;
    while (a + 1 < r.axes && 8 * v >= r.sec_end[a]) ++a;
    return r.positions + a * r.pos_stride;
}
// Cosines and sines of pairs 8 v .. 8 v + 7 at a position of the table.
__device__ __forceinline__ void rope_row(const RopeParams& r, int v, int pos, float (&c)[8], float (&s)[8]) {
    const float* row = r.table + static_cast<long long>(pos) * r.rot + 8 * v;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float4 x = reinterpret_cast<const float4*>(row)[k];
        const float4 y = reinterpret_cast<const float4*>(row + (r.rot >> 1))[k];
        c[4 * k] = x.x, c[4 * k + 1] = x.y, c[4 * k + 2] = x.z, c[4 * k + 3] = x.w;
        s[4 * k] = y.x, s[4 * k + 1] = y.y, s[4 * k + 2] = y.z, s[4 * k + 3] = y.w;
    }
}

// Cosines and (signed) sines of pairs 8 v .. 8 v + 7 of token `tok` (own_pos
// stands in where there is no position array). False where a position of these
// pairs is outside the table, which is then not read. SPLIT: sections may end
// inside the eight pairs (rope_split); without it they share one axis, and the
// table is read in 16-byte pieces.
template <bool SPLIT>
__device__ __forceinline__ bool rope_coeffs(const RopeParams& r, int v, long long tok, int own_pos,
                                            float (&c)[8], float (&s)[8]) {
    if constexpr (!SPLIT) {
        const int pos = r.positions ? rope_axis(r, v)[tok] : own_pos;
        if (static_cast<unsigned>(pos) >= static_cast<unsigned>(r.max_pos)) return false;
        rope_row(r, v, pos, c, s);
    } else {
        // The row of the first pair's axis, then over its end those of the axes behind it
        // (an axis without pairs is not read).
        const int i0 = 8 * v;
        int a = 0;
        while (a + 1 < r.axes && i0 >= r.sec_end[a]) ++a;
        const int pos = r.positions[a * r.pos_stride + tok];
        if (static_cast<unsigned>(pos) >= static_cast<unsigned>(r.max_pos)) return false;
        rope_row(r, v, pos, c, s);
#pragma unroll 1
        for (++a; a < r.axes && r.sec_end[a - 1] < i0 + 8; ++a) {
            if (r.sec_end[a] == r.sec_end[a - 1]) continue;
            const int next = r.positions[a * r.pos_stride + tok];
            if (static_cast<unsigned>(next) >= static_cast<unsigned>(r.max_pos)) return false;
            const float* row = r.table + static_cast<long long>(next) * r.rot + i0;
            const int from = r.sec_end[a - 1] - i0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 x = reinterpret_cast<const float4*>(row)[k];
                const float4 y = reinterpret_cast<const float4*>(row + (r.rot >> 1))[k];
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * k + e >= from) c[4 * k + e] = xs[e], s[4 * k + e] = ys[e];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] *= r.sign;
    return true;
}

// Whether `ok` holds for all threads of a token, 2^log_parts neighbours of a
// warp whose threads all come here.
__device__ __forceinline__ bool token_ok(bool ok, int log_parts) {
    const unsigned bad = __ballot_sync(0xffffffffu, !ok);
    const unsigned mine = ((1u << (1 << log_parts)) - 1u) << (threadIdx.x & 31 & ~((1 << log_parts) - 1));
    return (bad & mine) == 0u;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void rope_turn(float& a, float& b, float c, float s) {
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// Both vectors of part v, turned in place (pairs only).
__device__ __forceinline__ void rope_apply(bool interleaved, const float (&c)[8], const float (&s)[8], float (&x)[8],
                                           float (&y)[8]) {
    if (interleaved) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            rope_turn(x[2 * k], x[2 * k + 1], c[k], s[k]);
            rope_turn(y[2 * k], y[2 * k + 1], c[4 + k], s[4 + k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) rope_turn(x[k], y[k], c[k], s[k]);
    }
}

// Heads h0, h0 + step, ... below h1 of one token, part v: read at x, rotated,
// written at y (element pointers of the token's head 0; strides between heads
// in elements). Four heads' loads are in flight at once.
__device__ __forceinline__ void rope_heads(const RopeParams& r, int v, bool turn, const float (&c)[8],
                                           const float (&s)[8], const __nv_bfloat16* x, __nv_bfloat16* y,
                                           long long xh, long long yh, int h0, int h1, int step) {
    int c0, c1;
    rope_columns(r, v, c0, c1);
    constexpr int U = 4;
    for (int h = h0; h < h1; h += U * step) {
        uint4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u * step < h1) {
                const __nv_bfloat16* p = x + (h + u * step) * xh;
                a[u] = *reinterpret_cast<const uint4*>(p + c0);
                b[u] = *reinterpret_cast<const uint4*>(p + c1);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u * step < h1) {
                if (turn) {
                    float fa[8], fb[8];
                    unpack_bf16x8(a[u], fa);
                    unpack_bf16x8(b[u], fb);
                    rope_apply(r.interleaved != 0, c, s, fa, fb);
                    a[u] = pack_bf16x8(fa);
                    b[u] = pack_bf16x8(fb);
                }
                __nv_bfloat16* p = y + (h + u * step) * yh;
                *reinterpret_cast<uint4*>(p + c0) = a[u];
                *reinterpret_cast<uint4*>(p + c1) = b[u];
            }
        }
    }
}

// Host side: whether a section ends inside a thread's eight pairs.
inline bool rope_split(const RopeParams& r) {
    for (int a = 0; a + 1 < r.axes; ++a)
        if (r.sec_end[a] % 8 != 0) return true;
    return false;
}
// Host side: checks a rotation's description (fa_rope.cu).
fa_status check_rope(const fa_rotation* rope, int d);
RopeParams rope_params(const fa_rotation* rope, long long tokens, bool inverse);

}  // namespace fa
