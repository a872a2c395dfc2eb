// fa_rope.cu — fa_rope: rotary positions with one to four axes on two tensors
// (queries and keys) in one launch, forward or inverse. The mathematics and
// the columns of a thread are in fa_rope.cuh.
//
// Memory-bound: every value is read and written once; the table rows of a
// token are read once per head group and stay in L1/L2. A block of 256 threads
// takes `tb` tokens (d / 16 threads each) and 256 / (tb * d / 16) heads at a
// time, and walks a chunk of the heads of both tensors.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa.h"
#include "fa_rope.cuh"

namespace fa {
namespace {

struct RopeTensor {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    int H;
    long long xs[3], ys[3];  // batch, head, token
};

struct RopeLaunch {
    RopeParams r;
    RopeTensor t[2];
    long long tokens;  // B * N
    int N;
    int log_parts;     // log2(d / 16): threads per token
    int log_tb;        // log2(tokens per block)
    int heads_chunk;   // heads (of both tensors in sequence) per block
    unsigned* status;
};

constexpr int kRopeThreads = 256;

template <bool SPLIT>
__global__ void __launch_bounds__(kRopeThreads, 3) fa_rope_kernel(const __grid_constant__ RopeLaunch p) {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int v = threadIdx.x & ((1 << p.log_parts) - 1);
    const int rest = threadIdx.x >> p.log_parts;
    const long long tok = (static_cast<long long>(blockIdx.x) << p.log_tb) + (rest & ((1 << p.log_tb) - 1));
    const int hs = rest >> p.log_tb;
    const int hstep = kRopeThreads >> (p.log_parts + p.log_tb);
    const bool turn = v < (p.r.rot >> 4);
    float c[8], s[8];
    const bool in = tok < p.tokens;
    bool ok = true;
    if (in && turn) ok = rope_coeffs<SPLIT>(p.r, v, tok, 0, c, s);
    ok = token_ok(ok, p.log_parts);
    if (!in) return;
    if (!ok) {
        if (v == 0 && hs == 0 && blockIdx.y == 0) atomicOr(p.status, kStatusBadPosition);
        return;
    }
    const long long b = tok / p.N;
    const long long n = tok - b * p.N;
    const int lo = blockIdx.y * p.heads_chunk;
    const int hi = lo + p.heads_chunk;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const RopeTensor& t = p.t[i];
        const int base = i ? p.t[0].H : 0;  // this tensor's heads are [base, base + H) of the sequence
        const int h0 = max(lo - base, 0), h1 = min(hi - base, t.H);
        if (h0 < h1)
            rope_heads(p.r, v, turn, c, s, t.x + b * t.xs[0] + n * t.xs[2], t.y + b * t.ys[0] + n * t.ys[2], t.xs[1],
                       t.ys[1], h0 + hs, h1, hstep);
    }
}

}  // namespace

fa_status check_rope(const fa_rotation* rope, int d) {
    if (!rope->table) return FA_ERR_NULL;
    if (!aligned(rope->table, 16) || !aligned(rope->positions, 4)) return FA_ERR_ALIGN;
    if (rope->rot < 16 || rope->rot > d || rope->rot % 16 != 0) return FA_ERR_ROPE;
    if (rope->axes < 1 || rope->axes > FA_MAX_AXES || rope->max_pos < 1) return FA_ERR_ROPE;
    if (!rope->positions && rope->axes != 1) return FA_ERR_ROPE;
    if (rope->axes > 1) {
        long long sum = 0;
        for (int a = 0; a < rope->axes; ++a) {
            if (rope->sections[a] < 0) return FA_ERR_ROPE;
            sum += rope->sections[a];
        }
        if (sum != rope->rot / 2) return FA_ERR_ROPE;
    }
    return FA_OK;
}

RopeParams rope_params(const fa_rotation* rope, long long tokens, bool inverse) {
    RopeParams r;
    std::memset(&r, 0, sizeof(r));
    if (!rope) return r;
    r.table = rope->table;
    r.positions = rope->positions;
    r.pos_stride = tokens;
    r.rot = rope->rot;
    r.axes = rope->axes;
    r.max_pos = rope->max_pos;
    r.interleaved = rope->interleaved ? 1 : 0;
    r.sign = inverse ? -1.f : 1.f;
    int end = 0;
    for (int a = 0; a < FA_MAX_AXES; ++a) {
        if (a < rope->axes) end += rope->axes == 1 ? rope->rot / 2 : rope->sections[a];
        r.sec_end[a] = end;
    }
    return r;
}

}  // namespace fa

extern "C" fa_status fa_rope(const fa_rope_tensor* q, const fa_rope_tensor* k, const fa_rotation* rope, int B, int N,
                             int d, int inverse, cudaStream_t stream) {
    if (!q || !rope || !rope->positions) return FA_ERR_NULL;
    if (B < 1 || N < 1 || static_cast<long long>(B) * N > 0x7fffffffll) return FA_ERR_SHAPE;
    if (!fa::valid_d(d)) return FA_ERR_HEADDIM;
    const long long tokens = static_cast<long long>(B) * N;
    const fa_status s = fa::check_rope(rope, d);
    if (s != FA_OK) return s;
    fa::RopeLaunch p;
    std::memset(&p, 0, sizeof(p));
    int heads = 0;
    for (int i = 0; i < 2; ++i) {
        const fa_rope_tensor* t = i ? k : q;
        if (!t) continue;
        if (!t->x || !t->y) return FA_ERR_NULL;
        if (t->H < 1 || t->H > 65535) return FA_ERR_SHAPE;
        if (!fa::aligned(t->x, 16) || !fa::aligned(t->y, 16)) return FA_ERR_ALIGN;
        for (int j = 0; j < 3; ++j) {
            // Sixteen-byte vectors; the byte offsets must stay far from 64 bits.
            if (t->x_stride[j] % 8 != 0 || t->y_stride[j] % 8 != 0) return FA_ERR_STRIDE;
            if (t->x_stride[j] < 0 || t->y_stride[j] < 0 || t->x_stride[j] > (1ll << 40) ||
                t->y_stride[j] > (1ll << 40))
                return FA_ERR_STRIDE;
            // (Inputs may be expanded; outputs would be written many times.)
            if (t->y_stride[j] == 0 && (j == 0 ? B : j == 1 ? t->H : N) > 1) return FA_ERR_STRIDE;
            p.t[i].xs[j] = t->x_stride[j];
            p.t[i].ys[j] = t->y_stride[j];
        }
        p.t[i].x = static_cast<const __nv_bfloat16*>(t->x);
        p.t[i].y = static_cast<__nv_bfloat16*>(t->y);
        p.t[i].H = t->H;
        heads += t->H;
    }
    p.r = fa::rope_params(rope, tokens, inverse != 0);
    p.tokens = tokens;
    p.N = N;
    p.log_parts = d == 64 ? 2 : d == 128 ? 3 : 4;
    const int room = 8 - p.log_parts;  // log2 of (token, head) pairs per block
    p.log_tb = 0;
    while (p.log_tb < room && (1ll << p.log_tb) < tokens) ++p.log_tb;
    const long long bx = (tokens + (1ll << p.log_tb) - 1) >> p.log_tb;
    // Heads per block: as many as keep four blocks per SM in the grid.
    const int hstep = 1 << (room - p.log_tb);
    int chunk = 8 * hstep;
    while (chunk > hstep && bx * ((heads + chunk - 1) / chunk) < 4ll * 152) chunk >>= 1;
    p.heads_chunk = chunk;
    if (fa::device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>((heads + chunk - 1) / chunk), 1);
    const cudaError_t e = fa::launch_dependent(
        fa::rope_split(p.r) ? fa::fa_rope_kernel<true> : fa::fa_rope_kernel<false>, grid, fa::kRopeThreads, 0, stream, p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
