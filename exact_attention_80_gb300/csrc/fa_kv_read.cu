// fa_kv_read.cu — fa_kv_read_fp8: keys and values of cached tokens back from the paged
// e4m3 cache, as packed bf16 rows.
//
// x = code * scale of its page and head, formed in fp32 and rounded to bf16 once: exact
// for the power-of-two scales of the append, since a code has four significant bits.
// Bound by memory: a code is read once and written twice its size (six bytes a value of
// K and V together). A thread holds one token's sixteen codes at a time, of one head's K
// or V after the other: sixteen bytes loaded, 32 written, all loads of a thread
// independent of one another behind the token's page. Which sequence a token belongs to
// is found once per block, so the chain is offsets, page, codes. A thread's 32 bytes go
// out as one store where the outputs and their tokens lie at multiples of 32 bytes (WIDE):
// as two of sixteen, each leaves half of every sector to the other (eight contexts of up
// to 16200 tokens, 8 heads of 128: 84.7 us against 64.6, 6.35 TB/s).
#include <algorithm>
#include <cstring>

#include "fa.h"
#include "fa_launch.h"
#include "fa_paged.cuh"

namespace fa {
namespace {

struct ReadParams {
    const uint8_t* codes[2];   // [num_pages][Hkv][page_size][d]: K, V
    const float* scale[2];     // [num_pages][Hkv]
    __nv_bfloat16* out[2];     // [total][Hkv][d], tokens stride elements apart
    long long stride[2];
    const int* page_table;     // [B][max_pages]
    const int* cu;             // [B + 1]
    const int* starts;         // [B] or null
    int B, Hkv, total, num_pages, log_page, max_pages, fill;
    int items, per_block;      // 2 Hkv (head, K or V) pairs, and how many a block takes
    unsigned* status;
};

constexpr int kReadThreads = 256;

template <int D, bool WIDE>
__global__ void __launch_bounds__(kReadThreads) fa_kv_read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int LANES = D / 16, TOKENS = kReadThreads / LANES, UNROLL = 16;
    __shared__ int seq_of[TOKENS];
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int t0 = blockIdx.x * TOKENS, t1 = min(p.total, t0 + TOKENS);
    if (threadIdx.x < TOKENS) seq_of[threadIdx.x] = -1;
    __syncthreads();
    // The sequences that have tokens here; a broken one has none.
    const long long slots = static_cast<long long>(p.max_pages) << p.log_page;
    for (int b = threadIdx.x; b < p.B; b += kReadThreads) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1], s = p.starts ? p.starts[b] : 0;
        const bool ok = 0 <= c0 && c0 <= c1 && c1 <= p.total && s >= 0 && s <= slots - (c1 - c0);
        if (!ok) {
            if (blockIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, kStatusBadSeqlens);
            continue;
        }
        for (int t = max(c0, t0); t < min(c1, t1); ++t) seq_of[t - t0] = b;
    }
    __syncthreads();
    const int lane = threadIdx.x % LANES, at = threadIdx.x / LANES, token = t0 + at;
    if (token >= p.total) return;
    const int b = seq_of[at];
    const int first = blockIdx.y * p.per_block, last = min(p.items, first + p.per_block);
    auto dst = [&](int item) {
        const int w = item & 1;
        return p.out[w] + static_cast<long long>(token) * p.stride[w] + static_cast<long long>(item >> 1) * D +
               lane * 16;
    };
    auto put = [&](__nv_bfloat16* to, const uint32_t (&x)[8]) {
        if constexpr (WIDE) {
            st_global_v8(to, x);
        } else {
            reinterpret_cast<uint4*>(to)[0] = make_uint4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<uint4*>(to)[1] = make_uint4(x[4], x[5], x[6], x[7]);
        }
    };
    if (b < 0) {
        if (!p.fill) return;
        const int c0 = p.cu[0], c1 = p.cu[p.B];
        // (A broken sequence's tokens stay as they are.)
        if (!(0 <= c0 && c0 <= c1 && c1 <= p.total) || (token >= c0 && token < c1)) return;
        const uint32_t zero[8] = {};
        for (int i = first; i < last; ++i) put(dst(i), zero);
        return;
    }
    const int pos = token - p.cu[b] + (p.starts ? p.starts[b] : 0);
    const int page = p.page_table[static_cast<long long>(b) * p.max_pages + (pos >> p.log_page)];
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.status, kStatusBadPage);
        return;
    }
    const int slot = pos & ((1 << p.log_page) - 1);
    for (int i0 = first; i0 < last; i0 += UNROLL) {
        uint4 c[UNROLL];
        float f[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int i = i0 + u;
            if (i >= last) break;
            const long long cell = static_cast<long long>(page) * p.Hkv + (i >> 1);
            c[u] = __ldcs(
                reinterpret_cast<const uint4*>(p.codes[i & 1] + ((cell << p.log_page) + slot) * D + lane * 16));
            f[u] = p.scale[i & 1][cell];
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (i0 + u >= last) break;
            const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
            uint32_t x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y[4];
                decode_e4m3x4(w[e], y);
                x[2 * e] = pack_bf16x2(y[0] * f[u], y[1] * f[u]);
                x[2 * e + 1] = pack_bf16x2(y[2] * f[u], y[3] * f[u]);
            }
            put(dst(i0 + u), x);
        }
    }
}

template <int D>
cudaError_t launch_read(const ReadParams& p, dim3 grid, cudaStream_t stream) {
    const bool wide = aligned(p.out[0], 32) && aligned(p.out[1], 32) && p.stride[0] % 16 == 0 && p.stride[1] % 16 == 0;
    return launch_dependent(wide ? fa_kv_read_kernel<D, true> : fa_kv_read_kernel<D, false>, grid, kReadThreads, 0,
                            stream, p);
}

}  // namespace
}  // namespace fa

extern "C" fa_status fa_kv_read_fp8(const fa_paged_cache* cache, const int* page_table, const int* cu_seqlens,
                                    const int* starts, void* k_out, void* v_out, int B, int total, int max_pages,
                                    long long k_stride, long long v_stride, int fill, cudaStream_t stream) {
    if (!cache || !page_table || !cu_seqlens || !k_out || !v_out) return FA_ERR_NULL;
    const fa_status s = fa::check_cache(cache);
    if (s != FA_OK) return s;
    const int d = cache->d, Hkv = cache->Hkv;
    if (B < 1 || total < 1 || total > 0x3fffffff || max_pages < 1) return FA_ERR_SHAPE;
    if (static_cast<long long>(max_pages) * cache->page_size > 0x7fffffffll - 4096) return FA_ERR_SHAPE;
    if (!fa::aligned(k_out, 16) || !fa::aligned(v_out, 16) || !fa::aligned(page_table, 4) ||
        !fa::aligned(cu_seqlens, 4) || !fa::aligned(starts, 4))
        return FA_ERR_ALIGN;
    if (!fa::token_stride(k_stride, Hkv, d) || !fa::token_stride(v_stride, Hkv, d)) return FA_ERR_STRIDE;
    // Few tokens: their heads go to several blocks, until there are about four per SM.
    const int tokens = fa::kReadThreads / (d / 16);
    const long long blocks = (static_cast<long long>(total) + tokens - 1) / tokens;
    const int items = 2 * Hkv;
    int per_block = items;
    while (per_block > 1 && (blocks * ((items + per_block - 1) / per_block) < 4 * 152 ||
                             (items + per_block - 1) / per_block < (items + 65534) / 65535))
        per_block = (per_block + 1) / 2;
    const long long parts = (items + per_block - 1) / per_block;
    // A block looks through all sequences, at 320 to 570 of them a nanosecond on the whole
    // GPU (65536, a million tokens of one head of 64: 2.7 ms); 2^41 take 4 to 7 s.
    if (blocks * parts > (1ll << 41) / B) return FA_ERR_SHAPE;
    fa::ReadParams p;
    std::memset(&p, 0, sizeof(p));
    p.items = items;
    p.per_block = per_block;
    p.codes[0] = static_cast<const uint8_t*>(cache->k);
    p.codes[1] = static_cast<const uint8_t*>(cache->v);
    p.scale[0] = cache->k_scale;
    p.scale[1] = cache->v_scale;
    p.out[0] = static_cast<__nv_bfloat16*>(k_out);
    p.out[1] = static_cast<__nv_bfloat16*>(v_out);
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.page_table = page_table;
    p.cu = cu_seqlens;
    p.starts = starts;
    p.B = B;
    p.Hkv = Hkv;
    p.total = total;
    p.num_pages = cache->num_pages;
    p.log_page = fa::log2_exact(cache->page_size);
    p.max_pages = max_pages;
    p.fill = fill ? 1 : 0;
    if (fa::device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(parts), 1);
    const cudaError_t e = d == 64    ? fa::launch_read<64>(p, grid, stream)
                          : d == 128 ? fa::launch_read<128>(p, grid, stream)
                                     : fa::launch_read<256>(p, grid, stream);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
