// fa_kv_append.cu — fa_kv_append_fp8: new keys (rotated) and values appended to
// a paged e4m3 cache, and the new queries rotated, in one launch.
//
// A page holds page_size tokens of one sequence; page and head share one scale
// 2^e, e the least exponent with amax <= 448 * 2^e over the block's tokens, so
// no code saturates and a code times its scale is exact in fp32 and bf16. An
// append to a page that holds earlier tokens of the sequence keeps the larger
// of the old and the new scale; where it grows, the earlier codes are rounded
// again to the new scale (a power of two apart: only values that become
// subnormal in e4m3 change). The first slot of a page starts a new block: what
// the page's scale was for an earlier owner does not count.
//
// An item is (sequence, page it touches, kv head, K or V). Its threads hold the
// item's new values in registers (sixteen columns of up to four tokens each), so
// the input is read once: rotate, reduce |.| over the item, form the scale,
// round, store. Launch-bound for single tokens; for prompts bound by the loads
// in flight, since positions and table rows are two loads behind the offsets:
// hence four tokens a thread rather than one (141 us with one, for the prompts
// measured at the kernel). An item's threads are a power of two: within a warp
// (a single token at d = 128 takes eight threads, so one warp serves four
// items; a page of 16 takes one warp), or a whole block of up to 512.
#include <algorithm>
#include <cstring>

#include <cuda_fp16.h>

#include "fa.h"
#include "fa_paged.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

struct AppendLaunch {
    RopeParams r;
    const __nv_bfloat16* q;      // [total][H][d], token stride q_stride; null: no queries
    const __nv_bfloat16* kv[2];  // k, v: [total][Hkv][d], token strides kv_stride
    __nv_bfloat16* q_out;        // [total][H][d]
    long long q_stride, kv_stride[2];
    uint8_t* cache[2];           // [num_pages][Hkv][page_size][d]
    float* scale[2];             // [num_pages][Hkv]
    const int* page_table;       // [B][max_pages]
    const int* cu;               // [B + 1] new tokens
    const int* lens;             // [B] cache lengths, the new tokens among them
    int B, H, Hkv, total, max_new, num_pages, log_page, max_pages, d;
    int log_parts;               // log2(d / 16)
    int log_slots;               // log2(token slots an item's threads cover)
    int log_group;               // log2(threads per item)
    int touch;                   // pages a sequence can touch
    unsigned items;              // B * touch * Hkv * 2
    unsigned item_blocks;        // blocks that take items; the others take queries
    int q_log_tb, q_chunks;      // queries: log2(tokens per block), token blocks per sequence
    int q_heads_chunk, q_heads_blocks;
    unsigned* status;
};

// Largest finite absolute value of a thread's two vectors: |x| + 0 x is NaN where x is
// not finite, and fmaxf drops NaN.
__device__ __forceinline__ float amax16(const float (&x)[8], const float (&y)[8]) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fmaxf(fmaf(x[k], 0.f, fabsf(x[k])), fmaf(y[k], 0.f, fabsf(y[k]))));
    return m;
}

// Least e with a <= 448 * 2^e = 1.75 * 2^(e + 8), within [kScaleExpMin, kScaleExpMax].
__device__ __forceinline__ int scale_exponent(float a) {
    const uint32_t bits = __float_as_uint(a);
    const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return a > 0.f ? min(max(e, kScaleExpMin), kScaleExpMax) : kScaleExpMin;
}

// Eight codes of x inv; what is not finite becomes e4m3's NaN (x inv + 0 x is NaN for an
// infinity, which the conversion alone would make 448).
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = fmaf(x[k], inv, x[k] * 0.f);
    return make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
}

// Sixteen codes times `f` (a power of two below one), rounded to e4m3 again.
__device__ __forceinline__ uint4 recode16(const uint4& u, float f) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float x[4];
        decode_e4m3x4(w[k], x);
        w[k] = pack_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The queries of one token block: rotated (or copied) into q_out.
template <bool SPLIT>
__device__ __forceinline__ void append_queries(const AppendLaunch& p, unsigned lin) {
    const int hb = static_cast<int>(lin % static_cast<unsigned>(p.q_heads_blocks));
    lin /= static_cast<unsigned>(p.q_heads_blocks);
    const int b = static_cast<int>(lin / static_cast<unsigned>(p.q_chunks));
    const int chunk = static_cast<int>(lin % static_cast<unsigned>(p.q_chunks));
    const int v = threadIdx.x & ((1 << p.log_parts) - 1);
    const int rest = threadIdx.x >> p.log_parts;
    const int i = (chunk << p.q_log_tb) + (rest & ((1 << p.q_log_tb) - 1));
    const int hs = rest >> p.q_log_tb;
    const int hstep = blockDim.x >> (p.log_parts + p.q_log_tb);
    NewTokens t;
    const bool in = new_tokens(p.cu, p.lens, b, p.total, p.max_new, p.max_pages << p.log_page, t) && i < t.n;
    const long long tok = t.first + i;
    const bool turn = p.r.table && v < (p.r.rot >> 4);
    float c[8], s[8];
    bool ok = true;
    if (in && turn) ok = rope_coeffs<SPLIT>(p.r, v, tok, t.len - t.n + i, c, s);
    ok = token_ok(ok, p.log_parts);
    if (!in) return;
    if (!ok) {
        if (v == 0 && hs == 0) atomicOr(p.status, kStatusBadPosition);
        return;
    }
    const int lo = hb * p.q_heads_chunk;
    const int hi = min(lo + p.q_heads_chunk, p.H);
    rope_heads(p.r, v, turn, c, s, p.q + tok * p.q_stride, p.q_out + tok * static_cast<long long>(p.H) * p.d, p.d,
               p.d, lo + hs, hi, hstep);
}

// PER: token slots of an item held by one thread.
// BLOCK: an item is a whole block (its reduction goes through shared memory);
// otherwise a power-of-two group within a warp.
// SPLIT: sections that end inside a thread's eight pairs; the second row of the table
// costs registers (two blocks per SM 109 us, three 113, for the prompts above).
template <int PER, bool BLOCK, bool SPLIT>
__global__ void __launch_bounds__(BLOCK ? 512 : 256, BLOCK ? 1 : SPLIT && PER == 4 ? 2 : 3)
    fa_kv_append_kernel(const __grid_constant__ AppendLaunch p) {
    __shared__ float red[16];
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    // Item blocks are spread evenly among the query blocks: items wait for long
    // chains of loads, queries for bandwidth, so each fills the other's gaps
    // (six ragged prompts of 4001 tokens, 32 + 2 * 8 heads, d = 128: 83 us; the
    // items alone took 47, the queries 52, when both took 87).
    const unsigned long long total_blocks = gridDim.x;
    const unsigned before = static_cast<unsigned>(blockIdx.x * static_cast<unsigned long long>(p.item_blocks) / total_blocks);
    const unsigned after =
        static_cast<unsigned>((blockIdx.x + 1ull) * static_cast<unsigned long long>(p.item_blocks) / total_blocks);
    if (before == after) {
        append_queries<SPLIT>(p, blockIdx.x - before);
        return;
    }
    const unsigned item = before * (blockDim.x >> p.log_group) + (threadIdx.x >> p.log_group);
    const int g = threadIdx.x & ((1 << p.log_group) - 1);
    // An item's threads agree on everything below up to the item's end; in a
    // group within a warp the whole warp runs the reduction.
    bool live = item < p.items;
    unsigned lin = live ? item : 0u;
    const int which = lin >= p.items / 2 ? 1 : 0;  // all of K's items, then V's
    if (which) lin -= p.items / 2;
    const int h = static_cast<int>(lin % static_cast<unsigned>(p.Hkv));
    lin /= static_cast<unsigned>(p.Hkv);
    const int touch = static_cast<int>(lin % static_cast<unsigned>(p.touch));
    const int b = static_cast<int>(lin / static_cast<unsigned>(p.touch));

    NewTokens t;
    const bool valid = new_tokens(p.cu, p.lens, b, p.total, p.max_new, p.max_pages << p.log_page, t);
    if (!valid && live && g == 0 && which == 0 && h == 0 && touch == 0) atomicOr(p.status, kStatusBadSeqlens);
    const int page_size = 1 << p.log_page;
    const int start = t.len - t.n;                    // slot of the sequence's first new token
    const int blk = (start >> p.log_page) + touch;    // page index within the sequence
    // (Page indices past the table would overflow as slots where max_new is large.)
    live = live && valid && t.n > 0 && blk < p.max_pages;
    const int lo = touch == 0 ? (start & (page_size - 1)) : 0;             // first new slot of the page
    const int hi = min(page_size, t.len - (blk << p.log_page));            // end of the new slots
    live = live && lo < hi;
    const int v = g & ((1 << p.log_parts) - 1);
    const int slot0 = g >> p.log_parts;
    const int slot_step = 1 << (p.log_group - p.log_parts);
    const bool turn = which == 0 && p.r.table && v < (p.r.rot >> 4);
    int c0, c1;
    if (which == 0 && p.r.table) rope_columns(p.r, v, c0, c1);
    else c0 = 16 * v, c1 = 16 * v + 8;

    // The new values stay packed in registers: rotating them twice, for the
    // maximum and for the codes, costs less than the registers of their fp32
    // values (101 against 118 us for the prompts above: three blocks per SM
    // rather than two).
    uint4 a[PER], c[PER];
    const __nv_bfloat16* src = which ? p.kv[1] : p.kv[0];
    const long long stride = which ? p.kv_stride[1] : p.kv_stride[0];
    const long long tok0 = static_cast<long long>(t.first) + (blk << p.log_page) - start;  // token of slot 0
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int slot = lo + slot0 + i * slot_step;
        a[i] = c[i] = make_uint4(0u, 0u, 0u, 0u);
        if (live && slot < hi) {
            const __nv_bfloat16* row = src + (tok0 + slot) * stride + static_cast<long long>(h) * p.d;
            a[i] = *reinterpret_cast<const uint4*>(row + c0);
            c[i] = *reinterpret_cast<const uint4*>(row + c1);
        }
    }
    // The slots' positions, all at once; a slot without a token takes row 0.
    int at[PER];
    if constexpr (!SPLIT) {
        if (turn && live) {
            const int* axis = rope_axis(p.r, v);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int slot = lo + slot0 + i * slot_step;
                at[i] = slot >= hi ? 0 : p.r.positions ? axis[tok0 + slot] : (blk << p.log_page) + slot;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const bool outside = static_cast<unsigned>(at[i]) >= static_cast<unsigned>(p.r.max_pos);
                bad = bad || outside;
                at[i] = outside ? 0 : at[i];
            }
        }
    }
    int page = -1;
    if (live) {
        page = p.page_table[static_cast<long long>(b) * p.max_pages + blk];
        if (page < 0 || page >= p.num_pages) {
            if (g == 0 && which == 0 && h == 0) atomicOr(p.status, kStatusBadPage);
            live = false;
        }
    }
    // A position outside the table spoils the whole item: found by the threads
    // that hold its pairs, agreed on with the reduction.
    auto values = [&](int i, float (&x)[8], float (&y)[8]) {
        const int slot = lo + slot0 + i * slot_step;
        unpack_bf16x8(a[i], x);
        unpack_bf16x8(c[i], y);
        if constexpr (!SPLIT) {
            if (turn && live) {
                float co[8], si[8];
                rope_row(p.r, v, at[i], co, si);
                rope_apply(p.r.interleaved != 0, co, si, x, y);
            }
        } else if (turn && live && slot < hi && !bad) {
            float co[8], si[8];
            if (rope_coeffs<SPLIT>(p.r, v, tok0 + slot, (blk << p.log_page) + slot, co, si))
                rope_apply(p.r.interleaved != 0, co, si, x, y);
            else bad = true;
        }
    };
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        float x[8], y[8];
        values(i, x, y);
        amax = fmaxf(amax, amax16(x, y));
    }
    if (bad) amax = -1.f;  // marks the item: the reduction below keeps it apart

    // Item-wide maximum, and whether any thread found a bad position.
    float* sc = which ? p.scale[1] : p.scale[0];
    const long long cell = static_cast<long long>(page) * p.Hkv + h;
    const float s_old = (live && lo > 0) ? sc[cell] : 0.f;
    float mx = amax, mn = amax;
    const int width = BLOCK ? 32 : (1 << p.log_group);
    for (int o = width >> 1; o > 0; o >>= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    if constexpr (BLOCK) {
        const int warps = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mn < 0.f ? -1.f : mx;
        __syncthreads();
        mx = 0.f, mn = 0.f;
        for (int w = 0; w < warps; ++w) {
            mx = fmaxf(mx, red[w]);
            mn = fminf(mn, red[w]);
        }
    } else {
        __syncwarp();
    }
    if (!live) return;
    // The codes below read the table again: keeping every cosine and sine across
    // the reduction would take more registers than there are.
    asm volatile("" ::: "memory");
    if (mn < 0.f) {
        if (g == 0) atomicOr(p.status, kStatusBadPosition);
        return;
    }
    const float s_new = fmaxf(exp2i(scale_exponent(mx)), s_old);
    const float inv = 1.f / s_new;  // exact: a power of two (old scales are the caller's)
    uint8_t* base = (which ? p.cache[1] : p.cache[0]) + (cell << p.log_page) * p.d;
    if (lo > 0 && s_new > s_old) {
        // The earlier tokens of the block, at its new scale. Their bytes are
        // this item's alone, and no thread reads a slot that another writes.
        const float f = s_old / s_new;
        const int vecs = (lo * p.d) >> 4;
        for (int k = g; k < vecs; k += 1 << p.log_group) {
            uint4* at = reinterpret_cast<uint4*>(base) + k;
            *at = recode16(*at, f);
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int slot = lo + slot0 + i * slot_step;
        if (slot < hi) {
            float x[8], y[8];
            values(i, x, y);
            uint8_t* row = base + slot * p.d;
            *reinterpret_cast<uint2*>(row + c0) = encode8(x, inv);
            *reinterpret_cast<uint2*>(row + c1) = encode8(y, inv);
        }
    }
    if (g == 0) sc[cell] = s_new;
}

}  // namespace
}  // namespace fa

extern "C" fa_status fa_kv_append_fp8(const void* q, const void* k, const void* v, void* q_out,
                                      const fa_rotation* rope, const fa_paged_cache* cache, const int* page_table,
                                      const int* cu_seqlens, const int* seqlens_k, int B, int H, int total_new,
                                      int max_new, int max_pages, long long q_stride, long long k_stride,
                                      long long v_stride, cudaStream_t stream) {
    if (!k || !v || !cache || !page_table || !cu_seqlens || !seqlens_k) return FA_ERR_NULL;
    if ((q == nullptr) != (q_out == nullptr)) return FA_ERR_NULL;
    const fa_status sc = fa::check_cache(cache);
    if (sc != FA_OK) return sc;
    const int d = cache->d, Hkv = cache->Hkv;
    if (B < 1 || total_new < 1 || max_new < 1 || max_new > total_new || max_pages < 1) return FA_ERR_SHAPE;
    if (total_new > 0x7fffffff - 4096) return FA_ERR_SHAPE;  // token indices of whole blocks are int
    if (q && (H < 1 || H > 65535)) return FA_ERR_SHAPE;
    if (static_cast<long long>(max_pages) * cache->page_size > 0x7fffffffll - 4096) return FA_ERR_SHAPE;
    if (!fa::aligned(k, 16) || !fa::aligned(v, 16) || !fa::aligned(q, 16) || !fa::aligned(q_out, 16) ||
        !fa::aligned(page_table, 4) || !fa::aligned(cu_seqlens, 4) || !fa::aligned(seqlens_k, 4))
        return FA_ERR_ALIGN;
    const long long most = 1ll << 32;  // elements between tokens: offsets stay far from 64 bits
    if (k_stride % 8 || v_stride % 8 || k_stride < 0 || v_stride < 0 || k_stride > most || v_stride > most)
        return FA_ERR_STRIDE;
    if (q && (q_stride % 8 || q_stride < 0 || q_stride > most)) return FA_ERR_STRIDE;
    if (rope) {
        const fa_status s = fa::check_rope(rope, d);
        if (s != FA_OK) return s;
    }
    fa::AppendLaunch p;
    std::memset(&p, 0, sizeof(p));
    p.r = fa::rope_params(rope, total_new, false);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.kv[0] = static_cast<const __nv_bfloat16*>(k);
    p.kv[1] = static_cast<const __nv_bfloat16*>(v);
    p.q_stride = q_stride;
    p.kv_stride[0] = k_stride;
    p.kv_stride[1] = v_stride;
    p.cache[0] = static_cast<uint8_t*>(cache->k);
    p.cache[1] = static_cast<uint8_t*>(cache->v);
    p.scale[0] = cache->k_scale;
    p.scale[1] = cache->v_scale;
    p.page_table = page_table;
    p.cu = cu_seqlens;
    p.lens = seqlens_k;
    p.B = B;
    p.H = q ? H : 0;
    p.Hkv = Hkv;
    p.total = total_new;
    p.max_new = max_new;
    p.num_pages = cache->num_pages;
    p.log_page = fa::log2_exact(cache->page_size);
    p.max_pages = max_pages;
    p.d = d;
    p.log_parts = d == 64 ? 2 : d == 128 ? 3 : 4;
    // Slots of a page that one append can fill, rounded up to a power of two.
    p.log_slots = 0;
    while (p.log_slots < p.log_page && (1 << p.log_slots) < max_new) ++p.log_slots;
    const int log_lanes = p.log_parts + p.log_slots;  // sixteen-column pieces of an item: at most 2^11
    const int log_per = std::min(std::max(log_lanes - 5, 0), 2);
    p.log_group = log_lanes - log_per;
    const int per = 1 << log_per;
    p.touch = static_cast<int>((static_cast<long long>(cache->page_size) - 1 + max_new + cache->page_size - 1) >>
                               p.log_page);
    const long long items = static_cast<long long>(B) * p.touch * Hkv * 2;
    if (items > 0x7fffffffll) return FA_ERR_SHAPE;
    p.items = static_cast<unsigned>(items);
    const unsigned threads = p.log_group > 5 ? 1u << p.log_group : (q ? 256u : 128u);
    const long long per_block = static_cast<long long>(threads) >> p.log_group;
    const long long item_blocks = (items + per_block - 1) / per_block;
    long long q_blocks = 0;
    if (q) {
        int log_threads = 0;
        while ((1u << log_threads) < threads) ++log_threads;
        const int room = std::max(0, log_threads - p.log_parts);
        while (p.q_log_tb < room && (1 << p.q_log_tb) < max_new) ++p.q_log_tb;
        p.q_chunks = (max_new + (1 << p.q_log_tb) - 1) >> p.q_log_tb;
        q_blocks = static_cast<long long>(B) * p.q_chunks;
        const int hstep = 1 << (room - p.q_log_tb);
        int chunk = 16 * hstep;
        while (chunk > hstep && q_blocks * ((H + chunk - 1) / chunk) < 4ll * 152) chunk >>= 1;
        p.q_heads_chunk = chunk;
        p.q_heads_blocks = (H + chunk - 1) / chunk;
        q_blocks *= p.q_heads_blocks;
    }
    if (item_blocks + q_blocks > 0x7fffffffll) return FA_ERR_SHAPE;
    p.item_blocks = static_cast<unsigned>(item_blocks);
    if (fa::device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(item_blocks + q_blocks), 1, 1);
    const bool split = fa::rope_split(p.r);
    auto kernel = p.log_group > 5 ? (split ? fa::fa_kv_append_kernel<4, true, true> : fa::fa_kv_append_kernel<4, true, false>)
                  : per == 1 ? (split ? fa::fa_kv_append_kernel<1, false, true> : fa::fa_kv_append_kernel<1, false, false>)
                  : per == 2 ? (split ? fa::fa_kv_append_kernel<2, false, true> : fa::fa_kv_append_kernel<2, false, false>)
                             : (split ? fa::fa_kv_append_kernel<4, false, true> : fa::fa_kv_append_kernel<4, false, false>);
    const cudaError_t e = fa::launch_dependent(kernel, grid, threads, 0, stream, p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
