// fa_paged.cuh — pieces shared by the append to the paged e4m3 cache and the
// attention over it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <utility>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

// Exponents of a block's scale: 448 * 2^120 covers bf16's largest value, and
// 2^-100 keeps the reciprocal and sums of it far inside fp32.
constexpr int kScaleExpMin = -100;
constexpr int kScaleExpMax = 120;

// A V scale as the kernels use it (its logarithm and reciprocal): within the
// range of a scale, so that a block whose scale was never set, or is zero
// because its values are, counts as values next to zero.
__device__ __forceinline__ float usable_scale(float s) { return fminf(fmaxf(s, 0x1p-100f), 0x1p+120f); }

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The scale of a query row, from the bits of its largest |element| as an unsigned
// maximum (where every NaN and infinity lies above all finite values): f, a power of
// two, brings that element to [2^7, 2^8); f and 1 / f stay normal. The scores' factor
// back is 1 / f, or NaN where the row holds an element that is not finite: the operands would make
// a finite number of it (e4m3 has no infinity), so the row's scores are made NaN.
__device__ __forceinline__ uint32_t abs_bits_max(uint32_t m, const float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
    return m;
}
__device__ __forceinline__ int query_exponent(uint32_t bits) {  // of f
    const int ex = bits > 0u ? min(max(static_cast<int>(bits >> 23) - 127, -100), 120) : 0;
    return min(7 - ex, 120);
}
__device__ __forceinline__ float query_undo(uint32_t bits, float inverse) {
    return bits < 0x7f800000u ? inverse : __uint_as_float(0x7fffffffu);
}

// Four e4m3 codes as two packed f16 pairs (codes 0 and 1, 2 and 3): exact.
__device__ __forceinline__ void decode_e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void decode_e4m3x4(uint32_t w, float (&x)[4]) {
    uint32_t lo, hi;
    decode_e4m3x4_f16(w, lo, hi);
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

constexpr float kPShift = 7.f;  // p = 2^(x - m + 7)
constexpr float kPSlack = 8.f;  // the reference moves when x passes it by more, so p <= 2^15

struct PagedParams {
    CUtensorMap tm_k, tm_v;  // e4m3 [num_pages * Hkv * page_size][d], box {row part, keys per copy}
    const __nv_bfloat16* q;  // [total_q][H][d]
    __nv_bfloat16* o;
    float* lse;              // [H][total_q]
    const float* k_scale;    // [num_pages][Hkv]
    const float* v_scale;
    const int* page_table;   // [B][max_pages]
    const int* cu;
    const int* lens;
    float* ws_o;             // [splits][total_q * H][d]
    float* ws_m;             // base-2 units of the scaled score
    float* ws_l;
    int B, H, Hkv, G, total_q, max_q, max_k, num_pages, log_page, max_pages;
    int window, sinks;
    int row_blocks, num_splits, tiles_per_split;  // row blocks of block_rows rows, tiles of block_keys keys
    int block_rows, block_keys;
    // fa_paged_tc.cu: shares of a key tile's columns that copies of the rows take
    // (1, 2 or 4; 0: full tiles); softmax warps of a tile slot; whether the CTAs
    // choose the pieces' length.
    int shares, slot_warps, balance;
    float scale_log2;
    long long wait_limit;
    unsigned* status;
    // A batch that shares a prefix (fa_fwd_prefix_fp8; the kernels' PART forms): its keys
    // up to base_len, in the first base_pages entries of the table, are one part, the
    // sequences' own keys the other. `whole`: this launch is the first part, one problem
    // of all total_q rows that see all max_k keys. Either part leaves its states for a
    // merge in any case, as numbers state0 .. state0 + num_splits - 1.
    int base_len, base_pages, whole, state0;
    int own_q, own_k;  // bounds of a sequence's new tokens and of its own keys, in either part's launch
    // A launch of fa_paged_rows_kernel that takes both parts: the first `whole_ctas`
    // CTAs have the prefix, cut as `shared` says, the others the sequences' own keys;
    // `solo`: each warp of those a unit of its own (paged_unit), `places` of them, or twice
    // as many as run at once beside a launch that has part of the SMs.
    unsigned whole_ctas;
    int solo, places;
    // The second launch of a call that takes two: it need not wait for the first one, whose
    // CTAs have all waited for what came before when this grid may start, so the two run
    // side by side; one CTA more, the last, waits for the first launch, and by it the merge
    // does. What came before is visible to a grid that waits, and starting says nothing of
    // it, so it is passed on: the first launch's CTA 0 adds to `gate` behind its wait, before
    // it allows this grid, and every thread of this one reads that count first (`gate` is the
    // device's; all that ever happens to it is such adds, so a call's own or a later one
    // is what is read).
    int early;
    unsigned* gate;
    struct {
        int max_q, max_k, row_blocks, num_splits, tiles_per_split, state0;
    } shared;
};

// Waits for the grid before this one in the stream; false for the CTA that is there for
// that alone.
template <bool PART>
__device__ __forceinline__ bool paged_wait(const PagedParams& p) {
    if (PART && p.early) {
        if (blockIdx.x + 1 < gridDim.x) {
            gate_acquire(p.gate);
            return true;
        }
        griddep_wait();
        return false;
    }
    griddep_wait();
    return true;
}
// Lets the next grid start.
template <bool PART>
__device__ __forceinline__ void paged_allow(const PagedParams& p) {
    if (threadIdx.x == 0) {
        // (The test makes it wait for the add; a grid whose CTA 0 says nothing is allowed by its end.)
        const bool add = PART && p.gate && !p.early && blockIdx.x == 0;
        if (!add || gate_release(p.gate) != 0xffffffffu) griddep_launch_dependents();
    }
}
// The new tokens of sequence b (of the one problem where `whole`), positions and lengths
// without the keys of a shared prefix. False where they are broken.
template <bool PART>
__device__ __forceinline__ bool paged_tokens(const PagedParams& p, bool whole, int b, NewTokens& t) {
    if constexpr (!PART) return new_tokens(p.cu, p.lens, b, p.total_q, p.max_q, p.max_k, t);
    if (whole) {
        t = {0, p.total_q, p.base_len};
        return true;
    }
    // (All three loads at once. A sequence that brings nothing need not hold the prefix.)
    const int c0 = p.cu[b], n = p.cu[b + 1] - c0, len = p.lens[b] - p.base_len;
    const bool ok = (0 <= c0) & (n >= 0) & (n <= p.total_q - c0) & (n <= p.own_q) & ((n == 0) | ((n <= len) & (len <= p.own_k)));
    t.first = ok ? c0 : 0;
    t.n = ok ? n : 0;
    t.len = ok && n > 0 ? len : 0;
    return ok;
}
// Position of the first row's token (`whole`: the last key's, for all rows).
__device__ __forceinline__ int paged_start(bool whole, const NewTokens& t) { return whole ? t.len - 1 : t.len - t.n; }
// The pages of the table's row b that the part reads.
template <bool PART>
__device__ __forceinline__ const int* paged_table(const PagedParams& p, bool whole, int b) {
    return p.page_table + static_cast<long long>(b) * p.max_pages + (PART && !whole ? p.base_pages : 0);
}

// A unit of the sequences' own parts: sequence b, its split `split` of `used`, key tiles
// i0 .. i1 - 1. Splits are as long as lets all units run at once, of which there may be
// `most` per kv head, and at least p.tiles_per_split tiles, so that the workspace holds
// them. Unit `r` in the order of the sequences, found by a whole warp; false where there
// is none. (Lengths are divided in floats, rounded about right: every warp gets the
// same numbers, and never more splits than tiles / length, rounded up.)
struct PagedUnit {
    int b, split, used, i0, i1;
};
template <int KEYS>
__device__ __forceinline__ bool paged_unit(const PagedParams& p, int r, int most, int lane, PagedUnit& u) {
    auto tiles_of = [&](int i) {  // -1: none
        NewTokens t;
        if (i >= p.B) return -1;
        if (!paged_tokens<true>(p, false, i, t)) return 0;  // broken: one unit, which reports it
        return t.n > 0 ? (t.len + KEYS - 1) / KEYS : -1;
    };
    const int t0 = tiles_of(lane), t1 = p.B > 32 ? tiles_of(32 + lane) : -1;  // the others are read again
    int sum = 0, live = 0;
    auto each = [&](auto&& f) {
        f(t0);
        if (p.B > 32) f(t1);
#pragma unroll 1
        for (int c = 64; c < p.B; c += 32) f(tiles_of(c + lane));
    };
    each([&](int t) { sum += max(t, 0), live += t >= 0 ? 1 : 0; });
    sum = __reduce_add_sync(0xffffffffu, sum);
    live = __reduce_add_sync(0xffffffffu, live);
    float inv;
    auto pieces = [&](int t) { return t < 0 ? 0 : max(1, static_cast<int>(fmaf(static_cast<float>(t), inv, 0.999f))); };
    // A sequence's last split is half full on average: tried first. One whole length per
    // sequence on top of its share never is too many.
    int length = max((p.max_k + KEYS - 1) / KEYS, 1);
#pragma unroll 1
    for (int round = 0; round < 2 && most > live; ++round) {
        const int room = most - (round ? live : live / 2);
        const int at = (sum + room - 1) / room;
        inv = 1.f / static_cast<float>(at);
        int k = 0;
        each([&](int t) { k += pieces(t); });
        if (round || __reduce_add_sync(0xffffffffu, k) <= most) {
            length = at;
            break;
        }
    }
    inv = 1.f / static_cast<float>(max(length, p.tiles_per_split));
#pragma unroll 1
    for (int c = 0; c < p.B; c += 32) {
        int tiles = c == 0 ? t0 : c == 32 ? t1 : tiles_of(c + lane);
        const int k = pieces(tiles);
        int upto = k;  // units of this and the lower lanes
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const unsigned here = __ballot_sync(0xffffffffu, r < upto);
        if (here) {
            const int who = __ffs(here) - 1;
            u.b = c + who;
            u.split = r - __shfl_sync(0xffffffffu, upto - k, who);
            u.used = __shfl_sync(0xffffffffu, k, who);
            tiles = max(__shfl_sync(0xffffffffu, tiles, who), 0);
            // Even parts.
            u.i0 = static_cast<int>(static_cast<long long>(tiles) * u.split / u.used);
            u.i1 = static_cast<int>(static_cast<long long>(tiles) * (u.split + 1) / u.used);
            return true;
        }
        r -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

// The first sequence that brings tokens and is not broken (-1: none): the prefix's pages are
// those of its row. Called by a whole warp.
__device__ __forceinline__ int paged_first(const PagedParams& p, int lane) {
    for (int c = 0; c < p.B; c += 32) {
        const int at = c + lane;
        NewTokens t;
        const bool sound = paged_tokens<true>(p, false, min(at, p.B - 1), t);
        const unsigned who = __ballot_sync(0xffffffffu, sound & (t.n > 0) & (at < p.B));
        if (who) return c + __ffs(who) - 1;
    }
    return -1;
}
// Reports a table of sequence b that does not begin with the shared prefix's pages, those
// of the first one (paged_first). Called by a whole warp.
__device__ __forceinline__ void paged_check_prefix(const PagedParams& p, int b, int lane) {
    const int first = paged_first(p, lane);
    if (first < 0 || first == b) return;
    const int* x = p.page_table + static_cast<long long>(first) * p.max_pages;
    const int* y = p.page_table + static_cast<long long>(b) * p.max_pages;
    bool same = true;
    for (int i0 = lane; i0 < p.base_pages; i0 += 256) {  // eight loads of each in flight
        int u[8], v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + 32 * k;
            u[k] = i < p.base_pages ? x[i] : 0;
            v[k] = i < p.base_pages ? y[i] : 0;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) same = same && u[k] == v[k];
    }
    if (!same) atomicOr(p.status, kStatusBadPage);
}

// What a partial state leaves as its reference m: -inf marks a state that saw no
// key, or that no CTA filled; a NaN sum stays one through the merge.
__device__ __forceinline__ float state_ref(float m, float l) { return l > 0.f ? m : l == 0.f ? -INFINITY : l; }
// LSE of a row's reference and sum (of 2^(x - m + 7): the shift comes out again).
__device__ __forceinline__ float state_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * 0.69314718055994530942f;
}

// The key tiles a row block visits, as a list: tiles 0 .. ns - 1 (sinks), then
// tile `lo` on, n in all. Positions p0 .. p1 are the block's first and last.
struct KeyList {
    int ns, lo, n;
    __device__ __forceinline__ int tile(int i) const { return i < ns ? i : lo + (i - ns); }
};
template <int KEYS>
__device__ __forceinline__ KeyList key_list(int window, int sinks, int p0, int p1) {
    KeyList k;
    const int end = p1 < 0 ? 0 : p1 / KEYS + 1;
    k.ns = 0, k.lo = 0;
    if (window > 0) {
        const int first = max(0, p0 - window + 1) / KEYS;
        const int st = min((sinks + KEYS - 1) / KEYS, end);
        if (first > st) k.ns = st, k.lo = first;
    }
    k.n = k.ns + max(0, end - k.lo);
    return k;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

// 16-byte shared-memory accesses at a register plus a constant.
template <int OFF>
__device__ __forceinline__ void ld_shared_v4_at(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFF)
                 : "memory");
}
template <int OFF>
__device__ __forceinline__ void st_shared_v4_at(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0 + %1], {%2, %3, %4, %5};" ::"r"(addr), "n"(OFF), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// f(Index<0>) .. f(Index<N - 1>): a loop whose index is a constant, for immediate
// operands.
template <int V>
struct Index {
    static constexpr int value = V;
    __host__ __device__ constexpr operator int() const { return V; }
};
template <int... I, typename F>
__device__ __forceinline__ void static_for_impl(std::integer_sequence<int, I...>, F&& f) {
    (f(Index<I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    static_for_impl(std::make_integer_sequence<int, N>{}, f);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Host side (fa_paged.cu): checks a cache's description.
fa_status check_cache(const fa_paged_cache* cache);
// The kernel for many query rows (fa_paged_tc.cu): rows per tile (a CTA takes two
// tiles, or one tile twice over two splits), keys per tile.
constexpr int kTcRows = 128;
constexpr int kTcKeys = 128;
constexpr int kTcAtOnce = 152;      // its CTAs running at a time: one per SM
constexpr int kTcStart = 5;         // start and end of a CTA, in key tiles of a pair of slots
constexpr int kTcBalance = 64;      // sequences up to which a call's pieces are balanced
cudaError_t launch_paged_tc(const PagedParams& p, int d, bool part, cudaStream_t stream);
inline int log2_exact(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

}  // namespace fa
