// fa_paged.cu — attention over the paged e4m3 cache: the kernel for up to 16 query
// rows per kv head (single tokens, a few drafted ones), the merge of key splits, and
// the C entry points.
//
// A CTA owns (sequence, kv head, 16 query rows, key split). Its rows are the
// (query token, head of the group) pairs of the kv head, so a group's heads
// share every byte of K and V that is read. What bounds it is that reading: a
// key costs 2 d bytes and at 16 rows only 64 d multiply-adds, so the products
// run on mma.sync (m16n8k16, f16 operands, fp32 sums), which needs no tile of
// 128 rows.
//
// Each of the CTA's four warps takes every fourth tile of 32 (16) keys with a ring of
// its own: TMA copies of whole pages (or their parts) into swizzled
// shared memory, one mbarrier per slot, no barrier between the warps until
// their states meet at the end. e4m3 codes convert to f16 exactly (one
// instruction per two codes), in the registers of the fragments:
//   * K as the B operand of S = Q K^T. The contraction index may be permuted at
//     will if Q is permuted alike, so a lane reads 16 consecutive codes of a
//     key row with one 16-byte load and feeds four MMAs with them.
//   * V as the B operand of O += P V, through ldmatrix.trans on pairs of codes:
//     a 32-bit result holds two keys of two neighbouring columns; one byte
//     permute separates the columns, which go to two MMAs.
// Q (bf16) enters as f16 after a power-of-two scale per row that brings its
// largest element to [2^7, 2^8): elements down to 2^-22 of it stay exact.
//
// The recurrence in base 2, with a tile's K scale ks and V scale vs per key:
//   x_j = s_j * (ks_j * scale * log2 e) + log2 vs_j,  p_j = 2^(x_j - m + 7),
//   O += p_j code_j,  l += p_j / vs_j:  O / l = sum_j softmax_j vs_j code_j.
// The V scale sits in the exponent, so P stays in f16's range whatever the
// scales are; the reference m moves only when a row's largest x passes it by
// more than 8 (p <= 2^15), so O is seldom rescaled.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "fa.h"
#include "fa_paged.cuh"
#include "fa_paged_phases.h"
#include "fa_rope.cuh"

namespace fa {

fa_status check_cache(const fa_paged_cache* c) {
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return FA_ERR_NULL;
    if (!valid_d(c->d)) return FA_ERR_HEADDIM;
    if (c->page_size < 16 || c->page_size > 128 || (c->page_size & (c->page_size - 1))) return FA_ERR_PAGE_SIZE;
    // Row indices of the cache seen as [num_pages * Hkv * page_size][d] are
    // 32-bit TMA coordinates.
    if (c->num_pages < 1 || c->Hkv < 1 || c->Hkv > 65535) return FA_ERR_SHAPE;
    const unsigned long long rows = static_cast<unsigned long long>(c->num_pages) * c->Hkv;
    if (rows > 0x7fffffffull / c->page_size) return FA_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return FA_ERR_ALIGN;
    return FA_OK;
}

namespace {

constexpr int kRows = 16;      // query rows per CTA
constexpr int kWarps = 4;
constexpr int kPlaces = 152;   // SMs
constexpr int kClusterSplits = 8;  // splits that can be a cluster (the portable size)
// Keys of a warp's tile, and CTAs an SM holds. A warp's tile is a chain of
// dependent steps, so throughput comes from the warps beside it: short tiles and
// two- or three-slot rings, for as many CTAs as the registers allow. Measured on
// 64 contexts of 8192 to 32768 tokens (32 of 4096 to 16384 at d = 256), 32 + 8 heads,
// TB/s:
//   d = 64:  two CTAs of six-slot rings 3.4, three of four 4.2, four of three 4.8,
//            five of two 4.6; tiles of 64 keys, three CTAs, 4.6
//   d = 128: two CTAs of three-slot rings 5.7, three of two slots 6.3
//   d = 256: tiles of 32 keys, one CTA, 4.5; of 16 keys, two CTAs, 5.5
__host__ __device__ constexpr int rows_keys(int d) { return d == 256 ? 16 : 32; }
__host__ __device__ constexpr int rows_ctas(int d) { return d == 64 ? 4 : d == 128 ? 3 : 2; }
template <int D, bool PART = false>
struct PagedLayout {
    static constexpr int ROW_BYTES = D < 128 ? D : 128;  // bytes of a swizzled row
    static constexpr int PARTS = D / ROW_BYTES;          // row parts (128-byte columns of a key)
    static constexpr int KEYS = rows_keys(D);            // keys of a warp's tile
    static constexpr int GROUPS = KEYS / 16;             // scales of a tile: one per 16 keys, the smallest page
    static constexpr uint32_t TILE = KEYS * D;           // bytes of K (or V) of a tile
    static constexpr uint32_t SLOT = 2 * TILE;
    static constexpr int STAGES = D == 64 ? 3 : 2;
    static constexpr uint32_t RING = STAGES * SLOT;      // per warp
    static constexpr bool Q_SHARED = D == 256;           // Q fragments in shared memory, not registers
    static constexpr uint32_t Q_BYTES = Q_SHARED ? kRows * D * 2 : 0;  // (PART: each warp its own)
    static constexpr uint32_t Q_OFF = kWarps * RING;
    static constexpr uint32_t BAR_OFF = Q_OFF + (PART ? kWarps : 1) * Q_BYTES;
    static constexpr uint32_t ML_OFF = BAR_OFF + kWarps * STAGES * 8;  // [warp][m, l][16 rows]
    static constexpr uint32_t CTA_ML_OFF = ML_OFF + kWarps * 2 * kRows * 4;  // [m, l][16 rows] of the CTA
    static constexpr uint32_t BYTES = CTA_ML_OFF + 2 * kRows * 4;
    static constexpr size_t ALLOC = BYTES + 1024;
    static_assert(RING >= kRows * D * 4, "a warp's O is staged in its ring");
    static_assert(TILE % 1024 == 0, "swizzle atoms are 1024-byte aligned");
};

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, long long limit, unsigned* status,
                                             unsigned what) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long start = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (clock64() - start > limit) {
            atomicOr(status, what);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Byte offset of 16-byte unit `unit` of key row `row` in a swizzled tile: rows
// of 128 bytes (units XOR row mod 8; further row parts a tile's rows behind), or of
// 64 bytes (units XOR row / 2 mod 4).
template <int D>
__device__ __forceinline__ uint32_t tile_unit(int row, int unit) {
    if constexpr (D == 64) return row * 64 + ((unit ^ ((row >> 1) & 3)) << 4);
    else return (unit >> 3) * (rows_keys(D) * 128) + row * 128 + (((unit & 7) ^ (row & 7)) << 4);
}
// Key row (0..7 of an 8-key group) behind fragment index j: with 128-byte rows
// the two rows that one quarter of a warp reads together lie four apart, so
// that their swizzled units fall into different banks.
template <int D>
__device__ __forceinline__ int key_of(int j) {
    return D == 64 ? j : (j >> 1) | ((j & 1) << 2);
}

// Shared memory of the cluster's CTA `rank` at this CTA's address.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "r"(addr)
                 : "memory");
    return x;
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// CLUSTER: the splits of a unit are a cluster, whose CTAs read one another's
// states at the end: no workspace traffic and no second launch (one token for 8
// heads of 64 over 516 keys, five splits: 6.1 us against 7.4 through the workspace,
// replayed from a graph; 9.5 with one split). Every CTA of a cluster comes to both
// of its meetings, whatever it found.
// PART: a part of a batch that shares a prefix (PagedParams).
template <int D, bool CLUSTER, bool PART>
__global__ void __launch_bounds__(kWarps * 32, rows_ctas(D))
    fa_paged_rows_kernel(const __grid_constant__ PagedParams p) {
    using L = PagedLayout<D, PART>;
    constexpr int KEYS = L::KEYS, NT = KEYS / 8, GROUPS = L::GROUPS;
    constexpr int C = D / 64;    // 64-column parts of the contraction: one 16-byte load each
    constexpr int X = D / 16;    // 16-column units of O
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = sbase + warp * L::RING;
    const uint32_t q_off = L::Q_OFF + (PART ? warp * L::Q_BYTES : 0);
    const uint32_t bar0 = sbase + L::BAR_OFF + warp * L::STAGES * 8;
    if (lane == 0) {
        for (int s = 0; s < L::STAGES; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_mbar_init();
        if (warp == 0) {
            tma_prefetch_desc(&p.tm_k);
            tma_prefetch_desc(&p.tm_v);
        }
    }
    __syncwarp();
    if (!paged_wait<PART>(p)) return;
    paged_allow<PART>(p);

    // Unit: row blocks fastest (they share K and V in L2), then splits, heads.
    // (A cluster's CTAs are consecutive: its splits.) PART: the sequences' own units have
    // one row block. Where those fill the GPU (solo), every warp has one of its own, heads
    // fastest: their lengths differ, and one wave of short units ends together, where
    // four warps a unit took 2.7 uneven waves (64 sequences of 260 to 2000 keys, 8 kv
    // heads).
    const bool whole = PART && blockIdx.x < p.whole_ctas, solo = PART && !whole && p.solo;
    const int num_splits = whole ? p.shared.num_splits : p.num_splits;
    const int state0 = whole ? p.shared.state0 : 0;
    unsigned lin = CLUSTER ? blockIdx.x / num_splits : blockIdx.x;
    int rb = 0, split, h, b;
    PagedUnit unit = {};
    if constexpr (PART) {
        if (!whole) lin -= p.whole_ctas;
        if (solo) {
            lin = lin * kWarps + warp;
            if (!paged_unit<KEYS>(p, static_cast<int>(lin / p.Hkv), p.places / p.Hkv, lane, unit)) return;
            b = unit.b;
            split = unit.split;
        } else {
            if (whole) {
                rb = static_cast<int>(lin % p.shared.row_blocks);
                lin /= p.shared.row_blocks;
            }
            split = static_cast<int>(lin % num_splits);
            lin /= num_splits;
            b = whole ? 0 : static_cast<int>(lin / p.Hkv);
        }
        h = static_cast<int>(lin % p.Hkv);
    } else {
        rb = static_cast<int>(lin % p.row_blocks);
        lin /= p.row_blocks;
        split = static_cast<int>(CLUSTER ? blockIdx.x % num_splits : lin % num_splits);
        if (!CLUSTER) lin /= num_splits;
        h = static_cast<int>(lin % p.Hkv);
        b = static_cast<int>(lin / p.Hkv);
    }
    // (All CTAs of a cluster agree on the returns below.)
    NewTokens nt;
    if (!paged_tokens<PART>(p, whole, b, nt)) {
        if (solo ? lane == 0 : threadIdx.x == 0) atomicOr(p.status, kStatusBadSeqlens);
        return;
    }
    const int rows = nt.n * p.G;
    const int r0 = rb * kRows;
    if (r0 >= rows) return;
    if constexpr (PART) {
        if (whole) b = paged_first(p, lane);
        else if (h == 0 && split == 0) paged_check_prefix(p, b, lane);
        if (b < 0) return;
    }
    const int start = paged_start(whole, nt), step = whole ? 0 : 1;  // position of the first query
    const int p0 = start + step * (r0 / p.G);
    const int p1 = start + step * ((min(r0 + kRows, rows) - 1) / p.G);
    const KeyList list = key_list<KEYS>(p.window, p.sinks, p0, p1);
    const int tiles_per_split = whole ? p.shared.tiles_per_split : p.tiles_per_split;
    const int used = solo ? unit.used : max(1, (list.n + tiles_per_split - 1) / tiles_per_split);
    if (!CLUSTER && split >= used) return;
    const int i0 = solo ? unit.i0 : split * tiles_per_split;
    const int i1 = solo ? unit.i1 : min(list.n, i0 + tiles_per_split);
    // This warp's tiles: first + stride k.
    const int first = solo ? i0 : i0 + warp, stride = solo ? 1 : kWarps;
    const int mine = max(0, (i1 - first + stride - 1) / stride);
    const int* table = paged_table<PART>(p, whole, b);
    const int page_size = 1 << p.log_page;
    const int last_page = (nt.len - 1) >> p.log_page;

    // Page i of the tile's pages (or the one page it lies in), or -1 where the
    // sequence has none there (nothing is read) or its entry is bad.
    const int per = page_size < KEYS ? KEYS >> p.log_page : 1;  // pages of a tile
    auto page_of = [&](int kt, int i) -> int {
        const int idx = ((kt * KEYS) >> p.log_page) + i;
        if (idx > last_page) return -1;
        const int id = table[idx];
        if (id < 0 || id >= p.num_pages) {
            atomicOr(p.status, kStatusBadPage);
            return -1;
        }
        return id;
    };
    // Page ids of the warp's next 32 tiles to copy, one tile per lane.
    int ids[GROUPS];
    auto fetch_ids = [&](int k) {
        const int i = first + stride * (k + lane);
#pragma unroll
        for (int e = 0; e < GROUPS; ++e) ids[e] = i < i1 && e < per ? page_of(list.tile(i), e) : -1;
    };
    // Copies of tile number k of the warp into its slot: a page that is not there
    // is left out, and its keys are masked.
    auto issue_next = [&](int k) {
        if ((k & 31) == 0) fetch_ids(k);
        int id[GROUPS], there = 0;
#pragma unroll
        for (int e = 0; e < GROUPS; ++e) {
            id[e] = __shfl_sync(0xffffffffu, ids[e], k & 31);
            there += id[e] >= 0 ? 1 : 0;
        }
        const int s = ring_slot(k, L::STAGES);
        const uint32_t dst = ring + s * L::SLOT, bar = bar0 + 8 * s;
        const int rows_each = min(page_size, KEYS);
        if (lane == 0) mbar_arrive_expect_tx(bar, there * rows_each * D * 2);
        __syncwarp();
        // A lane per page and tensor.
        const int e = lane >> 1;
        int page = id[0];
#pragma unroll
        for (int i = 1; i < GROUPS; ++i)
            if (e == i) page = id[i];
        if (e < GROUPS && page >= 0) {
            const int key0 = list.tile(first + stride * k) * KEYS;
            const int row = ((page * p.Hkv + h) << p.log_page) + (per == 1 ? key0 & (page_size - 1) : 0);
            const CUtensorMap* map = (lane & 1) ? &p.tm_v : &p.tm_k;
#pragma unroll
            for (int c = 0; c < L::PARTS; ++c)
                tma_load_2d(dst + (lane & 1) * L::TILE + c * (KEYS * 128) + e * rows_each * L::ROW_BYTES, map, bar, c * 128,
                            row);
        }
        __syncwarp();
    };
    const int ahead = min(mine, L::STAGES);
    for (int k = 0; k < ahead; ++k) issue_next(k);

    // Q rows r0 + g and r0 + g + 8 as f16 A fragments: contraction index 2 t, 2 t + 1
    // (and + 8) of step (c, ks) is column 64 c + 16 t + 4 ks + 0, 1 (and 2, 3).
    float rowf[2];  // scale of a row's scores, base 2, without the K scale
    int pos[2];     // its position (rows past the last one repeat the first; they are not written)
    uint32_t qf[L::Q_SHARED ? 1 : C][4][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = r0 + g + 8 * e;
        const bool ok = r < rows;
        const int i = (ok ? r : r0) / p.G, j = (ok ? r : r0) - i * p.G;
        pos[e] = ok ? start + step * i : p1;
        const __nv_bfloat16* src =
            p.q + (static_cast<long long>(nt.first + i) * p.H + h * p.G + j) * D + 16 * t;
        uint4 raw[C][2];
        uint32_t mx = 0u;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                raw[c][u] = *reinterpret_cast<const uint4*>(src + 64 * c + 8 * u);
                float x[8];
                unpack_bf16x8(raw[c][u], x);
                mx = abs_bits_max(mx, x);
            }
        }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float f = exp2i(query_exponent(mx));
        // (Exact, as the inverse exponent's power would be, which lets the loop below
        // be scheduled worse: 441 us for 64 contexts of up to 32768 keys against 437.)
        rowf[e] = p.scale_log2 * query_undo(mx, 1.f / f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x[8];
                unpack_bf16x8(raw[c][u], x);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t a = pack_f16x2(x[4 * k] * f, x[4 * k + 1] * f);
                    const uint32_t z = pack_f16x2(x[4 * k + 2] * f, x[4 * k + 3] * f);
                    const int ks = 2 * u + k;
                    if constexpr (L::Q_SHARED) {
                        if (PART || warp == 0) {
                            uint32_t* dst = reinterpret_cast<uint32_t*>(smem + q_off) + ((c * 4 + ks) * 32 + lane) * 4;
                            dst[e] = a;
                            dst[2 + e] = z;
                        }
                    } else {
                        qf[c][ks][e] = a;
                        qf[c][ks][2 + e] = z;
                    }
                }
            }
        }
    }
    if constexpr (L::Q_SHARED) {
        if constexpr (PART) __syncwarp();
        else __syncthreads();
    }

    float o[X][2][4];  // [16-column unit][even, odd column of a pair][row g: 2, row g + 8: 2]
#pragma unroll
    for (int x = 0; x < X; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[x][e][k] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int pmin = p0, pmax = p1;
    // Scales of the warp's current 32 tiles, one tile per lane: K scale, log2 of
    // the V scale and its reciprocal for each page of the tile.
    float sk[GROUPS], sv[GROUPS], si[GROUPS];
    const int group_shift = per == 1 ? 31 : p.log_page - 4;  // 16-key group to page of the tile
    bool ok = true;
    // The lane's parts of its shared-memory addresses: K's 16-byte loads of 64
    // columns each, V's ldmatrix rows of 32 columns each.
    uint32_t k_lane[C], v_lane[X / 2];
#pragma unroll
    for (int c = 0; c < C; ++c) k_lane[c] = tile_unit<D>(key_of<D>(g), 4 * c + t);
#pragma unroll
    for (int x = 0; x < X; x += 2)
        v_lane[x / 2] = tile_unit<D>(8 * ((lane >> 3) & 1) + key_of<D>(lane & 7), x + (lane >> 4));

    int k = 0;
    for (; k < mine; ++k) {
        if ((k & 31) == 0) {
            const int i = first + stride * (k + lane);
#pragma unroll
            for (int e = 0; e < GROUPS; ++e) {
                const int id = i < i1 && e < per ? page_of(list.tile(i), e) : -1;
                const long long cell = static_cast<long long>(id) * p.Hkv + h;
                const float vs = id >= 0 ? usable_scale(p.v_scale[cell]) : 1.f;
                sk[e] = id >= 0 ? p.k_scale[cell] : 1.f;
                sv[e] = log2f(vs);
                si[e] = 1.f / vs;
            }
        }
        const int slot = ring_slot(k, L::STAGES);
        ok = __all_sync(0xffffffffu, wait_bounded(bar0 + 8 * slot, ring_parity(k, L::STAGES), p.wait_limit, p.status,
                                                  kStatusWaitKvFull));
        if (!ok) break;
        const int key0 = list.tile(first + stride * k) * KEYS;
        const uint32_t ks_at = ring + slot * L::SLOT, vs_at = ks_at + L::TILE;

        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t kw[NT][4];
            const uint32_t at = ks_at + k_lane[c];
            static_for<NT>([&](auto n) { ld_shared_v4_at<n * 8 * L::ROW_BYTES>(kw[n], at); });
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint32_t a[4];
                if constexpr (L::Q_SHARED) {
                    ld_shared_v4(a, sbase + q_off + ((c * 4 + ks) * 32 + lane) * 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = qf[c][ks][e];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t b0, b1;
                    decode_e4m3x4_f16(kw[n][ks], b0, b1);
                    mma_f16(s[n], a, b0, b1);
                }
            }
        }

        // x = s * (ks scale log2 e) + log2 vs, masked where a row does not see the key.
        float kc[GROUPS], kv[GROUPS], ki[GROUPS];
#pragma unroll
        for (int e = 0; e < GROUPS; ++e) {
            // (The tile's page behind group e; the arrays keep constant indices.)
            const int page = e >> group_shift;
            float a = sk[0], b = sv[0], c = si[0];
#pragma unroll
            for (int i = 1; i < GROUPS; ++i)
                if (page == i) a = sk[i], b = sv[i], c = si[i];
            kc[e] = __shfl_sync(0xffffffffu, a, k & 31);
            kv[e] = __shfl_sync(0xffffffffu, b, k & 31);
            ki[e] = __shfl_sync(0xffffffffu, c, k & 31);
        }
        const bool masked = !(key0 + KEYS - 1 <= pmin &&
                              (p.window <= 0 || key0 > pmax - p.window || key0 + KEYS <= p.sinks));
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = fmaf(s[n][e], rowf[e >> 1] * kc[n >> 1], kv[n >> 1]);
                if (masked) {
                    const int key = key0 + 8 * n + key_of<D>(2 * t + (e & 1));
                    const int q = pos[e >> 1];
                    if (!(key <= q && (p.window <= 0 || key > q - p.window || key < p.sinks))) x = -INFINITY;
                }
                s[n][e] = x;
                top[e >> 1] = fmaxf(top[e >> 1], x);
            }
        }
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
            const bool move = top[e] > m[e] + kPSlack;
            const float mn = move ? top[e] : m[e];
            alpha[e] = move ? ex2(m[e] - mn) : 1.f;
            m[e] = mn;
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[x][e][j] *= alpha[j >> 1];
            l[0] *= alpha[0];
            l[1] *= alpha[1];
        }
        const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0] - kPShift, m[1] == -INFINITY ? 0.f : m[1] - kPShift};
        uint32_t pf[GROUPS][4];  // P of 16 keys as an A fragment
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float e0 = ex2(s[n][0] - ref[0]), e1 = ex2(s[n][1] - ref[0]);
            float e2 = ex2(s[n][2] - ref[1]), e3 = ex2(s[n][3] - ref[1]);
            l[0] = fmaf(e0 + e1, ki[n >> 1], l[0]);
            l[1] = fmaf(e2 + e3, ki[n >> 1], l[1]);
            pf[n >> 1][2 * (n & 1)] = pack_f16x2(e0, e1);
            pf[n >> 1][2 * (n & 1) + 1] = pack_f16x2(e2, e3);
        }

        // O += P V. Fragment index kk of 8 keys is key row key_of(kk); a key that
        // no row sees may hold anything (a slot never written, a NaN): its bytes
        // are cleared.
#pragma unroll
        for (int kk = 0; kk < GROUPS; ++kk) {
            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
            if (masked) {
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                    keep[hi] = 0u;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = key0 + 16 * kk + 8 * hi + key_of<D>(2 * t + e);
                        const bool seen = key <= pmax && (p.window <= 0 || key > pmin - p.window || key < p.sinks);
                        if (seen) keep[hi] |= e ? 0xffff0000u : 0x0000ffffu;
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < X; x += 2) {
                uint32_t w[4];
                ldmatrix_x4_trans(w, vs_at + v_lane[x / 2] + kk * 16 * L::ROW_BYTES);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t lo = w[2 * u], hi = w[2 * u + 1];
                    if (masked) lo &= keep[0], hi &= keep[1];
                    uint32_t e0, e1, d0, d1;  // even and odd columns, keys 0-7 and 8-15
                    decode_e4m3x4_f16(__byte_perm(lo, 0u, 0x3120), e0, d0);
                    decode_e4m3x4_f16(__byte_perm(hi, 0u, 0x3120), e1, d1);
                    mma_f16(o[x + u][0], pf[kk], e0, e1);
                    mma_f16(o[x + u][1], pf[kk], d0, d1);
                }
            }
        }
        __syncwarp();
        if (k + L::STAGES < mine) issue_next(k + L::STAGES);
    }
    if (!ok) {
        // Copies still in flight land before the ring is used again and the CTA goes
        // away: those of the tile that was waited for and of the ones behind it.
        for (const int end = ring_issued(k, L::STAGES, mine); k < end; ++k)
            wait_bounded(bar0 + 8 * ring_slot(k, L::STAGES), ring_parity(k, L::STAGES), p.wait_limit, p.status,
                         kStatusWaitDrain);
    }

    // The warps' states meet: O rows staged in each warp's ring, m and l beside.
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    float* ml = reinterpret_cast<float*>(smem + L::ML_OFF) + warp * 2 * kRows;
    if (t == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ml[g + 8 * e] = m[e];
            ml[kRows + g + 8 * e] = l[e];
        }
    }
    float* stage = reinterpret_cast<float*>(smem + warp * L::RING);
#pragma unroll
    for (int x = 0; x < X; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(stage + (g + 8 * e) * D + 16 * x + 4 * t) =
                make_float4(o[x][0][2 * e], o[x][1][2 * e], o[x][0][2 * e + 1], o[x][1][2 * e + 1]);
    auto place = [&](int r) -> long long {
        const int i = (r0 + r) / p.G, j = (r0 + r) - i * p.G;
        return static_cast<long long>(nt.first + i) * p.H + h * p.G + j;
    };
    if constexpr (PART) {
        if (solo) {
            // The warp's own state.
            __syncwarp();
            for (int u = lane; u < kRows * (D / 4) && ok; u += 32) {
                const int r = u / (D / 4), c = u - r * (D / 4);
                if (r >= rows) break;
                const long long row = place(r), at = static_cast<long long>(split) * p.total_q * p.H + row;
                *reinterpret_cast<float4*>(p.ws_o + at * D + 4 * c) = *reinterpret_cast<const float4*>(stage + r * D + 4 * c);
                if (c == 0) {
                    p.ws_m[at] = state_ref(ml[r], ml[kRows + r]);
                    p.ws_l[at] = ml[kRows + r];
                }
                // States that the row does not use are marked as empty for the merge.
                for (int s = used + c; s < num_splits && split == 0; s += D / 4)
                    p.ws_m[static_cast<long long>(s) * p.total_q * p.H + row] = -INFINITY;
            }
            return;
        }
    }
    const bool failed = __syncthreads_or(!ok);
    if (!CLUSTER && failed) return;

    const float* mls = reinterpret_cast<const float*>(smem + L::ML_OFF);
    constexpr int VEC = D / 4;  // float4 units of a row
    auto put = [&](int r, int c, const float4& a, float mm, float ll) {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        *reinterpret_cast<uint2*>(p.o + place(r) * D + 4 * c) =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        if (c == 0) {
            const int i = (r0 + r) / p.G, j = (r0 + r) - i * p.G;
            p.lse[static_cast<long long>(h * p.G + j) * p.total_q + nt.first + i] = state_lse(mm, ll);
        }
    };
    for (int u = threadIdx.x; u < kRows * VEC; u += kWarps * 32) {
        const int r = u / VEC, c = u - r * VEC;
        if (r0 + r >= rows) break;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, mls[w * 2 * kRows + r]);
        float ll = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = mls[w * 2 * kRows + r];
            const float f = mw == -INFINITY ? 0.f : ex2(mw - mm);
            const float4 x = *reinterpret_cast<const float4*>(smem + w * L::RING + (r * VEC + c) * 16);
            ll = fmaf(f, mls[w * 2 * kRows + kRows + r], ll);
            a.x = fmaf(f, x.x, a.x), a.y = fmaf(f, x.y, a.y), a.z = fmaf(f, x.z, a.z), a.w = fmaf(f, x.w, a.w);
        }
        if constexpr (CLUSTER) {
            // (Over warp 0's state of this unit, which this thread alone reads.)
            *reinterpret_cast<float4*>(smem + (r * VEC + c) * 16) = a;
            if (c == 0) {
                float* own = reinterpret_cast<float*>(smem + L::CTA_ML_OFF);
                own[r] = state_ref(mm, ll);
                own[kRows + r] = ll;
            }
            continue;
        }
        const long long row = place(r);
        // States that the row does not use are marked as empty for the merge.
        const bool done = used == 1 && !PART;
        if (split == 0 && num_splits > 1)
            for (int s = (done ? 0 : used) + c; s < num_splits; s += VEC)
                p.ws_m[static_cast<long long>(state0 + s) * p.total_q * p.H + row] = -INFINITY;
        if (done) {
            put(r, c, a, mm, ll);
        } else {
            const long long at = static_cast<long long>(state0 + split) * p.total_q * p.H + row;
            *reinterpret_cast<float4*>(p.ws_o + at * D + 4 * c) = a;
            if (c == 0) {
                p.ws_m[at] = state_ref(mm, ll);
                p.ws_l[at] = ll;
            }
        }
    }
    if constexpr (CLUSTER) {
        __syncwarp();
        cluster_meet();
        // The CTAs take units of the rows in turn; a failed wait leaves them out.
        for (int u = split * kWarps * 32 + threadIdx.x; u < kRows * VEC && !failed; u += p.num_splits * kWarps * 32) {
            const int r = u / VEC, c = u - r * VEC;
            if (r0 + r >= rows) break;
            float m_of[kClusterSplits], l_of[kClusterSplits];
            float4 x[kClusterSplits];
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int s = 0; s < kClusterSplits; ++s) {
                m_of[s] = -INFINITY;
                if (s < used) {
                    m_of[s] = ld_cluster(map_rank(sbase + L::CTA_ML_OFF + r * 4, s));
                    l_of[s] = ld_cluster(map_rank(sbase + L::CTA_ML_OFF + (kRows + r) * 4, s));
                    x[s] = ld_cluster_v4(map_rank(sbase + (r * VEC + c) * 16, s));
                }
            }
#pragma unroll
            for (int s = 0; s < kClusterSplits; ++s) mm = fmaxf(mm, m_of[s]);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < kClusterSplits; ++s) {
                if (m_of[s] == -INFINITY) continue;  // no key, or no such split
                const float f = ex2(m_of[s] - mm);
                ll = fmaf(f, l_of[s], ll);
                a.x = fmaf(f, x[s].x, a.x), a.y = fmaf(f, x[s].y, a.y);
                a.z = fmaf(f, x[s].z, a.z), a.w = fmaf(f, x[s].w, a.w);
            }
            put(r, c, a, mm, ll);
        }
        __syncwarp();
        cluster_meet();  // no CTA leaves while another reads its states
    }
}

// Merge of the key splits of the (token, head) rows whose block used more than
// one: M = max m_s, O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s. States with
// m = -inf were not used (all of them where the row is finished already) or
// saw no key. W warps (1 or 4) share a row, each with eight partial rows in
// flight: the merge of a single sequence's few rows over many splits is a matter
// of latency alone.
template <int D, int W, bool PART>
__global__ void __launch_bounds__(128) fa_paged_merge_kernel(const __grid_constant__ PagedParams p) {
    constexpr int PER = D / 32, U = 8;
    __shared__ float weight[4][FA_MAX_SPLITS];
    __shared__ float sums[W > 1 ? 4 : 1][W > 1 ? D : 1];
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wi = warp % W;
    const long long unit = static_cast<long long>(blockIdx.x) * (4 / W) + warp / W;
    const int head = static_cast<int>(unit % p.H);
    const long long rest = unit / p.H;
    const int i = static_cast<int>(rest % p.max_q);
    const int b = static_cast<int>(rest / p.max_q);
    NewTokens nt;
    bool live = b < p.B && paged_tokens<PART>(p, false, b, nt) && i < nt.n;
    const long long row = live ? static_cast<long long>(nt.first + i) * p.H + head : 0;
    const long long stride = static_cast<long long>(p.total_q) * p.H;
    const int states = live ? p.num_splits : 0;
    const float* src = p.ws_o + row * D + lane * PER;
    float x[U][PER];
    auto load = [&](int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * W;
#pragma unroll
            for (int e = 0; e < PER; e += 2) {
                const float2 a = s < states ? *reinterpret_cast<const float2*>(src + s * stride * D + e) : make_float2(0.f, 0.f);
                x[u][e] = a.x;
                x[u][e + 1] = a.y;
            }
        }
    };
    load(wi);
    int used = 0;
    float mm = -INFINITY, ll = 0.f, ref;
    if (PART && p.num_splits <= 32) {
        // A state a lane: m and l in one trip to memory.
        const float m = lane < states ? p.ws_m[lane * stride + row] : -INFINITY;
        const float l = lane < states ? p.ws_l[lane * stride + row] : 0.f;
        if (m != -INFINITY) used = lane + 1;
        used = __reduce_max_sync(0xffffffffu, used);
        live = used > 0;
        mm = m;
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        ref = mm == -INFINITY ? 0.f : mm;
        const float f = ex2(m - ref);
        weight[warp][lane] = f;
        if (m != -INFINITY) ll = f * l;
    } else {
        for (int s = lane; s < states; s += 32) {
            const float m = p.ws_m[s * stride + row];
            if (m != -INFINITY) used = s + 1, mm = fmaxf(mm, m);
        }
        used = __reduce_max_sync(0xffffffffu, used);
        live = used > 0;
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        ref = mm == -INFINITY ? 0.f : mm;
        for (int s = lane; s < used; s += 32) {
            const float m = p.ws_m[s * stride + row];
            const float f = ex2(m - ref);
            weight[warp][s] = f;
            if (m != -INFINITY) ll = fmaf(f, p.ws_l[s * stride + row], ll);
        }
    }
    for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
    __syncwarp();
    float acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int s0 = wi; s0 < used; s0 += U * W) {
        if (s0 != wi) load(s0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * W;
            const float f = s < used ? weight[warp][s] : 0.f;
            if (f == 0.f) continue;  // an unused state holds anything
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = fmaf(f, x[u][e], acc[e]);
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < PER; ++e) sums[warp][lane * PER + e] = acc[e];
        __syncthreads();
        if (wi != 0) return;
        for (int k = 1; k < W; ++k)
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] += sums[warp + k][lane * PER + e];
    }
    if (!live) return;
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + lane * PER);
#pragma unroll
    for (int e = 0; e < PER; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0)
        p.lse[static_cast<long long>(head) * p.total_q + nt.first + i] = state_lse(ref, ll);
}

// e4m3 cache as [rows][d], box {min(d, 128), box_rows}, swizzled by row size.
bool encode_cache_map(CUtensorMap* map, const void* base, int d, long long rows, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(d < 128 ? d : 128), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call is cut: by the tensor-core kernel of fa_paged_tc.cu, or by this
// file's.
struct Plan {
    bool tc, dual;
    int block_rows, block_keys;
    long long row_blocks;
    long long tiles;  // most key tiles a row block can list
};
Plan plan_of(int G, int max_q, int max_k, int d, int window, int sinks) {
    Plan c;
    const long long rows = static_cast<long long>(max_q) * G;
    // The tensor-core kernel from 17 rows on. One block of 16 rows is no slower here,
    // two, which read K and V twice, are (32 + 8 heads, 16 sequences of 4600 to 16200
    // keys, us here and there: 16 rows 87 and 85 at d = 128, 61 and 69 at d = 64; 20
    // rows 132 and 87, 93 and 70; of 2000 to 8000 keys at d = 256: 16 rows 94 and 113,
    // 20 rows 137 and 113, 40 rows 202 and 114).
    c.tc = rows > kRows;
    c.dual = c.tc && rows <= kTcRows && d <= 128;
    c.block_rows = !c.tc ? kRows : c.dual || d == 256 ? kTcRows : 2 * kTcRows;
    c.block_keys = c.tc ? kTcKeys : rows_keys(d);
    c.row_blocks = (rows + c.block_rows - 1) / c.block_rows;
    const long long K = c.block_keys;
    c.tiles = (max_k + K - 1) / K;
    if (window > 0) {
        const long long span = std::min(max_q, c.block_rows);  // tokens a block's rows can cover
        c.tiles = std::min(c.tiles, (window + span + K - 1) / K + 1 + (sinks + K - 1) / K);
    }
    return c;
}

// Splits that finish earliest, in rounds of 128 keys; a CTA's start and end cost
// about two, leaving and merging partial states some more. While the CTAs leave half
// of the places free, only the longest one counts, and the merge costs two rounds,
// or half a one in a cluster (replayed from a graph, one token for 8 heads of 64 over
// 516 keys: 9.5 us with one split, 7.1 with three, 6.1 with five; four contexts of
// up to 700: 11.5 and 6.6 with six). One sequence in several waves: CTAs of equal
// length. Several sequences: their lengths differ, so the longest CTA comes on top
// of an even share of all of them, at two thirds of the longest length (64 contexts
// of 8192 to 32768, 512 units: 582 us with one split, 479 with three, 426 with eight,
// 438 with the 16 proposed; all of 20480, 542, 429, 415, and 423 with the ten
// proposed; one of 131072, 8 units: 55 us in one wave of splits, 80 in four).
//
// Pairs of slots (dual): of 2 to 64 sequences (kTcBalance) a CTA takes pieces of
// whatever length balances those at hand (tc_piece), so only the most pieces of a
// sequence are chosen here: an even share of all of them, ten rounds a piece for its
// start and end, and half a piece for the last ones, with sequences at two thirds of
// the longest on average (five drafted tokens, pieces of the longest and us: 16
// contexts of 4600 to 16200 keys, 1: 103, 2: 104, 3: 87, 4: 90; 64 of up to 32768, 1:
// 535, 2: 529, 3: 561; 80 of 8192, 1: 195, 2: 229; 2 of 16200, 8: 26, 10: 25, 12: 28).
// Lengths are not known here: sequences of one length would rather stay whole (16 of
// 10125 keys, 1: 71, the three proposed: 83; of 16200, 106 and 117), and a bound above
// the lengths at hand cuts them more coarsely than they need (one token for one
// sequence of 8192 keys: 18 us at a bound of 8192, 25 at 32768, 34 at 131072; for 16:
// 66, 72, 83).
int best_splits(int B, long long units, long long rounds, int slots, bool dual, bool many_rows) {
    if (dual && B > 1) {
        int best = 1;
        double best_cost = -1.;
        const double R = static_cast<double>(rounds), start = 10.;
        for (int c = 1; c <= FA_MAX_SPLITS / 2 && (c == 1 || 2 * c <= rounds); ++c) {
            const double even = units * (0.65 * R + (c == 1 ? 1. : 0.65 * c + 0.35) * start) / kTcAtOnce + 0.5 * R / c;
            const double cost = std::max(even, R / c + start);
            if (best_cost < 0. || cost < best_cost) best = c, best_cost = cost;
        }
        return best;
    }
    // (Partial sums of 256 rows cost more than they even out: two chunks of 2048
    // tokens over 16384 keys, 398 us with one split, 477 with four.)
    if (many_rows && units >= slots) return 1;
    // (A split of less than one round leaves warps idle, of less than two a slot.)
    const long long most =
        std::max(1ll, std::min(static_cast<long long>(FA_MAX_SPLITS), dual || many_rows ? rounds / 2 : rounds));
    const double start = many_rows ? 8. : 2.;
    long long best = 1;
    double best_cost = -1.;
    for (long long s = 1; s <= most; ++s) {
        const long long ctas = units * s;
        const double each = static_cast<double>((rounds + s - 1) / s) + start;
        if (!many_rows && 2 * ctas <= slots) {
            const double merge = s == 1 ? 0. : !dual && s <= kClusterSplits ? 0.5 : 2. + 0.02 * static_cast<double>(s);
            const double cost = each + merge;
            if (best_cost < 0. || cost < best_cost) best = s, best_cost = cost;
            continue;
        }
        const double cost = (B == 1 || many_rows ? static_cast<double>((ctas + slots - 1) / slots) * each
                                                 : (1. + 0.65 * static_cast<double>(ctas) / slots) * each) +
                            (s > 1 ? 4. + 0.1 * static_cast<double>(B == 1 ? s : 4 * s) : 0.);
        if (best_cost < 0. || cost < best_cost) best = s, best_cost = cost;
    }
    return static_cast<int>(best);
}

template <int D, bool CLUSTER, bool PART>
cudaError_t launch_rows(const PagedParams& p, cudaStream_t stream) {
    using L = PagedLayout<D, PART>;
    static ContextCache<int> attr_set;
    int done = 0;
    const cudaError_t e = attr_set.get(&done, [](int* out) {
        *out = 1;
        return cudaFuncSetAttribute(fa_paged_rows_kernel<D, CLUSTER, PART>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(L::ALLOC));
    });
    if (e != cudaSuccess) return e;
    long long ctas = static_cast<long long>(p.B) * p.Hkv * p.num_splits * p.row_blocks;
    if constexpr (PART) {
        // Warps for the sequences' own parts, as paged_unit counts them.
        const long long units = std::min(ctas, std::max(static_cast<long long>(p.places), static_cast<long long>(p.B) * p.Hkv));
        ctas = p.whole_ctas + (p.whole ? 0 : p.solo ? (units + kWarps - 1) / kWarps : ctas) + p.early;
    }
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_dependent_clusters(fa_paged_rows_kernel<D, CLUSTER, PART>, dim3(static_cast<unsigned>(ctas)),
                                     CLUSTER ? static_cast<unsigned>(p.num_splits) : 1u, kWarps * 32, L::ALLOC, stream,
                                     p);
}
// How a shared prefix is cut, where the sequences' own parts are cut as `own`. Beyond 16
// rows by blocks of 16 all the same, in one launch with the own parts, while a warp gets
// no more than two key tiles where all run at once: a launch, Q's way into shared memory
// and 128 rows of partial sums less (us, so and on the tensor cores; warps with 0.03
// tiles, 17 sequences, 464 keys, 4 heads of 64 over one: 11.8 and 16.4; 0.35, 29, 1280, 8
// heads of 128 over 4: 12.3 and 17.9; 2.6, 25 of four tokens, 14400, 2 heads of 64: 18.5
// and 19.0; 3.3, 12, 5360, 56 heads of 64 over 8: 20.5 and 18.9; 5, 31, 10432, 14 heads of
// 128 over 2: 30 and 22).
Plan prefix_plan(const Plan& own, int total_q, int G, int Hkv, int prefix_len, int d) {
    Plan c = plan_of(G, total_q, prefix_len, d, 0, 0);
    const long long rows = static_cast<long long>(total_q) * G, blocks = (rows + kRows - 1) / kRows;
    const long long tiles = (static_cast<long long>(prefix_len) + rows_keys(d) - 1) / rows_keys(d);
    const long long warps = static_cast<long long>(kPlaces) * rows_ctas(d) * kWarps;
    if (!c.tc || own.tc || tiles > 2 * warps || blocks * Hkv > 2 * warps / tiles) return c;
    c.tc = c.dual = false;
    c.block_rows = kRows;
    c.block_keys = rows_keys(d);
    c.row_blocks = blocks;
    c.tiles = tiles;
    return c;
}
// Sequences behind a prefix at most: each that brings tokens looks for the first one, past
// those before it that do not (the second half of 131072 sequences past the first: 52 ms,
// with 32 heads on one 224; 2^19 would take 0.8 and 3.6 s).
constexpr int kPrefixSeqs = 1 << 19;

// Whether the warps of the sequences' own parts behind a prefix take units alone: where
// there is a unit for every CTA that runs at once (and all key tiles can be counted in int),
// up to 1024 sequences, all of which every warp looks through (us so and with a CTA a unit,
// one token behind 512 keys with 9 of its own, 8 kv heads of 128: 512 sequences 50 and 71,
// 1024 110 and 131, 2048 340 and 252, 4096 1252 and 512).
bool solo_units(const Plan& own, int B, int Hkv, int d) {
    return !own.tc && static_cast<long long>(B) * Hkv >= static_cast<long long>(kPlaces) * rows_ctas(d) && B <= 1024 &&
           own.tiles <= 0x3fffffff / B;
}
// The splits of a shared prefix that the tensor-core kernel takes beside the sequences'
// own parts (its SMs hold nothing else): both cut so that the whole ends earliest, with
// the prefix on a part of the SMs, in microseconds of CTAs fitted to 21 batches on a GB300,
// B x prefix + own keys from 2 x 2900 + 50 to 64 x 65536 + 2000. (64 sequences, 16384 + up
// to 2000 keys, 32 + 8 heads, d = 128: 73 us with the prefix on all SMs first, in 19 parts,
// 61 with six, before the merge's last steps; 16 of five tokens, 8160 + up to 4000: 67
// with eight, 55 with three. All of those have lengths spread up to the longest; for
// others it is further off: 64 of 16384 + 2000 each, 104 as proposed and 81 at best, one
// of 2000 among 63 of 50, 53 and 37.)
int prefix_splits_beside(const Plan& w, const Plan& own, int B, int H, int Hkv, int total_q, int max_own, int d,
                         int* prefix_splits) {
    const double start = d == 64 ? 6. : d == 128 ? 8. : 24., tile = 1.6;  // a prefix CTA, a key tile of it
    const bool solo = solo_units(own, B, Hkv, d);
    const int at_once = own.tc ? 1 : rows_ctas(d);  // own CTAs of an SM
    const double own_start = own.tc ? 12. : solo ? 12. : 10.;
    const double own_key = own.tc ? 0.003 : solo ? (d == 64 ? 0.03 : d == 128 ? 0.04 : 0.07) : d == 64 ? 0.01 : d == 128 ? 0.02 : 0.035;
    const double merge = 0.5e-6 * total_q * H * d;  // per split
    const double units = static_cast<double>(B) * Hkv * own.row_blocks;
    const long long whole = static_cast<long long>(Hkv) * w.row_blocks;
    int best = 1;
    double least = -1.;
    for (const int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
        if (s > 1 && s > w.tiles) break;
        const long long ctas = whole * s;
        const double each = start + tile * static_cast<double>((w.tiles + s - 1) / s);
        const double end = each * static_cast<double>((ctas + kPlaces - 1) / kPlaces);
        const double beside = static_cast<double>(std::max(0ll, kPlaces - ctas)) * at_once;
        for (const int a : {1, 2, 3, 4, 6, 8, 12, 16, 24}) {
            if (a > 1 && 128ll * a > max_own + 63) break;
            // Sequences of six tenths of the longest length on average; a warp is a quarter
            // of a CTA.
            const double parts = (a > 1 ? units * (0.6 * a + 0.5) : units) / (solo ? kWarps : 1);
            const double part = own_start + own_key * max_own / a;
            const double even = (static_cast<double>(ctas) * each + parts * part / at_once) / kPlaces + 0.45 * part;
            const double cost = std::max(parts <= beside ? part : even, end) + merge * (s + a);
            if (least < 0. || cost < least) least = cost, best = a, *prefix_splits = s;
        }
    }
    return best;
}
// The splits of a call as clusters: where all of its CTAs run at once, since a
// CTA that is done holds its place until the others of its cluster are.
bool as_clusters(const Plan& c, long long units, int num_splits, int d) {
    return !c.tc && num_splits > 1 && num_splits <= kClusterSplits && units * num_splits <= 152 * rows_ctas(d);
}

template <int D, bool PART>
cudaError_t launch_merge(const PagedParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.B) * p.max_q * p.H;
    // Four warps a row while that leaves the grid within about one wave (of the merge of a
    // prefix's states, which holds more registers, a smaller one: 2048 rows of nine states,
    // the whole call, 57 us with one warp, 60.5 with four).
    const bool four = p.num_splits > 8 && rows <= (PART ? 1024 : 4096);
    const long long blocks = four ? rows : (rows + 3) / 4;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_dependent(four ? fa_paged_merge_kernel<D, 4, PART> : fa_paged_merge_kernel<D, 1, PART>,
                            dim3(static_cast<unsigned>(blocks)), 128, 0, stream, p);
}

// What the paged calls check alike: the cache, the batch's arrays and bounds, the
// shape, the scale.
fa_status check_paged(const void* q, const fa_paged_cache* cache, const int* page_table, const int* cu_seqlens_q,
                      const int* seqlens_k, const void* o, const float* lse, int B, int H, int total_q,
                      int max_seqlen_q, int max_seqlen_k, int max_pages, float scale) {
    if (!q || !cache || !page_table || !cu_seqlens_q || !seqlens_k || !o || !lse) return FA_ERR_NULL;
    const fa_status sc = check_cache(cache);
    if (sc != FA_OK) return sc;
    const int Hkv = cache->Hkv;
    if (B < 1 || H < 1 || total_q < 1 || max_seqlen_q < 1 || max_seqlen_q > total_q || max_seqlen_k < 1 ||
        max_pages < 1)
        return FA_ERR_SHAPE;
    if (H < Hkv || H % Hkv) return FA_ERR_GROUP;
    if (static_cast<long long>(max_pages) * cache->page_size > 0x7fffffffll - 4096) return FA_ERR_SHAPE;
    if (max_seqlen_k > max_pages * cache->page_size) return FA_ERR_SHAPE;
    if (static_cast<long long>(max_seqlen_q) * (H / Hkv) > 0x7fffffffll - 4096) return FA_ERR_SHAPE;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_SCALE;
    return FA_OK;
}
bool paged_aligned(const void* q, const void* o, const float* lse, const int* page_table, const int* cu_seqlens_q,
                   const int* seqlens_k) {
    return aligned(q, 16) && aligned(o, 16) && aligned(lse, 4) && aligned(page_table, 4) && aligned(cu_seqlens_q, 4) &&
           aligned(seqlens_k, 4);
}

// PagedParams::gate on the current device.
__device__ unsigned g_fa_prefix_gate = 0u;
cudaError_t gate_ptr(unsigned** ptr) {
    static ContextCache<unsigned*> cache;
    return cache.get(ptr, [](unsigned** out) {
        void* p = nullptr;
        const cudaError_t e = cudaGetSymbolAddress(&p, g_fa_prefix_gate);
        *out = static_cast<unsigned*>(p);
        return e;
    });
}

// The parameters of a launch over `seqs` sequences of at most max_q new tokens and max_k
// keys, cut into num_splits; the cache's maps and the arrays are set already.
void cut_paged(PagedParams& p, const Plan& c, int seqs, int max_q, int max_k, int num_splits) {
    p.max_q = max_q;
    p.max_k = max_k;
    p.block_rows = c.block_rows;
    p.block_keys = c.block_keys;
    p.row_blocks = static_cast<int>(c.row_blocks);
    p.num_splits = num_splits;
    const long long row_warps = (static_cast<long long>(max_q) * p.G + 31) / 32;
    p.shares = !c.dual ? 0 : row_warps > 2 ? 1 : row_warps == 2 ? 2 : 4;
    p.slot_warps = p.shares == 1 ? static_cast<int>(row_warps) : 4;
    p.balance = c.dual && num_splits > 1 && seqs > 1 && seqs <= kTcBalance;
    p.tiles_per_split = static_cast<int>((c.tiles + num_splits - 1) / num_splits);
}
bool encode_cache(PagedParams& p, const fa_paged_cache* cache, const Plan& c) {
    const long long rows = static_cast<long long>(cache->num_pages) * cache->Hkv * cache->page_size;
    const int box = std::min(cache->page_size, c.block_keys);
    return encode_cache_map(&p.tm_k, cache->k, cache->d, rows, box) &&
           encode_cache_map(&p.tm_v, cache->v, cache->d, rows, box);
}
// Everything of a call that does not depend on how it is cut.
cudaError_t fill_paged(PagedParams& p, const void* q, const fa_paged_cache* cache, const int* page_table,
                       const int* cu_seqlens_q, const int* seqlens_k, void* o, float* lse, void* workspace, int B,
                       int H, int total_q, int max_pages, int states, float scale) {
    std::memset(&p, 0, sizeof(p));
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.page_table = page_table;
    p.cu = cu_seqlens_q;
    p.lens = seqlens_k;
    if (states > 1) {
        const size_t part = static_cast<size_t>(states) * total_q * H;
        p.ws_o = static_cast<float*>(workspace);
        p.ws_m = p.ws_o + part * cache->d;
        p.ws_l = p.ws_m + part;
    }
    p.B = B;
    p.H = H;
    p.Hkv = cache->Hkv;
    p.G = H / cache->Hkv;
    p.total_q = total_q;
    p.num_pages = cache->num_pages;
    p.log_page = log2_exact(cache->page_size);
    p.max_pages = max_pages;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_limit = kDefaultWaitLimit;
    return device_status_ptr(&p.status);
}
template <bool PART>
cudaError_t launch_paged(const PagedParams& p, const Plan& c, int d, cudaStream_t stream) {
    return c.tc       ? launch_paged_tc(p, d, PART, stream)
           : d == 64  ? launch_rows<64, false, PART>(p, stream)
           : d == 128 ? launch_rows<128, false, PART>(p, stream)
                      : launch_rows<256, false, PART>(p, stream);
}
template <bool PART>
cudaError_t launch_paged_merge(const PagedParams& p, int d, cudaStream_t stream) {
    return d == 64    ? launch_merge<64, PART>(p, stream)
           : d == 128 ? launch_merge<128, PART>(p, stream)
                      : launch_merge<256, PART>(p, stream);
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_paged_num_splits(int B, int H, int Hkv, int max_seqlen_q, int max_seqlen_k, int d, int window, int sinks) {
    if (B < 1 || Hkv < 1 || H < Hkv || H % Hkv || max_seqlen_q < 1 || max_seqlen_k < 1 || !fa::valid_d(d)) return 0;
    const fa::Plan c = fa::plan_of(H / Hkv, max_seqlen_q, max_seqlen_k, d, window, sinks);
    const long long units = static_cast<long long>(B) * Hkv * c.row_blocks;
    const long long rounds = (c.tiles * c.block_keys + 127) / 128;
    // CTAs at once: one per SM for the tensor-core kernel.
    return fa::best_splits(B, units, rounds, 152 * (c.tc ? 1 : fa::rows_ctas(d)), c.dual, c.tc && !c.dual);
}

size_t fa_paged_workspace_bytes(int total_q, int H, int d, int num_splits) {
    if (total_q < 1 || H < 1 || !fa::valid_d(d) || num_splits < 1 || num_splits > FA_MAX_SPLITS) return 0;
    if (num_splits == 1) return 0;
    return static_cast<size_t>(num_splits) * total_q * H * (static_cast<size_t>(d) + 2) * sizeof(float);
}

fa_status fa_fwd_paged_fp8(const void* q, const fa_paged_cache* cache, const int* page_table, const int* cu_seqlens_q,
                           const int* seqlens_k, void* o, float* lse, void* workspace, int B, int H, int total_q,
                           int max_seqlen_q, int max_seqlen_k, int max_pages, float scale, int window, int sinks,
                           int num_splits, cudaStream_t stream) {
    const fa_status sc = fa::check_paged(q, cache, page_table, cu_seqlens_q, seqlens_k, o, lse, B, H, total_q, max_seqlen_q,
                                         max_seqlen_k, max_pages, scale);
    if (sc != FA_OK) return sc;
    if (window < 0 || sinks < 0 || (window == 0 && sinks != 0) || sinks > 0x40000000 || window > 0x40000000)
        return FA_ERR_WINDOW;
    if (num_splits < 1 || num_splits > FA_MAX_SPLITS) return FA_ERR_SPLITS;
    if (!fa::paged_aligned(q, o, lse, page_table, cu_seqlens_q, seqlens_k)) return FA_ERR_ALIGN;
    if (num_splits > 1 && (!workspace || !fa::aligned(workspace, 16))) return FA_ERR_WORKSPACE;
    const int d = cache->d;
    fa::PagedParams p;
    if (fa::fill_paged(p, q, cache, page_table, cu_seqlens_q, seqlens_k, o, lse, workspace, B, H, total_q, max_pages,
                       num_splits, scale) != cudaSuccess)
        return FA_ERR_CUDA;
    p.window = window;
    p.sinks = sinks;
    const fa::Plan c = fa::plan_of(p.G, max_seqlen_q, max_seqlen_k, d, window, sinks);
    fa::cut_paged(p, c, B, max_seqlen_q, max_seqlen_k, num_splits);
    if (!fa::encode_cache(p, cache, c)) return FA_ERR_CUDA;
    if (fa::as_clusters(c, static_cast<long long>(B) * p.Hkv * c.row_blocks, num_splits, d)) {
        const cudaError_t e = d == 64    ? fa::launch_rows<64, true, false>(p, stream)
                              : d == 128 ? fa::launch_rows<128, true, false>(p, stream)
                                         : fa::launch_rows<256, true, false>(p, stream);
        return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    }
    cudaError_t e = fa::launch_paged<false>(p, c, d, stream);
    if (e == cudaSuccess && num_splits > 1) e = fa::launch_paged_merge<false>(p, d, stream);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_prefix_num_splits(int B, int H, int Hkv, int total_q, int max_seqlen_q, int max_seqlen_k, int prefix_len, int d,
                         int* prefix_splits) {
    if (!prefix_splits || prefix_len < 1 || prefix_len >= max_seqlen_k || total_q < max_seqlen_q || B < 1 ||
        B > fa::kPrefixSeqs || Hkv < 1 || H < Hkv || H % Hkv || max_seqlen_q < 1 || !fa::valid_d(d))
        return 0;
    const fa::Plan c = fa::plan_of(H / Hkv, max_seqlen_q, max_seqlen_k - prefix_len, d, 0, 0);
    const fa::Plan w = fa::prefix_plan(c, total_q, H / Hkv, Hkv, prefix_len, d);
    if (w.tc && !w.dual) return fa::prefix_splits_beside(w, c, B, H, Hkv, total_q, max_seqlen_k - prefix_len, d, prefix_splits);
    int own = fa_paged_num_splits(B, H, Hkv, max_seqlen_q, max_seqlen_k - prefix_len, d, 0, 0);
    const int shared = fa::best_splits(1, Hkv * w.row_blocks, (w.tiles * w.block_keys + 127) / 128,
                                       fa::kPlaces * (w.tc ? 1 : fa::rows_ctas(d)), w.dual, false);
    // Warps with units alone cut the sequences by their lengths at hand: room for
    // twice the mean number of splits.
    const long long warps = static_cast<long long>(fa::kPlaces) * fa::rows_ctas(d) * fa::kWarps;
    if (fa::solo_units(c, B, Hkv, d))
        own = static_cast<int>(std::min(c.tiles, 2 * warps / (static_cast<long long>(B) * Hkv) + 1));
    *prefix_splits = std::min(shared, FA_MAX_SPLITS / 2);
    return std::min(own, FA_MAX_SPLITS / 2);
}

fa_status fa_fwd_prefix_fp8(const void* q, const fa_paged_cache* cache, const int* page_table, const int* cu_seqlens_q,
                            const int* seqlens_k, void* o, float* lse, void* workspace, int B, int H, int total_q,
                            int max_seqlen_q, int max_seqlen_k, int max_pages, int prefix_len, float scale,
                            int num_splits, int prefix_splits, cudaStream_t stream) {
    const fa_status sc = fa::check_paged(q, cache, page_table, cu_seqlens_q, seqlens_k, o, lse, B, H, total_q, max_seqlen_q,
                                         max_seqlen_k, max_pages, scale);
    if (sc != FA_OK) return sc;
    const int d = cache->d;
    if (prefix_len < 1 || prefix_len % cache->page_size || prefix_len >= max_seqlen_k || B > fa::kPrefixSeqs) return FA_ERR_SHAPE;
    if (static_cast<long long>(total_q) * (H / cache->Hkv) > 0x7fffffffll - 4096) return FA_ERR_SHAPE;
    if (num_splits < 1 || prefix_splits < 1 || num_splits > FA_MAX_SPLITS || prefix_splits > FA_MAX_SPLITS - num_splits)
        return FA_ERR_SPLITS;
    if (!fa::paged_aligned(q, o, lse, page_table, cu_seqlens_q, seqlens_k)) return FA_ERR_ALIGN;
    if (!workspace || !fa::aligned(workspace, 16)) return FA_ERR_WORKSPACE;
    fa::PagedParams p;
    if (fa::fill_paged(p, q, cache, page_table, cu_seqlens_q, seqlens_k, o, lse, workspace, B, H, total_q, max_pages,
                       num_splits + prefix_splits, scale) != cudaSuccess)
        return FA_ERR_CUDA;
    p.base_len = prefix_len;
    p.base_pages = prefix_len / cache->page_size;
    p.own_q = max_seqlen_q;
    p.own_k = max_seqlen_k - prefix_len;
    // The prefix, for all rows at once, and the sequences' own keys, in one launch where
    // both are cut into blocks of 16 rows; then the merge.
    const fa::Plan own = fa::plan_of(p.G, max_seqlen_q, max_seqlen_k - prefix_len, d, 0, 0);
    const fa::Plan whole = fa::prefix_plan(own, total_q, p.G, p.Hkv, prefix_len, d);
    p.whole = 1;
    p.state0 = num_splits;
    fa::cut_paged(p, whole, 1, total_q, prefix_len, prefix_splits);
    const long long ctas = p.Hkv * whole.row_blocks * prefix_splits;
    if (ctas > 0x7fffffffll) return FA_ERR_SHAPE;
    if (!whole.tc) {
        p.whole_ctas = static_cast<unsigned>(ctas);
        p.shared = {p.max_q, p.max_k, p.row_blocks, p.num_splits, p.tiles_per_split, p.state0};
    }
    if (whole.tc || own.tc) {
        if (fa::gate_ptr(&p.gate) != cudaSuccess || !fa::encode_cache(p, cache, whole)) return FA_ERR_CUDA;
        if (fa::launch_paged<true>(p, whole, d, stream) != cudaSuccess) return FA_ERR_CUDA;
        p.whole_ctas = 0;
        p.early = 1;
    }
    p.whole = 0;
    p.state0 = 0;
    fa::cut_paged(p, own, B, max_seqlen_q, max_seqlen_k - prefix_len, num_splits);
    p.solo = fa::solo_units(own, B, p.Hkv, d);
    p.places = fa::kPlaces * fa::rows_ctas(d) * fa::kWarps * (p.early ? 2 : 1);
    if (!fa::encode_cache(p, cache, own)) return FA_ERR_CUDA;
    if (fa::launch_paged<true>(p, own, d, stream) != cudaSuccess) return FA_ERR_CUDA;
    p.num_splits = num_splits + prefix_splits;
    return fa::launch_paged_merge<true>(p, d, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
