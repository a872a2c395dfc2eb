// fa_bwd.cu — attention backward for head dims 64, 128 and 256: dQ, dK, dV. Holds the
// backward's kernels and its C entry points (fa_bwd_workspace_bytes, fa_bwd).
//
// What is computed (the plain definition of the forward differentiated; the
// FA-2 page, "AI 大模型之 FlashAttention_02", sections "warp之间怎样减少通信" and
// "训练与部署 切分与归约的反向一致性": the training backward needs dQ, dK, dV,
// with dK and dV accumulated across query rows):
//   P = exp(scale Q K^T - LSE) (the forward's row LSE; masked entries 0)
//   dV = P^T dO,  dP = dO V^T,  D_i = sum_c dO_ic O_ic,  dS = P * (dP - D)
//   dQ = scale dS K,  dK = scale dS^T Q.
//
// Responsibilities and accumulation (the page asks that they be written down):
//   * fa_bwd_pre_kernel: per query row (rows padded to whole 128-row tiles),
//     -LSE log2(e) and -D_i in fp32 (D_i from bf16 dO and O; padded rows and
//     rows that saw no key get -inf and 0); zeroes the fp32 dQ accumulator.
//   * fa_bwd_kernel: one CTA per (head, 128-key tile). It owns dK and dV of its
//     keys and accumulates them over every query tile in TMEM (fp32), so they
//     need no cross-CTA reduction. Its dQ contribution, dS K for its keys, is
//     added to the fp32 accumulator with atomic adds: dQ is the one quantity
//     summed across CTAs (across key tiles).
//   * fa_bwd_dq_kernel: dQ = scale * accumulator, to bf16.
//
// fa_bwd_kernel steps over the queries 64 at a time. Roles: warp 0 loads K
// and V once and, per step, Q, dO and the step's -LSE log2e and -D into a ring
// of three slots (TMA); warp 1 issues tcgen05 MMAs; warps 4-11 are the compute
// group, two warps per TMEM lane quarter, one per 32-query chunk of a step
// (thread = TMEM lane = key row); warps 12-15 read dQ^T out (lane = head dim).
// TMEM holds two step buffers of 128 columns beside dV and dK. Per step h
// (buffer h & 1):
//   S^T = K Q_h^T and dP^T = V dO_h^T (lanes = keys, 64 query columns each);
//   the compute group forms P^T = exp2(S^T scale log2e - LSE log2e) and
//   dS^T = P^T (dP^T - D), writes both as bf16 into TMEM over the first half
//   of each chunk's own columns, and dS^T into shared memory (128-byte
//   swizzle);
//   dV += P^T dO_h and dK += dS^T Q_h (A from TMEM, B = dO_h / Q_h MN-major);
//   dQ_h^T = K^T dS^T (A = K MN-major, B = dS^T from shared memory) over the
//   buffer's S^T columns; the readout group takes it out of TMEM, releases the
//   buffer and adds it to the fp32 accumulator, 32 consecutive floats per warp
//   instruction.
// The issuer runs the MMAs in pairs of steps, S^T and dP^T of two steps then
// dV, dK and dQ^T of the same two, so that each of the three groups (tensor
// core, compute, readout) always has the other step's work to overlap.
// Every mbarrier wait is bounded, as in the forward kernels.
//
// Head dim 64: the same steps with half-width K, V, Q and dO tiles and 64
// TMEM columns each for dV and dK. dQ^T keeps M = 128 (head-dim lanes): its A
// operand, K read MN-major, has a second 64-dim chunk of zeros that the CTA
// writes once, so lanes 64-127 of dQ^T are zero and only the readout warps of
// lanes 0-63 take it out.
//
// Head dim 256: dV and dK of 128 keys at d = 256 would take all 512 TMEM
// columns, so each key tile has two CTAs, one per 128-column half of the head
// dim. Both compute the whole S^T and dP^T (the contraction runs over all 256
// columns); each accumulates its half of dV and dK in TMEM and adds its half
// of dQ. K and V stay resident (64 KB each), which leaves shared memory for one
// Q/dO stage: the issuer then runs the steps one after another (S^T and dP^T
// of step h + 1 once step h's dV and dK have read the stage and its load has
// landed) instead of in pairs.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "fa.h"
#include "fa_internal.h"
#include "fa_launch.h"
#include "fa_packed.cuh"
#include "sm103_ptx.cuh"

namespace fa {

// Kernel parameters, filled by fa_bwd below.
struct BwdParams {
    CUtensorMap tm_q;   // bf16 [B*H][Nq][d], box {64, 64, 1} (64 head-dim columns)
    CUtensorMap tm_k;   // bf16 [B*H][Nk][d], box {64, 128, 1}
    CUtensorMap tm_v;   // same as tm_k
    CUtensorMap tm_do;  // same as tm_q (dO)
    const float* nlse2; // fp32 [B*H][Nq_pad]: -LSE log2(e); -inf past Nq or with no key
    const float* ndd;   // fp32 [B*H][Nq_pad]: -D_i = -sum_c dO_ic O_ic; 0 past Nq
    float* dq_acc;      // fp32 [B*H][Nq_pad][d], zeroed, unscaled dS K accumulated
    void* dk;           // bf16 [B*H][Nk][d]
    void* dv;           // bf16 [B*H][Nk][d]
    int BH, Nq, Nk;
    int Nq_pad;         // Nq rounded up to whole 128-row query tiles
    int causal, causal_br;
    int k_tiles;        // ceil(Nk / 128)
    int pair_tiles;     // 1: a CTA takes key tiles kt and k_tiles - 1 - kt (causal)
    int tile_units;     // key-tile units per head: k_tiles, or ceil(k_tiles / 2) when paired
    float scale;
    float scale_log2;   // scale * log2(e)
    long long wait_limit;
    unsigned* status;
    // Sliding window (bottom-right; 0: none) with sinks, and heads that share kv
    // heads in groups: K, V, dK, dV have BHkv = B * Hkv heads.
    int window, sinks, group, H, Hkv, BHkv;
    // A tile's steps (all heads of its group in turn) are cut into parts, each a
    // CTA's: sink_parts for the first sink_tiles tiles, parts for the others.
    // With more than one part the CTAs leave fp32 partial sums, [unit][dK, dV]
    // [128 keys][d], which the last launch adds in order.
    int sink_tiles, sink_parts, parts;
    float* dkv_part;
    // Packed sequences (the window's fields apply; tensors token-major [total][heads][d],
    // tokens these many elements apart): rows of nlse2, ndd and dq_acc are [H][rows_pad],
    // a sequence's at pad_row. Partial sums of the sinks' tiles (the first sink_tiles of
    // each sequence) come first, [b][tile], then the others', by tile_slot.
    PackedSeqs seqs;
    long long rows_pad;
    long long q_stride, k_stride, v_stride, do_stride, dq_stride, dk_stride, dv_stride;
    int fill, block_heads;
    int pack_heads;  // kv heads whose units are taken together
};

namespace {

constexpr int kBwdKeys = 128;   // keys per CTA (TMEM lanes of S^T, dP^T, dV, dK)
constexpr int kBwdHalf = 64;    // queries per step
constexpr float kLog2e = 1.4426950408889634f;

// WIN: the form under a window (and on packed sequences). At d = 64 TMEM then holds a
// third step buffer; the dense form gains nothing from it (1069 against 1063 us for 8 x 32
// heads of 2048 rows; under a window of 512 with heads in groups of four 406 against 448).
template <int D, bool WIN = false>
struct LayoutBwd {
    static_assert(D == 64 || D == 128 || D == 256, "head dim 64, 128 or 256");
    static constexpr int DH = D < 128 ? D : 128;        // head-dim columns of dV, dK, dQ a CTA owns
    static constexpr int HALVES = D / DH;               // CTAs per key tile
    static constexpr int BUFS = D == 64 && WIN ? 3 : 2;        // step buffers in TMEM
    static constexpr int STAGES = D == 256 ? 1 : BUFS == 3 ? 5 : 3;  // Q/dO (+ -LSE log2e, -D) ring slots
    // warp 0 producer, warp 1 issuer, warps 2-3 idle (packed sequences: warp 2 finds
    // the unit), warps 4-11 compute (two
    // per TMEM lane quarter, one per 32-query chunk of a step), warps 12-15
    // dQ readout (one per lane quarter; at D = 64 the first two only).
    static constexpr int COMPUTE_WARPS = 8;
    static constexpr int READOUT_WARPS = 4;
    static constexpr int READOUT_ACTIVE = DH / 32;                  // lane quarters holding dQ^T
    static constexpr int CHUNKS = D / 64;                           // 64-column chunks of a row
    static constexpr int DH_CHUNKS = DH / 64;                       // chunks of the CTA's head-dim part
    static constexpr int THREADS = 128 + 32 * (COMPUTE_WARPS + READOUT_WARPS);
    static constexpr uint32_t KV_CHUNK = kBwdKeys * 128;            // 16 KB: 64 columns of K or V
    // K spans at least two chunks: dQ^T reads it as an M = 128 operand, and at
    // D = 64 the second chunk is zeros.
    static constexpr uint32_t K_BYTES = (CHUNKS < 2 ? 2 : CHUNKS) * KV_CHUNK;
    static constexpr uint32_t V_BYTES = CHUNKS * KV_CHUNK;
    static constexpr uint32_t QH_CHUNK = kBwdHalf * 128;            // 8 KB: 64 columns of a step's Q or dO
    static constexpr uint32_t QH_BYTES = CHUNKS * QH_CHUNK;
    static constexpr uint32_t ROWS_BYTES = kBwdHalf * 4;            // 256 B of -LSE log2e (or -D)
    static constexpr uint32_t STAGE_BYTES = 2 * QH_BYTES;           // Q and dO of a step
    static constexpr uint32_t DS_BYTES = kBwdKeys * kBwdHalf * 2;   // 16 KB: dS^T bf16 [keys][64 queries]
    // Swizzled tiles start on 1024-byte boundaries (the MMA descriptors'
    // base offset is 0); the per-row arrays need 16 bytes.
    static constexpr uint32_t K_OFF = 0;
    static constexpr uint32_t V_OFF = K_OFF + K_BYTES;
    static constexpr uint32_t STAGE_OFF = V_OFF + V_BYTES;           // [stage]: Q, dO
    static constexpr uint32_t Q_IN = 0, DO_IN = QH_BYTES;
    static constexpr uint32_t DS_OFF = STAGE_OFF + STAGES * STAGE_BYTES;  // [buffer]
    static constexpr uint32_t ROWS_OFF = DS_OFF + BUFS * DS_BYTES;     // [stage]: -LSE log2e, -D
    static constexpr uint32_t NL_IN = 0, ND_IN = ROWS_BYTES;
    static constexpr uint32_t BAR_OFF = ROWS_OFF + STAGES * 2 * ROWS_BYTES;
    static_assert(STAGE_OFF % 1024 == 0 && STAGE_BYTES % 1024 == 0 && QH_CHUNK % 1024 == 0 &&
                      DS_OFF % 1024 == 0 && DS_BYTES % 1024 == 0, "swizzle atoms must be 1024-aligned");
    static constexpr int BAR_KV = 0;
    static constexpr int BAR_QFULL = 1;                    // [stage]
    static constexpr int BAR_QEMPTY = BAR_QFULL + STAGES;   // [stage]
    static constexpr int BAR_SFULL = BAR_QEMPTY + STAGES;   // [buffer] S^T, dP^T done
    static constexpr int BAR_PREADY = BAR_SFULL + BUFS;    // [buffer] P^T, dS^T written (one arrival per compute warp)
    static constexpr int BAR_DQFULL = BAR_PREADY + BUFS;   // [buffer] dQ^T done (and every earlier MMA)
    static constexpr int BAR_DQREAD = BAR_DQFULL + BUFS;   // [buffer] dQ^T read (one arrival per readout warp)
    static constexpr int BAR_KVFREE = BAR_DQREAD + BUFS;   // the first of two key tiles' MMAs done
    static constexpr int BAR_ACCFREE = BAR_KVFREE + 1;  // its dK, dV read out of TMEM (one arrival per compute warp)
    static constexpr int BAR_DRAIN = BAR_ACCFREE + 1;
    static constexpr int NUM_BARS = BAR_DRAIN + 1;
    static constexpr uint32_t MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr uint32_t BYTES = MISC_OFF + 16;
    static constexpr size_t ALLOC_BYTES = BYTES + 1024;
    // TMEM columns. Buffer b (b = step % BUFS) at 128 b: S^T in its first 64
    // columns (then P^T packed over their first halves, then dQ^T), dP^T in
    // the next 64 (then dS^T packed over their first halves). dV and dK last
    // (D columns each).
    __host__ __device__ static constexpr uint32_t BUF_COL(int b) { return 128u * static_cast<uint32_t>(b); }
    static constexpr uint32_t DP_IN = 64, DV_COL = 128 * BUFS, DK_COL = DV_COL + (512 - DV_COL) / 2;
    static_assert(DV_COL + 2 * DH <= 512 && DK_COL + DH <= 512, "dV and dK overflow TMEM");
    static_assert(ALLOC_BYTES <= 232448, "shared memory over the 227 KB per-CTA limit");
    static_assert(THREADS * 128 <= 65536, "registers: 128 per thread at most");
};

__device__ __forceinline__ bool bwd_wait(uint32_t bar, uint32_t parity, const BwdParams& p,
                                         volatile uint32_t* abort_flag, unsigned what,
                                         bool honor_abort = true) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long start = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (honor_abort && *abort_flag) return false;
        if (clock64() - start > p.wait_limit) {
            *abort_flag = 1u;
            atomicOr(p.status, what);
            return false;
        }
    }
}

// The 64-query steps a key tile sees: all of them, or (causal) those with a
// row at or after the tile's first key minus the alignment offset.
__device__ __forceinline__ void bwd_steps(const BwdParams& p, int kt, int& h0, int& n) {
    const int steps = (p.Nq + kBwdHalf - 1) / kBwdHalf;
    h0 = 0;
    if (p.causal) {
        const int off = p.causal_br ? p.Nk - p.Nq : 0;
        const int first_row = kt * kBwdKeys - off;  // key k is visible to rows >= k - off
        h0 = first_row <= 0 ? 0 : first_row / kBwdHalf;
    }
    n = max(0, steps - h0);
}

// The steps of a key tile under a window: rows from the one at its first key to
// the last whose window reaches its last key, or to the end where the tile
// holds a sink.
__device__ __forceinline__ void bwd_steps_win(const BwdParams& p, int Nq, int Nk, int kt, int& h0, int& n) {
    const int off = Nk - Nq;
    const int k0 = kt * kBwdKeys;
    const int k1 = min(k0 + kBwdKeys, Nk) - 1;
    const int first = max(0, k0 - off);
    int last = Nq - 1;
    if (p.window > 0 && k0 >= p.sinks) last = min(last, k1 - off + p.window - 1);
    h0 = first / kBwdHalf;
    n = last < first ? 0 : last / kBwdHalf - h0 + 1;
}

// P^T and dS^T of one 32-query chunk for this thread's key row: s and dp are
// the chunk's S^T and dP^T columns, nl and nd the chunk's -LSE log2e and -D in
// shared memory (the same addresses for every lane: broadcast loads). MASK:
// `lim` is the first visible chunk column (causal) and `key_ok` whether the
// key exists; without MASK every entry is visible. WIN: `end` is the first
// column past the key's window.
template <bool MASK, bool WIN = false>
__device__ __forceinline__ void bwd_chunk(const uint32_t (&s)[32], const uint32_t (&dp)[32], uint32_t nl,
                                          uint32_t nd, float sl2, int lim, bool key_ok, uint32_t (&pk)[16],
                                          uint32_t (&dk)[16], int end = 0) {
    const uint64_t sl2x2 = f2pack(sl2, sl2);
    // (One bit per column rather than two comparisons each.)
    const uint32_t seen = WIN && key_ok ? low_bits(end) & ~low_bits(lim) : 0u;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        float l4[4], d4[4];
        ld_shared_v4f(nl + 16 * u, l4);
        ld_shared_v4f(nd + 16 * u, d4);
        const uint64_t x01 = ffma2(f2pack(__uint_as_float(s[4 * u]), __uint_as_float(s[4 * u + 1])), sl2x2,
                                   f2pack(l4[0], l4[1]));
        const uint64_t x23 = ffma2(f2pack(__uint_as_float(s[4 * u + 2]), __uint_as_float(s[4 * u + 3])), sl2x2,
                                   f2pack(l4[2], l4[3]));
        float x[4];
        f2unpack(x01, x[0], x[1]);
        f2unpack(x23, x[2], x[3]);
        float pv[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            // The exponential runs for every element and the mask selects after
            // it (x is finite or -inf: no NaN), so there are no branches.
            const float ex = ex2(x[h]);
            if constexpr (WIN && MASK) pv[h] = (seen & (1u << (4 * u + h))) ? ex : 0.f;
            else pv[h] = MASK ? ((key_ok && 4 * u + h >= lim) ? ex : 0.f) : ex;
        }
        const uint64_t g01 = fadd2(f2pack(__uint_as_float(dp[4 * u]), __uint_as_float(dp[4 * u + 1])),
                                   f2pack(d4[0], d4[1]));
        const uint64_t g23 = fadd2(f2pack(__uint_as_float(dp[4 * u + 2]), __uint_as_float(dp[4 * u + 3])),
                                   f2pack(d4[2], d4[3]));
        float ds[4];
        f2unpack(fmul2(f2pack(pv[0], pv[1]), g01), ds[0], ds[1]);
        f2unpack(fmul2(f2pack(pv[2], pv[3]), g23), ds[2], ds[3]);
        pk[2 * u] = pack_bf16x2(pv[0], pv[1]);
        pk[2 * u + 1] = pack_bf16x2(pv[2], pv[3]);
        dk[2 * u] = pack_bf16x2(ds[0], ds[1]);
        dk[2 * u + 1] = pack_bf16x2(ds[2], ds[3]);
    }
}

// A packed batch's unit: its sequence (number b), key tile and part, and the number of
// its first part's partial sums.
struct BwdUnit {
    PackedSeq s;
    int b, h, kt, part, parts;
    long long sums;
    bool live;
};
__device__ __forceinline__ int key_tiles(const PackedSeq& s) { return (s.m + kBwdKeys - 1) / kBwdKeys; }
// Number of the partial sums of tile kt, kv head h.
__device__ __forceinline__ long long bwd_sums(const BwdParams& p, const PackedSeq& s, int b, int kt, int h) {
    if (kt < p.sink_tiles) return ((static_cast<long long>(b) * p.sink_tiles + kt) * p.Hkv + h) * p.sink_parts;
    const long long sinks = p.sink_parts > 1 ? static_cast<long long>(p.seqs.B) * p.sink_tiles * p.Hkv * p.sink_parts : 0;
    return sinks + ((tile_slot(s.k0, b) + kt) * p.Hkv + h) * p.parts;
}
// Unit number `lin`, found by one warp: the sinks' tiles first, then the others; of each, a
// tile's parts beside one another.
__device__ __forceinline__ void bwd_pack_unit(const BwdParams& p, long long lin, int lane, BwdUnit* u) {
    PackedSeq s;
    if (blockIdx.x == 0)
        for (int b = lane; b < p.seqs.B; b += 32)
            if (!packed_seq(p.seqs, b, s)) atomicOr(p.status, kStatusBadSeqlens);
    int sinks = 0, all = 0;  // a kv head's units of the sinks' tiles, and of the others
    if (p.sink_tiles > 0)
        sinks = p.sink_parts * packed_total(p.seqs.B, lane, [&](int b) {
            PackedSeq y;
            packed_seq(p.seqs, b, y);
            return min(key_tiles(y), p.sink_tiles);
        });
    const long long sink_units = static_cast<long long>(sinks) * p.Hkv;
    const bool sink = lin < sink_units;
    const int parts = sink ? p.sink_parts : p.parts, together = sink ? p.Hkv : p.pack_heads;
    if (together < p.Hkv)
        all = p.parts * packed_total(p.seqs.B, lane, [&](int b) {
            PackedSeq y;
            packed_seq(p.seqs, b, y);
            return max(key_tiles(y) - p.sink_tiles, 0);
        });
    PackedCursor first = {0, 0};
    int h = 0, at = 0;
    const bool there = packed_head(sink ? lin : lin - sink_units, p.Hkv, together, all, h, at);
    const int r = at / parts;
    // Levels count a sequence's tiles from its last one up.
    auto runs = [&](int b, int& a, int& n) {
        PackedSeq y;
        packed_seq(p.seqs, b, y);
        const int tiles = key_tiles(y), first = min(tiles, p.sink_tiles);
        a = sink ? tiles - first : 0;
        n = sink ? first : tiles - first;
    };
    int b = 0, level = 0;
    const bool live = there && packed_pick(p.seqs.B, r, lane, runs, b, level, first);
    if (lane == 0) {
        *u = {};
        u->live = live;
        if (live) {
            packed_seq(p.seqs, b, u->s);
            u->b = b;
            u->kt = key_tiles(u->s) - 1 - level;
            u->parts = parts;
            u->h = h;
            u->part = at % parts;
            u->sums = bwd_sums(p, u->s, b, u->kt, h);
        }
    }
}

// One CTA per (head, key-tile unit, head-dim part), stepping over the queries
// 64 at a time. A unit is one 128-key tile, or under a causal mask the pair of
// tiles kt and k_tiles - 1 - kt, run one after the other: the steps of a tile
// fall with its index, so every pair has about the same number of steps and no
// CTA is left with the few steps of a last tile alone. The two tiles share the
// step sequence: global step G (over both tiles) uses TMEM buffer G % BUFS and
// ring slot G % STAGES. Between the tiles K and V are reloaded once the first
// tile's MMAs are done (KVFREE) and the first MMA into dV and dK waits until
// the compute group has read the first tile's out of TMEM (ACCFREE).
//   The issuer runs each tile's MMAs in pairs of steps: S^T and dP^T of steps
// 2k+2 and 2k+3 (each needs its buffer's dQ^T of two steps back read out),
// then dV, dK and dQ^T of steps 2k+2 and 2k+3 (each needs its P^T and dS^T).
// While the tensor core runs one step's MMAs, the compute group forms P^T and
// dS^T of the other and the readout group adds the previous dQ^T to the
// accumulator. With one ring slot (d = 256) the steps run in order.
//   WIN: sliding window with sinks and grouped heads. A CTA takes one key tile
// of a kv head and walks the steps of every query head of the group in turn,
// K and V staying resident and dV and dK accumulating over the whole group; or
// a part of those steps, where the units would not fill the GPU otherwise, and
// for the tiles of the sinks, which see every row behind them (16 heads of 8192
// rows in groups of four, window 1024, 4 sinks, d = 128: a sink tile has 512
// steps, another 72). Units are ordered tile by tile over all kv heads, the
// sinks' first. P and dS are rounded to bf16 for their products here as well: the
// other operands (dO, Q, K) are bf16, which f16 does not hold, and kind::f16 takes
// both in one type.
//   PACK: the same on packed sequences. Units are taken longest first over all
// sequences (packed_pick: a key tile sees the more rows the further it lies from its
// sequence's end), the sinks' first. Rows of a tile that are not the sequence's (its
// last keys', its last step's queries') hold other tokens: the issuer overwrites them
// with zeros before the MMAs read them, since a weight of zero does not undo an
// infinity or a NaN.
template <int D, bool WIN = false, bool PACK = false>
__global__ void __launch_bounds__(LayoutBwd<D, WIN>::THREADS, 1) fa_bwd_kernel(const __grid_constant__ BwdParams p) {
    static_assert(WIN || !PACK, "packed sequences take the window's form");
    using L = LayoutBwd<D, WIN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
    volatile uint32_t* abort_flag = misc + 1;
    auto bar = [&](int i) -> uint32_t { return sbase + L::BAR_OFF + 8u * i; };
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // CTA = (head, key-tile unit, head-dim part), the part fastest.
    const int hd = static_cast<int>(blockIdx.x % L::HALVES);
    const int unit_lin = static_cast<int>(blockIdx.x / L::HALVES);
    int bh = WIN ? unit_lin % p.BHkv : unit_lin / p.tile_units;  // (PACK: the unit's kv head)
    int ui = WIN ? unit_lin / p.BHkv : unit_lin % p.tile_units;
    int part = 0, parts = 1;
    BwdUnit u = {};
    if constexpr (PACK) {
        griddep_wait();
        if (threadIdx.x == 0) griddep_launch_dependents();
        __shared__ BwdUnit unit;
        if (warp == 2) bwd_pack_unit(p, unit_lin, lane, &unit);
        __syncthreads();
        u = unit;
        if (!u.live) return;
        bh = u.h;
        ui = u.kt;
        part = u.part;
        parts = u.parts;
    }
    const int Nq = PACK ? u.s.n : p.Nq, Nk = PACK ? u.s.m : p.Nk;
    if constexpr (WIN && !PACK) {
        const int sink_units = p.sink_tiles * p.sink_parts;
        const bool sink = ui < sink_units;
        parts = sink ? p.sink_parts : p.parts;
        if (!sink) ui -= sink_units;
        part = ui % parts;
        ui = ui / parts + (sink ? 0 : p.sink_tiles);
    }
    int kts[2], h0s[2], ns[2];
    int nt = 1;
    kts[0] = ui;
    if (p.pair_tiles && p.k_tiles - 1 - ui != ui) {
        kts[1] = p.k_tiles - 1 - ui;
        nt = 2;
    } else {
        kts[1] = ui;
    }
    if constexpr (WIN) bwd_steps_win(p, Nq, Nk, kts[0], h0s[0], ns[0]);
    else bwd_steps(p, kts[0], h0s[0], ns[0]);
    if (nt == 2) bwd_steps(p, kts[1], h0s[1], ns[1]);
    else ns[1] = 0, h0s[1] = 0;
    // WIN: this part's steps, s0 .. s1 - 1 of the group's ns[0] * group, as
    // passes over consecutive heads from head_first on.
    int s0 = 0, s1 = 0, head_first = 0;
    if constexpr (WIN) {
        const int all = ns[0] * p.group;
        const int each = (all + parts - 1) / parts;
        s0 = min(part * each, all);
        s1 = min(s0 + each, all);
        head_first = ns[0] > 0 ? s0 / ns[0] : 0;
        nt = s1 > s0 ? (s1 - 1) / ns[0] - head_first + 1 : 1;
    }
    const int n_all = WIN ? s1 - s0 : ns[0] + ns[1];
    // The second tile reuses K/V, dV and dK only if both tiles have steps.
    const bool handoff = !WIN && nt == 2 && ns[0] > 0 && ns[1] > 0;
    // Pass tt of a CTA: its key tile, first step and number of steps; the head
    // of Q, dO and the accumulator.
    auto KT = [&](int tt) { return WIN ? kts[0] : kts[tt]; };
    auto HB = [&](int tt) { return max(s0 - (head_first + tt) * ns[0], 0); };
    auto H0 = [&](int tt) { return WIN ? h0s[0] + HB(tt) : h0s[tt]; };
    auto NS = [&](int tt) {
        return WIN ? max(0, min(s1 - (head_first + tt) * ns[0], ns[0]) - HB(tt)) : ns[tt];
    };
    auto ZQ = [&](int tt) {
        return PACK ? bh * p.group + head_first + tt
                    : WIN ? (bh / p.Hkv) * p.H + (bh % p.Hkv) * p.group + head_first + tt : bh;
    };
    auto ROW0 = [&](int tt) {
        return PACK ? static_cast<size_t>(ZQ(tt)) * p.rows_pad + pad_row(u.s.q0, u.b)
                    : static_cast<size_t>(ZQ(tt)) * p.Nq_pad;
    };

    if (threadIdx.x == 0) {
        mbar_init(bar(L::BAR_KV), 1);
        mbar_init(bar(L::BAR_KVFREE), 1);
        mbar_init(bar(L::BAR_ACCFREE), L::COMPUTE_WARPS);
        for (int st = 0; st < L::STAGES; ++st) {
            mbar_init(bar(L::BAR_QFULL + st), 1);
            mbar_init(bar(L::BAR_QEMPTY + st), 1);
        }
        for (int b = 0; b < L::BUFS; ++b) {
            mbar_init(bar(L::BAR_SFULL + b), 1);
            mbar_init(bar(L::BAR_PREADY + b), L::COMPUTE_WARPS);
            mbar_init(bar(L::BAR_DQFULL + b), 1);
            mbar_init(bar(L::BAR_DQREAD + b), L::READOUT_ACTIVE);
        }
        mbar_init(bar(L::BAR_DRAIN), 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&p.tm_q);
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
        tma_prefetch_desc(&p.tm_do);
    }
    if (warp == 1) {
        tmem_alloc(sbase + L::MISC_OFF, 512);
        tmem_relinquish();
    }
    if constexpr (D == 64) {
        // The zero second chunk of K (head dims 64-127 of dQ^T's A operand),
        // written through the generic proxy and fenced for the MMAs. Only the
        // first chunk is ever loaded.
        const uint32_t z = sbase + L::K_OFF + L::KV_CHUNK + 32u * threadIdx.x;
        static_assert(L::THREADS * 32 == L::KV_CHUNK, "one 32-byte piece per thread");
        st_shared_v4(z, 0u, 0u, 0u, 0u);
        st_shared_v4(z + 16, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (warp == 0 && n_all > 0) {
        // ------------------------------------------------------------ producer
        const bool leader = elect_one();
        bool ok = true;
        int issued = 0;    // global steps whose Q/dO loads were issued
        int kv_loads = 0;
        for (int tt = 0; tt < nt && ok; ++tt) {
            const int n = NS(tt);
            if (n == 0) continue;
            const int zq = ZQ(tt);
            const size_t row0 = ROW0(tt);
            if (!WIN && kv_loads > 0)  // the previous tile's MMAs are done with K and V
                ok = __all_sync(0xffffffffu, bwd_wait(bar(L::BAR_KVFREE), (kv_loads - 1) & 1, p, abort_flag,
                                                      kStatusWaitKvEmpty));
            if (!ok) break;
            if (leader && (!WIN || tt == 0)) {
                const int k0 = (PACK ? u.s.k0 : 0) + KT(tt) * kBwdKeys;
                mbar_arrive_expect_tx(bar(L::BAR_KV), 2 * L::V_BYTES);
                for (int c = 0; c < L::CHUNKS; ++c) {
                    tma_load_3d(sbase + L::K_OFF + c * L::KV_CHUNK, &p.tm_k, bar(L::BAR_KV), 64 * c, k0, bh);
                    tma_load_3d(sbase + L::V_OFF + c * L::KV_CHUNK, &p.tm_v, bar(L::BAR_KV), 64 * c, k0, bh);
                }
            }
            if (!WIN || tt == 0) ++kv_loads;
            for (int h = 0; h < n && ok; ++h) {
                const int G = issued;
                const int st = G % L::STAGES;
                if (G >= L::STAGES)
                    ok = __all_sync(0xffffffffu, bwd_wait(bar(L::BAR_QEMPTY + st), ((G / L::STAGES) - 1) & 1, p,
                                                          abort_flag, kStatusWaitKvEmpty));
                if (!ok) break;
                if (leader) {
                    const int q0 = (H0(tt) + h) * kBwdHalf;
                    const uint32_t sb = sbase + L::STAGE_OFF + st * L::STAGE_BYTES;
                    const uint32_t rb = sbase + L::ROWS_OFF + st * 2 * L::ROWS_BYTES;
                    mbar_arrive_expect_tx(bar(L::BAR_QFULL + st), L::STAGE_BYTES + 2 * L::ROWS_BYTES);
                    const int y = (PACK ? u.s.q0 : 0) + q0;
                    for (int c = 0; c < L::CHUNKS; ++c) {
                        tma_load_3d(sb + L::Q_IN + c * L::QH_CHUNK, &p.tm_q, bar(L::BAR_QFULL + st), 64 * c, y, zq);
                        tma_load_3d(sb + L::DO_IN + c * L::QH_CHUNK, &p.tm_do, bar(L::BAR_QFULL + st), 64 * c, y,
                                    zq);
                    }
                    bulk_load(rb + L::NL_IN, p.nlse2 + row0 + q0, L::ROWS_BYTES, bar(L::BAR_QFULL + st));
                    bulk_load(rb + L::ND_IN, p.ndd + row0 + q0, L::ROWS_BYTES, bar(L::BAR_QFULL + st));
                }
                issued = G + 1;
            }
        }
        if (ok) {
            // The issuer's last slot releases: no commit arrival may still be in
            // flight when the CTA exits.
            for (int G = max(0, n_all - L::STAGES); G < n_all && ok; ++G)
                ok = __all_sync(0xffffffffu, bwd_wait(bar(L::BAR_QEMPTY + G % L::STAGES), (G / L::STAGES) & 1, p,
                                                      abort_flag, kStatusWaitKvEmpty));
        } else {
            if (kv_loads > 0) bwd_wait(bar(L::BAR_KV), (kv_loads - 1) & 1, p, abort_flag, kStatusWaitDrain, false);
            for (int G = max(0, issued - L::STAGES); G < issued; ++G)
                bwd_wait(bar(L::BAR_QFULL + G % L::STAGES), (G / L::STAGES) & 1, p, abort_flag,
                         kStatusWaitDrain, false);
        }
    } else if (warp == 1 && n_all > 0) {
        // ------------------------------------------------------------ MMA issuer
        const bool leader = elect_one();
        auto wait_all = [&](uint32_t b, uint32_t parity, unsigned what) {
            return __all_sync(0xffffffffu, bwd_wait(b, parity, p, abort_flag, what));
        };
        constexpr uint32_t IDESC_S = make_idesc_bf16(128, kBwdHalf, false, false);  // S^T, dP^T
        constexpr uint32_t IDESC_ACC = make_idesc_bf16(128, L::DH, false, true);    // dV, dK (this CTA's part)
        constexpr uint32_t IDESC_DQ = make_idesc_bf16(128, kBwdHalf, true, true);   // dQ^T
        // K-major operands (8-row groups 1024 bytes apart); MN-major ones with
        // their 64-element chunks KV_CHUNK (K as A of dQ^T) or QH_CHUNK (Q, dO
        // as B of dK, dV) apart; dS^T is one 64-query chunk.
        const uint64_t kmaj0 = make_sdesc_sw128(sbase, 16, 1024);
        const uint64_t kmn0 = make_sdesc_sw128(sbase, L::KV_CHUNK, 1024);
        const uint64_t qmn0 = make_sdesc_sw128(sbase, L::QH_CHUNK, 1024);
        const uint32_t kmaj_lo = static_cast<uint32_t>(kmaj0), kmaj_hi = static_cast<uint32_t>(kmaj0 >> 32);
        const uint32_t kmn_lo = static_cast<uint32_t>(kmn0), kmn_hi = static_cast<uint32_t>(kmn0 >> 32);
        const uint32_t qmn_lo = static_cast<uint32_t>(qmn0), qmn_hi = static_cast<uint32_t>(qmn0 >> 32);
        auto desc = [](uint32_t lo, uint32_t hi, uint32_t off) -> uint64_t {
            return (static_cast<uint64_t>(hi) << 32) | (lo + (off >> 4));
        };
        // S^T_G = K Q_G^T and dP^T_G = V dO_G^T into buffer G % BUFS (lanes = keys,
        // 64 query columns each), reading ring slot G % STAGES; first, from
        // G = BUFS on, the readout group must have taken that buffer's dQ^T of BUFS
        // steps back out. `rows`: the step's queries that the sequence has (PACK).
        auto clear_rows = [&](uint32_t tile, int from, int rows) {  // rows from .. rows - 1 of 128 bytes
            for (int at = from * 128 + lane * 16; at < rows * 128; at += 512)
                st_shared_v4(sbase + tile + at, 0u, 0u, 0u, 0u);
        };
        auto issue_sdp = [&](int G, int rows) -> bool {
            if (G >= L::BUFS) {
                if (!wait_all(bar(L::BAR_DQREAD + G % L::BUFS), (G / L::BUFS - 1) & 1, kStatusWaitO)) return false;
            }
            const int st = G % L::STAGES;
            if (!wait_all(bar(L::BAR_QFULL + st), (G / L::STAGES) & 1, kStatusWaitQ)) return false;
            tc_fence_after();
            const uint32_t sb = L::STAGE_OFF + st * L::STAGE_BYTES;
            if constexpr (PACK) {
                if (rows < kBwdHalf) {
                    for (int c = 0; c < 2 * L::CHUNKS; ++c) clear_rows(sb + c * L::QH_CHUNK, rows, kBwdHalf);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            const uint32_t col = L::BUF_COL(G % L::BUFS);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t in_a = (kk & 3) * 32 + (kk >> 2) * L::KV_CHUNK;
                const uint32_t in_b = (kk & 3) * 32 + (kk >> 2) * L::QH_CHUNK;
                const uint64_t ak = desc(kmaj_lo, kmaj_hi, L::K_OFF + in_a);
                const uint64_t av = desc(kmaj_lo, kmaj_hi, L::V_OFF + in_a);
                const uint64_t bq = desc(kmaj_lo, kmaj_hi, sb + L::Q_IN + in_b);
                const uint64_t bdo = desc(kmaj_lo, kmaj_hi, sb + L::DO_IN + in_b);
                if (leader) {
                    umma_ss(tmem + col, ak, bq, IDESC_S, kk > 0 ? 1u : 0u);
                    umma_ss(tmem + col + L::DP_IN, av, bdo, IDESC_S, kk > 0 ? 1u : 0u);
                }
            }
            if (leader) umma_commit(bar(L::BAR_SFULL + G % L::BUFS));
            return true;
        };
        // dV += P^T_G dO_G, dK += dS^T_G Q_G (A from TMEM: 16 queries = 8 packed
        // columns, each 32-query chunk packed into the first 16 of its own 32;
        // B MN-major, 16 query rows = 2048 bytes), then dQ^T_G = K^T dS^T_G
        // over the buffer's S^T columns (after the dV MMAs that read P^T
        // there, in issue order): A = K MN-major (M = head dim), B = dS^T
        // MN-major (N = queries), 16 keys = 2048 bytes per MMA. `first`: the
        // tile's first step, which starts dV and dK.
        auto issue_vkq = [&](int G, bool first) -> bool {
            const int b = G % L::BUFS;
            if (!wait_all(bar(L::BAR_PREADY + b), (G / L::BUFS) & 1, kStatusWaitP)) return false;
            tc_fence_after();
            const int st = G % L::STAGES;
            // B of dV and dK: this CTA's head-dim part of dO_G and Q_G.
            const uint32_t sb = L::STAGE_OFF + st * L::STAGE_BYTES + hd * L::DH_CHUNKS * L::QH_CHUNK;
            const uint32_t col = L::BUF_COL(b);
#pragma unroll
            for (int kk = 0; kk < kBwdHalf / 16; ++kk) {
                const uint32_t acc = (!first || kk > 0) ? 1u : 0u;
                const uint32_t pcol = col + 32 * (kk >> 1) + 8 * (kk & 1);
                const uint64_t bdo = desc(qmn_lo, qmn_hi, sb + L::DO_IN + kk * 2048);
                const uint64_t bq = desc(qmn_lo, qmn_hi, sb + L::Q_IN + kk * 2048);
                if (leader) {
                    umma_ts(tmem + L::DV_COL, tmem + pcol, bdo, IDESC_ACC, acc);
                    umma_ts(tmem + L::DK_COL, tmem + pcol + L::DP_IN, bq, IDESC_ACC, acc);
                }
            }
            if (leader) umma_commit(bar(L::BAR_QEMPTY + st));
            const uint32_t dsb = L::DS_OFF + b * L::DS_BYTES;
#pragma unroll
            for (int kk = 0; kk < kBwdKeys / 16; ++kk) {
                // A: this CTA's head-dim part of K (M = 128 head dims).
                const uint64_t a = desc(kmn_lo, kmn_hi, L::K_OFF + hd * L::DH_CHUNKS * L::KV_CHUNK + kk * 2048);
                const uint64_t bds = desc(qmn_lo, qmn_hi, dsb + kk * 2048);
                if (leader) umma_ss(tmem + col, a, bds, IDESC_DQ, kk > 0 ? 1u : 0u);
            }
            if (leader) umma_commit(bar(L::BAR_DQFULL + b));
            return true;
        };
        bool ok = true;
        // The MMAs of n steps, in an order that leaves the compute and readout groups
        // another step's work while one step's MMAs run.
        auto run = [&](int n, auto&& sdp, auto&& vkq) {
            if constexpr (L::BUFS == 3) {
                // S^T and dP^T two steps ahead, into the buffer whose dQ^T was read out
                // while the last step's MMAs ran: the issuer never waits for a readout.
                ok = sdp(0);
                if (ok && n > 1) ok = sdp(1);
                for (int a = 0; a < n && ok; ++a) {
                    ok = vkq(a);
                    if (ok && a + 2 < n) ok = sdp(a + 2);
                }
            } else if constexpr (L::STAGES >= 3) {
                ok = sdp(0);
                if (ok && n > 1) ok = sdp(1);
                for (int a = 0; a < n && ok; a += 2) {
                    ok = vkq(a);
                    if (ok && a + 1 < n) ok = vkq(a + 1);
                    // The next pair's S^T and dP^T.
                    for (int h = a + 2; h < a + 4 && h < n && ok; ++h) ok = sdp(h);
                }
            } else {
                // One stage: step G + 1's Q and dO load once step G's dV and dK
                // MMAs have read the stage, so its S^T and dP^T follow step G's
                // MMAs.
                ok = sdp(0);
                for (int h = 0; h < n && ok; ++h) {
                    ok = vkq(h);
                    if (ok && h + 1 < n) ok = sdp(h + 1);
                }
            }
        };
        if constexpr (PACK || L::BUFS == 3) {
            ok = wait_all(bar(L::BAR_KV), 0, kStatusWaitKvFull);
            if (ok) tc_fence_after();
            if constexpr (PACK) {
                const int keys = Nk - KT(0) * kBwdKeys;
                if (ok && keys < kBwdKeys) {
                    for (int c = 0; c < L::CHUNKS; ++c) {
                        clear_rows(L::K_OFF + c * L::KV_CHUNK, keys, kBwdKeys);
                        clear_rows(L::V_OFF + c * L::KV_CHUNK, keys, kBwdKeys);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            // The passes' steps follow one another without a break. `pos`: the next
            // step's place among the head's.
            int pos = s0 % ns[0];
            auto sdp = [&](int G) {
                const int rows = PACK ? Nq - (h0s[0] + pos) * kBwdHalf : kBwdHalf;
                if (++pos == ns[0]) pos = 0;
                return issue_sdp(G, rows);
            };
            if (ok) run(n_all, sdp, [&](int G) { return issue_vkq(G, G == 0); });
        } else {
            int gb = 0;        // global index of the tile's first step
            int kv_loads = 0;
            for (int tt = 0; tt < nt && ok; ++tt) {
                const int n = NS(tt);
                if (n == 0) continue;
                if (!WIN || tt == 0) {
                    ok = wait_all(bar(L::BAR_KV), kv_loads & 1, kStatusWaitKvFull);
                    ++kv_loads;
                }
                if (!ok) break;
                tc_fence_after();
                // The tile's first MMA into dV and dK waits until the compute group
                // has read the previous tile's out of TMEM.
                auto vkq = [&](int h) -> bool {
                    if (h == 0 && tt > 0 && handoff) {
                        if (!wait_all(bar(L::BAR_ACCFREE), 0, kStatusWaitO)) return false;
                        tc_fence_after();
                    }
                    return issue_vkq(gb + h, h == 0 && (!WIN || tt == 0));
                };
                run(n, [&](int h) { return issue_sdp(gb + h, kBwdHalf); }, vkq);
                // K and V free for the next tile once every MMA so far is done.
                if (ok && tt == 0 && handoff && leader) umma_commit(bar(L::BAR_KVFREE));
                gb += n;
            }
        }
        if (leader) umma_commit(bar(L::BAR_DRAIN));
        bwd_wait(bar(L::BAR_DRAIN), 0, p, abort_flag, kStatusWaitDrain, false);
    } else if (warp >= 4 && warp < 4 + L::COMPUTE_WARPS) {
        // ------------------------------------------------------------ compute group
        const int quarter = warp & 3;
        const int g = (warp - 4) >> 2;       // 32-query chunk of each step
        const int r = quarter * 32 + lane;   // TMEM lane: key row
        const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
        const int off = p.causal_br ? Nk - Nq : 0;
        const float sl2 = p.scale_log2;
        bool ok = true;
        int gb = 0;
        for (int tt = 0; tt < nt && ok; ++tt) {
            const int n = NS(tt);
            const int h0 = H0(tt);
            const int k0 = KT(tt) * kBwdKeys;
            const int key = k0 + r;
            const bool key_ok = key < Nk;
            const bool key_tail = k0 + kBwdKeys > Nk;
            for (int h = 0; h < n && ok; ++h) {
                const int G = gb + h;
                const int b = G % L::BUFS;
                const int q0 = (h0 + h) * kBwdHalf;
                // Every entry of the step is visible unless the tile holds missing
                // keys or (causal) crosses the diagonal; padded query rows carry
                // -inf as -LSE log2e, so their P is 0 either way.
                bool masked = key_tail || (p.causal && k0 + kBwdKeys - 1 > q0 + off);
                if constexpr (WIN)  // the step's last row has left the window of the tile's first key
                    masked = masked || (p.window > 0 && k0 <= q0 + kBwdHalf - 1 + off - p.window);
                ok = __all_sync(0xffffffffu, bwd_wait(bar(L::BAR_SFULL + b), (G / L::BUFS) & 1, p, abort_flag, kStatusWaitS));
                if (!ok) break;
                tc_fence_after();
                const uint32_t col = L::BUF_COL(b) + 32 * g;
                uint32_t sraw[32], draw[32];
                tmem_ld32(tmem + lane_field + col, sraw);
                tmem_ld32(tmem + lane_field + col + L::DP_IN, draw);
                tmem_wait_ld();
                // The slot's -LSE log2e and -D for this chunk's 32 queries (the S^T
                // commit implies the slot's loads landed: the issuer waited for them).
                const uint32_t rb = sbase + L::ROWS_OFF + (G % L::STAGES) * 2 * L::ROWS_BYTES;
                const uint32_t nl = rb + L::NL_IN + 128 * g;
                const uint32_t nd = rb + L::ND_IN + 128 * g;
                uint32_t pk[16], dk[16];
                if (masked) {
                    // Key row `key` is visible to query q iff key <= q + off.
                    const int lim = p.causal ? key - off - q0 - 32 * g : -1;
                    if constexpr (WIN) {
                        const int end = p.window > 0 && key >= p.sinks ? lim + p.window : 64;
                        bwd_chunk<true, true>(sraw, draw, nl, nd, sl2, lim, key_ok, pk, dk, end);
                    } else {
                        bwd_chunk<true>(sraw, draw, nl, nd, sl2, lim, key_ok, pk, dk);
                    }
                } else {
                    bwd_chunk<false>(sraw, draw, nl, nd, sl2, 0, true, pk, dk);
                }
                // P^T and dS^T over the first 16 of the chunk's own 32 columns (no
                // other warp reads or writes them).
                tmem_st16(tmem + lane_field + col, pk);
                tmem_st16(tmem + lane_field + col + L::DP_IN, dk);
                // dS^T into shared memory: row r, queries 32 g .. 32 g + 31 of the
                // step's 128-byte row (128-byte swizzle).
                const uint32_t line = sbase + L::DS_OFF + b * L::DS_BYTES + r * 128;
                const uint32_t swz = static_cast<uint32_t>(r & 7);
#pragma unroll
                for (int uu = 0; uu < 4; ++uu) {
                    const uint32_t u = static_cast<uint32_t>(g * 4 + uu);
                    st_shared_v4(line + ((u ^ swz) << 4), dk[4 * uu], dk[4 * uu + 1], dk[4 * uu + 2], dk[4 * uu + 3]);
                }
                fence_proxy_async_smem();
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::BAR_PREADY + b));
            }
            // dK (scaled) and dV of this key row, columns DH/2 g .. DH/2 g + DH/2 - 1 of
            // the CTA's head-dim part, once every MMA of the tile has finished (its
            // last dQ^T commit covers them all); zero when no query step sees the
            // key tile. tcgen05.ld is warp-collective: the loads run for the whole
            // warp (`ok` is warp-uniform), and only the stores check that the key
            // exists. After the first of two tiles the TMEM reads are handed back
            // (ACCFREE) before the stores.
            const bool last_pass = !WIN || tt == nt - 1;
            if (ok && n > 0 && last_pass) {
                const int G = gb + n - 1;
                ok = __all_sync(0xffffffffu, bwd_wait(bar(L::BAR_DQFULL + G % L::BUFS), (G / L::BUFS) & 1, p, abort_flag,
                                                      kStatusWaitO));
                if (ok) tc_fence_after();
            }
            if (ok && last_pass) {
                // This CTA's head-dim part of the key row's dK and dV.
                size_t at_k = (static_cast<size_t>(bh) * p.Nk + key) * D, at_v = at_k;
                if constexpr (PACK) {
                    at_k = static_cast<size_t>(u.s.k0 + key) * p.dk_stride + static_cast<size_t>(bh) * D;
                    at_v = static_cast<size_t>(u.s.k0 + key) * p.dv_stride + static_cast<size_t>(bh) * D;
                }
                __nv_bfloat16* dkp = static_cast<__nv_bfloat16*>(p.dk) + at_k + hd * L::DH;
                __nv_bfloat16* dvp = static_cast<__nv_bfloat16*>(p.dv) + at_v + hd * L::DH;
#pragma unroll 1
                for (int j = 0; j < L::DH_CHUNKS; ++j) {
                    const int cc = L::DH_CHUNKS * g + j;
                    uint32_t kr[32], vr[32];
                    if (n > 0) {
                        tmem_ld32(tmem + lane_field + L::DK_COL + cc * 32, kr);
                        tmem_ld32(tmem + lane_field + L::DV_COL + cc * 32, vr);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) kr[e] = vr[e] = 0u;
                    }
                    if (j == L::DH_CHUNKS - 1 && tt == 0 && handoff) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(L::BAR_ACCFREE));
                    }
                    if constexpr (WIN) {
                        if (parts > 1) {
                            const size_t unit = PACK ? static_cast<size_t>(u.sums + part)
                                                     : static_cast<size_t>(unit_lin);
                            float* at = p.dkv_part + (unit * 2 * kBwdKeys + r) * D + hd * L::DH + cc * 32;
                            uint4* dk4 = reinterpret_cast<uint4*>(at);
                            uint4* dv4 = reinterpret_cast<uint4*>(at + kBwdKeys * D);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                dk4[e] = make_uint4(kr[4 * e], kr[4 * e + 1], kr[4 * e + 2], kr[4 * e + 3]);
                                dv4[e] = make_uint4(vr[4 * e], vr[4 * e + 1], vr[4 * e + 2], vr[4 * e + 3]);
                            }
                            continue;
                        }
                    }
                    uint32_t kp[16], vp[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        kp[e] = pack_bf16x2(__uint_as_float(kr[2 * e]) * p.scale, __uint_as_float(kr[2 * e + 1]) * p.scale);
                        vp[e] = pack_bf16x2(__uint_as_float(vr[2 * e]), __uint_as_float(vr[2 * e + 1]));
                    }
                    if (key_ok) {
                        uint4* dk4 = reinterpret_cast<uint4*>(dkp + cc * 32);
                        uint4* dv4 = reinterpret_cast<uint4*>(dvp + cc * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            dk4[e] = make_uint4(kp[4 * e], kp[4 * e + 1], kp[4 * e + 2], kp[4 * e + 3]);
                            dv4[e] = make_uint4(vp[4 * e], vp[4 * e + 1], vp[4 * e + 2], vp[4 * e + 3]);
                        }
                    }
                }
            }
            gb += n;
        }
    } else if (warp >= 4 + L::COMPUTE_WARPS && (warp & 3) < L::READOUT_ACTIVE && n_all > 0) {
        // ------------------------------------------------------------ dQ readout
        // Lane r = head dim r; columns = the step's 64 queries. The TMEM loads
        // finish before the buffer is released; the atomic adds follow. The
        // accumulator has rows for whole 128-row tiles, so every add is in
        // bounds. (Warps 12-15 cover lane quarters 0-3: warp & 3 is the
        // quarter.)
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
        bool ok = true;
        int gb = 0;
        for (int tt = 0; tt < nt && ok; ++tt) {
            const int n = NS(tt);
            const size_t row0 = ROW0(tt);
            for (int h = 0; h < n && ok; ++h) {
                const int G = gb + h;
                const int b = G % L::BUFS;
                ok = __all_sync(0xffffffffu, bwd_wait(bar(L::BAR_DQFULL + b), (G / L::BUFS) & 1, p, abort_flag, kStatusWaitO));
                if (!ok) break;
                tc_fence_after();
                uint32_t lo[32], hi[32];
                tmem_ld32(tmem + lane_field + L::BUF_COL(b), lo);
                tmem_ld32(tmem + lane_field + L::BUF_COL(b) + 32, hi);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::BAR_DQREAD + b));
                float* dst = p.dq_acc + (row0 + static_cast<size_t>(H0(tt) + h) * kBwdHalf) * D + hd * L::DH + r;
#pragma unroll
                for (int e = 0; e < 32; ++e) atomicAdd(dst + e * D, __uint_as_float(lo[e]));
#pragma unroll
                for (int e = 0; e < 32; ++e) atomicAdd(dst + (32 + e) * D, __uint_as_float(hi[e]));
            }
            gb += n;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Per padded query row (one warp per row, D / 32 columns per lane): -D_i =
// -sum_c dO_ic O_ic (fp32 from bf16), -LSE log2e, and a zeroed dQ accumulator
// row. Rows past Nq get -inf and 0; so do rows whose LSE is -inf (no key).
template <int D>
__global__ void __launch_bounds__(256) fa_bwd_pre_kernel(const __nv_bfloat16* __restrict__ o,
                                                         const __nv_bfloat16* __restrict__ dout,
                                                         const float* __restrict__ lse,
                                                         float* __restrict__ nlse2, float* __restrict__ ndd,
                                                         float* __restrict__ dq_acc, long long rows_pad,
                                                         int Nq, int Nq_pad) {
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows_pad) return;
    const long long bh = row / Nq_pad;
    const int q = static_cast<int>(row - bh * Nq_pad);
    float s = 0.f, nl = -INFINITY;
    if (q < Nq) {
        const size_t src_row = static_cast<size_t>(bh) * Nq + q;
        const size_t base = src_row * D + lane * (D / 32);
        const __nv_bfloat162* o2 = reinterpret_cast<const __nv_bfloat162*>(o + base);
        const __nv_bfloat162* d2 = reinterpret_cast<const __nv_bfloat162*>(dout + base);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
            const float2 a = __bfloat1622float2(o2[e]);
            const float2 b = __bfloat1622float2(d2[e]);
            s = fmaf(a.x, b.x, s);
            s = fmaf(a.y, b.y, s);
        }
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const float l = lse[src_row];
        nl = (l == -INFINITY) ? -INFINITY : -(l * kLog2e);
    }
    if (lane == 0) {
        ndd[row] = -s;
        nlse2[row] = nl;
    }
    float* z = dq_acc + static_cast<size_t>(row) * D + lane * (D / 32);
    if constexpr (D >= 128) {
#pragma unroll
        for (int e = 0; e < D / 128; ++e) reinterpret_cast<float4*>(z)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        *reinterpret_cast<float2*>(z) = make_float2(0.f, 0.f);
    }
}

// Rows that see at most this many keys form D from P and dP (below).
constexpr int kFewKeys = 16;

// fa_bwd_pre_kernel under a window. A row that sees few keys has an O about as
// large as a single V row, and where one weight is near 1 that key's dP - D is
// a small difference: the rounding of bf16 O then dominates dS (measured on
// N(0, 1) inputs with two visible keys: dQ, dK off by 3.8e-3 against 2.3e-3).
// Such a row gets D = sum_j P_j dP_j from q, K, V and dO in fp32, at two dot
// products per key; from about sixteen keys on the rounding averages out, and D
// comes from O as in the dense backward (an error of up to 2^-8 sum_c |dO_c O_c|,
// the larger part of what dQ and dK are off by).
template <int D>
__global__ void __launch_bounds__(256) fa_bwd_win_pre_kernel(const __nv_bfloat16* __restrict__ q,
                                                             const __nv_bfloat16* __restrict__ k,
                                                             const __nv_bfloat16* __restrict__ v,
                                                             const __nv_bfloat16* __restrict__ o,
                                                             const __nv_bfloat16* __restrict__ dout,
                                                             const float* __restrict__ lse,
                                                             const __grid_constant__ BwdParams p, long long rows_pad) {
    // D / 8 threads per row, sixteen bytes of it each.
    constexpr int LANES = D / 8;
    const long long row = static_cast<long long>(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    if (row >= rows_pad) return;  // rows_pad is a multiple of 128: whole blocks
    const unsigned mine = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << ((threadIdx.x & 31) & ~(LANES - 1));
    const long long bh = row / p.Nq_pad;
    const int i = static_cast<int>(row - bh * p.Nq_pad);
    auto load = [&](const __nv_bfloat16* src, float (&x)[8]) {
        const uint4 u = reinterpret_cast<const uint4*>(src)[lane];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    };
    auto dot = [&](const float (&a)[8], const float (&b)[8]) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(a[e], b[e], s);
        for (int w = LANES / 2; w > 0; w >>= 1) s += __shfl_xor_sync(mine, s, w);
        return s;
    };
    float4* z = reinterpret_cast<float4*>(p.dq_acc + static_cast<size_t>(row) * D);
    z[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    z[lane + LANES] = make_float4(0.f, 0.f, 0.f, 0.f);
    float dd = 0.f, nl = -INFINITY;
    if (i < p.Nq) {
        const size_t src_row = static_cast<size_t>(bh) * p.Nq + i;
        const float l = lse[src_row];
        float g[8], a[8];
        load(dout + src_row * D, g);
        nl = (l == -INFINITY) ? -INFINITY : -(l * kLog2e);
        // Visible keys: [0, ns) and [w0, pos].
        const int pos = i + p.Nk - p.Nq;
        const int w0 = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        const int ns = min(p.sinks, w0);
        const int seen = pos < 0 ? 0 : ns + pos + 1 - w0;
        if (seen > kFewKeys) {
            load(o + src_row * D, a);
            dd = dot(a, g);
        } else if (nl != -INFINITY) {
            load(q + src_row * D, a);
            const long long b = bh / p.H;
            const size_t base = static_cast<size_t>(b * p.Hkv + (bh - b * p.H) / p.group) * p.Nk;
            for (int n = 0; n < seen; ++n) {
                const size_t key = base + (n < ns ? n : w0 + (n - ns));
                float kr[8], vr[8];
                load(k + key * D, kr);
                load(v + key * D, vr);
                dd = fmaf(ex2(fmaf(dot(a, kr), p.scale_log2, nl)), dot(g, vr), dd);
            }
        }
    }
    if (lane == 0) {
        const_cast<float*>(p.ndd)[row] = -dd;
        const_cast<float*>(p.nlse2)[row] = nl;
    }
}

// dQ = scale * accumulator, to bf16: one warp per query row, D / 32 columns
// per lane, reading the accumulator's padded rows.
template <int D>
__global__ void __launch_bounds__(256) fa_bwd_dq_kernel(const float* __restrict__ acc,
                                                        __nv_bfloat16* __restrict__ dq, long long rows,
                                                        int Nq, int Nq_pad, float scale) {
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const long long bh = row / Nq;
    const long long arow = bh * Nq_pad + (row - bh * Nq);
    const float* src = acc + static_cast<size_t>(arow) * D + lane * (D / 32);
    __nv_bfloat16* dst = dq + static_cast<size_t>(row) * D + lane * (D / 32);
    if constexpr (D >= 128) {
#pragma unroll
        for (int e = 0; e < D / 128; ++e) {
            const float4 a = reinterpret_cast<const float4*>(src)[e];
            __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * scale, a.y * scale);
            __nv_bfloat162 hi = __floats2bfloat162_rn(a.z * scale, a.w * scale);
            uint2 out;
            out.x = *reinterpret_cast<uint32_t*>(&lo);
            out.y = *reinterpret_cast<uint32_t*>(&hi);
            reinterpret_cast<uint2*>(dst)[e] = out;
        }
    } else {
        const float2 a = *reinterpret_cast<const float2*>(src);
        *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(a.x * scale, a.y * scale);
    }
}

// The last launch under a window: dQ as fa_bwd_dq_kernel, and behind its rows
// the keys of the tiles whose dK and dV were left in parts, added part by part
// (a fixed order) and written in bf16. D / 8 threads per row, 16-byte stores.
template <int D>
__global__ void __launch_bounds__(256) fa_bwd_win_post_kernel(const __grid_constant__ BwdParams p,
                                                              __nv_bfloat16* __restrict__ dq, long long q_rows,
                                                              long long k_rows) {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    constexpr int LANES = D / 8;
    const long long lin = static_cast<long long>(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
    const int c = (threadIdx.x % LANES) * 8;
    float x[8];
    auto add = [&](const float* src, bool first) {
        const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
        const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = first ? y[e] : x[e] + y[e];
    };
    auto put = [&](__nv_bfloat16* dst, float f) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f),
                                                    pack_bf16x2(x[4] * f, x[5] * f), pack_bf16x2(x[6] * f, x[7] * f));
    };
    if (lin < q_rows) {
        const long long bh = lin / p.Nq;
        add(p.dq_acc + (bh * p.Nq_pad + (lin - bh * p.Nq)) * D + c, true);
        put(dq + lin * D + c, p.scale);
        return;
    }
    long long k = lin - q_rows;
    if (k >= k_rows) return;
    // Row k of (tensor, tile in parts, kv head, key of the tile).
    const int r = static_cast<int>(k % kBwdKeys);
    k /= kBwdKeys;
    const int bh = static_cast<int>(k % p.BHkv);
    k /= p.BHkv;
    const int is_v = static_cast<int>(k & 1);
    const int first = p.sink_parts > 1 ? 0 : p.sink_tiles;  // first tile in parts
    const int kt = first + static_cast<int>(k >> 1);
    const int key = kt * kBwdKeys + r;
    if (key >= p.Nk) return;
    const bool sink = kt < p.sink_tiles;
    const int parts = sink ? p.sink_parts : p.parts;
    const long long unit0 = sink ? static_cast<long long>(kt) * parts
                                 : static_cast<long long>(p.sink_tiles) * p.sink_parts +
                                       static_cast<long long>(kt - p.sink_tiles) * parts;
    for (int i = 0; i < parts; ++i)
        add(p.dkv_part + ((((unit0 + i) * p.BHkv + bh) * 2 + is_v) * kBwdKeys + r) * D + c, i == 0);
    put(static_cast<__nv_bfloat16*>(is_v ? p.dv : p.dk) + (static_cast<long long>(bh) * p.Nk + key) * D + c,
        is_v ? 1.f : p.scale);
}

// The sequence that padded row `row` (a multiple of 64) or, by `tiles`, key tile `row`
// belongs to, found by one warp: its number, or -1. Sixty-four padded rows or a tile
// have one sequence at most.
__device__ __forceinline__ int bwd_pack_find(const BwdParams& p, long long row, bool tiles, int lane, PackedSeq& s) {
    // (128 sequences at a time: their loads are in flight together.)
    for (int c = 0; c < p.seqs.B; c += 128) {
        PackedSeq y[4];
        bool here[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int b = c + 32 * u + lane;
            y[u] = {0, 0, 0, 0};
            here[u] = b < p.seqs.B && packed_seq(p.seqs, b, y[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int b = c + 32 * u + lane;
            if (here[u]) {
                const long long at = row - (tiles ? tile_slot(y[u].k0, b) : pad_row(y[u].q0, b));
                here[u] = at >= 0 && at < (tiles ? key_tiles(y[u]) : y[u].n);
            }
            const unsigned who = __ballot_sync(0xffffffffu, here[u]);
            if (who) {
                const int from = __ffs(who) - 1;
                s.q0 = __shfl_sync(0xffffffffu, y[u].q0, from);
                s.n = __shfl_sync(0xffffffffu, y[u].n, from);
                s.k0 = __shfl_sync(0xffffffffu, y[u].k0, from);
                s.m = __shfl_sync(0xffffffffu, y[u].m, from);
                return c + 32 * u + from;
            }
        }
    }
    return -1;
}
struct BwdPlace {
    PackedSeq s;
    int b;
};

// Sixteen bytes of a row in fp32, and the dot product over a row's LANES threads.
__device__ __forceinline__ void bwd_unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ void bwd_load8(const __nv_bfloat16* src, float (&x)[8]) {
    bwd_unpack8(*reinterpret_cast<const uint4*>(src), x);
}
template <int LANES>
__device__ __forceinline__ float bwd_dot(unsigned mine, const float (&a)[8], const float (&b)[8]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(a[e], b[e], s);
    for (int w = LANES / 2; w > 0; w >>= 1) s += __shfl_xor_sync(mine, s, w);
    return s;
}

// fa_bwd_win_pre_kernel on packed sequences: a block takes 64 padded rows, which are one
// sequence's, of block_heads heads. Bound by memory (O and dO are read, the fp32 dQ is
// zeroed; 63 us, 6.8 TB/s, for 24 documents of up to 2047 tokens, 16 heads of 128): four
// rows of a thread are loaded before the first is used. Rows that see few keys come in a
// loop of their own behind, four keys at a time: one key after the other they took longer
// than all other rows (the same documents: 88 us).
// (pre_heads(D) heads where those blocks fill the SMs twice, one where they do not: 240
// tokens in twelve documents, 14 heads of 128, 13 us with two.)
constexpr int pre_heads(int d) { return d == 64 ? 4 : d == 128 ? 2 : 1; }
template <int D>
__global__ void __launch_bounds__(256, 4) fa_bwd_pack_pre_kernel(const __nv_bfloat16* __restrict__ q,
                                                                 const __nv_bfloat16* __restrict__ k,
                                                                 const __nv_bfloat16* __restrict__ v,
                                                                 const __nv_bfloat16* __restrict__ o,
                                                                 const __nv_bfloat16* __restrict__ dout,
                                                                 const float* __restrict__ lse,
                                                                 const __grid_constant__ BwdParams p) {
    constexpr int LANES = D / 8, ROWS = 256 / LANES, PASSES = kBwdHalf / ROWS, U = 4;
    __shared__ BwdPlace place;
    const int lane = threadIdx.x % LANES, c = lane * 8, r0 = threadIdx.x / LANES;
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    // (Heads fastest: the blocks at hand read whole tokens.)
    const unsigned parts = (p.H + p.block_heads - 1) / p.block_heads;
    const long long first = static_cast<long long>(blockIdx.x / parts) * kBwdHalf;
    const int h0 = static_cast<int>(blockIdx.x % parts) * p.block_heads, h1 = min(p.H, h0 + p.block_heads);
    if (threadIdx.x < 32) {
        BwdPlace x = {};
        x.b = bwd_pack_find(p, first, false, threadIdx.x, x.s);
        if (threadIdx.x == 0) place = x;
    }
    __syncthreads();
    if (place.b < 0) return;
    const PackedSeq s = place.s;
    const int i0 = static_cast<int>(first - pad_row(s.q0, place.b));
    const unsigned mine = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << ((threadIdx.x & 31) & ~(LANES - 1));
    const uint32_t zero[8] = {};
    const bool wide = reinterpret_cast<uintptr_t>(p.dq_acc) % 32 == 0;  // whole sectors a store
    // Visible keys of row i: [0, ns) and [w0, w0 + seen - ns).
    auto visible = [&](int i, int& ns, int& w0) {
        const int pos = i + s.m - s.n;
        w0 = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        ns = min(p.sinks, w0);
        return pos < 0 ? 0 : ns + pos + 1 - w0;
    };
    bool few = false;
    const int items = PASSES * (h1 - h0);
#pragma unroll 1
    for (int e0 = 0; e0 < items; e0 += U) {
        uint4 g_raw[U], o_raw[U];
        float l[U];
#pragma unroll
        for (int e = 0; e < U; ++e) {
            const int x = min(e0 + e, items - 1), h = h0 + x / PASSES;
            const long long token = s.q0 + min(i0 + r0 + x % PASSES * ROWS, s.n - 1);
            l[e] = lse[static_cast<long long>(h) * p.seqs.total_q + token];
            g_raw[e] = *reinterpret_cast<const uint4*>(dout + token * p.do_stride + static_cast<long long>(h) * D + c);
            o_raw[e] = *reinterpret_cast<const uint4*>(o + (token * p.H + h) * D + c);
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
            const int x = e0 + e, h = h0 + x / PASSES, r = r0 + x % PASSES * ROWS, i = i0 + r;
            if (x >= items) break;  // (the whole block)
            const long long row = static_cast<long long>(h) * p.rows_pad + first + r;
            float* sums = p.dq_acc + row * D + c;
            if (i < s.n && wide) {
                st_global_v8(sums, zero);
            } else if (i < s.n) {
                reinterpret_cast<float4*>(sums)[0] = reinterpret_cast<float4*>(sums)[1] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float g[8], a[8];
            bwd_unpack8(g_raw[e], g);
            bwd_unpack8(o_raw[e], a);
            const float dd = bwd_dot<LANES>(mine, a, g);
            int ns, w0;
            const int seen = visible(i, ns, w0);
            const bool by_keys = i < s.n && seen > 0 && seen <= kFewKeys;
            few = few || by_keys;
            if (lane == 0) {
                if (!by_keys) const_cast<float*>(p.ndd)[row] = i < s.n && seen > 0 ? -dd : 0.f;
                const_cast<float*>(p.nlse2)[row] = i < s.n && l[e] != -INFINITY ? -(l[e] * kLog2e) : -INFINITY;
            }
        }
    }
    if (!few) return;
#pragma unroll 1
    for (int e = 0; e < PASSES * (h1 - h0); ++e) {
        const int h = h0 + e / PASSES, r = r0 + e % PASSES * ROWS, i = i0 + r;
        int ns, w0;
        const int seen = visible(i, ns, w0);
        if (i >= s.n || seen == 0 || seen > kFewKeys) continue;
        const long long token = s.q0 + i, head = static_cast<long long>(h / p.group) * D + c;
        const float l = lse[static_cast<long long>(h) * p.seqs.total_q + token];
        const float nl = l == -INFINITY ? -INFINITY : -(l * kLog2e);
        float a[8], g[8], dd = 0.f;
        bwd_load8(q + token * p.q_stride + static_cast<long long>(h) * D + c, a);
        bwd_load8(dout + token * p.do_stride + static_cast<long long>(h) * D + c, g);
#pragma unroll 1
        for (int n0 = 0; n0 < seen; n0 += 4) {
            uint4 k_raw[4], v_raw[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int n = min(n0 + u, seen - 1);
                const long long key = s.k0 + (n < ns ? n : w0 + (n - ns));
                k_raw[u] = *reinterpret_cast<const uint4*>(k + key * p.k_stride + head);
                v_raw[u] = *reinterpret_cast<const uint4*>(v + key * p.v_stride + head);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float kr[8], vr[8];
                bwd_unpack8(k_raw[u], kr);
                bwd_unpack8(v_raw[u], vr);
                const float w = ex2(fmaf(bwd_dot<LANES>(mine, a, kr), p.scale_log2, nl)), dp = bwd_dot<LANES>(mine, g, vr);
                if (n0 + u < seen) dd = fmaf(w, dp, dd);
            }
        }
        if (lane == 0) const_cast<float*>(p.ndd)[static_cast<long long>(h) * p.rows_pad + first + r] = -dd;
    }
}

// The last launch on packed sequences: a block writes dQ of 64 padded rows of block_heads
// heads, or, behind those, dK or dV of kPostKeys keys of a tile whose sums were left in
// parts, added part by part in order. Four rows of a thread, or parts of one, are loaded
// before the first is used; bound by memory (38000 tokens in six documents, 16 heads of 64,
// window 1024, 4 sinks: 35 us, 6.7 TB/s; with a head and a tile per block, a row after the
// other, 61). Rows that belong to no sequence get zeros where the call asks for it.
constexpr int kPostKeys = 32;
template <int D>
__global__ void __launch_bounds__(256, 4) fa_bwd_pack_post_kernel(const __grid_constant__ BwdParams p,
                                                                  __nv_bfloat16* __restrict__ dq, long long q_blocks) {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
    constexpr int LANES = D / 8, ROWS = 256 / LANES, PASSES = kBwdHalf / ROWS, U = 4;
    __shared__ BwdPlace place;
    const int lane = threadIdx.x % LANES, c = lane * 8, r0 = threadIdx.x / LANES;
    auto put = [&](__nv_bfloat16* dst, const float (&x)[8], float f) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f),
                                                    pack_bf16x2(x[4] * f, x[5] * f), pack_bf16x2(x[6] * f, x[7] * f));
    };
    auto get = [&](const float* src, float (&x)[8]) {
        const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    };
    const bool is_q = blockIdx.x < q_blocks;
    long long lin = is_q ? blockIdx.x : blockIdx.x - q_blocks;
    const int heads = is_q ? (p.H + p.block_heads - 1) / p.block_heads : 2 * p.Hkv * (kBwdKeys / kPostKeys);
    const int h = static_cast<int>(lin % heads);
    lin /= heads;
    // The padded row, or the tile by its number (the sinks' alone: by theirs).
    const long long first = is_q ? lin * kBwdHalf : lin;
    if (threadIdx.x < 32) {
        BwdPlace x = {};
        if (is_q || p.parts > 1) {
            x.b = bwd_pack_find(p, first, !is_q, threadIdx.x, x.s);
        } else {
            x.b = static_cast<int>(lin / p.sink_tiles);
            packed_seq(p.seqs, x.b, x.s);
        }
        if (threadIdx.x == 0) place = x;
    }
    __syncthreads();
    const PackedSeq s = place.s;
    if (place.b >= 0 && is_q) {
        const int i0 = static_cast<int>(first - pad_row(s.q0, place.b));
        const int h0 = h * p.block_heads, items = PASSES * (min(p.H, h0 + p.block_heads) - h0);
#pragma unroll 1
        for (int e0 = 0; e0 < items; e0 += U) {
            float x[U][8];
#pragma unroll
            for (int e = 0; e < U; ++e) {
                const int at = min(e0 + e, items - 1), r = min(r0 + at % PASSES * ROWS, s.n - 1 - i0);
                get(p.dq_acc + (static_cast<long long>(h0 + at / PASSES) * p.rows_pad + first + r) * D + c, x[e]);
            }
#pragma unroll
            for (int e = 0; e < U; ++e) {
                const int at = e0 + e, r = r0 + at % PASSES * ROWS;
                if (at < items && i0 + r < s.n)
                    put(dq + (static_cast<long long>(s.q0) + i0 + r) * p.dq_stride +
                            static_cast<long long>(h0 + at / PASSES) * D + c,
                        x[e], p.scale);
            }
        }
    } else if (place.b >= 0) {
        const int kt = static_cast<int>(p.parts > 1 ? first - tile_slot(s.k0, place.b) : lin % p.sink_tiles);
        const int quarter = h % (kBwdKeys / kPostKeys), head = h / (kBwdKeys / kPostKeys) >> 1;
        const int is_v = h / (kBwdKeys / kPostKeys) & 1;
        const int parts = kt < p.sink_tiles ? p.sink_parts : p.parts;
        const long long sums = bwd_sums(p, s, place.b, kt, head);
#pragma unroll 1
        for (int r = quarter * kPostKeys + r0; r < (quarter + 1) * kPostKeys && parts > 1; r += ROWS) {
            const int key = kt * kBwdKeys + r;
            if (key >= s.m) break;
            float x[8];
#pragma unroll 1
            for (int n0 = 0; n0 < parts; n0 += U) {
                float y[U][8];
#pragma unroll
                for (int n = 0; n < U; ++n)
                    get(p.dkv_part + (((sums + min(n0 + n, parts - 1)) * 2 + is_v) * kBwdKeys + r) * D + c, y[n]);
#pragma unroll
                for (int n = 0; n < U; ++n)
                    if (n0 + n < parts)
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = n0 + n == 0 ? y[n][e] : x[e] + y[n][e];
            }
            put(static_cast<__nv_bfloat16*>(is_v ? p.dv : p.dk) +
                    (static_cast<long long>(s.k0) + key) * (is_v ? p.dv_stride : p.dk_stride) +
                    static_cast<long long>(head) * D + c,
                x, is_v ? 1.f : p.scale);
        }
    }
    if (!p.fill) return;
    auto zeros = [&](__nv_bfloat16* dst, const int* cu, int total, int n, long long stride) {
        const int c0 = cu[0], c1 = cu[p.seqs.B];
        if (!(0 <= c0 && c0 <= c1 && c1 <= total)) return;
        for (long long i = blockIdx.x; i < total - (c1 - c0); i += gridDim.x)
            for (int e = threadIdx.x; e < n * LANES; e += 256)
                *reinterpret_cast<uint4*>(dst + (i < c0 ? i : i + (c1 - c0)) * stride + e * 8) = make_uint4(0u, 0u, 0u, 0u);
    };
    zeros(dq, p.seqs.cu_q, p.seqs.total_q, p.H, p.dq_stride);
    zeros(static_cast<__nv_bfloat16*>(p.dk), p.seqs.cu_k, p.seqs.total_k, p.Hkv, p.dk_stride);
    zeros(static_cast<__nv_bfloat16*>(p.dv), p.seqs.cu_k, p.seqs.total_k, p.Hkv, p.dv_stride);
}

// How a windowed backward is cut into parts (host side). Each step of a CTA
// takes about as long as any other, a CTA's start and end about kUnitCost
// steps, leaving and adding partial sums kPartCost more; 152 CTAs run at once.
// `parts` minimises the waves' length, and a sink tile is cut into pieces of
// about the same number of steps.
struct BwdParts {
    int sink_tiles, sink_parts, parts;
    size_t part_floats;  // floats of the partial sums
};
BwdParts bwd_parts(int B, int H, int Hkv, int Nq, int Nk, int d, int window, int sinks) {
    constexpr long long kUnitCost = 4, kPartCost = 6;
    BwdParts c = {0, 1, 1, 0};
    const int halves = d == 256 ? 2 : 1;
    const long long k_tiles = (static_cast<long long>(Nk) + kBwdKeys - 1) / kBwdKeys;
    const long long all = (static_cast<long long>(Nq) + kBwdHalf - 1) / kBwdHalf;
    const long long G = H / Hkv, heads = static_cast<long long>(B) * Hkv;
    if (window > 0) c.sink_tiles = static_cast<int>(std::min(k_tiles, (static_cast<long long>(sinks) + kBwdKeys - 1) / kBwdKeys));
    const long long reach = window > 0 ? std::min(all, (kBwdKeys + static_cast<long long>(window) + kBwdHalf - 2) / kBwdHalf + 1) : all;
    const long long steps = G * reach, sink_steps = G * all;
    long long best = -1;
    for (int p = 1; p <= 16 && (p == 1 || p <= steps); ++p) {
        const long long piece = std::max(8ll, (steps + p - 1) / p);
        const long long sp = c.sink_tiles > 0 ? std::min(64ll, (sink_steps + piece - 1) / piece) : 1;
        const long long ctas = heads * halves * ((k_tiles - c.sink_tiles) * p + c.sink_tiles * sp);
        const long long longest = std::max((steps + p - 1) / p, c.sink_tiles > 0 ? (sink_steps + sp - 1) / sp : 0);
        const long long cost = (ctas + 151) / 152 * (longest + kUnitCost + (p > 1 ? kPartCost : 0));
        if (best < 0 || cost < best) {
            best = cost;
            c.parts = p;
            c.sink_parts = static_cast<int>(sp);
        }
    }
    const long long units = heads * (c.sink_tiles * static_cast<long long>(c.sink_parts) +
                                     (c.parts > 1 ? (k_tiles - c.sink_tiles) * c.parts : 0));
    if (c.parts > 1 || (c.sink_tiles > 0 && c.sink_parts > 1))
        c.part_floats = static_cast<size_t>(units) * 2 * kBwdKeys * d;
    return c;
}

// The same for a packed batch, whose lengths the host does not know: the longest CTA
// against an even share of the steps that sequences of the longest length would have.
struct BwdPackParts {
    int sink_tiles, sink_parts, parts;
    long long tiles, slots;  // key tiles at most, and the numbers that tile_slot gives them
    size_t part_floats;
};
BwdPackParts bwd_pack_parts(int B, int total_k, int max_q, int max_k, int H, int Hkv, int d, int window, int sinks) {
    // (At d = 256 a step takes more than twice as long, a CTA's start and end do not.)
    const double kUnitCost = d == 256 ? 2. : 4., kPartCost = d == 256 ? 2. : 6.;
    BwdPackParts c = {0, 1, 1, 0, 0, 0};
    const long long halves = d == 256 ? 2 : 1, G = H / Hkv, seqs = std::min(B, total_k);
    const long long k_tiles = (static_cast<long long>(max_k) + kBwdKeys - 1) / kBwdKeys;
    c.tiles = std::min((total_k + seqs * (kBwdKeys - 1)) / kBwdKeys, seqs * k_tiles);
    c.slots = total_k / kBwdKeys + static_cast<long long>(B) + 1;
    const long long all = (static_cast<long long>(max_q) + kBwdHalf - 1) / kBwdHalf;
    if (window > 0)
        c.sink_tiles = static_cast<int>(std::min(k_tiles, (static_cast<long long>(sinks) + kBwdKeys - 1) / kBwdKeys));
    const long long reach =
        window > 0 ? std::min(all, (kBwdKeys + static_cast<long long>(window) + kBwdHalf - 2) / kBwdHalf + 1) : all;
    const long long steps = G * reach, sink_steps = G * all, heads = Hkv * halves;
    const long long sink_units = std::min(c.tiles, seqs * c.sink_tiles), others = c.tiles - sink_units;
    // (Without a window half of a causal sequence's steps are not there.)
    const double work = static_cast<double>(heads) * (static_cast<double>(others) * steps * (window > 0 ? 1. : 0.5) +
                                                      static_cast<double>(sink_units) * sink_steps * 0.5);
    double best = -1.;
    for (long long p = 1; p <= 16 && (p == 1 || p <= steps); ++p) {
        const long long piece = std::max(8ll, (steps + p - 1) / p);
        const long long sp = c.sink_tiles > 0 ? std::min(64ll, (sink_steps + piece - 1) / piece) : 1;
        const double extra = kUnitCost + (p > 1 ? kPartCost : 0.);
        const double longest = static_cast<double>(
            std::max((steps + p - 1) / p, c.sink_tiles > 0 ? (sink_steps + sp - 1) / sp : 0)) + extra;
        const double even = (work + static_cast<double>(heads) * (others * p + sink_units * sp) * extra) / 152.;
        const double cost = std::max(longest, even);
        if (best < 0. || cost < 0.9 * best) best = cost, c.parts = static_cast<int>(p), c.sink_parts = static_cast<int>(sp);
    }
    const long long sums = (c.sink_parts > 1 ? static_cast<long long>(B) * c.sink_tiles * Hkv * c.sink_parts : 0) +
                           (c.parts > 1 ? c.slots * Hkv * c.parts : 0);
    c.part_floats = static_cast<size_t>(sums) * 2 * kBwdKeys * d;
    return c;
}
long long packed_rows_pad(int total_q, int B) { return (total_q + 64ll * (B + 1ll) + 127) / 128 * 128; }
// Units of a kv head at most: no more sinks' tiles than the sequences have, the others for
// the rest.
long long bwd_pack_units(const BwdPackParts& c, int B, int total_k) {
    return std::min(c.tiles, static_cast<long long>(std::min(B, total_k)) * c.sink_tiles) * c.sink_parts + c.tiles * c.parts;
}
// The tiles whose sums the last launch adds up (numbers of tile_slot, or the sinks' alone).
long long bwd_pack_summed(const BwdPackParts& c, int B) {
    return c.parts > 1 ? c.slots : c.sink_parts > 1 ? static_cast<long long>(B) * c.sink_tiles : 0;
}
// Whether the three launches' searches through the sequences end in time: the first and the
// last launch's blocks go through half of them on average.
bool bwd_pack_search(const BwdPackParts& c, int B, int total_q, int total_k, int H, int Hkv, int d) {
    const long long rows = packed_rows_pad(total_q, B) / kBwdHalf * ((H + pre_heads(d) - 1) / pre_heads(d));
    return packed_search(bwd_pack_units(c, B, total_k) * Hkv * (d == 256 ? 2 : 1) + rows +
                             bwd_pack_summed(c, B) * Hkv * (kBwdKeys / kPostKeys), B);
}

}  // namespace

template <int D>
cudaError_t launch_bwd_pre(const void* o, const void* dout, const float* lse, float* nlse2, float* ndd,
                           float* dq_acc, int BH, int Nq, int Nq_pad, cudaStream_t stream) {
    const long long rows_pad = static_cast<long long>(BH) * Nq_pad;
    const long long blocks = (rows_pad + 7) / 8;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    fa_bwd_pre_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dout), lse, nlse2, ndd,
        dq_acc, rows_pad, Nq, Nq_pad);
    return cudaGetLastError();
}

template <int D, bool WIN, bool PACK = false>
cudaError_t launch_bwd_main(const BwdParams& p, cudaStream_t stream) {
    using L = LayoutBwd<D, WIN>;
    // Kernel attributes belong to the context: set once per device and context.
    static ContextCache<int> attr_set;
    int done = 0;
    const cudaError_t e = attr_set.get(&done, [](int* out) {
        *out = 1;
        return cudaFuncSetAttribute(fa_bwd_kernel<D, WIN, PACK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(L::ALLOC_BYTES));
    });
    if (e != cudaSuccess) return e;
    const long long units = PACK  ? p.tile_units * static_cast<long long>(p.Hkv)
                            : WIN ? static_cast<long long>(p.BHkv) * (p.sink_tiles * p.sink_parts +
                                                                      (p.k_tiles - p.sink_tiles) * p.parts)
                                : static_cast<long long>(p.BH) * p.tile_units;
    const long long ctas = units * L::HALVES;
    if (ctas < 1 || ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    // (Packed sequences: its start under the first launch's end, 1 to 3 us less at any size.)
    if constexpr (PACK)
        return launch_dependent(fa_bwd_kernel<D, WIN, PACK>, dim3(static_cast<unsigned>(ctas)), L::THREADS, L::ALLOC_BYTES,
                                stream, p);
    fa_bwd_kernel<D, WIN, PACK><<<static_cast<unsigned>(ctas), L::THREADS, L::ALLOC_BYTES, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_bwd_dq(const float* dq_acc, void* dq, int BH, int Nq, int Nq_pad, float scale,
                          cudaStream_t stream) {
    const long long rows = static_cast<long long>(BH) * Nq;
    const long long blocks = (rows + 7) / 8;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    fa_bwd_dq_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        dq_acc, static_cast<__nv_bfloat16*>(dq), rows, Nq, Nq_pad, scale);
    return cudaGetLastError();
}

// The three launches of one backward call at head dim D.
template <int D>
cudaError_t launch_bwd(const BwdParams& p, const void* o, const void* dout, const float* lse, void* dq,
                       cudaStream_t stream) {
    cudaError_t e = launch_bwd_pre<D>(o, dout, lse, const_cast<float*>(p.nlse2), const_cast<float*>(p.ndd),
                                      p.dq_acc, p.BH, p.Nq, p.Nq_pad, stream);
    if (e == cudaSuccess) e = launch_bwd_main<D, false>(p, stream);
    if (e == cudaSuccess) e = launch_bwd_dq<D>(p.dq_acc, dq, p.BH, p.Nq, p.Nq_pad, p.scale, stream);
    return e;
}

// The same under a window.
template <int D>
cudaError_t launch_bwd_win(const BwdParams& p, const void* q, const void* k, const void* v, const void* o,
                           const void* dout, const float* lse, void* dq, cudaStream_t stream) {
    const long long rows_pad = static_cast<long long>(p.BH) * p.Nq_pad;
    const long long per_pre = 256 / (D / 8);
    const long long blocks = (rows_pad + per_pre - 1) / per_pre;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    using T = const __nv_bfloat16*;
    fa_bwd_win_pre_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        static_cast<T>(q), static_cast<T>(k), static_cast<T>(v), static_cast<T>(o), static_cast<T>(dout), lse, p,
        rows_pad);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_bwd_main<D, true>(p, stream);
    if (e != cudaSuccess) return e;
    const long long q_rows = static_cast<long long>(p.BH) * p.Nq;
    const long long in_parts = (p.sink_parts > 1 ? p.sink_tiles : 0) + (p.parts > 1 ? p.k_tiles - p.sink_tiles : 0);
    const long long k_rows = in_parts * 2 * p.BHkv * kBwdKeys;
    const long long per_block = 256 / (D / 8);
    const long long post = (q_rows + k_rows + per_block - 1) / per_block;
    if (post > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_dependent(fa_bwd_win_post_kernel<D>, dim3(static_cast<unsigned>(post)), 256, 0, stream, p,
                            static_cast<__nv_bfloat16*>(dq), q_rows, k_rows);
}

// The three launches on packed sequences.
template <int D>
cudaError_t launch_bwd_pack(BwdParams p, const void* q, const void* k, const void* v, const void* o,
                            const void* dout, const float* lse, void* dq, long long k_tiles, cudaStream_t stream) {
    using T = const __nv_bfloat16*;
    p.block_heads = pre_heads(D);
    long long blocks = p.rows_pad / kBwdHalf * ((p.H + p.block_heads - 1) / p.block_heads);
    if (blocks < 2 * 152) p.block_heads = 1, blocks = p.rows_pad / kBwdHalf * p.H;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    // A grid below the number of SMs starts under the end of the one before it (9 to 320
    // tokens: up to 2 us less; 534 tokens of 32 heads, 176 blocks: 2.5 us more, 24 documents
    // 16).
    cudaError_t e;
    if (blocks <= 128) {
        e = launch_dependent(fa_bwd_pack_pre_kernel<D>, dim3(static_cast<unsigned>(blocks)), 256, 0, stream, static_cast<T>(q),
                             static_cast<T>(k), static_cast<T>(v), static_cast<T>(o), static_cast<T>(dout), lse, p);
    } else {
        fa_bwd_pack_pre_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
            static_cast<T>(q), static_cast<T>(k), static_cast<T>(v), static_cast<T>(o), static_cast<T>(dout), lse, p);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = launch_bwd_main<D, true, true>(p, stream);
    if (e != cudaSuccess) return e;
    const long long q_blocks = blocks;
    const long long k_blocks = k_tiles * 2 * p.Hkv * (kBwdKeys / kPostKeys);
    if (q_blocks + k_blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_dependent(fa_bwd_pack_post_kernel<D>, dim3(static_cast<unsigned>(q_blocks + k_blocks)), 256, 0, stream,
                            p, static_cast<__nv_bfloat16*>(dq), q_blocks);
}

}  // namespace fa

extern "C" {

size_t fa_bwd_workspace_bytes(int B, int H, int Nq, int d) {
    if (B < 1 || H < 1 || Nq < 1 || (d != 64 && d != 128 && d != 256)) return 0;
    const size_t rows_pad = static_cast<size_t>(B) * H * ((static_cast<size_t>(Nq) + 127) / 128 * 128);
    return rows_pad * (static_cast<size_t>(d) + 2) * sizeof(float);
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                 const float* lse, void* dq, void* dk, void* dv, void* workspace, int B, int H,
                 int Nq, int Nk, int d, float scale, int causal, cudaStream_t stream) {
    fa_status s = fa::check_common(q, k, v, B, H, Nq, Nk, d, scale);
    if (s != FA_OK) return s;
    // Query rows are padded to whole 128-row tiles and key tiles counted in
    // int: both lengths must leave room for that rounding.
    if (Nq > 0x7fffffff - 127 || Nk > 0x7fffffff - 127) return FA_ERR_SHAPE;
    if (d != 64 && d != 128 && d != 256) return FA_ERR_HEADDIM;
    if (!fa::valid_causal(causal)) return FA_ERR_CAUSAL;
    if (!o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_NULL;
    if (!fa::aligned(o, 16) || !fa::aligned(dout, 16) || !fa::aligned(lse, 4) ||
        !fa::aligned(dq, 16) || !fa::aligned(dk, 16) || !fa::aligned(dv, 16))
        return FA_ERR_ALIGN;
    if (!workspace || !fa::aligned(workspace, 16)) return FA_ERR_WORKSPACE;
    const int BH = B * H;
    const int Nq_pad = (Nq + 127) / 128 * 128;
    const size_t rows_pad = static_cast<size_t>(BH) * Nq_pad;
    float* dq_acc = static_cast<float*>(workspace);
    float* nlse2 = dq_acc + rows_pad * d;
    float* ndd = nlse2 + rows_pad;
    fa::BwdParams p;
    std::memset(&p, 0, sizeof(p));
    if (!fa::encode_rows_map(&p.tm_q, q, d, Nq, BH, 64) ||
        !fa::encode_rows_map(&p.tm_k, k, d, Nk, BH, 128) ||
        !fa::encode_rows_map(&p.tm_v, v, d, Nk, BH, 128) ||
        !fa::encode_rows_map(&p.tm_do, dout, d, Nq, BH, 64))
        return FA_ERR_CUDA;
    p.nlse2 = nlse2;
    p.ndd = ndd;
    p.dq_acc = dq_acc;
    p.dk = dk;
    p.dv = dv;
    p.BH = BH;
    p.Nq = Nq;
    p.Nk = Nk;
    p.Nq_pad = Nq_pad;
    p.causal = causal ? 1 : 0;
    p.causal_br = (causal == FA_CAUSAL_BOTTOM_RIGHT) ? 1 : 0;
    p.k_tiles = (Nk + 127) / 128;
    // Under a causal mask a key tile's query steps fall with its index: pairs
    // of tiles from both ends give every CTA about the same work (measured on
    // the C2 shape: 1-2.5 % faster at d = 64 and 128; at d = 256, whose single
    // Q/dO stage leaves the hand-over between the tiles exposed, 2 % slower).
    p.pair_tiles = (causal && d <= 128) ? 1 : 0;
    p.tile_units = p.pair_tiles ? (p.k_tiles + 1) / 2 : p.k_tiles;
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_limit = fa::kDefaultWaitLimit;
    if (fa::device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    const cudaError_t e = d == 64    ? fa::launch_bwd<64>(p, o, dout, lse, dq, stream)
                          : d == 128 ? fa::launch_bwd<128>(p, o, dout, lse, dq, stream)
                                     : fa::launch_bwd<256>(p, o, dout, lse, dq, stream);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_window_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d, int window, int sinks) {
    if (Nk < 1 || fa::check_window(H, Hkv, Nq, Nk, window, sinks) != FA_OK) return 0;
    const size_t base = fa_bwd_workspace_bytes(B, H, Nq, d);
    if (base == 0) return 0;
    return base + fa::bwd_parts(B, H, Hkv, Nq, Nk, d, window, sinks).part_floats * sizeof(float);
}

fa_status fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, void* workspace, int B, int H, int Hkv,
                        int Nq, int Nk, int d, float scale, int window, int sinks, cudaStream_t stream) {
    fa_status s = fa::check_common(q, k, v, B, H, Nq, Nk, d, scale);
    if (s != FA_OK) return s;
    s = fa::check_window(H, Hkv, Nq, Nk, window, sinks);
    if (s != FA_OK) return s;
    if (!o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_NULL;
    if (!fa::aligned(o, 16) || !fa::aligned(dout, 16) || !fa::aligned(lse, 4) || !fa::aligned(dq, 16) ||
        !fa::aligned(dk, 16) || !fa::aligned(dv, 16))
        return FA_ERR_ALIGN;
    if (!workspace || !fa::aligned(workspace, 16)) return FA_ERR_WORKSPACE;
    const int BH = B * H;
    const int Nq_pad = (Nq + 127) / 128 * 128;
    const size_t rows_pad = static_cast<size_t>(BH) * Nq_pad;
    float* dq_acc = static_cast<float*>(workspace);
    float* nlse2 = dq_acc + rows_pad * d;
    float* ndd = nlse2 + rows_pad;
    fa::BwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.BHkv = B * Hkv;
    if (!fa::encode_rows_map(&p.tm_q, q, d, Nq, BH, 64) || !fa::encode_rows_map(&p.tm_k, k, d, Nk, p.BHkv, 128) ||
        !fa::encode_rows_map(&p.tm_v, v, d, Nk, p.BHkv, 128) || !fa::encode_rows_map(&p.tm_do, dout, d, Nq, BH, 64))
        return FA_ERR_CUDA;
    p.nlse2 = nlse2;
    p.ndd = ndd;
    p.dq_acc = dq_acc;
    p.dk = dk;
    p.dv = dv;
    p.BH = BH;
    p.H = H;
    p.Hkv = Hkv;
    p.group = H / Hkv;
    p.Nq = Nq;
    p.Nk = Nk;
    p.Nq_pad = Nq_pad;
    p.causal = 1;
    p.causal_br = 1;
    p.window = window;
    p.sinks = sinks;
    p.k_tiles = (Nk + 127) / 128;
    p.tile_units = p.k_tiles;
    const fa::BwdParts c = fa::bwd_parts(B, H, Hkv, Nq, Nk, d, window, sinks);
    p.sink_tiles = c.sink_tiles;
    p.sink_parts = c.sink_parts;
    p.parts = c.parts;
    p.dkv_part = ndd + rows_pad;  // 16-byte aligned: rows_pad is a multiple of 128
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_limit = fa::kDefaultWaitLimit;
    if (fa::device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    const cudaError_t e = d == 64    ? fa::launch_bwd_win<64>(p, q, k, v, o, dout, lse, dq, stream)
                          : d == 128 ? fa::launch_bwd_win<128>(p, q, k, v, o, dout, lse, dq, stream)
                                     : fa::launch_bwd_win<256>(p, q, k, v, o, dout, lse, dq, stream);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_packed_workspace_bytes(int B, int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int H, int Hkv,
                                     int d, int window, int sinks) {
    const int none = 0;
    const fa_packed_batch c = {&none, &none, B, total_q, total_k, max_seqlen_q, max_seqlen_k};
    if (fa::check_packed(&c, H, Hkv, d, 1.f, window, sinks) != FA_OK) return 0;
    const size_t rows = static_cast<size_t>(fa::packed_rows_pad(total_q, B)) * H;
    const fa::BwdPackParts parts = fa::bwd_pack_parts(B, total_k, max_seqlen_q, max_seqlen_k, H, Hkv, d, window, sinks);
    if (!fa::bwd_pack_search(parts, B, total_q, total_k, H, Hkv, d)) return 0;
    return (rows * (static_cast<size_t>(d) + 2) + parts.part_floats) * sizeof(float);
}

fa_status fa_bwd_packed(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                        void* dq, void* dk, void* dv, void* workspace, const fa_packed_batch* batch, int H, int Hkv,
                        int d, const fa_packed_strides* strides, float scale, int window, int sinks, int fill,
                        cudaStream_t stream) {
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !strides) return FA_ERR_NULL;
    const fa_status s = fa::check_packed(batch, H, Hkv, d, scale, window, sinks);
    if (s != FA_OK) return s;
    for (const void* x : {q, k, v, o, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv)})
        if (!fa::aligned(x, 16)) return FA_ERR_ALIGN;
    if (!fa::aligned(lse, 4)) return FA_ERR_ALIGN;
    for (long long x : {strides->q, strides->dout, strides->dq})
        if (!fa::token_stride(x, H, d)) return FA_ERR_STRIDE;
    for (long long x : {strides->k, strides->v, strides->dk, strides->dv})
        if (!fa::token_stride(x, Hkv, d)) return FA_ERR_STRIDE;
    if (!workspace || !fa::aligned(workspace, 16)) return FA_ERR_WORKSPACE;
    const fa::BwdPackParts c = fa::bwd_pack_parts(batch->B, batch->total_k, batch->max_seqlen_q, batch->max_seqlen_k, H,
                                                  Hkv, d, window, sinks);
    if (!fa::bwd_pack_search(c, batch->B, batch->total_q, batch->total_k, H, Hkv, d)) return FA_ERR_SHAPE;
    fa::BwdParams p;
    std::memset(&p, 0, sizeof(p));
    if (!fa::encode_strided_tokens_map(&p.tm_q, q, d, batch->total_q, H, strides->q, fa::kBwdHalf) ||
        !fa::encode_strided_tokens_map(&p.tm_do, dout, d, batch->total_q, H, strides->dout, fa::kBwdHalf) ||
        !fa::encode_strided_tokens_map(&p.tm_k, k, d, batch->total_k, Hkv, strides->k, fa::kBwdKeys) ||
        !fa::encode_strided_tokens_map(&p.tm_v, v, d, batch->total_k, Hkv, strides->v, fa::kBwdKeys))
        return FA_ERR_CUDA;
    p.rows_pad = fa::packed_rows_pad(batch->total_q, batch->B);
    const size_t rows = static_cast<size_t>(p.rows_pad) * H;
    float* ws = static_cast<float*>(workspace);
    p.dq_acc = ws;
    p.nlse2 = ws + rows * d;
    p.ndd = p.nlse2 + rows;
    p.dkv_part = ws + rows * (static_cast<size_t>(d) + 2);  // 16-byte aligned: rows_pad is a multiple of 128
    p.dk = dk;
    p.dv = dv;
    p.H = H;
    p.Hkv = p.BHkv = Hkv;
    p.group = H / Hkv;
    p.causal = 1;
    p.causal_br = 1;
    p.window = window;
    p.sinks = sinks;
    p.seqs = {batch->cu_seqlens_q, batch->cu_seqlens_k, batch->B,           batch->total_q,
              batch->total_k,      batch->max_seqlen_q, batch->max_seqlen_k};
    p.q_stride = strides->q;
    p.k_stride = strides->k;
    p.v_stride = strides->v;
    p.do_stride = strides->dout;
    p.dq_stride = strides->dq;
    p.dk_stride = strides->dk;
    p.dv_stride = strides->dv;
    p.fill = fill ? 1 : 0;
    p.sink_tiles = c.sink_tiles;
    p.sink_parts = c.sink_parts;
    p.parts = c.parts;
    // Kv heads whose Q, dO and dQ sums (8 bytes a value) stay in L2 together are taken before
    // the next ones (32 heads of 128 without groups, eight documents of 2048: 1229 -> 950 us;
    // 16 heads of 256, four of 4096: 3047 -> 2580), where that leaves two waves of units, the
    // longest first (one document of 8192, 32 heads over 8, a head after the other: 1275 ->
    // 1516), and without a window, whose tiles' rows lie close together (986 -> 1001).
    const double head_bytes = 8. * d * p.group * batch->total_q;
    const int together = static_cast<int>(std::min<double>(Hkv, 64e6 / head_bytes));
    p.pack_heads = window > 0 || static_cast<double>(c.tiles) * c.parts * together < 2 * 152 ? Hkv : together;
    const long long units = fa::bwd_pack_units(c, batch->B, batch->total_k);
    if (units * Hkv * 2 > 0x7fffffffll) return FA_ERR_SHAPE;
    p.tile_units = static_cast<int>(units);
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_limit = fa::kDefaultWaitLimit;
    if (fa::device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    const long long summed = fa::bwd_pack_summed(c, batch->B);
    const cudaError_t e = d == 64    ? fa::launch_bwd_pack<64>(p, q, k, v, o, dout, lse, dq, summed, stream)
                          : d == 128 ? fa::launch_bwd_pack<128>(p, q, k, v, o, dout, lse, dq, summed, stream)
                                     : fa::launch_bwd_pack<256>(p, q, k, v, o, dout, lse, dq, summed, stream);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
