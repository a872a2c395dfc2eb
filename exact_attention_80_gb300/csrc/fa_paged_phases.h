// fa_paged_phases.h — which mbarrier phases the paged kernels wait for. Plain C++
// beside CUDA, so that the host can walk every order of completions.
//
// A wait for parity q passes when the barrier's phase in progress has the other
// parity: a barrier that is two phases on looks as it did before either of them.
// So a wait by parity is right only where the barrier can be at most one phase
// past the one that is waited for.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define FA_PHASES_FN __host__ __device__ __forceinline__
#else
#define FA_PHASES_FN inline
#endif

namespace fa {

// fa_paged_tc.cu, d = 256: the end of PV_j of n key tiles is told on barrier 0, phase
// j, but that of the last tile on barrier 1, phase 0. PV_j starts when all softmax
// warps have handed P_j over, so at step j, before that, barrier 0 is at most one
// phase past PV_{j-1}'s. Behind a warp's last arrival it is not: there only the last
// tile's own barrier tells anything.
FA_PHASES_FN int wide_pv_barrier(int j, int n) { return j == n - 1 ? 1 : 0; }
FA_PHASES_FN uint32_t wide_pv_parity(int j, int n) { return j == n - 1 ? 0u : static_cast<uint32_t>(j & 1); }

// fa_paged.cu: the copies of a warp's tile k complete phase k / stages of slot
// k % stages of its ring. At the wait for tile k the copies of the tiles up to
// ring_issued have started (tile k + stages follows when tile k's slot is free).
FA_PHASES_FN int ring_slot(int k, int stages) { return k % stages; }
FA_PHASES_FN uint32_t ring_parity(int k, int stages) { return static_cast<uint32_t>(k / stages & 1); }
FA_PHASES_FN int ring_issued(int k, int stages, int tiles) { return k + stages < tiles ? k + stages : tiles; }

}  // namespace fa
