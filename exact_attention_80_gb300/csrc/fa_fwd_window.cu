// fa_fwd_window.cu — fa_fwd_window: sliding-window attention with sinks and
// grouped heads; instantiations of the forward kernels (fa_fwd_win.cuh has what
// the window changes) and the C entry point.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa_fwd_kernel.cuh"

namespace fa {

cudaError_t launch_fwd_win_d64(const FwdParams& p, unsigned grid, cudaStream_t stream) {
    return launch_fwd<64, false, false, false, false, true>(p, grid, stream);
}
cudaError_t launch_fwd_win_d128(const FwdParams& p, unsigned grid, cudaStream_t stream) {
    return launch_fwd<128, false, false, false, false, true>(p, grid, stream);
}
cudaError_t launch_fwd_win_d64_persist(const FwdParams& p, unsigned grid, cudaStream_t stream) {
    return launch_fwd<64, false, false, true, false, true>(p, grid, stream);
}
cudaError_t launch_fwd_win_d128_persist(const FwdParams& p, unsigned grid, cudaStream_t stream) {
    return launch_fwd<128, false, false, true, false, true>(p, grid, stream);
}
cudaError_t launch_fwd_win_d256(const FwdParams& p, unsigned grid, cudaStream_t stream) {
    return launch_fwd<256, false, false, false, false, true>(p, grid, stream);
}

fa_status check_window(int H, int Hkv, int Nq, int Nk, int window, int sinks) {
    if (Hkv < 1) return FA_ERR_SHAPE;
    if (H < Hkv || H % Hkv) return FA_ERR_GROUP;
    // Positions and tile bounds are computed in int: room for a whole unit.
    if (Nq > 0x3fffffff || Nk > 0x3fffffff) return FA_ERR_SHAPE;
    if (window < 0 || window > 0x3fffffff || sinks < 0 || sinks > 0x3fffffff || (window == 0 && sinks != 0))
        return FA_ERR_WINDOW;
    return FA_OK;
}

namespace {

// Time of a call in steps of a CTA (one key tile, about 1.1 us): its waves of CTAs,
// four steps for a CTA's start and end, and for split keys the second launch and
// the partial states, which are written and read. Few rows over many keys leave
// most SMs idle otherwise (one row of 8 heads of 64 over 4096 keys, replayed from a
// graph: 36 us in one part, 9.2 in sixteen; 2 heads of 4096 rows, no window: 42 us,
// 29 in four).
int window_splits(long long units, long long tiles, long long rows, int d, int sms) {
    if (units >= sms) return 1;
    long long best = 1;
    double best_cost = -1., whole = 0.;
    for (long long s = 1; s <= std::min<long long>({tiles, 64, FA_MAX_SPLITS}); ++s) {
        const double waves = static_cast<double>((units * s + sms - 1) / sms);
        const double cost = waves * (static_cast<double>((tiles + s - 1) / s) + 4.) +
                            (s > 1 ? 3. + 0.05 * s + 1e-6 * static_cast<double>(s) * rows * d : 0.);
        if (best_cost < 0. || cost < best_cost) best = s, best_cost = cost;
        if (s == 1) whole = cost;
    }
    // (Less than a quarter is not worth a workspace and another order of sums.)
    return best_cost < 0.75 * whole ? static_cast<int>(best) : 1;
}
// Key tiles a unit of `rows` rows lists at most.
long long window_tiles(int Nk, int rows, int window, int sinks) {
    const long long all = (static_cast<long long>(Nk) + 127) / 128;
    return window > 0 ? std::min<long long>(all, (static_cast<long long>(window) + rows + 126) / 128 + 1 + (sinks + 127) / 128)
                      : all;
}

fa_status window_forward(const void* q, const void* k, const void* v, void* o, float* lse, float* workspace, int B,
                         int H, int Hkv, int Nq, int Nk, int d, float scale, int window, int sinks, int num_splits,
                         cudaStream_t stream) {
    const FwdConfig c = fwd_config(d);
    FwdParams p;
    std::memset(&p, 0, sizeof(p));
    const int BH = B * H;
    if (!encode_rows_map(&p.tm_q, q, d, Nq, BH, 128) || !encode_rows_map(&p.tm_k, k, d, Nk, B * Hkv, c.bn) ||
        !encode_rows_map(&p.tm_v, v, d, Nk, B * Hkv, c.bn))
        return FA_ERR_CUDA;
    if (!workspace && !encode_rows_map(&p.tm_o, o, d, Nq, BH, d == 256 ? 128 : 32)) return FA_ERR_CUDA;
    p.o = o;
    p.lse = lse;
    if (workspace) {
        const size_t rows = static_cast<size_t>(num_splits) * BH * Nq;
        p.ws_o = workspace;
        p.ws_m = p.ws_o + rows * d;
        p.ws_l = p.ws_m + rows;
        p.split_mode = 1;
    }
    p.BH = BH;
    p.H = H;
    p.Hkv = Hkv;
    p.group = H / Hkv;
    p.Nq = Nq;
    p.Nk = Nk;
    p.causal = 1;
    p.causal_br = 1;
    p.window = window;
    p.sinks = sinks;
    p.num_splits = num_splits;
    p.tiles_per_cta = c.q_tiles;
    const int rows = c.q_tiles * 128;
    p.n_units = (Nq + rows - 1) / rows;
    const long long ctas = static_cast<long long>(BH) * p.n_units * num_splits;
    if (ctas > 0x7fffffffll) return FA_ERR_SHAPE;
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) return FA_ERR_CUDA;
    p.head_group = std::max(1, std::min(BH, sms / p.n_units));
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o_scale = 1.f;
    p.wait_limit = kDefaultWaitLimit;
    if (device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    // Persistent CTAs where the units fill at least four waves (three if they list
    // four key tiles at most) and list few key tiles, as for the dense forward: the
    // start and end of a unit overlap its neighbours' (2 x 32 heads of 8192, d = 64,
    // us, persistent and not: window 1024 and 4 sinks 206 and 216, window 128 76 and
    // 105; 16 heads, d = 128, 3.4 waves: 77 and 76, window 128 29 and 35).
    const long long listed =
        window > 0 ? std::min<long long>((Nk + 127) / 128, (window + 126) / 128 + 2 + (sinks + 127) / 128)
                   : (Nk + 127) / 128;
    p.total_units = ctas;
    if (!workspace && d <= 128 && ctas >= (listed <= 4 ? 3ll : 4ll) * sms && listed <= 16) {
        const unsigned all = static_cast<unsigned>(sms);
        const cudaError_t e = d == 64 ? launch_fwd_win_d64_persist(p, all, stream)
                                      : launch_fwd_win_d128_persist(p, all, stream);
        return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    }
    const unsigned grid = static_cast<unsigned>(ctas);
    const cudaError_t e = d == 64    ? launch_fwd_win_d64(p, grid, stream)
                          : d == 128 ? launch_fwd_win_d128(p, grid, stream)
                                     : launch_fwd_win_d256(p, grid, stream);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Hkv, int Nq,
                        int Nk, int d, float scale, int window, int sinks, cudaStream_t stream) {
    fa_status s = fa::check_common(q, k, v, B, H, Nq, Nk, d, scale);
    if (s != FA_OK) return s;
    s = fa::check_window(H, Hkv, Nq, Nk, window, sinks);
    if (s != FA_OK) return s;
    if (!o || !lse) return FA_ERR_NULL;
    if (!fa::aligned(o, 16) || !fa::aligned(lse, 4)) return FA_ERR_ALIGN;
    return fa::window_forward(q, k, v, o, lse, nullptr, B, H, Hkv, Nq, Nk, d, scale, window, sinks, 1, stream);
}

fa_status fa_fwd_window_splitkv(const void* q, const void* k, const void* v, void* workspace, int B, int H, int Hkv,
                                int Nq, int Nk, int d, float scale, int window, int sinks, int num_splits,
                                cudaStream_t stream) {
    fa_status s = fa::check_common(q, k, v, B, H, Nq, Nk, d, scale);
    if (s != FA_OK) return s;
    s = fa::check_window(H, Hkv, Nq, Nk, window, sinks);
    if (s != FA_OK) return s;
    if (num_splits < 1 || num_splits > FA_MAX_SPLITS) return FA_ERR_SPLITS;
    if (!workspace || !fa::aligned(workspace, 16)) return FA_ERR_WORKSPACE;
    return fa::window_forward(q, k, v, nullptr, nullptr, static_cast<float*>(workspace), B, H, Hkv, Nq, Nk, d, scale,
                              window, sinks, num_splits, stream);
}

int fa_window_num_splits(int B, int H, int Hkv, int Nq, int Nk, int d, int window, int sinks) {
    if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || !fa::valid_d(d) ||
        fa::check_window(H, Hkv, Nq, Nk, window, sinks) != FA_OK)
        return 0;
    const int rows = fa::fwd_config(d).q_tiles * 128;
    const long long bh = static_cast<long long>(B) * H;
    return fa::window_splits(bh * ((Nq + rows - 1) / rows), fa::window_tiles(Nk, std::min(Nq, rows), window, sinks),
                             bh * Nq, d, 152);
}

}  // extern "C"
