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

}  // namespace fa

extern "C" fa_status fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                                   int Hkv, int Nq, int Nk, int d, float scale, int window, int sinks,
                                   cudaStream_t stream) {
    fa_status s = fa::check_common(q, k, v, B, H, Nq, Nk, d, scale);
    if (s != FA_OK) return s;
    s = fa::check_window(H, Hkv, Nq, Nk, window, sinks);
    if (s != FA_OK) return s;
    if (!o || !lse) return FA_ERR_NULL;
    if (!fa::aligned(o, 16) || !fa::aligned(lse, 4)) return FA_ERR_ALIGN;
    const fa::FwdConfig c = fa::fwd_config(d);
    fa::FwdParams p;
    std::memset(&p, 0, sizeof(p));
    const int BH = B * H;
    if (!fa::encode_rows_map(&p.tm_q, q, d, Nq, BH, 128) || !fa::encode_rows_map(&p.tm_k, k, d, Nk, B * Hkv, c.bn) ||
        !fa::encode_rows_map(&p.tm_v, v, d, Nk, B * Hkv, c.bn) ||
        !fa::encode_rows_map(&p.tm_o, o, d, Nq, BH, d == 256 ? 128 : 32))
        return FA_ERR_CUDA;
    p.o = o;
    p.lse = lse;
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
    p.num_splits = 1;
    p.tiles_per_cta = c.q_tiles;
    const int rows = c.q_tiles * 128;
    p.n_units = (Nq + rows - 1) / rows;
    const long long ctas = static_cast<long long>(BH) * p.n_units;
    if (ctas > 0x7fffffffll) return FA_ERR_SHAPE;
    int sms = 0;
    if (fa::sm_count(&sms) != cudaSuccess) return FA_ERR_CUDA;
    p.head_group = std::max(1, std::min(BH, sms / p.n_units));
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o_scale = 1.f;
    p.wait_limit = fa::kDefaultWaitLimit;
    if (fa::device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    // Persistent CTAs where the units fill at least four waves and list few key
    // tiles, as for the dense forward: the start and end of a unit overlap its
    // neighbours' (2 x 32 heads of 8192, window 1024, d = 64: 216 against 225 us;
    // window 128: 83 against 107; with 3.4 waves 79 against 76).
    const long long listed =
        window > 0 ? std::min<long long>((Nk + 127) / 128, (window + 126) / 128 + 2 + (sinks + 127) / 128)
                   : (Nk + 127) / 128;
    p.total_units = ctas;
    if (d <= 128 && ctas >= 4ll * sms && listed <= 16) {
        const unsigned all = static_cast<unsigned>(sms);
        const cudaError_t e = d == 64 ? fa::launch_fwd_win_d64_persist(p, all, stream)
                                      : fa::launch_fwd_win_d128_persist(p, all, stream);
        return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    }
    const unsigned grid = static_cast<unsigned>(ctas);
    const cudaError_t e = d == 64    ? fa::launch_fwd_win_d64(p, grid, stream)
                          : d == 128 ? fa::launch_fwd_win_d128(p, grid, stream)
                                     : fa::launch_fwd_win_d256(p, grid, stream);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
