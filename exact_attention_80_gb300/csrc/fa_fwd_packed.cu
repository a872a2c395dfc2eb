// fa_fwd_packed.cu — fa_fwd_packed: causal attention over packed sequences of
// different lengths with grouped heads, a window and sinks; instantiations of the
// forward kernels (fa_fwd_pack.cuh has what the packing changes) and the C entry point.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa_fwd_kernel.cuh"

namespace fa {

cudaError_t launch_fwd_packed(const FwdParams& p, int d, bool persist, unsigned grid, cudaStream_t stream) {
    if (persist)
        return d == 64 ? launch_fwd<64, false, false, true, false, true, true>(p, grid, stream)
                       : launch_fwd<128, false, false, true, false, true, true>(p, grid, stream);
    return d == 64    ? launch_fwd<64, false, false, false, false, true, true>(p, grid, stream)
           : d == 128 ? launch_fwd<128, false, false, false, false, true, true>(p, grid, stream)
                      : launch_fwd<256, false, false, false, false, true, true>(p, grid, stream);
}

fa_status check_packed(const fa_packed_batch* c, int H, int Hkv, int d, float scale, int window, int sinks) {
    if (!c || !c->cu_seqlens_q || !c->cu_seqlens_k) return FA_ERR_NULL;
    if (c->B < 1 || H < 1 || H > 65535 || Hkv < 1) return FA_ERR_SHAPE;
    // Positions, units and tiles are counted in int, with room for a tile per sequence.
    const int most = 0x3fffffff;
    if (c->total_q < 1 || c->total_k < 1 || c->total_q > most || c->total_k > most || c->B > (1 << 22))
        return FA_ERR_SHAPE;
    if (c->max_seqlen_q < 1 || c->max_seqlen_q > c->total_q || c->max_seqlen_k < 1 || c->max_seqlen_k > c->total_k)
        return FA_ERR_SHAPE;
    if (!valid_d(d)) return FA_ERR_HEADDIM;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_SCALE;
    if (!aligned(c->cu_seqlens_q, 4) || !aligned(c->cu_seqlens_k, 4)) return FA_ERR_ALIGN;
    const fa_status s = check_window(H, Hkv, c->max_seqlen_q, c->max_seqlen_k, window, sinks);
    if (s != FA_OK) return s;
    return H / Hkv <= 128 ? FA_OK : FA_ERR_GROUP;
}

bool token_stride(long long stride, int heads, int d) {
    return stride % 8 == 0 && stride >= static_cast<long long>(heads) * d && stride <= (1ll << 32);
}

}  // namespace fa

extern "C" fa_status fa_fwd_packed(const void* q, const void* k, const void* v, void* o, float* lse,
                                   const fa_packed_batch* batch, int H, int Hkv, int d, long long q_stride,
                                   long long k_stride, long long v_stride, float scale, int window, int sinks, int fill,
                                   cudaStream_t stream) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
    const fa_status s = fa::check_packed(batch, H, Hkv, d, scale, window, sinks);
    if (s != FA_OK) return s;
    if (!fa::aligned(q, 16) || !fa::aligned(k, 16) || !fa::aligned(v, 16) || !fa::aligned(o, 16) ||
        !fa::aligned(lse, 4))
        return FA_ERR_ALIGN;
    if (!fa::token_stride(q_stride, H, d) || !fa::token_stride(k_stride, Hkv, d) || !fa::token_stride(v_stride, Hkv, d))
        return FA_ERR_STRIDE;
    const fa::FwdConfig c = fa::fwd_config(d);
    const int G = H / Hkv, tokens = 128 / G;
    // Units: at most one that is not full per sequence that has a token.
    const long long unit = static_cast<long long>(c.q_tiles) * tokens, B = std::min(batch->B, batch->total_q);
    const long long units = std::min((batch->total_q + B * (unit - 1)) / unit,
                                     B * ((batch->max_seqlen_q + unit - 1) / unit));
    const long long ctas = units * Hkv;
    if (ctas > 0x7fffffffll) return FA_ERR_SHAPE;
    if (d == 256 && !fa::packed_search(ctas, batch->B)) return FA_ERR_SHAPE;
    fa::FwdParams p;
    std::memset(&p, 0, sizeof(p));
    if (!fa::encode_token_heads_map(&p.tm_q, q, d, batch->total_q, H, q_stride, G, tokens) ||
        !fa::encode_strided_tokens_map(&p.tm_k, k, d, batch->total_k, Hkv, k_stride, c.bn) ||
        !fa::encode_strided_tokens_map(&p.tm_v, v, d, batch->total_k, Hkv, v_stride, c.bn))
        return FA_ERR_CUDA;
    p.store_boxes = 32 % G == 0;
    if (p.store_boxes &&
        !fa::encode_token_heads_map(&p.tm_o, o, d, batch->total_q, H, static_cast<long long>(H) * d, G, 32 / G))
        return FA_ERR_CUDA;
    p.o = o;
    p.lse = lse;
    p.H = H;
    p.Hkv = Hkv;
    p.group = G;
    p.B = batch->B;
    p.Nq = batch->max_seqlen_q;
    p.max_k = batch->max_seqlen_k;
    p.Nk = batch->total_k;
    p.total_q = batch->total_q;
    p.cu_q = batch->cu_seqlens_q;
    p.cu_k = batch->cu_seqlens_k;
    p.tile_tokens = tokens;
    p.q_bytes = static_cast<uint32_t>(G) * tokens * d * 2;
    p.fill = fill ? 1 : 0;
    p.causal = 1;
    p.causal_br = 1;
    p.window = window;
    p.sinks = sinks;
    p.num_splits = 1;
    p.tiles_per_cta = c.q_tiles;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o_scale = 1.f;
    p.wait_limit = fa::kDefaultWaitLimit;
    if (fa::device_status_ptr(&p.status) != cudaSuccess) return FA_ERR_CUDA;
    int sms = 0;
    if (fa::sm_count(&sms) != cudaSuccess) return FA_ERR_CUDA;
    // Persistent CTAs where the units fill two waves, at d = 128 with lists of up to 64 key
    // tiles: a unit's start and end overlap its neighbours', its steps take a little longer
    // (us, one unit per CTA and persistent: d = 64, 16 + 4 heads, four prompts of 8000 tokens
    // 561 and 542, 32 + 8, ten of 2000 262 and 217; d = 128, 16 heads, 64 of 500 152 and 144,
    // 16 + 4, 2.5 waves in three of 2047 58 and 55; 1.6 waves in three of up to 1500, 16 + 8,
    // 29.3 and 30.5; one of 16000 with one of 9000, 16 + 4, 900 and 934). Longer lists too
    // where each unit's search through the sequences would take longest: persistent CTAs go
    // through them once.
    const long long reach = std::min<long long>(batch->max_seqlen_k, window > 0 ? window + unit + sinks : 1ll << 30);
    // (A unit's time bounds the wait for the next but three: 2^24 keys take 0.1 s.)
    const bool long_lists = d == 64 || !fa::packed_search(ctas, batch->B);
    const bool persist = d <= 128 && ctas >= 2ll * sms && reach <= (long_lists ? 1 << 24 : 64 * 128);
    if (!persist && !fa::packed_search(ctas, batch->B)) return FA_ERR_SHAPE;
    const unsigned grid = static_cast<unsigned>(persist ? sms : ctas);
    return fa::launch_fwd_packed(p, d, persist, grid, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
