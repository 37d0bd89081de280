// Host side of the expert FFN's forward pass: tile choices, tensor maps and the launches of the grouped
// GEMM in expert_gemm.cuh (bf16, e4m3, router logits).
#include "expert_gemm.cuh"

namespace smoe {

#ifndef SMOE_SHARED_FIRST
#define SMOE_SHARED_FIRST 1   // small-tile gate/up launches list the shared expert's tiles first
#endif

// Largest token tile of a launch: the smallest power of two >= 1.25 x the mean rows per routed
// expert, 16..256. Groups with fewer rows use smaller tiles inside the kernel.
#ifndef SMOE_TILE_FACTOR
#define SMOE_TILE_FACTOR 1.25
#endif
int choose_token_tile(const smoe_config_t& c, int64_t T) {
    const double mean = (double)T * c.top_k / c.n_experts;
    int nt = 16;
    while (nt < SMOE_MAX_TOKEN_TILE && nt < SMOE_TILE_FACTOR * mean) nt *= 2;
    return nt;
}

// Shared units before the wait only when all of them fit in one round of CTAs (decode-sized
// batches): with more (the MTP batch's 16 tiles), the GEMM launched early competes with the
// top-k kernel's CTAs for the SMs and the routing takes longer than the overlap saves.
bool shared_prewait_fits(const smoe_config_t& c, int64_t T, int num_sms) {
    const int nt = choose_token_tile(c, T);
    int nt_sh = 16;
    while (nt_sh < T && nt_sh < nt) nt_sh *= 2;
    return (T + nt_sh - 1) / nt_sh * (c.inter / 128) <= num_sms;
}

size_t packed_gateup_bytes(const smoe_config_t& c) {
    return (size_t)(c.n_experts + 1) * 2 * c.inter * c.hidden * 2;
}
size_t packed_down_bytes(const smoe_config_t& c) { return (size_t)(c.n_experts + 1) * c.hidden * c.inter * 2; }

cudaError_t launch_expert_ffn(const smoe_config_t& c, const uint16_t* x, const uint16_t* x_perm,
                              const int32_t* row_token, const int32_t* offsets, int64_t T, const void* packed,
                              uint16_t* y, uint16_t* h, int32_t* err, int num_sms, cudaStream_t s,
                              bool shared_prewait, const Checkpoint* ck) {
    constexpr int BK = SMOE_GEMM_BK;
    const int E = c.n_experts, H = c.hidden, I = c.inter, k = c.top_k;
    const int64_t routed = T * k;
    const int nt = choose_token_tile(c, T);
    const uint8_t* wgu = static_cast<const uint8_t*>(packed);
    const uint8_t* wdn = wgu + packed_gateup_bytes(c);

    GemmMaps m1, m2;
    const bool gather = x_perm == nullptr;
    // CTA pairs for large token tiles (each pair handles 256 output features)
    const bool pairs = nt >= kPairMinTile && I % 256 == 0 && H % 256 == 0;
    auto act_maps = [&](CUtensorMap* maps, const void* base, uint64_t rows, uint64_t cols) {
        return pairs ? make_half_act_maps(maps, base, rows, cols, nt, BK) : make_act_maps(maps, base, rows, cols, nt, BK);
    };
    bool ok_act = gather ? make_map(&m1.act[0], x, (uint64_t)T, H, 1, BK) : act_maps(m1.act, x_perm, (uint64_t)routed, H);
    if (gather)
        for (int i = 1; i < kNumTiles; ++i) m1.act[i] = m1.act[0];
    // packed weights, tile-major: viewed as [rows][64] with 256-row (gate/up) / 128-row (down) tiles
    if (!ok_act || !make_map(&m1.w, wgu, (uint64_t)(E + 1) * 2 * I * (H / 64), 64, 256, BK) ||
        !act_maps(m1.sh, x, (uint64_t)T, H) ||
        !make_map(&m2.w, wdn, (uint64_t)(E + 1) * H * (I / 64), 64, 128, BK) ||
        !act_maps(m2.act, h, (uint64_t)(routed + T), I))
        return cudaErrorNotSupported;
    for (int i = 0; i < kNumTiles; ++i) m2.sh[i] = m2.act[i];

    GemmParams p1{offsets, E, (int)T, (int)routed, H, I, 0, (int)routed, nt, 0, 0, I, I, gather ? row_token : nullptr,
                  c.swiglu_limit, c.swiglu_limit_shared, 1, 0, h, nullptr, err};
    p1.shared_first = gather && !pairs && SMOE_SHARED_FIRST ? 1 : 0;
    p1.shared_prewait = gather && !pairs && shared_prewait && shared_prewait_fits(c, T, num_sms) ? 1 : 0;
    cudaError_t e;
    if (ck != nullptr) {
        p1.codes = ck->codes;
        p1.scales = ck->scales;
        p1.ck_rows = routed + T;
        e = pairs ? run_gemm_pair<MODE_GATEUP_SAVE>(m1, p1, num_sms, s)
                  : run_gemm<MODE_GATEUP_SAVE>(m1, p1, num_sms, s);
    } else {
        e = pairs ? run_gemm_pair<MODE_GATEUP>(m1, p1, num_sms, s) : run_gemm<MODE_GATEUP>(m1, p1, num_sms, s);
    }
    if (e != cudaSuccess) return e;
    GemmParams p2{offsets, E, (int)T, (int)routed, I, H, (int)routed, (int)routed, nt, 0, 0, H, H, nullptr, 0.f, 0.f, 1,
                  0, y, nullptr, err};
    e = pairs ? run_gemm_pair<MODE_DOWN>(m2, p2, num_sms, s) : run_gemm<MODE_DOWN>(m2, p2, num_sms, s);
    if (e == cudaSuccess) launches_add(2);
    return e;
}

cudaError_t launch_expert_ffn_fp8(const smoe_config_t& c, const uint8_t* x_q, const uint8_t* x_q_perm,
                                  const float* s_x, const int32_t* row_token, const int32_t* offsets, int64_t T,
                                  const void* packed_fp8, uint16_t* y, uint16_t* h, uint8_t* h_q, float* s_h,
                                  int32_t* err, int num_sms, cudaStream_t s) {
    constexpr int BK = SMOE_GEMM_BK;
    const int E = c.n_experts, H = c.hidden, I = c.inter, k = c.top_k;
    const int64_t routed = T * k;
    const int nt = choose_token_tile(c, T);
    const Fp8Layout L = fp8_layout(c);
    const uint8_t* pk = static_cast<const uint8_t*>(packed_fp8);

    GemmMaps m1, m2;
    const bool gather = x_q_perm == nullptr;
    const bool pairs = nt >= kPairMinTile && I % 256 == 0 && H % 256 == 0;
    auto act_maps = [&](CUtensorMap* maps, const void* base, uint64_t rows, uint64_t cols) {
        return pairs ? make_half_act_maps(maps, base, rows, cols, nt, BK, true)
                     : make_act_maps(maps, base, rows, cols, nt, BK, true);
    };
    bool ok_act = gather ? make_map_u8(&m1.act[0], x_q, (uint64_t)T, H, 1) : act_maps(m1.act, x_q_perm, (uint64_t)routed, H);
    if (gather)
        for (int i = 1; i < kNumTiles; ++i) m1.act[i] = m1.act[0];
    // packed codes, tile-major: viewed as [rows][128] with 256-row (gate/up) / 128-row (down) tiles
    if (!ok_act || !make_map_u8(&m1.w, pk + L.gateup, (uint64_t)(E + 1) * 2 * I * (H / 128), 128, 256) ||
        !act_maps(m1.sh, x_q, (uint64_t)T, H) ||
        !make_map_u8(&m2.w, pk + L.down, (uint64_t)(E + 1) * H * (I / 128), 128, 128) ||
        !act_maps(m2.act, h_q, (uint64_t)(routed + T), I))
        return cudaErrorNotSupported;
    for (int i = 0; i < kNumTiles; ++i) m2.sh[i] = m2.act[i];

    GemmParams p1{offsets, E, (int)T, (int)routed, H, I, 0, (int)routed, nt, 0, 0, I, I, gather ? row_token : nullptr,
                  c.swiglu_limit, c.swiglu_limit_shared, 1, 0, h, nullptr, err};
    p1.w_scale = reinterpret_cast<const float*>(pk + L.gateup_scale);
    p1.act_scale = s_x;
    p1.scale_tok = row_token;
    p1.scale_shared_base = 0;
    p1.shared_first = gather && !pairs && SMOE_SHARED_FIRST ? 1 : 0;
    cudaError_t e = pairs ? run_gemm_pair<MODE_GATEUP, true>(m1, p1, num_sms, s)
                          : run_gemm<MODE_GATEUP, true>(m1, p1, num_sms, s);
    if (e != cudaSuccess) return e;
    e = launch_quantize_rows(h, routed + T, I, h_q, s_h, K_QUANT_H, s);
    if (e != cudaSuccess) return e;
    GemmParams p2{offsets, E, (int)T, (int)routed, I, H, (int)routed, (int)routed, nt, 0, 0, H, H, nullptr, 0.f, 0.f, 1,
                  0, y, nullptr, err};
    p2.w_scale = reinterpret_cast<const float*>(pk + L.down_scale);
    p2.act_scale = s_h;
    p2.scale_tok = nullptr;
    p2.scale_shared_base = (int)routed;
    e = pairs ? run_gemm_pair<MODE_DOWN, true>(m2, p2, num_sms, s) : run_gemm<MODE_DOWN, true>(m2, p2, num_sms, s);
    if (e == cudaSuccess) launches_add(2);
    return e;
}

// Router logits on the tensor cores: partial[p][T][E] = x [T][H] . W_p^T for the three bf16
// pieces p = hi, mid, lo of W_r; w_split [e_pad][3H] holds the pieces of each fp32 router row
// side by side (rows >= E are zero). One group of T rows; each unit covers one piece's K range
// (x's K coordinate wraps), so the three partials are summed later in a fixed order.
cudaError_t launch_router_gemm(const uint16_t* x, int64_t T, int H, const uint16_t* w_split, int e_pad, int E,
                               float* logits, int nt, int ksplit, int num_sms, cudaStream_t s) {
    constexpr int BK = SMOE_GEMM_BK;
    GemmMaps m;
    if (!make_map(&m.w, w_split, (uint64_t)e_pad, (uint64_t)3 * H, 128, BK) ||
        !make_act_maps(m.sh, x, (uint64_t)T, H, nt, BK))
        return cudaErrorNotSupported;
    for (int i = 0; i < kNumTiles; ++i) m.act[i] = m.sh[i];
    GemmParams p{nullptr, 0, (int)T, 0, 3 * H, e_pad, 0, 0, nt, 0, H / BK, E, E, nullptr, 0.f, 0.f, ksplit, (size_t)T * E,
                 nullptr, logits, nullptr};
    return run_gemm<MODE_ROUTER>(m, p, num_sms, s);
}

}  // namespace smoe
