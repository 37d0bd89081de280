// Backward pass of the expert FFNs (smoe_expert_ffn_backward). With the checkpoint's g, u of every row
// (expert_gemm.cuh, epi_load_save), dY the gradient of the expert outputs and F(x) = W_d (SiLU(g) u):
//   dh = dY W_d;  h, dG, dU from dh, g, u (expert_gemm.cuh, epi_swiglu_backward)       one grouped GEMM
//   dX = dG W_g + dU W_u                                                                one grouped GEMM
//   dW_g = dG^T X,  dW_u = dU^T X,  dW_d = dY^T h, for every expert over its own rows   two launches
// (SwiGLU experts: Step 3.5 Flash summary, paperlayer.ai, §B.) dh and dx run on the forward pass's
// kernels and read its packed weights in place, through M-major operand tiles.
//
// Weight gradients: a persistent, warp-specialised grouped GEMM whose contraction runs over an
// expert's rows. Unit = (group, 128 x 256 block of the gradient); both operands are M-major tiles of
// 64 rows x 64 columns boxes straight from the row-major activations, so nothing is transposed. A
// group's rows start anywhere and rarely end on a tile: the last stage also holds rows of the next
// group, which may be infinite or NaN, so up to the next multiple of 16 they are overwritten with
// zeros in shared memory and the products beyond are not issued. Groups without rows get zeros.
#include "expert_gemm.cuh"

namespace smoe {

namespace {

constexpr int kWgThreads = 192;      // producer warp, MMA warp, four epilogue warps
constexpr int kWgN = 256;            // gradient columns of a unit (128 for the last block of an odd width)
constexpr int kWgKRows = 64;         // rows of a pipeline stage
constexpr int kWgABytes = 2 * kMnBoxBytes;
constexpr int kWgStageBytes = kWgABytes + (kWgN / 64) * kMnBoxBytes;
constexpr int kWgStages = 4;
constexpr int kWgStoreBytes = 32 * 128;   // an epilogue warp's staging box: 32 gradient rows x 64 columns

struct WgradMaps {
    CUtensorMap a, a_sh;        // M side [rows][M] of the routed groups and of the shared one: box {64, 64}
    CUtensorMap b, b_sh;        // N side [rows][N]: box {64, 64}
    CUtensorMap out[2];         // gradients [E * M'][N]: rows m < m_split go to out[0], the others to out[1]
    CUtensorMap out_sh[2];      // the shared expert's [M'][N]: box {64, 32}
};

struct WgradParams {
    const int32_t* offsets;   // [E+1] routed row offsets
    int E, T, routed_rows;
    int M, N;                 // gradient rows (over both outputs) and columns
    int m_split;              // rows of an output (M or M / 2)
    int a_sh_row, b_sh_row;   // first row of the shared group in a_sh / b_sh
    int32_t* err;
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int32_t c0, int32_t c1, uint32_t src, uint64_t pol) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2}], [%3], %4;" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src), "l"(pol)
                 : "memory");
}

size_t wgrad_smem_bytes(int E) {
    return 1024 + (size_t)kWgStages * kWgStageBytes + 4 * kWgStoreBytes + sizeof(uint64_t) * (2 * kWgStages + 5) + 16 +
           sizeof(int32_t) * (size_t)(E + 1);
}

__global__ void __launch_bounds__(kWgThreads, 1)
expert_wgrad_kernel(const __grid_constant__ WgradMaps maps, const WgradParams p) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int S = kWgStages;
    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = tiles + (size_t)S * kWgStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + 4 * kWgStoreBytes);
    uint64_t* empty = full + S;
    uint64_t* tfull = empty + S;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* offs = reinterpret_cast<int32_t*>(tmem_slot + 4);   // [E+1]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;
    const int MB = p.M / 128, NB = (p.N + kWgN - 1) / kWgN;
    const int upg = MB * NB;                 // units of a group
    const int total = (E + 1) * upg;         // at most 1025 * 512 * 128: fits
    const int W = gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 4);
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 2) {
        // corrupt offsets: no routed rows (their gradients are zeros), the error word set
        bool bad = false;
        for (int i = lane; i <= E; i += 32) {
            int v = p.offsets[i];
            if (v < 0 || v > p.routed_rows) { bad = true; v = 0; }
            offs[i] = v;
        }
        __syncwarp();
        for (int i = lane; i < E; i += 32)
            if (offs[i + 1] < offs[i]) bad = true;
        if (__any_sync(0xFFFFFFFFu, bad)) {
            for (int i = lane; i <= E; i += 32) offs[i] = 0;
            if (lane == 0) record_error(p.err, SMOE_ERR_DEVICE);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // unit u: the shared group's first (it has the most rows), then the routed groups in order; the
    // units of a group run at the same time on neighbouring SMs and share its rows in L2
    struct WUnit { int g, mb, nb, rows, ncols; };
    auto unit_at = [&](int u) {
        WUnit w;
        const int o = u / upg, r = u % upg;
        w.g = o == 0 ? E : o - 1;
        w.mb = r / NB;
        w.nb = r % NB;
        w.rows = group_rows(w.g, E, p.T, offs);
        w.ncols = min(kWgN, p.N - w.nb * kWgN);
        return w;
    };

    if (warp == 0 && lane == 0) {
        // ---------------------------------------------------------------- TMA producer
        const uint64_t pol = l2_policy_evict_last();
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_par = 0;
        bool ok = true;
        for (int i = 0; ok && i * W < total; ++i) {
            const int u = snake_unit(i, blockIdx.x, W, total);
            if (u < 0) continue;
            const WUnit w = unit_at(u);
            const CUtensorMap* am = w.g < E ? &maps.a : &maps.a_sh;
            const CUtensorMap* bm = w.g < E ? &maps.b : &maps.b_sh;
            const int a_row = w.g < E ? offs[w.g] : p.a_sh_row, b_row = w.g < E ? offs[w.g] : p.b_sh_row;
            const uint32_t tx = (uint32_t)(kWgABytes + w.ncols / 64 * kMnBoxBytes);
            for (int k = 0; k < w.rows; k += kWgKRows) {
                ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, p.err, abort_flag, true);
                if (!ok) break;
                const uint32_t fb = smem_u32(&full[stage]);
                const uint32_t a_s = smem_u32(tiles + (size_t)stage * kWgStageBytes);
                mbar_arrive_expect_tx(fb, tx);
                for (int j = 0; j < 2; ++j)
                    tma_load_2d(a_s + j * kMnBoxBytes, am, w.mb * 128 + 64 * j, a_row + k, fb, pol);
                for (int j = 0; j < w.ncols / 64; ++j)
                    tma_load_2d(a_s + kWgABytes + j * kMnBoxBytes, bm, w.nb * kWgN + 64 * j, b_row + k, fb, pol);
                armed |= 1u << stage;
                armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
        }
        for (int s = 0; s < S; ++s)   // every load issued must land before the CTA may exit
            if ((armed >> s) & 1u) mbar_wait(smem_u32(&full[s]), (armed_par >> s) & 1u, p.err, abort_flag, false);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA (lane 0; all lanes clear row tails)
        const uint32_t idesc0 = idesc_bf16_f32(128, 0) | kIdescAMajorM | kIdescBMajorN;
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int i = 0; ok && i * W < total; ++i) {
            const int u = snake_unit(i, blockIdx.x, W, total);
            if (u < 0) continue;
            const WUnit w = unit_at(u);
            const uint32_t idesc = idesc0 | ((uint32_t)(w.ncols >> 3) << 17);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, p.err, abort_flag, true));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(acc * kWgN);
            for (int k = 0; k < w.rows; k += kWgKRows) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&full[stage]), phase, p.err, abort_flag, true));
                if (!ok) break;
                uint8_t* st = tiles + (size_t)stage * kWgStageBytes;
                const int valid = min(kWgKRows, w.rows - k), ksteps = (valid + 15) / 16;
                if (valid & 15) {
                    // rows valid .. 16 ksteps - 1 of every box: whole 128-byte lines, whatever the swizzle
                    const int n = 8 * (16 * ksteps - valid), boxes = 2 + w.ncols / 64;
                    for (int z = lane; z < n * boxes; z += 32)
                        *reinterpret_cast<uint4*>(st + (z / n) * kMnBoxBytes + valid * 128 + (z % n) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t a_s = smem_u32(st), b_s = a_s + kWgABytes;
                    for (int kk = 0; kk < ksteps; ++kk)
                        umma_f16_ss(d, smem_desc_mnmajor(a_s + kk * kMnKStep, kMnBoxBytes),
                                    smem_desc_mnmajor(b_s + kk * kMnKStep, kMnBoxBytes), idesc, (k | kk) != 0 ? 1u : 0u);
                    umma_commit(smem_u32(&empty[stage]));
                }
                __syncwarp();
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            if (lane == 0) umma_commit(smem_u32(&tfull[acc]));
            __syncwarp();
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (lane == 0) {   // all MMAs issued must finish before TMEM is released
            umma_commit(smem_u32(drain));
            mbar_wait(smem_u32(drain), 0u, p.err, abort_flag, false);
        }
        __syncwarp();
    } else if (warp >= 2) {
        // ---------------------------------------------------------------- epilogue: TMEM -> bf16 -> TMA store
        const int q = warp & 3;
        uint8_t* stg = staging + q * kWgStoreBytes;
        const uint64_t pol = l2_policy_evict_first();
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int i = 0; i * W < total; ++i) {
            const int u = snake_unit(i, blockIdx.x, W, total);
            if (u < 0) continue;
            const WUnit w = unit_at(u);
            const int m = w.mb * 128 + q * 32;
            const int part = m >= p.m_split ? 1 : 0;
            const CUtensorMap* om = w.g < E ? &maps.out[part] : &maps.out_sh[part];
            const int y = (w.g < E ? w.g * p.m_split : 0) + m - part * p.m_split;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&tfull[acc]), acc_phase, p.err, abort_flag, true))) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kWgN);
            for (int c = 0; c < w.ncols; c += 64) {
                uint32_t v[32];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t a[32];
                    if (w.rows > 0) {
                        tmem_ld_x32_wait(t_row + c + 32 * z, a);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) a[j] = 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[16 * z + j] = pack_bf16x2(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]));
                }
                if (c + 64 >= w.ncols) {   // all of this warp's accumulator has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&tempty[acc]));
                }
                // the previous box has left the staging buffer
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 8; ++x)   // the 128-byte swizzle: 16-byte chunk x of row l lies at x ^ (l & 7)
                    *reinterpret_cast<uint4*>(stg + lane * 128 + ((x ^ (lane & 7)) << 4)) =
                        make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(om, w.nb * kWgN + c, y, smem_u32(stg), pol);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

cudaError_t run_wgrad(const WgradMaps& maps, const WgradParams& p, KernelId id, int num_sms, cudaStream_t s) {
    const size_t smem = wgrad_smem_bytes(p.E);
    cudaError_t e = cudaFuncSetAttribute(expert_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    LaunchTimer lt(id, s);
    return launch_pdl(expert_wgrad_kernel, dim3(num_sms), dim3(kWgThreads), smem, s, maps, p);
}

}  // namespace

cudaError_t launch_expert_ffn_backward(const smoe_config_t& c, const ExpertBackward& b, int64_t T, int32_t* err,
                                       int num_sms, cudaStream_t s) {
    constexpr int BK = SMOE_GEMM_BK;
    const int E = c.n_experts, H = c.hidden, I = c.inter, k = c.top_k;
    const int64_t routed = T * k, rows = routed + T;
    const int nt = choose_token_tile(c, T);
    const uint8_t* wgu = static_cast<const uint8_t*>(b.packed);
    const uint8_t* wdn = wgu + packed_gateup_bytes(c);
    const bool pairs = nt >= kPairMinTile && I % 256 == 0 && H % 256 == 0;   // as in the forward pass
    auto act_maps = [&](CUtensorMap* maps, const void* base, uint64_t n, uint64_t cols) {
        return pairs ? make_half_act_maps(maps, base, n, cols, nt, BK) : make_act_maps(maps, base, n, cols, nt, BK);
    };

    GemmMaps m1, m2;
    WgradMaps wd, wg;
    // packed weights viewed as rows of 64 columns, loaded in boxes of 64 rows
    if (!make_map(&m1.w, wdn, (uint64_t)(E + 1) * H * (I / 64), 64, 64, BK) || !act_maps(m1.act, b.dy, routed, H) ||
        !act_maps(m1.sh, b.dout, T, H) ||
        !make_map(&m2.w, wgu, (uint64_t)(E + 1) * 2 * I * (H / 64), 64, 64, BK) ||
        !act_maps(m2.act, b.dgu, rows, 2 * I) ||
        !make_map(&wd.a, b.dy, routed, H, 64, BK) || !make_map(&wd.a_sh, b.dout, T, H, 64, BK) ||
        !make_map(&wd.b, b.h, rows, I, 64, BK) || !make_map(&wd.out[0], b.dw_down, (uint64_t)E * H, I, 32, BK) ||
        !make_map(&wd.out_sh[0], b.dws_down, H, I, 32, BK) ||
        !make_map(&wg.a, b.dgu, rows, 2 * I, 64, BK) || !make_map(&wg.b, b.x_perm, routed, H, 64, BK) ||
        !make_map(&wg.b_sh, b.x, T, H, 64, BK) ||
        !make_map(&wg.out[0], b.dw_gate, (uint64_t)E * I, H, 32, BK) ||
        !make_map(&wg.out[1], b.dw_up, (uint64_t)E * I, H, 32, BK) ||
        !make_map(&wg.out_sh[0], b.dws_gate, I, H, 32, BK) || !make_map(&wg.out_sh[1], b.dws_up, I, H, 32, BK))
        return cudaErrorNotSupported;
    for (int i = 0; i < kNumTiles; ++i) m2.sh[i] = m2.act[i];
    wd.b_sh = wd.b;
    wd.out[1] = wd.out[0];
    wd.out_sh[1] = wd.out_sh[0];
    wg.a_sh = wg.a;

    GemmParams p1{b.offsets, E, (int)T, (int)routed, H, I, 0, (int)routed, nt, 0, 0, 2 * I, I, nullptr,
                  c.swiglu_limit, c.swiglu_limit_shared, 1, 0, b.dgu, nullptr, err};
    p1.codes = const_cast<uint8_t*>(b.codes);
    p1.scales = const_cast<uint8_t*>(b.scales);
    p1.ck_rows = rows;
    p1.h_out = b.h;
    cudaError_t e = pairs ? run_gemm_pair<MODE_DH>(m1, p1, num_sms, s) : run_gemm<MODE_DH>(m1, p1, num_sms, s);
    if (e != cudaSuccess) return e;
    GemmParams p2{b.offsets, E, (int)T, (int)routed, 2 * I, H, (int)routed, (int)routed, nt, 0, 0, H, H, nullptr, 0.f, 0.f,
                  1, 0, b.dx_rows, nullptr, err};
    e = pairs ? run_gemm_pair<MODE_DX>(m2, p2, num_sms, s) : run_gemm<MODE_DX>(m2, p2, num_sms, s);
    if (e != cudaSuccess) return e;
    e = run_wgrad(wg, WgradParams{b.offsets, E, (int)T, (int)routed, 2 * I, H, I, (int)routed, 0, err},
                  K_EXPERT_WGRAD_GATEUP, num_sms, s);
    if (e != cudaSuccess) return e;
    e = run_wgrad(wd, WgradParams{b.offsets, E, (int)T, (int)routed, H, I, H, 0, (int)routed, err},
                  K_EXPERT_WGRAD_DOWN, num_sms, s);
    if (e == cudaSuccess) launches_add(4);
    return e;
}

}  // namespace smoe
