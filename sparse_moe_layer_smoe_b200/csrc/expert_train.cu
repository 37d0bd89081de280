// Backward pass of the expert FFNs (smoe_expert_ffn_backward). With the checkpoint's g, u of every row
// (expert_gemm.cuh, epi_gateup_save), dY the gradient of the expert outputs and F(x) = W_d (SiLU(g) u):
//   dh = dY W_d;  h, dG, dU from dh, g, u (expert_gemm.cuh, epi_swiglu_backward)       one grouped GEMM
//   dX = dG W_g + dU W_u                                                                one grouped GEMM
//   dW_g = dG^T X,  dW_u = dU^T X,  dW_d = dY^T h, for every expert over its own rows   one launch
// (SwiGLU experts: Step 3.5 Flash summary, paperlayer.ai, §B.) dh and dx run on the forward pass's
// kernels and read its packed weights in place, through M-major operand tiles.
//
// Weight gradients: a persistent, warp-specialised grouped GEMM on CTA pairs whose contraction runs over
// an expert's rows. Unit = (group, 256 x 256 block of the gradient); both operands are M-major tiles
// (boxes of 64 rows x 64 columns) straight from the row-major activations, so nothing is transposed.
// Every CTA of the pair loads 128 of the block's rows' columns and 128 of its columns': 32 KB a stage for
// 512 clocks of MMA, where one CTA alone on 128 x 256 loads 48 KB. 8192 tokens of the full layer (2.3 TFLOP,
// 9.1 GB written) take 3.05 to 3.15 ms in a burst and 3.6 to 3.7 ms at the power limit; the library's batched
// GEMM on even groups of 256 rows takes 3.0 ms there.
// A group's rows start anywhere and rarely end on a tile: the last stage also holds rows of the next
// group, which may be infinite or NaN, so up to the next multiple of 16 they are overwritten with zeros
// in shared memory and the products beyond are not issued. Groups without rows get zeros.
#include "expert_gemm.cuh"

namespace smoe {

namespace {

constexpr int kWgEpiWarps = 8;       // two per quarter of the TMEM lanes, each every other 64-column box
constexpr int kWgThreads = 128 + 32 * kWgEpiWarps;  // two producer warps, MMA and tail warp, epilogue warps
constexpr int kWgTile = 256;         // gradient rows (128 a CTA) and columns of a unit
constexpr int kWgKRows = 64;         // rows of a pipeline stage
constexpr int kWgABytes = 2 * kMnBoxBytes;          // this CTA's 128 gradient rows
constexpr int kWgStageBytes = 2 * kWgABytes;        // and its half of the columns
constexpr int kWgMaxStages = 6;
// Stages that a row tail is loaded ahead of its turn. Its clearing, handed over between the CTAs, takes longer than
// the other rows' landing: 8192 tokens in a burst 3.22 ms at 0, 3.20 at 1, 3.17 at 2, 3.15 at 3 (at the power
// limit 3.90 and 3.73 at 0 and 3).
constexpr int kWgAhead = 3;
constexpr int kWgStoreBytes = 32 * 128;   // an epilogue warp's staging box (two each): 32 gradient rows x 64 columns

// A contraction over every group's rows: gradient [M][N] of group g = A_g^T B_g. A launch takes two: gate and
// up (A = dG | dU, B = X), then down (A = dY, B = h).
struct WgradProblem {
    // operands [rows][cols] viewed as {64 columns, rows, cols / 64}, box {64, 64, 2}: two M-major tiles a load
    CUtensorMap a, a_sh;        // M side of the routed groups and of the shared one
    CUtensorMap b, b_sh;        // N side
    CUtensorMap out[2];         // gradients [E * M'][N]: rows m < m_split go to out[0], the others to out[1]
    CUtensorMap out_sh[2];      // the shared expert's [M'][N]; boxes of 64 columns x 32 rows
    int M, N;                 // gradient rows (over both outputs) and columns
    int m_split;              // rows of an output (M or M / 2)
    int a_sh_row, b_sh_row;   // first row of the shared group in a_sh / b_sh
    int nb, upg;              // column blocks, units of a group
    uint32_t inv_nb, inv_upg; // 2^32 / those, rounded up
};

struct WgradParams {
    WgradProblem prob[2];
    const int32_t* offsets;   // [E+1] routed row offsets
    int E, T, routed_rows;
    int stages;               // pipeline depth
    int32_t* err;
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int32_t c0, int32_t c1, uint32_t src, uint64_t pol) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2}], [%3], %4;" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src), "l"(pol)
                 : "memory");
}

// Operand map (see WgradProblem) of a bf16 matrix [rows][cols], cols a multiple of 64.
bool make_wgrad_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {64, rows, cols / 64};
    cuuint64_t strides[2] = {cols * 2, 128};
    cuuint32_t box[3] = {64, kWgKRows, 2};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// tma_load_2d_pair for a 3D map.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                                 uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}

size_t wgrad_smem_bytes(int stages, int E) {
    return 1024 + (size_t)stages * kWgStageBytes + 2 * kWgEpiWarps * kWgStoreBytes +
           sizeof(uint64_t) * (4 * (size_t)stages + 5) + 16 + sizeof(int32_t) * (size_t)(E + 1);
}

// Hand-over of a cleared row tail between the pair's CTAs: the first CTA's MMA reads the second one's shared
// memory, so what the second one wrote there must be ordered across the cluster. The arrival releases at
// cluster scope and the wait acquires there; fence.proxy.async before the arrival makes the writes
// visible to the tensor cores.
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgThreads, 1)
expert_wgrad_kernel(const __grid_constant__ WgradParams p) {
    extern __shared__ uint8_t smem_raw[];
    const int S = p.stages;
    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = tiles + (size_t)S * kWgStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + 2 * kWgEpiWarps * kWgStoreBytes);
    // A stage's loads of both CTAs complete on the first CTA's full barrier. A stage with a row tail is
    // different: each CTA's loads complete on its own tail_full and its tail warp clears the tail; the
    // second CTA's then arrives on the first one's tail_ready, and the first one's, having seen that, on
    // full. The MMA thread waits for full alone, and the clearing is done well before it gets there.
    uint64_t* tail_full = full + S;
    uint64_t* tail_ready = tail_full + S;
    uint64_t* empty = tail_ready + S;
    uint64_t* tfull = empty + S;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* offs = reinterpret_cast<int32_t*>(tmem_slot + 4);   // [E+1]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int E = p.E;
    const int total0 = (E + 1) * p.prob[0].upg;              // at most 1025 * 256 * 128 each: fits
    const int total = total0 + (E + 1) * p.prob[1].upg;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&tail_full[s]), 1);
            mbar_init(smem_u32(&tail_ready[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 2 * kWgEpiWarps);   // epilogue warps of both CTAs
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish_pair();
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
    cluster_sync();   // barrier inits and TMEM allocation visible to both CTAs
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // unit u of a problem: the shared group's first (it has the most rows), then the routed groups in order;
    // the units of a group run at the same time on neighbouring pairs and share its rows in L2
    struct WUnit { int prob, g, mb, nb, rows, ncols; };
    // a / b by its rounded-up reciprocal: one too high at most (a < 2^32), which the remainder shows
    auto divide = [](int a, int b, uint32_t inv, int& rest) {
        int q = b == 1 ? a : (int)__umulhi((uint32_t)a, inv);
        rest = a - q * b;
        if (rest < 0) {
            --q;
            rest += b;
        }
        return q;
    };
    auto unit_at = [&](int u) {
        WUnit w;
        w.prob = u >= total0 ? 1 : 0;
        const WgradProblem& q = p.prob[w.prob];
        int r;
        const int o = divide(u - (w.prob ? total0 : 0), q.upg, q.inv_upg, r);
        w.g = o == 0 ? E : o - 1;
        w.mb = divide(r, q.nb, q.inv_nb, w.nb);
        w.rows = group_rows(w.g, E, p.T, offs);
        w.ncols = min(kWgTile, q.N - w.nb * kWgTile);
        return w;
    };
    // Stages of a unit, and the place of its row tail among their loads (none: -1); the products take it last.
    // Fewer than S stages ahead, so that the stage is free again before the ring comes round to it.
    auto stages_of = [](const WUnit& w) { return (w.rows + kWgKRows - 1) / kWgKRows; };
    auto tail_place = [&](const WUnit& w) {
        const int n = stages_of(w);
        return (w.rows & 15) == 0 ? -1 : max(n - 1 - min(kWgAhead, S - 2), 0);
    };

    if ((warp == 0 || warp == 3) && lane == 0) {
        // ---------------------------------------------------------------- TMA producers (both CTAs)
        // warp 0 arms a stage's barrier and loads the M side, warp 3 the N side (one thread for both: the
        // gate/up gradients of 8192 tokens in 2.13 ms instead of 2.04). Bytes may land before the barrier is
        // armed; the phase waits for the arming arrival.
        const bool m_side = warp == 0;
        const uint64_t pol = l2_policy_evict_last();
        const uint32_t dst0 = smem_u32(tiles) + (m_side ? 0 : kWgABytes);
        const uint32_t full0 = mapa_shared(smem_u32(full), 0), tail0 = mapa_shared(smem_u32(tail_full), rank);
        int stage = 0;
        // last use of each stage with a load that completes here (bits by stage): on which barrier and parity
        uint32_t phase = 0, armed = 0, on_tail = 0, full_par = 0, tail_par = 0;
        bool ok = true;
        for (int i = 0; ok && i * npairs < total; ++i) {
            const int u = snake_unit(i, pair, npairs, total);
            if (u < 0) continue;
            const WUnit w = unit_at(u);
            const WgradProblem& q = p.prob[w.prob];
            const CUtensorMap* map = m_side ? (w.g < E ? &q.a : &q.a_sh) : (w.g < E ? &q.b : &q.b_sh);
            const int row = w.g < E ? offs[w.g] : (m_side ? q.a_sh_row : q.b_sh_row);
            // first 64-column block: past M (zero fill) in the second CTA for an odd last block of M; for an odd
            // last block of N each CTA uses one of the two it loads
            const int blk = m_side ? w.mb * (kWgTile / 64) + 2 * rank : w.nb * (kWgTile / 64) + rank * (w.ncols / 128);
            const int n = stages_of(w), place = tail_place(w);
            for (int j = 0; j < n; ++j) {
                const uint32_t bit = 1u << stage;
                const bool tail = j == place;
                const int k = kWgKRows * (tail ? n - 1 : place >= 0 && j > place ? j - 1 : j);
                ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, p.err, abort_flag, true);
                if (!ok) break;
                if (m_side) {
                    if (tail) {
                        mbar_arrive_expect_tx(smem_u32(&tail_full[stage]), kWgStageBytes);
                        tail_par ^= bit;
                        on_tail |= bit;
                        armed |= bit;
                    } else if (rank == 0) {
                        mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * kWgStageBytes);
                        on_tail &= ~bit;
                        armed |= bit;
                    }
                    full_par = (full_par & ~bit) | (phase << stage);
                }
                tma_load_3d_pair(dst0 + (uint32_t)stage * kWgStageBytes, map, 0, row + k, blk,
                                 (tail ? tail0 : full0) + 8u * (uint32_t)stage, pol);
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
        }
        // every load that completes on a barrier of this CTA must land before the CTA may exit (an earlier
        // use of a stage has landed when the stage was used again); the M side waits for both
        for (int s = 0; s < S; ++s)
            if ((armed >> s) & 1u) {
                const bool t = (on_tail >> s) & 1u;
                mbar_wait(smem_u32(t ? &tail_full[s] : &full[s]), t ? ((tail_par >> s) & 1u) ^ 1u : (full_par >> s) & 1u,
                          p.err, abort_flag, false);
            }
    } else if (warp == 1 && rank == 0) {
        // ---------------------------------------------------------------- MMA issuer (first CTA)
        // The tensor cores take few MMAs ahead: whatever this warp does between one stage's MMAs and the
        // next's beyond the 512 clocks that they run is lost, and a lone warp needs some 5 clocks an
        // instruction. So its loop is one wait, four MMAs from two precomputed descriptors, one commit, with
        // the warp converged and one lane elected (a single running lane measured 7% slower).
        const uint32_t idesc0 = idesc_bf16_f32(256, 0) | kIdescAMajorM | kIdescBMajorN;
        const uint64_t a0 = smem_desc_mnmajor(smem_u32(tiles), kMnBoxBytes);
        const uint64_t b0 = smem_desc_mnmajor(smem_u32(tiles) + kWgABytes, kMnBoxBytes);
        const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), tfull0 = smem_u32(tfull), tempty0 = smem_u32(tempty);
        int stage = 0;
        uint32_t phase = 0, acc = 0, acc_phase = 1;
        bool ok = true;
        for (int i = 0; ok && i * npairs < total; ++i) {
            const int u = snake_unit(i, pair, npairs, total);
            if (u < 0) continue;
            const WUnit w = unit_at(u);
            const uint32_t idesc = idesc0 | ((uint32_t)(w.ncols >> 3) << 17);
            const uint32_t d = tmem_base + acc * kWgTile;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(tempty0 + 8 * acc, acc_phase, p.err, abort_flag, true));
            if (!ok) break;
            tc_fence_after();
            uint32_t accum = 0;
            const int n = stages_of(w), place = tail_place(w);
            int held = 0, left = w.rows;
            uint32_t held_phase = 0;
            for (int j = 0; j < n + (place >= 0 ? 1 : 0); ++j) {
                if (j == place) {   // the tail's stage: its turn comes last
                    held = stage;
                    held_phase = phase;
                    if (++stage == S) { stage = 0; phase ^= 1u; }
                    continue;
                }
                const bool tail = j == n;
                const int at = tail ? held : stage;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(full0 + 8 * at, tail ? held_phase : phase, p.err, abort_flag, true));
                if (!ok) break;
                tc_fence_after();
                const uint64_t a = a0 + (uint32_t)at * (kWgStageBytes >> 4), b = b0 + (uint32_t)at * (kWgStageBytes >> 4);
                if (elect_one()) {
                    umma_f16_ss_pair(d, a, b, idesc, accum);
                    if (left > 16) umma_f16_ss_pair(d, a + (kMnKStep >> 4), b + (kMnKStep >> 4), idesc, 1u);
                    if (left > 32) umma_f16_ss_pair(d, a + 2 * (kMnKStep >> 4), b + 2 * (kMnKStep >> 4), idesc, 1u);
                    if (left > 48) umma_f16_ss_pair(d, a + 3 * (kMnKStep >> 4), b + 3 * (kMnKStep >> 4), idesc, 1u);
                    umma_commit_pair_both(empty0 + 8 * at);
                }
                __syncwarp();
                accum = 1;
                left -= kWgKRows;
                if (!tail && ++stage == S) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            if (elect_one()) umma_commit_pair_both(tfull0 + 8 * acc);
            __syncwarp();
            acc ^= 1u;
            if (acc == 0) acc_phase ^= 1u;
        }
        // all MMAs issued must finish before TMEM is released
        if (elect_one()) {
            umma_commit_pair(mapa_shared(smem_u32(drain), 0));
            mbar_wait(smem_u32(drain), 0u, p.err, abort_flag, false);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------------------------------------------------------- row tails (both CTAs)
        int stage = 0;
        uint32_t tail_par = 0;
        bool ok = true;
        for (int i = 0; ok && i * npairs < total; ++i) {
            const int u = snake_unit(i, pair, npairs, total);
            if (u < 0) continue;
            const WUnit w = unit_at(u);
            const int n = stages_of(w), place = tail_place(w);
            const int last = (stage + place) % S, valid = w.rows - (n - 1) * kWgKRows;
            stage = (stage + n) % S;
            if (place < 0) continue;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&tail_full[last]), (tail_par >> last) & 1u, p.err, abort_flag, true));
            if (!ok) break;
            tail_par ^= 1u << last;
            // rows valid .. up to the next multiple of 16: whole 128-byte lines of every box, whatever the swizzle
            uint8_t* st = tiles + (size_t)last * kWgStageBytes + (lane & 7) * 16;
            const int end = (valid + 15) & ~15, boxes = 2 + w.ncols / 128;
            for (int r = valid + (lane >> 3); r < end; r += 4)
                for (int z = 0; z < boxes; ++z)
                    *reinterpret_cast<uint4*>(st + z * kMnBoxBytes + r * 128) = make_uint4(0u, 0u, 0u, 0u);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // for the tensor cores
            __syncwarp();
            if (rank != 0) {
                if (lane == 0) mbar_arrive_release_cluster(mapa_shared(smem_u32(&tail_ready[last]), 0));
            } else {
                const uint32_t bar = smem_u32(&tail_ready[last]), par = ((tail_par >> last) & 1u) ^ 1u;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait<kClusterScope>(bar, par, p.err, abort_flag, true));
                if (!ok) break;
                if (lane == 0) mbar_arrive(smem_u32(&full[last]));
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- epilogue: TMEM -> bf16 -> TMA store
        constexpr int G = kWgEpiWarps / 4;
        const int quarter = warp & 3, g0 = (warp - 4) >> 2;
        uint8_t* const stg0 = staging + (warp - 4) * 2 * kWgStoreBytes;
        int buf = 0;
        const uint64_t pol = l2_policy_evict_first();
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int i = 0; i * npairs < total; ++i) {
            const int u = snake_unit(i, pair, npairs, total);
            if (u < 0) continue;
            const WUnit w = unit_at(u);
            const WgradProblem& q = p.prob[w.prob];
            const int m = w.mb * kWgTile + rank * 128 + quarter * 32;
            const int part = m >= q.m_split ? 1 : 0;
            const CUtensorMap* om = w.g < E ? &q.out[part] : &q.out_sh[part];
            const int y = (w.g < E ? w.g * q.m_split : 0) + m - part * q.m_split;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&tfull[acc]), acc_phase, p.err, abort_flag, true))) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kWgTile);
            // the warp's boxes (64-column boxes g0, g0 + G, ..) into registers first, so that the accumulator
            // goes back before the stores
            constexpr int NBOX = kWgTile / 64 / G;
            uint32_t v[NBOX][32];
#pragma unroll
            for (int b = 0; b < NBOX; ++b) {
                const int c = 64 * (g0 + G * b);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t a[32];
                    if (w.rows > 0 && c < w.ncols) {
                        tmem_ld_x32_wait(t_row + c + 32 * z, a);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) a[j] = 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[b][16 * z + j] = pack_bf16x2(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]));
                }
            }
            // a relaxed arrive (tcgen05.wait::ld has completed every load), as in expert_gemm_pair_kernel
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tempty[acc]), 0));
#pragma unroll
            for (int b = 0; b < NBOX; ++b) {
                const int c = 64 * (g0 + G * b);
                if (c >= w.ncols || m >= q.M) break;
                // the store before the last has left this staging buffer
                uint8_t* stg = stg0 + buf * kWgStoreBytes;
                buf ^= 1;
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 8; ++x)   // the 128-byte swizzle: 16-byte chunk x of row l lies at x ^ (l & 7)
                    *reinterpret_cast<uint4*>(stg + lane * 128 + ((x ^ (lane & 7)) << 4)) =
                        make_uint4(v[b][4 * x], v[b][4 * x + 1], v[b][4 * x + 2], v[b][4 * x + 3]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(om, w.nb * kWgTile + c, y, smem_u32(stg), pol);
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
    if (*abort_flag) __nanosleep(100000);   // give loads still in flight after a timeout time to land
    cluster_sync();   // the peer's shared memory and TMEM stay alive until the pair's MMAs are done
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

cudaError_t run_wgrad(WgradParams& p, int num_sms, cudaStream_t s) {
    p.stages = kWgMaxStages;
    while (p.stages > 2 && wgrad_smem_bytes(p.stages, p.E) > (size_t)max_dynamic_smem()) --p.stages;
    for (WgradProblem& q : p.prob) {
        q.nb = (q.N + kWgTile - 1) / kWgTile;
        q.upg = q.nb * ((q.M + kWgTile - 1) / kWgTile);
        q.inv_nb = (uint32_t)(((1ull << 32) + q.nb - 1) / q.nb);   // 0 for 1, which is not divided by
        q.inv_upg = (uint32_t)(((1ull << 32) + q.upg - 1) / q.upg);
    }
    const size_t smem = wgrad_smem_bytes(p.stages, p.E);
    cudaError_t e = allow_smem(expert_wgrad_kernel, max_dynamic_smem());
    if (e != cudaSuccess) return e;
    static PerDevice resident;
    const int fit = resident_pairs(resident, expert_wgrad_kernel, kWgThreads, num_sms);
    if (fit == 0) return cudaErrorUnknown;
    LaunchTimer lt(K_EXPERT_WGRAD, s);
    return launch_pdl(expert_wgrad_kernel, dim3(2 * std::min(num_sms / 2, fit)), dim3(kWgThreads), smem, s, p);
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
    WgradParams pw = {};
    WgradProblem &wg = pw.prob[0], &wd = pw.prob[1];
    // packed weights viewed as rows of 64 columns, loaded in boxes of 64 rows
    if (!make_map(&m1.w, wdn, (uint64_t)(E + 1) * H * (I / 64), 64, 64, BK) || !act_maps(m1.act, b.dy, routed, H) ||
        !act_maps(m1.sh, b.dout, T, H) ||
        !make_map(&m2.w, wgu, (uint64_t)(E + 1) * 2 * I * (H / 64), 64, 64, BK) ||
        !act_maps(m2.act, b.dgu, rows, 2 * I) ||
        !make_wgrad_map(&wd.a, b.dy, routed, H) || !make_wgrad_map(&wd.a_sh, b.dout, T, H) ||
        !make_wgrad_map(&wd.b, b.h, rows, I) || !make_map(&wd.out[0], b.dw_down, (uint64_t)E * H, I, 32, BK) ||
        !make_map(&wd.out_sh[0], b.dws_down, H, I, 32, BK) ||
        !make_wgrad_map(&wg.a, b.dgu, rows, 2 * I) || !make_wgrad_map(&wg.b, b.x_perm, routed, H) ||
        !make_wgrad_map(&wg.b_sh, b.x, T, H) ||
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
    wg.M = 2 * I;
    wg.N = H;
    wg.m_split = I;
    wg.a_sh_row = (int)routed;
    wd.M = wd.m_split = H;
    wd.N = I;
    wd.b_sh_row = (int)routed;
    pw.offsets = b.offsets;
    pw.E = E;
    pw.T = (int)T;
    pw.routed_rows = (int)routed;
    pw.err = err;
    e = run_wgrad(pw, num_sms, s);
    if (e == cudaSuccess) launches_add(3);
    return e;
}

}  // namespace smoe
