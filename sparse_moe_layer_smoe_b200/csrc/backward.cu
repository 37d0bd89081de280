// Backward passes of the layer's routing steps, and the checkpoint's values.
//
//   combine_backward   out[t] = y_shared[t] + sum_j w[t,j] y[r(t,j)]  gives
//                      dy[r(t,j)] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[r(t,j)]>
//   permute_backward   every token's row went to k experts, the shared expert and the router:
//                      dx[t] = dx_rows[T*k + t] + sum_j dx_rows[r(t,j)] + sum_j dl[t,j] W_r[e(t,j)]
//   route_backward     w_j = c s_j / S with s = sigmoid(l), S = sum of the selected s:
//                      dl_j = w_j (1 - s_j) sum_i (w_i / c) (dw_j - dw_i)
//                      dW_r[e] = sum over the rows r of expert e of dl[r] x[token(r)]
//                      (the differences keep k = 1 exactly 0 and lose nothing where the dw are close;
//                      the selection and its bias have no gradient)
// Sources as for the forward steps: Step 3.5 Flash summary (hyper.ai), section "方法"; model card fields
// moe_router_activation sigmoid, norm_expert_weight, moe_router_scaling_factor.
// All sums are fp32 in a fixed order; every result is rounded once.
#include "common.cuh"
#include "internal.h"

namespace smoe {

namespace {

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

constexpr int kSlots = 8;      // slots a pass over a token's row takes (top-k 8; a larger k takes several passes)
constexpr int kMaxWarps = 8;
constexpr int kAhead = 2;      // router rows in flight beside the routed ones (1, 2 and 4 measure the same)

// One CTA per token; a thread owns 8 consecutive features of every row and has all k of them in flight.
// HBM-bound: 8192 tokens of H = 4096, k = 8 in 178 us, 6.4 TB/s (two CTAs an SM instead of three: 199 us;
// four spill: 241 us). y is read for the last time and passes through L2 (evict-first: 185 us without).
__global__ void __launch_bounds__(256, 3) combine_backward_kernel(const uint16_t* __restrict__ dout,
                                                               const uint16_t* __restrict__ y,
                                                               const int32_t* __restrict__ perm_row,
                                                               const float* __restrict__ topk_w, int T, int k, int H,
                                                               uint16_t* __restrict__ dy, float* __restrict__ dtopk_w,
                                                               int32_t* err) {
    __shared__ int32_t rows[kSlots];
    __shared__ float ws[kSlots];
    __shared__ float red[kMaxWarps][kSlots];
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int vec = H / 8;
    const int64_t nrouted = (int64_t)T * k;
    const uint4* d4 = reinterpret_cast<const uint4*>(dout) + (size_t)t * vec;
    const uint64_t pass = l2_policy_evict_first();
    for (int j0 = 0; j0 < k; j0 += kSlots) {
        const int n = min(kSlots, k - j0);
        if (threadIdx.x < kSlots) {
            int32_t r = -1;
            if ((int)threadIdx.x < n) {
                r = perm_row[(size_t)t * k + j0 + threadIdx.x];
                if (r < 0 || r >= nrouted) {
                    record_error(err, SMOE_ERR_DEVICE);
                    r = -1;
                }
                ws[threadIdx.x] = topk_w[(size_t)t * k + j0 + threadIdx.x];
            }
            rows[threadIdx.x] = r;
        }
        __syncthreads();
        float dot[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) dot[j] = 0.f;
        for (int c = threadIdx.x; c < vec; c += blockDim.x) {
            float d[8];
            unpack8(d4[c], d);
            uint4 v[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (rows[j] >= 0) v[j] = ld_global_hint(reinterpret_cast<const uint4*>(y) + (size_t)rows[j] * vec + c, pass);
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (rows[j] >= 0) {
                    float f[8], o[8];
                    unpack8(v[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[j] = fmaf(d[i], f[i], dot[j]);
                        o[i] = ws[j] * d[i];
                    }
                    reinterpret_cast<uint4*>(dy)[(size_t)rows[j] * vec + c] = pack8(o);
                }
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], off);
            if (lane == 0) red[warp][j] = dot[j];
        }
        __syncthreads();
        if ((int)threadIdx.x < n) {
            float s = 0.f;
            for (int q = 0; q < nw; ++q) s += red[q][threadIdx.x];
            dtopk_w[(size_t)t * k + j0 + threadIdx.x] = s;   // 0 for a skipped entry
        }
        __syncthreads();
    }
}

// One token's dx, by the threads of a CTA. rows, experts, dl: 32 slots each (rows, experts -1: none). PADDED:
// some of the slots that the loop takes have no expert (k no multiple of 8, skipped entries); without that check
// of every slot 8192 tokens take 128 us instead of 130.4.
template <bool ROUTER, bool PADDED>
__device__ __forceinline__ void permute_backward_row(const uint4* __restrict__ rows4, const uint4* __restrict__ own,
                                                     const float* __restrict__ w_router, const int32_t* rows,
                                                     const int32_t* experts, const float* dl, int k, int H,
                                                     uint4* __restrict__ out) {
    const int vec = H / 8;
    for (int c = threadIdx.x; c < vec; c += blockDim.x) {
        float acc[8];
        unpack8(own[c], acc);
        for (int j0 = 0; j0 < k; j0 += kSlots) {
            // the rows and the first router weights in flight together, then the rest of the weights
            uint4 v[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                v[j] = make_uint4(0u, 0u, 0u, 0u);
                if (rows[j0 + j] >= 0) v[j] = rows4[(size_t)rows[j0 + j] * vec + c];
            }
#pragma unroll
            for (int z = 0; z < kSlots; z += kAhead) {
                float4 a[kAhead], b[kAhead];
                if (ROUTER) {
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) {
                        const int32_t e = experts[j0 + z + j];
                        if (PADDED) a[j] = b[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (!PADDED || e >= 0) {
                            const float4* w4 = reinterpret_cast<const float4*>(w_router + (size_t)e * H) + 2 * c;
                            a[j] = w4[0];
                            b[j] = w4[1];
                        }
                    }
                }
                if (z == 0) {
#pragma unroll
                    for (int j = 0; j < kSlots; ++j) {
                        float f[8];
                        unpack8(v[j], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] += f[i];
                    }
                }
                if (ROUTER) {
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) {
                        const float g = dl[j0 + z + j];
                        acc[0] = fmaf(g, a[j].x, acc[0]);
                        acc[1] = fmaf(g, a[j].y, acc[1]);
                        acc[2] = fmaf(g, a[j].z, acc[2]);
                        acc[3] = fmaf(g, a[j].w, acc[3]);
                        acc[4] = fmaf(g, b[j].x, acc[4]);
                        acc[5] = fmaf(g, b[j].y, acc[5]);
                        acc[6] = fmaf(g, b[j].z, acc[6]);
                        acc[7] = fmaf(g, b[j].w, acc[7]);
                    }
                }
            }
        }
        out[c] = pack8(acc);
    }
}

// One CTA per token. The router's term is left out when dlogits is null. With it a token reads 16 KB of the
// router's weights for each of its experts (at H = 4096), more than the rows themselves, but from L2: 8192
// tokens take 137 to 142 us, 4.9 TB/s of HBM beside as much again and half from L2 (128 us where every pass writes
// the same output, which then stays in L2; the other figures here are of that kind). Four CTAs an SM matter
// (three: 139 us, two: 163). Keeping the weights of a 128-feature slice of all experts in shared memory, so
// that only the rows cross L2, was slower: 228 us, as rows are then read in 256-byte pieces.
__global__ void __launch_bounds__(256, 4) permute_backward_kernel(const uint16_t* __restrict__ dx_rows,
                                                               const int32_t* __restrict__ perm_row,
                                                               const int32_t* __restrict__ topk_idx,
                                                               const float* __restrict__ dlogits,
                                                               const float* __restrict__ w_router, int T, int k, int E,
                                                               int H, uint16_t* __restrict__ dx, int32_t* err) {
    __shared__ int32_t rows[32], experts[32];
    __shared__ float dl[32];
    __shared__ unsigned with_expert;   // slots, as bits
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x;
    const int vec = H / 8;
    const int64_t nrouted = (int64_t)T * k;
    if (threadIdx.x < 32) {
        const size_t i = (size_t)t * k + threadIdx.x;
        int32_t r = -1, e = -1;
        float g = 0.f;
        const bool entry = (int)threadIdx.x < k;
        if (entry) r = perm_row[i];
        if (entry && (r < 0 || r >= nrouted)) {
            record_error(err, SMOE_ERR_DEVICE);
            r = -1;
        }
        if (entry && dlogits != nullptr) {
            e = topk_idx[i];
            g = dlogits[i];
            if (e < 0 || e >= E) {
                record_error(err, SMOE_ERR_DEVICE);
                e = -1;
                g = 0.f;
            }
        }
        rows[threadIdx.x] = r;
        const unsigned valid = __ballot_sync(0xFFFFFFFFu, e >= 0);
        experts[threadIdx.x] = e;   // -1 past k and for skipped entries: nothing is read, and 0 * 0 added
        dl[threadIdx.x] = g;
        if (threadIdx.x == 0) with_expert = valid;
    }
    __syncthreads();
    const uint4* rows4 = reinterpret_cast<const uint4*>(dx_rows);
    const uint4* own = rows4 + (size_t)(nrouted + t) * vec;
    uint4* out = reinterpret_cast<uint4*>(dx) + (size_t)t * vec;
    if (with_expert == 0)   // also without dlogits
        permute_backward_row<false, false>(rows4, own, w_router, rows, experts, dl, k, H, out);
    else if (k % kSlots == 0 && __popc(with_expert) == k)
        permute_backward_row<true, false>(rows4, own, w_router, rows, experts, dl, k, H, out);
    else
        permute_backward_row<true, true>(rows4, own, w_router, rows, experts, dl, k, H, out);
}

// dl of entry i = t * k + j, whose selected logit is l.
__device__ __forceinline__ float dlogit(const float* __restrict__ w, const float* __restrict__ dw, int64_t t, int j, int k,
                                        float l, float inv_c) {
    const float dwj = dw[t * k + j];
    float sum = 0.f;
    for (int q = 0; q < k; ++q) sum = fmaf(w[t * k + q] * inv_c, dwj - dw[t * k + q], sum);
    return w[t * k + j] * (1.0f / (1.0f + expf(l))) * sum;   // 1 / (1 + e^l) = 1 - sigmoid(l)
}

constexpr int kRbThreads = 256;   // 8 features a thread: 2048 features a CTA
constexpr int kRbFlight = 8;      // rows in flight a thread

// One launch for both gradients. Item = up to kRouterItemRows rows of one expert, or all of them where the
// batch has no more tokens than that (an expert without rows has one empty item, which writes its zeros). CTA (x, y): for x below the item bound, item x's sum over
// its rows in order, for the 2048 features of slice y; it works out its item from the offsets and its
// rows' dl from the tokens' weights itself, so nothing has to run before it. Above the bound (y = 0):
// dlogits of 256 entries each. An expert of one item writes dW_r, the others' items partial sums. Rows
// are gathered from x in L2 (each is read by k experts), which bounds it: 4096 tokens read 268 MB in 31 us,
// 8.6 TB/s; 4 or 16 rows in flight and CTAs of 128 or 512 threads measure within 5% of that. Items of 256
// rows instead of 64: the same on even batches, but 46 us instead of 35 on a skewed one of 4096 tokens and
// 29 instead of 14 on one of 257, whose popular experts' long sums run alone at the end.
__global__ void __launch_bounds__(kRbThreads) router_backward_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const float* __restrict__ topk_w, const float* __restrict__ dtopk_w, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ perm_row, const int32_t* __restrict__ row_token, int T, int k, int E, int H, float inv_c,
    int max_items, float* __restrict__ dlogits, float* __restrict__ partial, float* __restrict__ dw_router, int32_t* err) {
    __shared__ int32_t tok[kRouterItemRows];
    __shared__ float g[kRouterItemRows];
    __shared__ int32_t warp_tot[kRbThreads / 32];
    __shared__ int4 found;   // expert, first row, rows, items of the expert
    const bool whole = T <= kRouterItemRows;   // an expert's rows are one item
    pdl_wait();
    pdl_launch_dependents();
    const int64_t nrouted = (int64_t)T * k;
    if ((int)blockIdx.x >= max_items) {
        const int64_t i = (int64_t)(blockIdx.x - max_items) * kRbThreads + threadIdx.x;
        if (blockIdx.y != 0 || i >= nrouted) return;
        const int64_t t = i / k;
        const int32_t e = topk_idx[i], r = perm_row[i];
        // an entry without a row is not in dw_router's sums, so its logit has no gradient either
        const bool has_row = e >= 0 && e < E && r >= 0 && r < nrouted;
        if (!has_row) record_error(err, SMOE_ERR_DEVICE);
        dlogits[i] = has_row ? dlogit(topk_w, dtopk_w, t, (int)(i % k), k, logits[t * E + e], inv_c) : 0.f;
        return;
    }
    // find the item: a scan of the experts' item counts, each thread a contiguous range of experts
    {
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
        const int chunk = (E + kRbThreads - 1) / kRbThreads, e0 = min((int)threadIdx.x * chunk, E), e1 = min(e0 + chunk, E);
        bool bad = false;
        int n = 0;
        for (int e = e0; e < e1; ++e) {
            const int a = offsets[e], b = offsets[e + 1];
            bad |= a < 0 || b < a || b > nrouted;
            n += whole ? 1 : max(1, (b - a + kRouterItemRows - 1) / kRouterItemRows);
        }
        bad = __syncthreads_or(bad);   // corrupt offsets: no rows, one empty item each
        if (bad) {
            n = e1 - e0;
            if (threadIdx.x == 0) record_error(err, SMOE_ERR_DEVICE);
        }
        int v = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, v, off);
            if (lane >= off) v += u;
        }
        if (lane == 31) warp_tot[w] = v;
        if (threadIdx.x == 0) found = make_int4(-1, 0, 0, 0);
        __syncthreads();
        int first = v - n;
        for (int q = 0; q < w; ++q) first += warp_tot[q];
        const int item = blockIdx.x;
        if (item >= first && item < first + n)
            for (int e = e0; e < e1; ++e) {
                const int a = bad ? 0 : offsets[e], b = bad ? 0 : offsets[e + 1];
                const int m = whole ? 1 : max(1, (b - a + kRouterItemRows - 1) / kRouterItemRows);
                if (item < first + m) {
                    const int r = (item - first) * kRouterItemRows;
                    found = make_int4(e, a + r, whole ? b - a : min(kRouterItemRows, b - a - r), m);
                    break;
                }
                first += m;
            }
        __syncthreads();
    }
    const int4 it = found;
    if (it.x < 0) return;
    static_assert(kRouterItemRows <= kRbThreads, "one row of an item a thread");
    const int c = blockIdx.y * kRbThreads + threadIdx.x;   // 8-feature vector
    const int vec = H / 8;
    const uint4* x4 = reinterpret_cast<const uint4*>(x) + c;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int row0 = 0; row0 < it.z; row0 += kRouterItemRows) {
        const int rows = min(kRouterItemRows, it.z - row0);
        int my_t = -1;
        if (row0 > 0) __syncthreads();   // the rows before these have been read
        if ((int)threadIdx.x < rows) {
            my_t = row_token[it.y + row0 + threadIdx.x];
            tok[threadIdx.x] = my_t >= 0 && my_t < T ? my_t : 0;
        }
        __syncthreads();
        if ((int)threadIdx.x < rows) {
            const int r = it.y + row0 + threadIdx.x, t = my_t;
            float d = 0.f;
            bool ok = t >= 0 && t < T;
            if (ok) {
                int j = -1;
                for (int q = 0; q < k; ++q)
                    if (perm_row[(int64_t)t * k + q] == r) j = q;
                ok = j >= 0;
                if (ok) d = dlogit(topk_w, dtopk_w, t, j, k, logits[(int64_t)t * E + it.x], inv_c);
            }
            if (!ok) record_error(err, SMOE_ERR_DEVICE);   // a row that is not its token's
            g[threadIdx.x] = d;
        }
        __syncthreads();
        if (c >= vec) continue;
        int r = 0;
        for (; r + kRbFlight <= rows; r += kRbFlight) {
            uint4 v[kRbFlight];
#pragma unroll
            for (int q = 0; q < kRbFlight; ++q) v[q] = x4[(size_t)tok[r + q] * vec];
#pragma unroll
            for (int q = 0; q < kRbFlight; ++q) {
                float f[8];
                unpack8(v[q], f);
                const float s = g[r + q];
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(s, f[i], acc[i]);
            }
        }
        for (; r < rows; ++r) {
            float f[8];
            unpack8(x4[(size_t)tok[r] * vec], f);
            const float s = g[r];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(s, f[i], acc[i]);
        }
    }
    if (c >= vec) return;
    float4* o = reinterpret_cast<float4*>((it.w == 1 ? dw_router + (size_t)it.x * H : partial + (size_t)blockIdx.x * H) + 8 * c);
    o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// Experts of several items: their partial sums added in a fixed order. The items before an expert's are
// counted from the offsets, as above.
__global__ void __launch_bounds__(256) router_wgrad_join_kernel(const float* __restrict__ partial,
                                                               const int32_t* __restrict__ offsets, int64_t nrouted, int H,
                                                               float* __restrict__ dw) {
    pdl_wait();
    pdl_launch_dependents();
    const int e = blockIdx.x, E = gridDim.x;
    // only for batches of more than kRouterItemRows tokens, whose items are of that many rows
    const int n = (offsets[e + 1] - offsets[e] + kRouterItemRows - 1) / kRouterItemRows;
    if (n <= 1) return;
    __shared__ int32_t part[8];
    int before = 0;
    bool bad = false;
    for (int q = threadIdx.x; q < E; q += 256) {
        const int a = offsets[q], b = offsets[q + 1];
        bad |= a < 0 || b < a || b > nrouted;
        if (q < e) before += max(1, (b - a + kRouterItemRows - 1) / kRouterItemRows);
    }
    if (__syncthreads_or(bad)) return;   // every expert had one empty item
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = before;
    __syncthreads();
    before = 0;
    for (int q = 0; q < 8; ++q) before += part[q];
    // two groups of threads take half of the items each
    __shared__ float4 half[128];
    const int col = threadIdx.x & 127, grp = threadIdx.x >> 7, per = (n + 1) / 2;
    const int c = blockIdx.y * 128 + col;   // 4-feature vector
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < H / 4) {
#pragma unroll 8
        for (int i = before + grp * per; i < before + min(n, (grp + 1) * per); ++i) {
            const float4 v = reinterpret_cast<const float4*>(partial + (size_t)i * H)[c];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    if (grp == 1) half[col] = s;
    __syncthreads();
    if (grp != 0 || c >= H / 4) return;
    s.x += half[col].x;
    s.y += half[col].y;
    s.z += half[col].z;
    s.w += half[col].w;
    reinterpret_cast<float4*>(dw + (size_t)e * H)[c] = s;
}

// Values of the checkpoint: bf16 holds a code times its scale exactly (short of bf16's own range). A lane
// takes 8 codes, so that a warp's stores are contiguous (16 codes and two stores: 150 us instead of 109 for
// 8192 tokens, 0.57 GB); a block 32 rows, so that a 32-byte sector of the column-wise scales serves all.
__global__ void __launch_bounds__(256) checkpoint_values_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t rows, int cols,
                                                               uint16_t* __restrict__ gu) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (blockIdx.y * 32 + lane) * 8;
    if (col >= cols) return;
    const int64_t r0 = (int64_t)blockIdx.x * 32 + warp * 4;
    uint2 q[4];
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (r0 + i < rows) {
            q[i] = *reinterpret_cast<const uint2*>(codes + (size_t)(r0 + i) * cols + col);
            e[i] = scales[(size_t)(col / 32) * rows + r0 + i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (r0 + i >= rows) return;
        const float s = __uint_as_float(e[i] << 23);
        const float2 a = e4m3x2_to_float2(q[i].x & 0xFFFFu), b = e4m3x2_to_float2(q[i].x >> 16);
        const float2 c = e4m3x2_to_float2(q[i].y & 0xFFFFu), d = e4m3x2_to_float2(q[i].y >> 16);
        *reinterpret_cast<uint4*>(gu + (size_t)(r0 + i) * cols + col) =
            make_uint4(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s), pack_bf16x2(c.x * s, c.y * s),
                       pack_bf16x2(d.x * s, d.y * s));
    }
}

int row_threads(int H) { return H / 8 >= 256 ? 256 : 128; }

}  // namespace

BwdLayout bwd_layout(const smoe_config_t& c, int64_t T) {
    BwdLayout L;
    const int64_t routed = T * c.top_k, rows = routed + T, items = router_max_items(T, c.top_k, c.n_experts);
    size_t o = kAlign;
    L.dgu = o;  o += align_up((size_t)rows * 2 * c.inter * 2);
    L.h = o;    o += align_up((size_t)rows * c.inter * 2);
    L.total = o;
    o = kAlign;
    L.partial = o;  o += align_up((size_t)items * c.hidden * 4);
    if (o > L.total) L.total = o;
    return L;
}

cudaError_t launch_combine_backward(const smoe_config_t& c, const uint16_t* dout, const uint16_t* y,
                                    const int32_t* perm_row, const float* topk_w, int64_t T, uint16_t* dy,
                                    float* dtopk_w, int32_t* err, cudaStream_t s) {
    cudaError_t e;
    {
        LaunchTimer lt(K_COMBINE_BACKWARD, s);
        e = launch_pdl(combine_backward_kernel, dim3((unsigned)T), dim3(row_threads(c.hidden)), 0, s, dout, y, perm_row,
                       topk_w, (int)T, c.top_k, c.hidden, dy, dtopk_w, err);
    }
    if (e == cudaSuccess) launches_add(1);
    return e;
}

cudaError_t launch_permute_backward(const smoe_config_t& c, const uint16_t* dx_rows, const int32_t* perm_row,
                                    const int32_t* topk_idx, const float* dlogits, const float* w_router, int64_t T,
                                    uint16_t* dx, int32_t* err, cudaStream_t s) {
    cudaError_t e;
    {
        LaunchTimer lt(K_PERMUTE_BACKWARD, s);
        e = launch_pdl(permute_backward_kernel, dim3((unsigned)T), dim3(row_threads(c.hidden)), 0, s, dx_rows, perm_row,
                       topk_idx, dlogits, w_router, (int)T, c.top_k, c.n_experts, c.hidden, dx, err);
    }
    if (e == cudaSuccess) launches_add(1);
    return e;
}

cudaError_t launch_route_backward(const smoe_config_t& c, const RouteBackward& b, int64_t T, int32_t* err,
                                  cudaStream_t s) {
    const int E = c.n_experts, H = c.hidden, k = c.top_k;
    const unsigned items = (unsigned)router_max_items(T, k, E), entries = (unsigned)((T * k + kRbThreads - 1) / kRbThreads);
    cudaError_t e;
    {
        LaunchTimer lt(K_ROUTER_BACKWARD, s);
        e = launch_pdl(router_backward_kernel, dim3(items + entries, (H / 8 + kRbThreads - 1) / kRbThreads), dim3(kRbThreads), 0, s, b.x,
                       b.logits, b.topk_idx, b.topk_w, b.dtopk_w, b.offsets, b.perm_row, b.row_token, (int)T, k, E, H,
                       1.0f / c.route_scale, (int)items, b.dlogits, b.partial, b.dw_router, err);
    }
    if (e != cudaSuccess) return e;
    launches_add(1);
    if (T <= kRouterItemRows) return cudaSuccess;   // one item an expert
    {
        LaunchTimer lt(K_ROUTER_WGRAD_JOIN, s);
        e = launch_pdl(router_wgrad_join_kernel, dim3(E, (H / 4 + 127) / 128), dim3(256), 0, s, (const float*)b.partial,
                       b.offsets, T * k, H, b.dw_router);
    }
    if (e == cudaSuccess) launches_add(1);
    return e;
}

cudaError_t launch_checkpoint_values(const smoe_config_t& c, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                     uint16_t* gu, cudaStream_t s) {
    const int cols = 2 * c.inter;
    cudaError_t e;
    {
        LaunchTimer lt(K_CHECKPOINT_VALUES, s);
        e = launch_pdl(checkpoint_values_kernel, dim3((unsigned)((rows + 31) / 32), (cols + 255) / 256), dim3(256), 0, s,
                       codes, scales, rows, cols, gu);
    }
    if (e == cudaSuccess) launches_add(1);
    return e;
}

}  // namespace smoe
