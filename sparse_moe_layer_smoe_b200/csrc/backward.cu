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

// One CTA per token; a thread owns 8 consecutive features of every row.
__global__ void __launch_bounds__(256) combine_backward_kernel(const uint16_t* __restrict__ dout,
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
                if (rows[j] >= 0) v[j] = reinterpret_cast<const uint4*>(y)[(size_t)rows[j] * vec + c];
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

// One CTA per token. The router's term is left out when dlogits is null.
__global__ void __launch_bounds__(256) permute_backward_kernel(const uint16_t* __restrict__ dx_rows,
                                                               const int32_t* __restrict__ perm_row,
                                                               const int32_t* __restrict__ topk_idx,
                                                               const float* __restrict__ dlogits,
                                                               const float* __restrict__ w_router, int T, int k, int E,
                                                               int H, uint16_t* __restrict__ dx, int32_t* err) {
    __shared__ int32_t rows[32], experts[32];
    __shared__ float dl[32];
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x;
    const int vec = H / 8;
    const int64_t nrouted = (int64_t)T * k;
    if ((int)threadIdx.x < k) {
        const size_t i = (size_t)t * k + threadIdx.x;
        int32_t r = perm_row[i], e = -1;
        float g = 0.f;
        if (r < 0 || r >= nrouted) {
            record_error(err, SMOE_ERR_DEVICE);
            r = -1;
        }
        if (dlogits != nullptr) {
            e = topk_idx[i];
            g = dlogits[i];
            if (e < 0 || e >= E) {
                record_error(err, SMOE_ERR_DEVICE);
                e = -1;
            }
        }
        rows[threadIdx.x] = r;
        experts[threadIdx.x] = e;
        dl[threadIdx.x] = g;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < vec; c += blockDim.x) {
        float acc[8];
        unpack8(reinterpret_cast<const uint4*>(dx_rows)[(size_t)(nrouted + t) * vec + c], acc);
        for (int j0 = 0; j0 < k; j0 += kSlots) {
            uint4 v[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (j0 + j < k && rows[j0 + j] >= 0)
                    v[j] = reinterpret_cast<const uint4*>(dx_rows)[(size_t)rows[j0 + j] * vec + c];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (j0 + j < k && rows[j0 + j] >= 0) {
                    float f[8];
                    unpack8(v[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] += f[i];
                }
        }
        for (int j = 0; j < k; ++j)
            if (experts[j] >= 0) {
                const float4* w4 = reinterpret_cast<const float4*>(w_router + (size_t)experts[j] * H) + 2 * c;
                const float4 a = w4[0], b = w4[1];
                const float g = dl[j];
                acc[0] = fmaf(g, a.x, acc[0]);
                acc[1] = fmaf(g, a.y, acc[1]);
                acc[2] = fmaf(g, a.z, acc[2]);
                acc[3] = fmaf(g, a.w, acc[3]);
                acc[4] = fmaf(g, b.x, acc[4]);
                acc[5] = fmaf(g, b.y, acc[5]);
                acc[6] = fmaf(g, b.z, acc[6]);
                acc[7] = fmaf(g, b.w, acc[7]);
            }
        reinterpret_cast<uint4*>(dx)[(size_t)t * vec + c] = pack8(acc);
    }
}

// Entry (t, j) per thread: dlogits, and the same value in row order for the weight gradient. The last
// block lists the items of the weight gradient instead: every expert's rows in pieces of
// kRouterItemRows (an expert without rows has one empty item, which writes its zeros).
__global__ void __launch_bounds__(1024) router_dlogits_kernel(const float* __restrict__ logits,
                                                             const int32_t* __restrict__ topk_idx,
                                                             const float* __restrict__ topk_w,
                                                             const float* __restrict__ dtopk_w,
                                                             const int32_t* __restrict__ offsets,
                                                             const int32_t* __restrict__ perm_row, int T, int k, int E,
                                                             float inv_c, float* __restrict__ dlogits,
                                                             float* __restrict__ dl_row, int4* __restrict__ items,
                                                             int32_t* __restrict__ first_item, int32_t* err) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t nrouted = (int64_t)T * k;
    if (blockIdx.x == gridDim.x - 1) {
        __shared__ int32_t warp_tot[32];
        __shared__ int bad;
        const int e = threadIdx.x, lane = e & 31, w = e >> 5;
        if (e == 0) bad = 0;
        __syncthreads();
        int32_t r0 = 0, r1 = 0;
        if (e < E) {
            r0 = offsets[e];
            r1 = offsets[e + 1];
            if (r0 < 0 || r1 < r0 || r1 > nrouted) bad = 1;
        }
        __syncthreads();
        if (bad) {   // corrupt offsets: no rows
            r0 = r1 = 0;
            if (e == 0) record_error(err, SMOE_ERR_DEVICE);
        }
        const int n = e < E ? max(1, (r1 - r0 + kRouterItemRows - 1) / kRouterItemRows) : 0;
        int32_t v = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, off);
            if (lane >= off) v += u;
        }
        if (lane == 31) warp_tot[w] = v;
        __syncthreads();
        if (w == 0) {
            int32_t tv = warp_tot[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t u = __shfl_up_sync(0xFFFFFFFFu, tv, off);
                if (lane >= off) tv += u;
            }
            warp_tot[lane] = tv;
        }
        __syncthreads();
        const int32_t first = v + (w > 0 ? warp_tot[w - 1] : 0) - n;
        if (e < E) {
            first_item[e] = first;
            for (int i = 0; i < n; ++i)
                items[first + i] = make_int4(e, r0 + i * kRouterItemRows,
                                             min(kRouterItemRows, r1 - r0 - i * kRouterItemRows), n);
            if (e == E - 1) first_item[E] = first + n;
        }
        return;
    }
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= nrouted) return;
    const int64_t t = i / k;
    const int32_t e = topk_idx[i];
    float g = 0.f;
    if (e >= 0 && e < E) {
        const float dwj = dtopk_w[i];
        float sum = 0.f;
        for (int q = 0; q < k; ++q) sum = fmaf(topk_w[t * k + q] * inv_c, dwj - dtopk_w[t * k + q], sum);
        const float rest = 1.0f / (1.0f + expf(logits[t * E + e]));   // 1 - sigmoid(l)
        g = topk_w[i] * rest * sum;
    } else {
        record_error(err, SMOE_ERR_DEVICE);
    }
    dlogits[i] = g;
    const int32_t r = perm_row[i];
    if (r >= 0 && r < nrouted)
        dl_row[r] = g;
    else
        record_error(err, SMOE_ERR_DEVICE);
}

constexpr int kWgThreadsRouter = 128;   // 8 features a thread: 1024 features a CTA

// CTA (item, 1024-feature slice): the item's rows in order, fp32. An expert of one item writes dW_r,
// others their partial sum.
__global__ void __launch_bounds__(kWgThreadsRouter) router_wgrad_kernel(const uint16_t* __restrict__ x,
                                                                        const float* __restrict__ dl_row,
                                                                        const int32_t* __restrict__ row_token,
                                                                        const int4* __restrict__ items,
                                                                        const int32_t* __restrict__ first_item, int T,
                                                                        int E, int H, float* __restrict__ partial,
                                                                        float* __restrict__ dw, int32_t* err) {
    __shared__ int32_t tok[kRouterItemRows];
    __shared__ float g[kRouterItemRows];
    pdl_wait();
    pdl_launch_dependents();
    const int item = blockIdx.x;
    if (item >= first_item[E]) return;
    const int4 it = items[item];
    for (int i = threadIdx.x; i < it.z; i += kWgThreadsRouter) {
        int32_t t = row_token[it.y + i];
        float v = dl_row[it.y + i];
        if (t < 0 || t >= T) {
            record_error(err, SMOE_ERR_DEVICE);
            t = 0;
            v = 0.f;
        }
        tok[i] = t;
        g[i] = v;
    }
    __syncthreads();
    const int c = blockIdx.y * kWgThreadsRouter + threadIdx.x;   // 8-feature vector
    if (c >= H / 8) return;
    const uint4* x4 = reinterpret_cast<const uint4*>(x) + c;
    const int vec = H / 8;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    int r = 0;
    for (; r + 8 <= it.z; r += 8) {
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = x4[(size_t)tok[r + q] * vec];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float f[8];
            unpack8(v[q], f);
            const float s = g[r + q];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(s, f[i], acc[i]);
        }
    }
    for (; r < it.z; ++r) {
        float f[8];
        unpack8(x4[(size_t)tok[r] * vec], f);
        const float s = g[r];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(s, f[i], acc[i]);
    }
    float4* o = reinterpret_cast<float4*>((it.w == 1 ? dw + (size_t)it.x * H : partial + (size_t)item * H) + 8 * c);
    o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// Experts of several items: their partial sums added in item order.
__global__ void __launch_bounds__(256) router_wgrad_join_kernel(const float* __restrict__ partial,
                                                               const int32_t* __restrict__ first_item, int H,
                                                               float* __restrict__ dw) {
    pdl_wait();
    pdl_launch_dependents();
    const int e = blockIdx.x;
    const int a = first_item[e], b = first_item[e + 1];
    if (b - a <= 1) return;
    const int c = blockIdx.y * 256 + threadIdx.x;   // 4-feature vector
    if (c >= H / 4) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = a; i < b; ++i) {
        const float4 v = reinterpret_cast<const float4*>(partial + (size_t)i * H)[c];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    reinterpret_cast<float4*>(dw + (size_t)e * H)[c] = s;
}

// Values of the checkpoint: bf16 holds a code times its scale exactly (short of bf16's own range). Block:
// 32 rows, so that a 32-byte sector of the column-wise scales serves all of them; a lane takes 16 codes.
__global__ void __launch_bounds__(256) checkpoint_values_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t rows, int cols,
                                                               uint16_t* __restrict__ gu) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (blockIdx.y * 32 + lane) * 16;
    if (col >= cols) return;
    for (int i = 0; i < 4; ++i) {
        const int64_t r = (int64_t)blockIdx.x * 32 + warp * 4 + i;
        if (r >= rows) return;
        const uint4 q = *reinterpret_cast<const uint4*>(codes + (size_t)r * cols + col);
        const float s = __uint_as_float((uint32_t)scales[(size_t)(col / 32) * rows + r] << 23);
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
        uint32_t o[8];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const float2 a = e4m3x2_to_float2(u[z] & 0xFFFFu), b = e4m3x2_to_float2(u[z] >> 16);
            o[2 * z] = pack_bf16x2(a.x * s, a.y * s);
            o[2 * z + 1] = pack_bf16x2(b.x * s, b.y * s);
        }
        uint4* d = reinterpret_cast<uint4*>(gu + (size_t)r * cols + col);
        d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        d[1] = make_uint4(o[4], o[5], o[6], o[7]);
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
    L.dl_row = o;   o += align_up((size_t)routed * 4);
    L.items = o;    o += align_up((size_t)items * sizeof(int4));
    L.n_items = o;  o += align_up((size_t)(c.n_experts + 1) * 4);
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
    const unsigned blocks = (unsigned)((T * k + 1023) / 1024);
    cudaError_t e;
    {
        LaunchTimer lt(K_ROUTER_DLOGITS, s);
        e = launch_pdl(router_dlogits_kernel, dim3(blocks + 1), dim3(1024), 0, s, b.logits, b.topk_idx, b.topk_w,
                       b.dtopk_w, b.offsets, b.perm_row, (int)T, k, E, 1.0f / c.route_scale, b.dlogits, b.dl_row, b.items,
                       b.n_items, err);
    }
    if (e != cudaSuccess) return e;
    {
        LaunchTimer lt(K_ROUTER_WGRAD, s);
        e = launch_pdl(router_wgrad_kernel, dim3((unsigned)router_max_items(T, k, E), (H + 1023) / 1024),
                       dim3(kWgThreadsRouter), 0, s, b.x, (const float*)b.dl_row, b.row_token, (const int4*)b.items,
                       (const int32_t*)b.n_items, (int)T, E, H, b.partial, b.dw_router, err);
    }
    if (e != cudaSuccess) return e;
    {
        LaunchTimer lt(K_ROUTER_WGRAD_JOIN, s);
        e = launch_pdl(router_wgrad_join_kernel, dim3(E, (H / 4 + 255) / 256), dim3(256), 0, s, (const float*)b.partial,
                       (const int32_t*)b.n_items, H, b.dw_router);
    }
    if (e == cudaSuccess) launches_add(3);
    return e;
}

cudaError_t launch_checkpoint_values(const smoe_config_t& c, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                     uint16_t* gu, cudaStream_t s) {
    const int cols = 2 * c.inter;
    cudaError_t e;
    {
        LaunchTimer lt(K_CHECKPOINT_VALUES, s);
        e = launch_pdl(checkpoint_values_kernel, dim3((unsigned)((rows + 31) / 32), (cols + 511) / 512), dim3(256), 0, s,
                       codes, scales, rows, cols, gu);
    }
    if (e == cudaSuccess) launches_add(1);
    return e;
}

}  // namespace smoe
