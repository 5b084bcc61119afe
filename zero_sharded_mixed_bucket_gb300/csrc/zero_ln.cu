// Layer norm of rows: the plan, the forward kernel, and the backward pass
// with the reduction of the weight's and the bias's gradient.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "dev_common.cuh"
#include "nvtx_ranges.h"

namespace zg {
namespace {

constexpr int kLnThreads = 256;

struct LnArgs {
    const void* x;
    const void* dy;
    const void* weight;
    const void* bias;
    const float* mean_in;
    const float* rstd_in;
    void* y;
    float* mean;
    float* rstd;
    void* dx;
    float* part;                 // [blocks][2][dim]: partial dweight, dbias
    int64_t rows, dim, x_stride, y_stride;
    float eps;
};

template <int DT>
__device__ __forceinline__ float ld1(const void* p, int64_t i)
{
    if constexpr (DT == kF32)
        return static_cast<const float*>(p)[i];
    else
        return to_f32<DT>(static_cast<const uint16_t*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void st1(void* p, int64_t i, float v)
{
    if constexpr (DT == kF32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = (uint16_t)from_f32<DT>(v);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the block, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float* sh)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int k = 0; k < kLnThreads / 32; k++)
        t += sh[k];
    return t;
}

template <int DT>
__global__ void __launch_bounds__(kLnThreads) k_ln_forward(const __grid_constant__ LnArgs a)
{
    __shared__ float sh[kLnThreads / 32];
    const float inv = 1.0f / (float)a.dim;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t xo = r * a.x_stride, yo = r * a.y_stride;
        float s = 0.0f;
        for (int64_t j = threadIdx.x; j < a.dim; j += kLnThreads)
            s += ld1<DT>(a.x, xo + j);
        const float mean = block_sum(s, sh) * inv;
        float q = 0.0f;
        for (int64_t j = threadIdx.x; j < a.dim; j += kLnThreads) {
            const float c = ld1<DT>(a.x, xo + j) - mean;
            q = fmaf(c, c, q);
        }
        const float rstd = 1.0f / sqrtf(block_sum(q, sh) * inv + a.eps);
        for (int64_t j = threadIdx.x; j < a.dim; j += kLnThreads) {
            const float w = a.weight ? ld1<DT>(a.weight, j) : 1.0f;
            const float b = a.bias ? ld1<DT>(a.bias, j) : 0.0f;
            st1<DT>(a.y, yo + j, fmaf((ld1<DT>(a.x, xo + j) - mean) * rstd, w, b));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kLnThreads) k_ln_dx(const __grid_constant__ LnArgs a)
{
    __shared__ float sh[kLnThreads / 32];
    const float inv = 1.0f / (float)a.dim;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t xo = r * a.x_stride, yo = r * a.y_stride;
        const float mean = a.mean_in[r], rstd = a.rstd_in[r];
        float s = 0.0f, q = 0.0f;
        for (int64_t j = threadIdx.x; j < a.dim; j += kLnThreads) {
            const float g = ld1<DT>(a.dy, yo + j) * (a.weight ? ld1<DT>(a.weight, j) : 1.0f);
            s += g;
            q = fmaf(g, (ld1<DT>(a.x, xo + j) - mean) * rstd, q);
        }
        const float c1 = block_sum(s, sh) * inv;
        const float c2 = block_sum(q, sh) * inv;
        for (int64_t j = threadIdx.x; j < a.dim; j += kLnThreads) {
            const float g = ld1<DT>(a.dy, yo + j) * (a.weight ? ld1<DT>(a.weight, j) : 1.0f);
            const float h = (ld1<DT>(a.x, xo + j) - mean) * rstd;
            st1<DT>(a.dx, xo + j, (g - c1 - h * c2) * rstd);
        }
    }
}

// Column sums over the row group blockIdx.y: one thread a column.
template <int DT>
__global__ void __launch_bounds__(kLnThreads) k_ln_dw_part(const __grid_constant__ LnArgs a)
{
    const int64_t j = (int64_t)blockIdx.x * kLnThreads + threadIdx.x;
    if (j >= a.dim) return;
    const int64_t G = gridDim.y, per = (a.rows + G - 1) / G;
    const int64_t lo = min(blockIdx.y * per, a.rows), hi = min(lo + per, a.rows);
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = lo; r < hi; r++) {
        const float dy = ld1<DT>(a.dy, r * a.y_stride + j);
        dw = fmaf(dy, (ld1<DT>(a.x, r * a.x_stride + j) - a.mean_in[r]) * a.rstd_in[r], dw);
        db += dy;
    }
    a.part[(2 * (int64_t)blockIdx.y) * a.dim + j] = dw;
    a.part[(2 * (int64_t)blockIdx.y + 1) * a.dim + j] = db;
}

// The groups' partial sums, in group order.
template <int DT>
__global__ void __launch_bounds__(kLnThreads) k_ln_dw_sum(const float* part, int groups, int64_t dim, void* dw, void* db)
{
    const int64_t j = (int64_t)blockIdx.x * kLnThreads + threadIdx.x;
    if (j >= dim) return;
    float s = 0.0f, t = 0.0f;
    for (int k = 0; k < groups; k++) {
        s += part[(2 * (int64_t)k) * dim + j];
        t += part[(2 * (int64_t)k + 1) * dim + j];
    }
    if (dw) st1<DT>(dw, j, s);
    if (db) st1<DT>(db, j, t);
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

zero_status_t cuda_failed(cudaError_t e, const char* what)
{
    char msg[200];
    std::snprintf(msg, sizeof msg, "%s: launch failed: %s", what, cudaGetErrorString(e));
    return set_error(ZERO_ECUDA, msg);
}

zero_status_t check_ln_plan(const zero_ln_plan_t* p)
{
    if (!p) return set_error(ZERO_EINVAL, "layer norm plan is NULL");
    zero_ln_plan_t fresh;
    const zero_status_t st = zero_ln_plan(p->rows, p->dim, p->dtype, p->x_stride, p->y_stride, &fresh);
    if (st != ZERO_OK) return st;
    if (std::memcmp(&fresh, p, sizeof fresh) != 0)
        return set_error(ZERO_EINVAL, "layer norm plan was not made by zero_ln_plan");
    return ZERO_OK;
}

template <int DT>
cudaError_t forward(const LnArgs& a, cudaStream_t s)
{
    const unsigned grid = (unsigned)(a.rows < 152 * 8 ? a.rows : 152 * 8);
    k_ln_forward<DT><<<grid, kLnThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int DT>
cudaError_t backward(const LnArgs& a, int groups, void* dw, void* db, cudaStream_t s)
{
    if (a.dx && a.rows) {
        const unsigned grid = (unsigned)(a.rows < 152 * 8 ? a.rows : 152 * 8);
        k_ln_dx<DT><<<grid, kLnThreads, 0, s>>>(a);
    }
    if (dw || db) {
        const unsigned cols = (unsigned)((a.dim + kLnThreads - 1) / kLnThreads);
        if (groups) k_ln_dw_part<DT><<<dim3(cols, (unsigned)groups), kLnThreads, 0, s>>>(a);
        k_ln_dw_sum<DT><<<cols, kLnThreads, 0, s>>>(a.part, groups, a.dim, dw, db);
    }
    return cudaGetLastError();
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

zero_status_t zero_ln_plan(int64_t rows, int64_t dim, int32_t dtype, int64_t x_stride, int64_t y_stride,
                           zero_ln_plan_t* out)
{
    if (!out) return set_error(ZERO_EINVAL, "zero_ln_plan: out is NULL");
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16 && dtype != ZERO_FP32)
        return set_error(ZERO_EINVAL, "zero_ln_plan: dtype unknown");
    if (rows < 0 || dim < 1) return set_error(ZERO_EINVAL, "zero_ln_plan: rows must be >= 0 and dim >= 1");
    if (rows > (int64_t(1) << 40) || dim > (int64_t(1) << 20))
        return set_error(ZERO_EUNSUPPORTED, "zero_ln_plan: rows exceed 2^40 or dim exceeds 2^20");
    const int64_t xs = x_stride ? x_stride : dim, ys = y_stride ? y_stride : dim;
    if (xs < dim || ys < dim || xs > (int64_t(1) << 40) || ys > (int64_t(1) << 40))
        return set_error(ZERO_EINVAL, "zero_ln_plan: a stride is below dim or above 2^40");
    if (rows && (xs > INT64_MAX / 8 / rows || ys > INT64_MAX / 8 / rows))
        return set_error(ZERO_EUNSUPPORTED, "zero_ln_plan: the rows span too many bytes");
    std::memset(out, 0, sizeof *out);
    out->rows = rows;
    out->dim = dim;
    out->x_stride = xs;
    out->y_stride = ys;
    out->dtype = dtype;
    const int64_t e = dtype == ZERO_FP32 ? 4 : 2;
    const int64_t groups = (rows + 31) / 32;
    out->blocks = (int32_t)(groups < 152 ? groups : 152);
    out->workspace_bytes = 16 + (int64_t)out->blocks * 2 * dim * 4;
    out->hbm_bytes_forward = rows * (2 * dim * e + 8) + 2 * dim * e;
    out->hbm_bytes_backward = rows * (3 * dim * e + 8) + 3 * dim * e;
    return ZERO_OK;
}

zero_status_t zero_ln_forward(const zero_ln_plan_t* plan, const void* x, const void* weight, const void* bias,
                              float eps, void* y, float* mean, float* rstd, void* stream)
{
    NvtxRange range("zero_ln_forward");
    const zero_status_t st = check_ln_plan(plan);
    if (st != ZERO_OK) return st;
    if (!(eps >= 0.0f)) return set_error(ZERO_EINVAL, "zero_ln_forward: eps must be >= 0");
    if (plan->rows == 0) return ZERO_OK;
    if (!x || !y) return set_error(ZERO_ENOMEM, "zero_ln_forward: x or y is NULL");
    const size_t e = plan->dtype == ZERO_FP32 ? 4 : 2;
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, e) || !aligned_to(bias, e) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return set_error(ZERO_EALIGN, "zero_ln_forward: a pointer is not aligned to its type");
    LnArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.rows = plan->rows; a.dim = plan->dim; a.x_stride = plan->x_stride; a.y_stride = plan->y_stride;
    a.eps = eps;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err = plan->dtype == ZERO_FP32   ? forward<kF32>(a, s)
                            : plan->dtype == ZERO_BF16 ? forward<kBF16>(a, s)
                                                       : forward<kF16>(a, s);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_ln_forward");
}

zero_status_t zero_ln_backward(const zero_ln_plan_t* plan, const void* dy, const void* x, const void* weight,
                               const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                               void* workspace, void* stream)
{
    NvtxRange range("zero_ln_backward");
    const zero_status_t st = check_ln_plan(plan);
    if (st != ZERO_OK) return st;
    if (plan->rows && (!dy || !x || !mean || !rstd))
        return set_error(ZERO_ENOMEM, "zero_ln_backward: dy, x, mean or rstd is NULL");
    if ((dweight || dbias) && !workspace) return set_error(ZERO_ENOMEM, "zero_ln_backward: workspace is NULL");
    const size_t e = plan->dtype == ZERO_FP32 ? 4 : 2;
    if (!aligned_to(x, e) || !aligned_to(dy, e) || !aligned_to(weight, e) || !aligned_to(dx, e) ||
        !aligned_to(dweight, e) || !aligned_to(dbias, e) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return set_error(ZERO_EALIGN, "zero_ln_backward: a pointer is not aligned to its type");
    if (!aligned_to(workspace, 16)) return set_error(ZERO_EALIGN, "zero_ln_backward: workspace is not 16-byte aligned");
    LnArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = x; a.dy = dy; a.weight = weight; a.mean_in = mean; a.rstd_in = rstd; a.dx = dx;
    a.rows = plan->rows; a.dim = plan->dim; a.x_stride = plan->x_stride; a.y_stride = plan->y_stride;
    a.part = static_cast<float*>(workspace) + 4;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err = plan->dtype == ZERO_FP32   ? backward<kF32>(a, plan->blocks, dweight, dbias, s)
                            : plan->dtype == ZERO_BF16 ? backward<kBF16>(a, plan->blocks, dweight, dbias, s)
                                                       : backward<kF16>(a, plan->blocks, dweight, dbias, s);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_ln_backward");
}

}  // extern "C"
