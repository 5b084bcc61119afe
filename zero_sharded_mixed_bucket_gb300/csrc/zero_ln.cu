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

// ---- rows in registers ---------------------------------------------------------------
// Rows on 16-byte boundaries are held in registers, as they were loaded, from
// the one time they are read: a group of 32 W lanes takes RB rows at a time,
// all their loads issued at once, V 16-byte vectors to a lane.  A row's ragged
// end is loaded value by value by the lane that has it.

// Values of vector v of lane gl that exist.
template <int DT, int W>
__device__ __forceinline__ int vec_count(int64_t dim, int v, int gl)
{
    constexpr int VE = kVecOf<DT>;
    return (int)max((int64_t)0, min((int64_t)VE, dim - (int64_t)(v * 32 * W + gl) * VE));
}

// Sums over the group of n values at once, the same in every lane.  sh: room
// for [2][8 warps][n] of the block; `turn` alternates, so one barrier a call.
template <int W, int N>
__device__ __forceinline__ void group_sum(float (&x)[N], float* sh, int& turn)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; k++)
            x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
    if constexpr (W > 1) {
        const int warp = threadIdx.x >> 5, first = warp / W * W;
        float* slot = sh + (turn & 1) * (kLnThreads / 32) * N;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < N; k++)
                slot[warp * N + k] = x[k];
        if constexpr (W == kLnThreads / 32)
            __syncthreads();
        else
            asm volatile("bar.sync %0, %1;" :: "r"(1 + first / W), "r"(32 * W) : "memory");
#pragma unroll
        for (int k = 0; k < N; k++) {
            float t = slot[first * N + k];
#pragma unroll
            for (int q = 1; q < W; q++)
                t += slot[(first + q) * N + k];
            x[k] = t;
        }
        turn++;
    }
}

template <int DT>
__device__ __forceinline__ void unpack(const Vals<DT>& v, float f[kVecOf<DT>])
{
    if constexpr (DT == kF32) {
#pragma unroll
        for (int k = 0; k < kVecOf<DT>; k++)
            f[k] = __uint_as_float(v.w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < kVecOf<DT> / 2; k++) {
            const float2 p = to_f32x2<DT>(v.w[k]);
            f[2 * k] = p.x;
            f[2 * k + 1] = p.y;
        }
    }
}

template <int DT>
__device__ __forceinline__ Vals<DT> pack(const float f[kVecOf<DT>])
{
    Vals<DT> v;
    if constexpr (DT == kF32) {
#pragma unroll
        for (int k = 0; k < kVecOf<DT>; k++)
            v.w[k] = __float_as_uint(f[k]);
    } else {
#pragma unroll
        for (int k = 0; k < kVecOf<DT> / 2; k++)
            v.w[k] = from_f32x2<DT>(f[2 * k], f[2 * k + 1]);
    }
    return v;
}

// Weights: kept in cache, `fill` where there are none.
template <int DT>
__device__ __forceinline__ void ld_weight(const void* p, int64_t i, int cnt, float fill, float f[kVecOf<DT>])
{
    constexpr int VE = kVecOf<DT>;
    if (!p) {
#pragma unroll
        for (int k = 0; k < VE; k++)
            f[k] = fill;
    } else if (cnt == VE) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (DT == kF32 ? 4 : 2));
        Vals<DT> v;
        v.w[0] = u.x; v.w[1] = u.y; v.w[2] = u.z; v.w[3] = u.w;
        unpack<DT>(v, f);
    } else {
#pragma unroll
        for (int k = 0; k < VE; k++)
            f[k] = k < cnt ? ld1<DT>(p, i + k) : 0.0f;
    }
}

template <int DT, int W, int V, int RB>
__global__ void __launch_bounds__(kLnThreads) k_ln_forward_reg(const __grid_constant__ LnArgs a)
{
    constexpr int VE = kVecOf<DT>, G = 32 * W, kGroups = kLnThreads / G;
    __shared__ float sh[2 * (kLnThreads / 32) * RB];
    const int gl = threadIdx.x % G;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    const int64_t stride = (int64_t)gridDim.x * kGroups * RB;
    for (int64_t r0 = ((int64_t)blockIdx.x * kGroups + threadIdx.x / G) * RB; r0 < a.rows; r0 += stride) {
        Vals<DT> q[RB][V];
        float mean[RB], rstd[RB];
#pragma unroll
        for (int b = 0; b < RB; b++)
#pragma unroll
            for (int v = 0; v < V; v++)               // rows past the end: the last one again, not written
                q[b][v] = ld_vals<DT>(a.x, min(r0 + b, a.rows - 1) * a.x_stride + (int64_t)(v * G + gl) * VE,
                                      vec_count<DT, W>(a.dim, v, gl));
#pragma unroll
        for (int b = 0; b < RB; b++) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) {
                float f[VE];
                unpack<DT>(q[b][v], f);               // values past the row's end are 0
#pragma unroll
                for (int k = 0; k < VE; k++)
                    s += f[k];
            }
            mean[b] = s;
        }
        group_sum<W, RB>(mean, sh, turn);
#pragma unroll
        for (int b = 0; b < RB; b++) {
            mean[b] *= inv;
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) {
                const int cnt = vec_count<DT, W>(a.dim, v, gl);
                float f[VE];
                unpack<DT>(q[b][v], f);
                if (cnt == VE) {
#pragma unroll
                    for (int k = 0; k < VE; k++) {
                        const float c = f[k] - mean[b];
                        s = fmaf(c, c, s);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < VE; k++) {
                        const float c = k < cnt ? f[k] - mean[b] : 0.0f;
                        s = fmaf(c, c, s);
                    }
                }
            }
            rstd[b] = s;
        }
        group_sum<W, RB>(rstd, sh, turn);
#pragma unroll
        for (int b = 0; b < RB; b++)
            rstd[b] = 1.0f / sqrtf(fmaf(rstd[b], inv, a.eps));
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int cnt = vec_count<DT, W>(a.dim, v, gl);
            const int64_t j = (int64_t)(v * G + gl) * VE;
            if (cnt == 0) continue;
            float w[VE], bias[VE];
            ld_weight<DT>(a.weight, j, cnt, 1.0f, w);
            ld_weight<DT>(a.bias, j, cnt, 0.0f, bias);
#pragma unroll
            for (int b = 0; b < RB; b++) {
                if (r0 + b >= a.rows) break;
                float f[VE];
                unpack<DT>(q[b][v], f);
#pragma unroll
                for (int k = 0; k < VE; k++)
                    f[k] = fmaf((f[k] - mean[b]) * rstd[b], w[k], bias[k]);
                st_vals<DT>(a.y, (r0 + b) * a.y_stride + j, pack<DT>(f), cnt);
            }
        }
        if (gl == 0) {
#pragma unroll
            for (int b = 0; b < RB; b++) {
                if (r0 + b >= a.rows) break;
                if (a.mean) a.mean[r0 + b] = mean[b];
                if (a.rstd) a.rstd[r0 + b] = rstd[b];
            }
        }
    }
}

// dx of a row group, and the column sums of dy * xhat and dy over all its
// rows in registers: x and dy are read once for both.  A block writes one
// pair of partial sums per column (its groups joined in group order).
template <int DT, int W, int V, int RB>
__global__ void __launch_bounds__(kLnThreads) k_ln_backward_reg(const __grid_constant__ LnArgs a)
{
    constexpr int VE = kVecOf<DT>, G = 32 * W, kGroups = kLnThreads / G;
    __shared__ float sh[2 * (kLnThreads / 32) * 2 * RB];
    __shared__ float join[kGroups > 1 ? 2 * V * G * VE : 1];
    const int gl = threadIdx.x % G, group = threadIdx.x / G;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    float dw[V][VE], db[V][VE];
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
        for (int k = 0; k < VE; k++)
            dw[v][k] = db[v][k] = 0.0f;
    const int64_t stride = (int64_t)gridDim.x * kGroups * RB;
    for (int64_t r0 = ((int64_t)blockIdx.x * kGroups + group) * RB; r0 < a.rows; r0 += stride) {
        Vals<DT> x[RB][V], dy[RB][V];
        float mean[RB], rstd[RB], c[2 * RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {
            const int64_t r = min(r0 + b, a.rows - 1);
#pragma unroll
            for (int v = 0; v < V; v++) {
                const int cnt = r0 + b < a.rows ? vec_count<DT, W>(a.dim, v, gl) : 0;   // rows past the end are 0
                const int64_t j = (int64_t)(v * G + gl) * VE;
                x[b][v] = ld_vals<DT>(a.x, r * a.x_stride + j, cnt);
                dy[b][v] = ld_vals<DT>(a.dy, r * a.y_stride + j, cnt);
            }
            mean[b] = a.mean_in[r];
            rstd[b] = a.rstd_in[r];
            c[2 * b] = c[2 * b + 1] = 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int cnt = vec_count<DT, W>(a.dim, v, gl);
            const int64_t j = (int64_t)(v * G + gl) * VE;
            float w[VE];
            ld_weight<DT>(a.weight, j, cnt, 1.0f, w);
#pragma unroll
            for (int b = 0; b < RB; b++) {
                float xf[VE], yf[VE];
                unpack<DT>(x[b][v], xf);
                unpack<DT>(dy[b][v], yf);             // 0 past the ends: adds nothing below, while x is finite
#pragma unroll
                for (int k = 0; k < VE; k++) {
                    const float h = (xf[k] - mean[b]) * rstd[b], g = yf[k] * w[k];
                    if (r0 + b < a.rows) {
                        dw[v][k] = fmaf(yf[k], h, dw[v][k]);
                        db[v][k] += yf[k];
                    }
                    c[2 * b] += g;
                    c[2 * b + 1] = fmaf(g, h, c[2 * b + 1]);
                }
            }
        }
        if (!a.dx) continue;
        group_sum<W, 2 * RB>(c, sh, turn);
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int cnt = vec_count<DT, W>(a.dim, v, gl);
            const int64_t j = (int64_t)(v * G + gl) * VE;
            if (cnt == 0) continue;
            float w[VE];
            ld_weight<DT>(a.weight, j, cnt, 1.0f, w);
#pragma unroll
            for (int b = 0; b < RB; b++) {
                if (r0 + b >= a.rows) break;
                float xf[VE], yf[VE];
                unpack<DT>(x[b][v], xf);
                unpack<DT>(dy[b][v], yf);
                const float c1 = c[2 * b] * inv, c2 = c[2 * b + 1] * inv;
#pragma unroll
                for (int k = 0; k < VE; k++) {
                    const float h = (xf[k] - mean[b]) * rstd[b];
                    xf[k] = (fmaf(yf[k], w[k], -c1) - h * c2) * rstd[b];
                }
                st_vals<DT>(a.dx, (r0 + b) * a.x_stride + j, pack<DT>(xf), cnt);
            }
        }
    }
    if (!a.part) return;
    if constexpr (kGroups > 1) {
        for (int g = 1; g < kGroups; g++) {           // group g's sums through shared memory to group 0
            __syncthreads();
            if (group == g)
#pragma unroll
                for (int v = 0; v < V; v++)
#pragma unroll
                    for (int k = 0; k < VE; k++) {
                        join[(v * VE + k) * G + gl] = dw[v][k];
                        join[((V + v) * VE + k) * G + gl] = db[v][k];
                    }
            __syncthreads();
            if (group == 0)
#pragma unroll
                for (int v = 0; v < V; v++)
#pragma unroll
                    for (int k = 0; k < VE; k++) {
                        dw[v][k] += join[(v * VE + k) * G + gl];
                        db[v][k] += join[((V + v) * VE + k) * G + gl];
                    }
        }
        if (group != 0) return;
    }
    float* pw = a.part + 2 * (int64_t)blockIdx.x * a.dim;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int cnt = vec_count<DT, W>(a.dim, v, gl);
        const int64_t j = (int64_t)(v * G + gl) * VE;
#pragma unroll
        for (int k = 0; k < VE; k++)
            if (k < cnt) {
                pw[j + k] = dw[v][k];
                pw[a.dim + j + k] = db[v][k];
            }
    }
}

// ---- any row -------------------------------------------------------------------------
// Rows off 16-byte boundaries, or longer than the registers hold: a block per
// row, values read again for every use (from cache).
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

// The blocks' partial sums: 32 columns a block, its 8 warps a part of the
// partial sums each, joined in warp order.
template <int DT>
__global__ void __launch_bounds__(kLnThreads) k_ln_dw_sum(const float* part, int blocks, int64_t dim, void* dw, void* db)
{
    wait_prev_grid();                                 // launched while the row kernel drains
    __shared__ float sh[2][kLnThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f, t = 0.0f;
    if (j < dim)
#pragma unroll 4
        for (int k = warp; k < blocks; k += kLnThreads / 32) {
            s += part[(2 * (int64_t)k) * dim + j];
            t += part[(2 * (int64_t)k + 1) * dim + j];
        }
    sh[0][warp][lane] = s;
    sh[1][warp][lane] = t;
    __syncthreads();
    if (warp > 0 || j >= dim) return;
    for (int k = 1; k < kLnThreads / 32; k++) {
        s += sh[0][k][lane];
        t += sh[1][k][lane];
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

template <typename K>
cudaError_t launch_rows(K kernel, const LnArgs& a, int64_t rows_per_block, int most, cudaStream_t s)
{
    const int64_t need = (a.rows + rows_per_block - 1) / rows_per_block;
    kernel<<<(unsigned)(need < most ? need : most), kLnThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// Blocks of a row kernel: as many as are resident at once on the GPU's 152
// SMs, each striding over the rows.
constexpr int kSms = 152;

template <int DT>
cudaError_t forward(const LnArgs& a, bool vec, cudaStream_t s)
{
    constexpr int VE = kVecOf<DT>;
    const int64_t vecs = (a.dim + VE - 1) / VE;
    // a warp per row while a lane's part fits its registers (16 vectors), then
    // a block; short rows several at a time
    if (vec && vecs <= 32) return launch_rows(k_ln_forward_reg<DT, 1, 1, 4>, a, 32, kSms * 8, s);
    if (vec && vecs <= 64) return launch_rows(k_ln_forward_reg<DT, 1, 2, 2>, a, 16, kSms * 8, s);
    if (vec && vecs <= 128) return launch_rows(k_ln_forward_reg<DT, 1, 4, 2>, a, 16, kSms * 4, s);
    if (vec && vecs <= 256) return launch_rows(k_ln_forward_reg<DT, 1, 8, 1>, a, 8, kSms * 4, s);
    if (vec && vecs <= 512) return launch_rows(k_ln_forward_reg<DT, 8, 2, 2>, a, 2, kSms * 6, s);
    if (vec && vecs <= 1024) return launch_rows(k_ln_forward_reg<DT, 8, 4, 1>, a, 1, kSms * 6, s);
    if (vec && vecs <= 2048) return launch_rows(k_ln_forward_reg<DT, 8, 8, 1>, a, 1, kSms * 4, s);
    return launch_rows(k_ln_forward<DT>, a, 1, kSms * 8, s);
}

template <int DT>
cudaError_t backward(LnArgs a, bool vec, int blocks, void* dw, void* db, cudaStream_t s)
{
    constexpr int VE = kVecOf<DT>;
    const int64_t vecs = (a.dim + VE - 1) / VE;
    const bool sums = dw || db;
    if (!sums) a.part = nullptr;
    cudaError_t e = cudaSuccess;
    if (blocks && vec && vecs <= 1024) {
        // the group's lanes hold one vector of the row each where they can: the
        // column sums take 2 registers a value beside the rows themselves
        if (vecs <= 32) k_ln_backward_reg<DT, 1, 1, 4><<<blocks, kLnThreads, 0, s>>>(a);
        else if (vecs <= 64) k_ln_backward_reg<DT, 2, 1, 4><<<blocks, kLnThreads, 0, s>>>(a);
        else if (vecs <= 128) k_ln_backward_reg<DT, 4, 1, 4><<<blocks, kLnThreads, 0, s>>>(a);
        else if (vecs <= 256) k_ln_backward_reg<DT, 8, 1, 4><<<blocks, kLnThreads, 0, s>>>(a);
        else if (vecs <= 512) k_ln_backward_reg<DT, 8, 2, 2><<<blocks, kLnThreads, 0, s>>>(a);
        else k_ln_backward_reg<DT, 8, 4, 1><<<blocks, kLnThreads, 0, s>>>(a);
        e = cudaGetLastError();
    } else {
        if (a.dx && a.rows) e = launch_rows(k_ln_dx<DT>, a, 1, kSms * 8, s);
        if (e == cudaSuccess && sums && blocks) {
            const unsigned cols = (unsigned)((a.dim + kLnThreads - 1) / kLnThreads);
            k_ln_dw_part<DT><<<dim3(cols, (unsigned)blocks), kLnThreads, 0, s>>>(a);
            e = cudaGetLastError();
        }
    }
    if (e == cudaSuccess && sums)
        e = launch_kernel(k_ln_dw_sum<DT>, (int)((a.dim + 31) / 32), kLnThreads, s, blocks > 0, (const float*)a.part,
                          blocks, a.dim, dw, db);
    return e;
}

// Rows of x and y (or dy, dx) and the vectors start on 16-byte boundaries.
bool on_vectors(const zero_ln_plan_t& p, const void* a, const void* b, const void* c, const void* d, const void* e)
{
    const int64_t ve = p.dtype == ZERO_FP32 ? 4 : 8;
    const uintptr_t any = (uintptr_t)a | (uintptr_t)b | (uintptr_t)c | (uintptr_t)d | (uintptr_t)e;
    return any % 16 == 0 && p.x_stride % ve == 0 && p.y_stride % ve == 0;
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
    // each block adds up its rows' weight gradients by itself: two blocks to an
    // SM of 152, and no more than the rows it takes at a time give
    const int64_t vecs = (dim * e + 15) / 16;
    const int64_t at_once = vecs <= 32 ? 32 : vecs <= 64 ? 16 : vecs <= 128 ? 8 : vecs <= 256 ? 4 : vecs <= 512 ? 2 : 1;
    const int64_t groups = (rows + at_once - 1) / at_once;
    out->blocks = (int32_t)(groups < 304 ? groups : 304);
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
    const bool vec = on_vectors(*plan, x, y, weight, bias, nullptr);
    const cudaError_t err = plan->dtype == ZERO_FP32   ? forward<kF32>(a, vec, s)
                            : plan->dtype == ZERO_BF16 ? forward<kBF16>(a, vec, s)
                                                       : forward<kF16>(a, vec, s);
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
    const bool vec = on_vectors(*plan, x, dy, weight, dx, nullptr);
    const cudaError_t err = plan->dtype == ZERO_FP32   ? backward<kF32>(a, vec, plan->blocks, dweight, dbias, s)
                            : plan->dtype == ZERO_BF16 ? backward<kBF16>(a, vec, plan->blocks, dweight, dbias, s)
                                                       : backward<kF16>(a, vec, plan->blocks, dweight, dbias, s);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_ln_backward");
}

}  // extern "C"
