// Layer norm of rows: the plan, the forward kernel, and the backward pass
// with the reduction of the weight's and the bias's gradient.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "dev_rows.cuh"
#include "nvtx_ranges.h"

namespace zg {

using namespace rows;

namespace {

constexpr int kLnThreads = kRowThreads;
constexpr int kLnFwdAhead = 2, kLnBwdAhead = 2;   // batches of rows on their way or in use
constexpr int kLnFwdRows = 8, kLnBwdRows = 4;     // rows of a batch, at one vector a lane
constexpr int kLnFwdBlocks = 3, kLnBwdBlocks = 2; // blocks of 256 threads resident on an SM

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
    int warps;                   // of a group (row kernels)
};

// s / n, where inv is 1 / n: the product, corrected by what it leaves of s (NaN
// for an infinite s).  The product alone is off by a unit in the last place for a
// quarter of all n, and a row of one value has to have that value as its mean:
// the unit is 0.02 of 1/rstd for a row of 1000 with eps = 1e-5.
__device__ __forceinline__ float quotient(float s, float n, float inv)
{
    const float q = s * inv;
    return fmaf(fmaf(-q, n, s), inv, q);
}

// A row's mean from its sum; of an infinite sum that infinity.
__device__ __forceinline__ float mean_of(float s, float n, float inv)
{
    return fabsf(s) < INFINITY ? quotient(s, n, inv) : s;
}

// ---- rows on 16-byte (or 4-byte) boundaries ---------------------------------------------
// A group of lanes takes RB rows at a time, V 16-byte vectors of a row to a
// lane: W warps (V > 1 only where 8 warps are not enough), or L < 32 lanes of
// one for short rows.  A block is as many groups as fit its T threads.  Each lane
// copies its vectors ahead of their use into slots of shared memory of its own
// (cp.async; a row's ragged end is filled with zeros), S batches deep: the
// bytes in flight do not depend on registers or on how far the other lanes
// are, and nothing waits but a lane for its own copies.  The rows stay there
// until they are done, read again for each use.
// What bounds these kernels is what few warps can issue: 17 instructions a value
// forward, 30 backward, so a batch is as large as registers allow (its sums,
// addresses and loop are shared by all its values), and registers leave 5.4 and
// 3.2 warps to a scheduler, which issues in 69 and 62 % of the cycles.  A warp's
// 5.1 cycles an instruction backward are 1 to issue, 1.1 in turn behind another,
// 0.75 of fixed latencies, 0.7 at the batch's barrier, 0.4 each for the arithmetic
// pipe and shared memory, 0.2 for loads; DRAM is half idle.  (Packed pairs of
// binary32 operations, fewer instructions, gained nothing: 79 us for 74.5.)
// 8192 x 4096 bfloat16 forward: 26.8 us, 5.0 TB/s (a device copy of the same
// bytes 23.5; rows in registers, a block to a row: 35).  32768 x 1600 binary16
// backward: 74.3 us, 4.2 TB/s (adding two arrays into a third of these sizes:
// 47.5; weight gradients in a pass of their own: 220; batches ahead in
// registers: 82).  In 32 bits: 8192 x 4096 forward 46.4 us, 5.8 TB/s, backward
// 85, 4.7.

// Forward.  A lane's values are unpacked once for both statistics: with the
// lane's own sum s and sum of squares m2 about its own mean, the row's sum of
// squares about its mean is the sum of m2 + n (s/n - mean)^2 over the lanes.
// RAGGED: dim is not a multiple of a vector's values.
template <int DT, int L, int V, int RB, int S, int T, int BLOCKS, bool RAGGED, int ALIGN>
__global__ void __launch_bounds__(T, BLOCKS) k_ln_forward_rows(const __grid_constant__ LnArgs a)
{
    constexpr int VE = kVecOf<DT>, E = DT == kF32 ? 4 : 2;
    extern __shared__ uint4 slots[];                  // [S][RB * V][T]
    __shared__ float sh[2 * (T / 32) * RB];
    const int lanes = L < 32 ? L : 32 * a.warps, gl = threadIdx.x % lanes, group = threadIdx.x / lanes;
    const int groups = blockDim.x / lanes;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    int cnt[V], have = 0;
#pragma unroll
    for (int v = 0; v < V; v++) {
        cnt[v] = vec_count<DT>(a.dim, v, gl, lanes);
        have += cnt[v];
    }
    const float n = (float)have, inv_n = have ? 1.0f / n : 0.0f;
    const int64_t stride = (int64_t)gridDim.x * groups * RB;
    int64_t r0 = ((int64_t)blockIdx.x * groups + group) * RB;
    int64_t ahead = r0;
    const int64_t x_row = a.x_stride * E, y_row = a.y_stride * E;
    const int apart = lanes * 16;                     // bytes between a lane's vectors
    const char* src = static_cast<const char*>(a.x) + r0 * x_row + gl * 16;
    char* dst = static_cast<char*>(a.y) + r0 * y_row + gl * 16;
    uint4* const mine = slots + threadIdx.x;
    auto fetch = [&](uint4* at) {
        const int here = rows_here(a.rows, ahead, RB);
        const char* p = src;
#pragma unroll
        for (int b = 0; b < RB; b++, p += x_row)
            if (b < here)
#pragma unroll
                for (int v = 0; v < V; v++)
                    if (cnt[v])
                        vec_ahead<ALIGN>(at + (b * V + v) * T, p + v * apart, RAGGED ? cnt[v] * E : 16);
        copies_issued();
        ahead += stride;
        src += stride * x_row;
    };
#pragma unroll
    for (int k = 0; k < S * RB * V; k++)              // vectors past the row's end are never copied: 0
        if (cnt[k % V] == 0) mine[k * T] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < S; k++)
        fetch(mine + k * RB * V * T);
    // groups of less than a warp go round together: their sums shuffle across the warp
    const int64_t first = L < 32 ? r0 - (int64_t)((threadIdx.x & 31) / L) * RB : r0;
    int slot = 0;
    for (int64_t rw = first; rw < a.rows; rw += stride) {
        copies_wait<S - 1>();
        uint4* const q = mine + slot * RB * V * T;    // rows past the end: whatever is there, not written
        float mean[RB], rstd[RB], own[RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {
            float f[V][VE], s = 0.0f, m2 = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) {
                unpack<DT>(from_slot<DT>(q + (b * V + v) * T), f[v]);
#pragma unroll
                for (int k = 0; k < VE; k++)
                    s += f[v][k];
            }
            own[b] = quotient(s, n, inv_n);
#pragma unroll
            for (int v = 0; v < V; v++) {
                if (!RAGGED && V > 1 && cnt[v] == 0) continue;    // no distance past the end
                if (RAGGED)
#pragma unroll
                    for (int k = 0; k < VE; k++)
                        f[v][k] = k < cnt[v] ? f[v][k] : own[b];
#pragma unroll
                for (int k = 0; k < VE; k++) {
                    const float c = f[v][k] - own[b];
                    m2 = fmaf(c, c, m2);
                }
            }
            mean[b] = s;
            rstd[b] = m2;
        }
        group_sum<L, RB, T>(mean, a.warps, sh, turn, [&](float t) { return mean_of(t, (float)a.dim, inv); });
#pragma unroll
        for (int b = 0; b < RB; b++) {
            const float c = own[b] - mean[b];
            rstd[b] = have ? fmaf(n * c, c, rstd[b]) : 0.0f;
        }
        group_sum<L, RB, T>(rstd, a.warps, sh, turn, [&](float t) { return rsqrtf(fmaf(t, inv, a.eps)); });
        const int here = rows_here(a.rows, r0, RB);
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (cnt[v] == 0) continue;
            const int64_t j = (int64_t)(v * lanes + gl) * VE;
            float w[VE], bias[VE];
            weight_vec<DT, RAGGED>(a.weight, j, cnt[v], 1.0f, w);
            weight_vec<DT, RAGGED>(a.bias, j, cnt[v], 0.0f, bias);
            char* p = dst + v * apart;
#pragma unroll
            for (int b = 0; b < RB; b++, p += y_row) {
                float f[VE];
                unpack<DT>(from_slot<DT>(q + (b * V + v) * T), f);
#pragma unroll
                for (int k = 0; k < VE; k++)
                    f[k] = fmaf((f[k] - mean[b]) * rstd[b], w[k], bias[k]);
                if (b < here) store_vec<DT, RAGGED, ALIGN>(p, pack<DT>(f), cnt[v]);
            }
        }
        if (gl == 0) {
#pragma unroll
            for (int b = 0; b < RB; b++) {
                if (b < here && a.mean) a.mean[r0 + b] = mean[b];
                if (b < here && a.rstd) a.rstd[r0 + b] = rstd[b];
            }
        }
        fetch(q);
        slot = slot == S - 1 ? 0 : slot + 1;
        r0 += stride;
        dst += stride * y_row;
    }
    copies_wait<0>();
}

// Backward: dx of the rows, and the column sums of dy * xhat and dy over all
// the rows of a lane in registers, so x and dy are read once for both.  A
// block writes one pair of partial sums per column (its groups joined in group
// order).  xhat = (x - mean) rstd is formed first, of order 1 whatever the row's
// size: the same with x - mean and powers of rstd in the averages is an
// operation less a value, and loses rows around 1e-22 or 1e17 to overflow and
// underflow.
template <int DT, int L, int V, int RB, int S, int T, int BLOCKS, bool RAGGED, int ALIGN>
__global__ void __launch_bounds__(T, BLOCKS) k_ln_backward_rows(const __grid_constant__ LnArgs a)
{
    constexpr int VE = kVecOf<DT>, E = DT == kF32 ? 4 : 2;
    extern __shared__ uint4 slots[];                  // [S][RB * V][x, dy][T]; at the end the groups' sums
    __shared__ float sh[2 * (T / 32) * 2 * RB];
    const int lanes = L < 32 ? L : 32 * a.warps, gl = threadIdx.x % lanes, group = threadIdx.x / lanes;
    const int groups = blockDim.x / lanes;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    int cnt[V];
    float dw[V][VE], db[V][VE];
#pragma unroll
    for (int v = 0; v < V; v++) {
        cnt[v] = vec_count<DT>(a.dim, v, gl, lanes);
#pragma unroll
        for (int k = 0; k < VE; k++)
            dw[v][k] = db[v][k] = 0.0f;
    }
    const int64_t stride = (int64_t)gridDim.x * groups * RB;
    int64_t r0 = ((int64_t)blockIdx.x * groups + group) * RB;
    int64_t ahead = r0;
    const int64_t x_row = a.x_stride * E, y_row = a.y_stride * E;
    const int apart = lanes * 16;
    const char* sx = static_cast<const char*>(a.x) + r0 * x_row + gl * 16;
    const char* sy = static_cast<const char*>(a.dy) + r0 * y_row + gl * 16;
    char* dst = static_cast<char*>(a.dx) + r0 * x_row + gl * 16;
    uint4* const mine = slots + threadIdx.x;
    auto fetch = [&](uint4* at) {
        const int here = rows_here(a.rows, ahead, RB);
        const char *px = sx, *py = sy;
#pragma unroll
        for (int b = 0; b < RB; b++, px += x_row, py += y_row)
#pragma unroll
            for (int v = 0; v < V; v++) {
                uint4* p = at + (b * V + v) * 2 * T;
                if (b < here) {
                    if (cnt[v]) {
                        vec_ahead<ALIGN>(p, px + v * apart, RAGGED ? cnt[v] * E : 16);
                        vec_ahead<ALIGN>(p + T, py + v * apart, RAGGED ? cnt[v] * E : 16);
                    }
                } else {                              // rows past the end: all 0
                    p[0] = p[T] = make_uint4(0, 0, 0, 0);
                }
            }
        copies_issued();
        ahead += stride;
        sx += stride * x_row;
        sy += stride * y_row;
    };
    float nmean[RB], nrstd[RB];
    auto fetch_stats = [&](int64_t from) {
        const int here = rows_here(a.rows, from, RB);
#pragma unroll
        for (int b = 0; b < RB; b++) {
            nmean[b] = b < here ? a.mean_in[from + b] : 0.0f;
            nrstd[b] = b < here ? a.rstd_in[from + b] : 0.0f;
        }
    };
#pragma unroll
    for (int k = 0; k < S * RB * V * 2; k++)          // vectors past the row's end are never copied: 0
        if (cnt[k / 2 % V] == 0) mine[k * T] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < S; k++)
        fetch(mine + k * RB * V * 2 * T);
    fetch_stats(r0);
    const int64_t first = L < 32 ? r0 - (int64_t)((threadIdx.x & 31) / L) * RB : r0;
    int slot = 0;
    for (int64_t rw = first; rw < a.rows; rw += stride) {
        copies_wait<S - 1>();
        uint4* const q = mine + slot * RB * V * 2 * T;
        float mean[RB], rstd[RB], c[2 * RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {
            mean[b] = nmean[b];
            rstd[b] = nrstd[b];
            c[2 * b] = c[2 * b + 1] = 0.0f;
        }
        fetch_stats(r0 + stride);
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (cnt[v] == 0) continue;
            float w[VE];
            weight_vec<DT, RAGGED>(a.weight, (int64_t)(v * lanes + gl) * VE, cnt[v], 1.0f, w);
#pragma unroll
            for (int b = 0; b < RB; b++) {
                float xf[VE], yf[VE];
                unpack<DT>(from_slot<DT>(q + (b * V + v) * 2 * T), xf);
                unpack<DT>(from_slot<DT>(q + ((b * V + v) * 2 + 1) * T), yf);   // 0 past the ends
#pragma unroll
                for (int k = 0; k < VE; k++) {
                    const float h = RAGGED && k >= cnt[v] ? 0.0f : (xf[k] - mean[b]) * rstd[b], g = yf[k] * w[k];
                    dw[v][k] = fmaf(yf[k], h, dw[v][k]);
                    db[v][k] += yf[k];
                    c[2 * b] += g;
                    c[2 * b + 1] = fmaf(g, h, c[2 * b + 1]);
                }
            }
        }
        if (a.dx) {
            group_sum<L, 2 * RB, T>(c, a.warps, sh, turn, [&](float t) { return t * -inv; });
            const int here = rows_here(a.rows, r0, RB);
#pragma unroll
            for (int v = 0; v < V; v++) {
                if (cnt[v] == 0) continue;
                float w[VE];
                weight_vec<DT, RAGGED>(a.weight, (int64_t)(v * lanes + gl) * VE, cnt[v], 1.0f, w);
                char* p = dst + v * apart;
#pragma unroll
                for (int b = 0; b < RB; b++, p += x_row) {
                    float xf[VE], yf[VE];
                    unpack<DT>(from_slot<DT>(q + (b * V + v) * 2 * T), xf);
                    unpack<DT>(from_slot<DT>(q + ((b * V + v) * 2 + 1) * T), yf);
#pragma unroll
                    for (int k = 0; k < VE; k++)
                        xf[k] = fmaf((xf[k] - mean[b]) * rstd[b], c[2 * b + 1], fmaf(yf[k], w[k], c[2 * b])) * rstd[b];
                    if (b < here) store_vec<DT, RAGGED, ALIGN>(p, pack<DT>(xf), cnt[v]);
                }
            }
        }
        fetch(q);
        slot = slot == S - 1 ? 0 : slot + 1;
        r0 += stride;
        dst += stride * x_row;
    }
    copies_wait<0>();
    if (!a.part) return;
    float* pw = a.part + 2 * (int64_t)blockIdx.x * a.dim;
    if (V == 1 && groups > 1) {
        float* join = reinterpret_cast<float*>(slots);            // [group][dw, db][VE][lanes]: no more than the slots
        const int one = 2 * VE * lanes;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < VE; k++) {
            join[group * one + k * lanes + gl] = dw[0][k];
            join[group * one + (VE + k) * lanes + gl] = db[0][k];
        }
        __syncthreads();
        for (int t = threadIdx.x; t < one; t += blockDim.x) {
            float s = 0.0f;
            for (int g = 0; g < groups; g++)
                s += join[g * one + t];
            const int k = t / lanes;                              // 0..2 VE - 1
            const int64_t j = (int64_t)(t - k * lanes) * VE + (k < VE ? k : k - VE);
            if (j < a.dim) pw[(k < VE ? 0 : a.dim) + j] = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; v++) {
            float* at = pw + (int64_t)(v * lanes + gl) * VE;
#pragma unroll
            for (int k = 0; k < VE; k++)
                if (k < cnt[v]) {
                    at[k] = dw[v][k];
                    at[a.dim + k] = db[v][k];
                }
        }
    }
}

// ---- other rows ------------------------------------------------------------------------
// The same groups, a lane's K values of a row one group of lanes apart: one
// access a value, neighbouring lanes neighbouring values, kept in registers as
// binary32.  What bounds these is the accesses: 8192 x 4095 bfloat16 forward 52
// us, 2.6 TB/s, backward 111; 16384 x 1023 binary32 30 and 57.  Whole 16-byte
// copies around a row, realigned in shared memory on the way in and by shuffles
// on the way out, take 59 and 92, and 39 and 62: the windows' ragged ends cost
// what the wide accesses save.  4-byte copies of 16-bit rows with the odd value
// shifted out: 57 and 91, and the rows on 4-byte boundaries lose by it.
template <int DT, int K>
__device__ __forceinline__ void ld_strided(const void* p, int64_t at, int gl, int lanes, int here, float f[K])
{
    // loads without branches, so that all of them are on their way at once: past
    // the row's end its first value again, dropped
    const char* row = static_cast<const char*>(p) + at * (DT == kF32 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < K; k++)
        f[k] = ld1<DT>(row, k < here ? gl + k * lanes : 0);
#pragma unroll
    for (int k = 0; k < K; k++)
        f[k] = k < here ? f[k] : 0.0f;
}

template <int DT, int L, int K, int RB>
__global__ void __launch_bounds__(kLnThreads, 2) k_ln_forward_any(const __grid_constant__ LnArgs a)
{
    __shared__ float sh[2 * (kLnThreads / 32) * RB];
    const int lanes = L < 32 ? L : 32 * a.warps, gl = threadIdx.x % lanes, group = threadIdx.x / lanes;
    const int groups = blockDim.x / lanes;
    const int here = gl < a.dim ? (int)((a.dim - 1 - gl) / lanes) + 1 : 0;         // values of the row that the lane has
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    const int64_t stride = (int64_t)gridDim.x * groups * RB;
    int64_t r0 = ((int64_t)blockIdx.x * groups + group) * RB;
    const int64_t first = L < 32 ? r0 - (int64_t)((threadIdx.x & 31) / L) * RB : r0;
    for (int64_t rw = first; rw < a.rows; rw += stride, r0 += stride) {
        const int rows = rows_here(a.rows, r0, RB);
        float f[RB][K], mean[RB], rstd[RB];
#pragma unroll
        for (int b = 0; b < RB; b++)
            ld_strided<DT, K>(a.x, min(r0 + b, a.rows - 1) * a.x_stride, gl, lanes, here, f[b]);   // past the end: not written
#pragma unroll
        for (int b = 0; b < RB; b++) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < K; k++)
                s += f[b][k];
            mean[b] = s;
        }
        group_sum<L, RB>(mean, a.warps, sh, turn, [&](float t) { return mean_of(t, (float)a.dim, inv); });
#pragma unroll
        for (int b = 0; b < RB; b++) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < K; k++) {
                f[b][k] -= mean[b];
                if (k < here) s = fmaf(f[b][k], f[b][k], s);
            }
            rstd[b] = s;
        }
        group_sum<L, RB>(rstd, a.warps, sh, turn, [&](float t) { return rsqrtf(fmaf(t, inv, a.eps)); });
#pragma unroll
        for (int k0 = 0; k0 < K; k0 += 8) {
            float w[8], bias[8];
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int j = k0 + k < here ? gl + (k0 + k) * lanes : 0;
                w[k] = a.weight ? ld1<DT>(a.weight, j) : 1.0f;
                bias[k] = a.bias ? ld1<DT>(a.bias, j) : 0.0f;
            }
#pragma unroll
            for (int b = 0; b < RB; b++) {
                char* row = static_cast<char*>(a.y) + (r0 + b) * a.y_stride * (DT == kF32 ? 4 : 2);
#pragma unroll
                for (int k = 0; k < 8; k++)
                    if (b < rows && k0 + k < here)
                        st1<DT>(row, gl + (k0 + k) * lanes, fmaf(f[b][k0 + k] * rstd[b], w[k], bias[k]));
            }
        }
        if (gl == 0) {
#pragma unroll
            for (int b = 0; b < RB; b++) {
                if (b < rows && a.mean) a.mean[r0 + b] = mean[b];
                if (b < rows && a.rstd) a.rstd[r0 + b] = rstd[b];
            }
        }
    }
}

template <int DT, int L, int K, int RB>
__global__ void __launch_bounds__(kLnThreads, 2) k_ln_backward_any(const __grid_constant__ LnArgs a)
{
    __shared__ float sh[2 * (kLnThreads / 32) * 2 * RB];
    __shared__ float join[K == 8 ? 2 * K * kLnThreads : 1];       // [group][dw, db][K][lanes]
    const int lanes = L < 32 ? L : 32 * a.warps, gl = threadIdx.x % lanes, group = threadIdx.x / lanes;
    const int groups = blockDim.x / lanes;
    const int here = gl < a.dim ? (int)((a.dim - 1 - gl) / lanes) + 1 : 0;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    float dw[K], db[K];
#pragma unroll
    for (int k = 0; k < K; k++)
        dw[k] = db[k] = 0.0f;
    const int64_t stride = (int64_t)gridDim.x * groups * RB;
    int64_t r0 = ((int64_t)blockIdx.x * groups + group) * RB;
    const int64_t first = L < 32 ? r0 - (int64_t)((threadIdx.x & 31) / L) * RB : r0;
    for (int64_t rw = first; rw < a.rows; rw += stride, r0 += stride) {
        const int rows = rows_here(a.rows, r0, RB);
        float x[RB][K], dy[RB][K], rstd[RB], c[2 * RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {
            const int64_t r = min(r0 + b, a.rows - 1);
            ld_strided<DT, K>(a.x, r * a.x_stride, gl, lanes, here, x[b]);
            ld_strided<DT, K>(a.dy, r * a.y_stride, gl, lanes, b < rows ? here : 0, dy[b]);
        }
#pragma unroll
        for (int b = 0; b < RB; b++) {
            const int64_t r = min(r0 + b, a.rows - 1);
            const float mean = a.mean_in[r];
            rstd[b] = a.rstd_in[r];
            c[2 * b] = c[2 * b + 1] = 0.0f;
#pragma unroll
            for (int k = 0; k < K; k++) {
                x[b][k] = ((k < here ? x[b][k] : mean) - mean) * rstd[b];            // xhat; 0 past the end
                if (b < rows) {
                    dw[k] = fmaf(dy[b][k], x[b][k], dw[k]);
                    db[k] += dy[b][k];
                }
            }
        }
        if (!a.dx) continue;
        if (a.weight) {
            float w[K];
            ld_strided<DT, K>(a.weight, 0, gl, lanes, here, w);
#pragma unroll
            for (int b = 0; b < RB; b++)
#pragma unroll
                for (int k = 0; k < K; k++)
                    dy[b][k] *= w[k];
        }
#pragma unroll
        for (int b = 0; b < RB; b++)
#pragma unroll
            for (int k = 0; k < K; k++) {
                c[2 * b] += dy[b][k];
                c[2 * b + 1] = fmaf(dy[b][k], x[b][k], c[2 * b + 1]);
            }
        group_sum<L, 2 * RB>(c, a.warps, sh, turn, [&](float t) { return t * -inv; });
#pragma unroll
        for (int b = 0; b < RB; b++) {
            const float k0 = c[2 * b] * rstd[b], k1 = c[2 * b + 1] * rstd[b];
            char* row = static_cast<char*>(a.dx) + (r0 + b) * a.x_stride * (DT == kF32 ? 4 : 2);
#pragma unroll
            for (int k = 0; k < K; k++)
                if (b < rows && k < here) st1<DT>(row, gl + k * lanes, fmaf(x[b][k], k1, fmaf(dy[b][k], rstd[b], k0)));
        }
    }
    if (!a.part) return;
    float* pw = a.part + 2 * (int64_t)blockIdx.x * a.dim;
    if (K == 8 && groups > 1) {
        const int one = 2 * K * lanes;
#pragma unroll
        for (int k = 0; k < K; k++) {
            join[group * one + k * lanes + gl] = dw[k];
            join[group * one + (K + k) * lanes + gl] = db[k];
        }
        __syncthreads();
        for (int t = threadIdx.x; t < one; t += blockDim.x) {
            float s = 0.0f;
            for (int g = 0; g < groups; g++)
                s += join[g * one + t];
            const int64_t j = t < K * lanes ? t : t - K * lanes;
            if (j < a.dim) pw[(t < K * lanes ? 0 : a.dim) + j] = s;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; k++)
            if (k < here) {
                pw[gl + (int64_t)k * lanes] = dw[k];
                pw[a.dim + gl + (int64_t)k * lanes] = db[k];
            }
    }
}

// ---- long rows -------------------------------------------------------------------------
// More than a block holds (forward over 4096 vectors of 16 bytes, backward over
// 2048): a block per row, values read again for every use (from cache), so the
// accesses bound it: 2048 x 40960 bfloat16 forward 274 us, 1.2 TB/s.  Backward in
// two kernels, rows for dx and columns for the weight gradients: 2048 x 20480 232
// us, 1.1 TB/s.  (Forward that size is in shared memory, one block of 10 warps
// an SM: 64 us, 2.6 TB/s.)
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
        const float mean = mean_of(block_sum(s, sh), (float)a.dim, inv);
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

// The blocks' partial sums: 32 columns a block, its 32 warps a part of the
// partial sums each, joined in warp order.  Bound by its own latency: 5.3 us
// alone for 32768 x 1600 as for 1003 x 771, part of it hidden by its early launch.
template <int DT>
__global__ void __launch_bounds__(1024) k_ln_dw_sum(const float* part, int blocks, int64_t dim, void* dw, void* db)
{
    wait_prev_grid();                                 // launched while the row kernel drains
    __shared__ float sh[2][32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f, t = 0.0f;
    if (j < dim)
#pragma unroll 5
        for (int k = warp; k < blocks; k += 32) {
            s += part[(2 * (int64_t)k) * dim + j];
            t += part[(2 * (int64_t)k + 1) * dim + j];
        }
    sh[0][warp][lane] = s;
    sh[1][warp][lane] = t;
    __syncthreads();
    if (warp > 0 || j >= dim) return;
    for (int k = 1; k < 32; k++) {
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

cudaError_t launch_rows(void (*kernel)(const LnArgs), const LnArgs& a, int64_t blocks, int threads, size_t smem,
                        cudaStream_t s)
{
    kernel<<<(unsigned)blocks, threads, smem, s>>>(a);
    return cudaGetLastError();
}

// A row kernel; SMEM bytes of slots, its static part with them over the
// default limit.
template <void (*KERNEL)(const LnArgs), size_t SMEM>
cudaError_t launch_slots(const LnArgs& a, int64_t blocks, int threads, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem((const void*)KERNEL, (int)SMEM, done);
    return e == cudaSuccess ? launch_rows(KERNEL, a, blocks, threads, SMEM, s) : e;
}

template <int DT, int L, int V, int RB, int S, int T, int BLOCKS>
cudaError_t forward_rows(LnArgs a, int64_t vecs, int align, cudaStream_t s)
{
    const RowShape h = shape_of(vecs, L, V, T);
    a.warps = h.warps;
    const int64_t at_once = (int64_t)h.groups * RB, need = (a.rows + at_once - 1) / at_once;
    const int64_t most = (int64_t)kSms * (BLOCKS * T / h.threads);            // resident at once
    const int64_t blocks = need < most ? need : most;
    constexpr size_t smem = (size_t)S * RB * V * T * 16;
    if constexpr (L == 32) {                          // fewer lanes: whole rows on 16-byte boundaries only
        if constexpr (DT != kF32)
            if (align < 16)
                return launch_slots<k_ln_forward_rows<DT, L, V, RB, S, T, BLOCKS, true, 4>, smem>(a, blocks, h.threads, s);
        if (a.dim % kVecOf<DT>)
            return launch_slots<k_ln_forward_rows<DT, L, V, RB, S, T, BLOCKS, true, 16>, smem>(a, blocks, h.threads, s);
    }
    return launch_slots<k_ln_forward_rows<DT, L, V, RB, S, T, BLOCKS, false, 16>, smem>(a, blocks, h.threads, s);
}

template <int DT, int L, int K, int RB>
cudaError_t forward_any(LnArgs a, int64_t eights, cudaStream_t s)
{
    const RowShape h = shape_of(eights, L, K / 8);
    a.warps = h.warps;
    const int64_t at_once = (int64_t)h.groups * RB, need = (a.rows + at_once - 1) / at_once;
    const int64_t most = (int64_t)kSms * (2 * kLnThreads / h.threads);
    return launch_rows(k_ln_forward_any<DT, L, K, RB>, a, need < most ? need : most, h.threads, 0, s);
}

// align: 16, 4 or 0, the boundary that every row starts on (of 0: its type's).
// 16-bit rows on 4-byte boundaries go the aligned rows' way in 4-byte copies of
// two values (32768 x 1602: 70 us against 84 value by value, backward 115 against
// 175); forward not the short ones (65536 x 134: 23 against 21, backward 35
// against 42).  In 32 bits such a copy is one value and loses (16384 x 1023:
// 43 against 30).
template <int DT>
cudaError_t forward(const LnArgs& a, int align, cudaStream_t s)
{
    constexpr int VE = kVecOf<DT>, T = kLnThreads, R = kLnFwdRows, S = kLnFwdAhead, B = kLnFwdBlocks;
    const int64_t vecs = (a.dim + VE - 1) / VE;
    const bool whole = a.dim % VE == 0 && align == 16;
    if (whole && vecs <= 8) return forward_rows<DT, 8, 1, 4, 3, T, 3>(a, vecs, align, s);
    if (whole && vecs <= 16) return forward_rows<DT, 16, 1, 4, 3, T, 3>(a, vecs, align, s);
    if (align == 16 || (DT != kF32 && align == 4 && vecs > 64)) {
        if (vecs <= 256) return forward_rows<DT, 32, 1, R, S, T, B>(a, vecs, align, s);
        if (vecs <= 512) return forward_rows<DT, 32, 2, R / 2, S, T, B>(a, vecs, align, s);
        if (vecs <= 1024) return forward_rows<DT, 32, 4, R / 4, S, T, B>(a, vecs, align, s);
        if (vecs <= 2048) return forward_rows<DT, 32, 8, 1, 2, T, 2>(a, vecs, align, s);
        if (vecs <= 4096) return forward_rows<DT, 32, 8, 1, 2, 2 * T, 1>(a, vecs, align, s);
    } else {
        const int64_t eights = (a.dim + 7) / 8;
        if (eights <= 8) return forward_any<DT, 8, 8, 4>(a, eights, s);
        if (eights <= 16) return forward_any<DT, 16, 8, 4>(a, eights, s);
        if (eights <= 256) return forward_any<DT, 32, 8, 4>(a, eights, s);
        if (eights <= 512) return forward_any<DT, 32, 16, 2>(a, eights, s);
        if (eights <= 1024) return forward_any<DT, 32, 32, 1>(a, eights, s);
    }
    return launch_rows(k_ln_forward<DT>, a, a.rows < kSms * 8 ? a.rows : kSms * 8, kLnThreads, 0, s);
}

// How the backward pass deals out a row: lanes of a group, vectors of a lane,
// threads and resident blocks, rows at a time.  The plan's blocks go by it
// (as for rows on 16-byte boundaries) whatever the pointers turn out to be.
struct BackwardShape {
    int L, V, T, blocks, rows;
};

BackwardShape backward_shape(int64_t vecs, bool whole)
{
    const int L = whole && vecs <= 8 ? 8 : whole && vecs <= 16 ? 16 : 32;
    if (vecs <= 256) return {L, 1, kLnThreads, kLnBwdBlocks, kLnBwdRows};
    if (vecs <= 512) return {L, 2, kLnThreads, kLnBwdBlocks, kLnBwdRows / 2};
    if (vecs <= 1024) return {L, 4, kLnThreads, kLnBwdBlocks, kLnBwdRows / 4};
    // up to 2048 vectors (8192 x 10464 of 16 bits: 158 us; x read twice, dy twice, in two kernels: 352)
    return {L, 4, 2 * kLnThreads, 1, kLnBwdRows / 4};
}

template <int DT, int L, int V, int RB, int T, int BLOCKS>
cudaError_t backward_rows(LnArgs a, int64_t vecs, int align, int blocks, cudaStream_t s)
{
    const RowShape h = shape_of(vecs, L, V, T);
    a.warps = h.warps;
    constexpr int S = kLnBwdAhead;
    constexpr size_t smem = (size_t)S * RB * V * 2 * T * 16;
    if constexpr (L == 32) {
        if constexpr (DT != kF32)
            if (align < 16)
                return launch_slots<k_ln_backward_rows<DT, L, V, RB, S, T, BLOCKS, true, 4>, smem>(a, blocks, h.threads, s);
        if (a.dim % kVecOf<DT>)
            return launch_slots<k_ln_backward_rows<DT, L, V, RB, S, T, BLOCKS, true, 16>, smem>(a, blocks, h.threads, s);
    }
    return launch_slots<k_ln_backward_rows<DT, L, V, RB, S, T, BLOCKS, false, 16>, smem>(a, blocks, h.threads, s);
}

// Blocks of the backward pass (the plan's): as many as are resident at once on
// 152 SMs, and no more than have rows.
int64_t backward_blocks(int64_t rows, int64_t vecs, bool whole)
{
    const BackwardShape b = backward_shape(vecs, whole);
    const RowShape h = shape_of(vecs <= 2048 ? vecs : 2048, b.L, b.V, b.T);
    const int64_t at_once = (int64_t)h.groups * b.rows, need = (rows + at_once - 1) / at_once;
    const int64_t most = (int64_t)kSms * (b.blocks * b.T / h.threads);
    return need < most ? need : most;
}

template <int DT, int L, int K, int RB>
cudaError_t backward_any(LnArgs a, int64_t eights, int blocks, cudaStream_t s)
{
    const RowShape h = shape_of(eights, L, K / 8);
    a.warps = h.warps;
    return launch_rows(k_ln_backward_any<DT, L, K, RB>, a, blocks, h.threads, 0, s);
}

template <int DT>
cudaError_t backward(LnArgs a, int align, int blocks, void* dw, void* db, cudaStream_t s)
{
    constexpr int VE = kVecOf<DT>, T = kLnThreads, R = kLnBwdRows, B = kLnBwdBlocks;
    const int64_t vecs = (a.dim + VE - 1) / VE, eights = (a.dim + 7) / 8;
    const bool sums = dw || db;
    if (!sums) a.part = nullptr;
    cudaError_t e = cudaSuccess;
    if (blocks && vecs <= 2048 && (align == 16 || (DT != kF32 && align == 4 && vecs > 16))) {
        const int L = align == 16 ? backward_shape(vecs, a.dim % VE == 0).L : 32;
        if (L == 8) e = backward_rows<DT, 8, 1, R, T, B>(a, vecs, align, blocks, s);
        else if (L == 16) e = backward_rows<DT, 16, 1, R, T, B>(a, vecs, align, blocks, s);
        else if (vecs <= 256) e = backward_rows<DT, 32, 1, R, T, B>(a, vecs, align, blocks, s);
        else if (vecs <= 512) e = backward_rows<DT, 32, 2, R / 2, T, B>(a, vecs, align, blocks, s);
        else if (vecs <= 1024) e = backward_rows<DT, 32, 4, R / 4, T, B>(a, vecs, align, blocks, s);
        else e = backward_rows<DT, 32, 4, R / 4, 2 * T, 1>(a, vecs, align, blocks, s);
    } else if (blocks && align < 16 && a.dim <= 4096) {
        if (eights <= 8) e = backward_any<DT, 8, 8, 2>(a, eights, blocks, s);
        else if (eights <= 16) e = backward_any<DT, 16, 8, 2>(a, eights, blocks, s);
        else if (eights <= 256) e = backward_any<DT, 32, 8, 2>(a, eights, blocks, s);
        else e = backward_any<DT, 32, 16, 1>(a, eights, blocks, s);
    } else {
        if (a.dx && a.rows) e = launch_rows(k_ln_dx<DT>, a, a.rows < kSms * 8 ? a.rows : kSms * 8, kLnThreads, 0, s);
        if (e == cudaSuccess && sums && blocks) {
            const unsigned cols = (unsigned)((a.dim + kLnThreads - 1) / kLnThreads);
            k_ln_dw_part<DT><<<dim3(cols, (unsigned)blocks), kLnThreads, 0, s>>>(a);
            e = cudaGetLastError();
        }
    }
    if (e == cudaSuccess && sums)
        e = launch_kernel(k_ln_dw_sum<DT>, (int)((a.dim + 31) / 32), 1024, s, blocks > 0, (const float*)a.part,
                          blocks, a.dim, dw, db);
    return e;
}

// The boundary that every row of x and y (or dy, dx: a, b, c) starts on: 16, 4
// or 0 bytes (their type's).  weight and bias off 16-byte boundaries count as 0.
int rows_align(const zero_ln_plan_t& p, const void* a, const void* b, const void* c, const void* weight, const void* bias)
{
    const uint64_t e = p.dtype == ZERO_FP32 ? 4 : 2;
    const uint64_t any = (uintptr_t)a | (uintptr_t)b | (uintptr_t)c | (uint64_t)p.x_stride * e | (uint64_t)p.y_stride * e;
    if (((uintptr_t)weight | (uintptr_t)bias) % 16) return 0;
    return any % 16 == 0 ? 16 : any % 4 == 0 ? 4 : 0;
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
    if (rows && (xs > INT64_MAX / 16 / rows || ys > INT64_MAX / 16 / rows))   // 3 * 4 bytes of each below INT64_MAX
        return set_error(ZERO_EUNSUPPORTED, "zero_ln_plan: the rows span too many bytes");
    std::memset(out, 0, sizeof *out);
    out->rows = rows;
    out->dim = dim;
    out->x_stride = xs;
    out->y_stride = ys;
    out->dtype = dtype;
    const int64_t e = dtype == ZERO_FP32 ? 4 : 2;
    out->blocks = (int32_t)backward_blocks(rows, (dim * e + 15) / 16, dim * e % 16 == 0);   // each adds up its rows' weight gradients
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
    const int align = rows_align(*plan, x, y, nullptr, weight, bias);
    const cudaError_t err = plan->dtype == ZERO_FP32   ? forward<kF32>(a, align, s)
                            : plan->dtype == ZERO_BF16 ? forward<kBF16>(a, align, s)
                                                       : forward<kF16>(a, align, s);
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
    const int align = rows_align(*plan, x, dy, dx, weight, nullptr);
    const cudaError_t err = plan->dtype == ZERO_FP32   ? backward<kF32>(a, align, plan->blocks, dweight, dbias, s)
                            : plan->dtype == ZERO_BF16 ? backward<kBF16>(a, align, plan->blocks, dweight, dbias, s)
                                                       : backward<kF16>(a, align, plan->blocks, dweight, dbias, s);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_ln_backward");
}

}  // extern "C"
