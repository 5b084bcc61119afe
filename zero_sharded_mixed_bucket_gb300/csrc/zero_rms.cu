// Root-mean-square norm of rows with the residual's addition: the plan, the
// forward kernels (results in the rows' type, or in 8 bits with a scale per
// block), the read-out of 8-bit results, and the backward pass.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "dev_rows.cuh"
#include "nvtx_ranges.h"

namespace zg {

using namespace rows;

namespace {

// Every kernel here is launched while its predecessor in the stream drains, and waits for
// its end before it reads or writes anything: 2 us less of a launch.
__device__ __forceinline__ void in_turn()
{
    wait_prev_grid();
    allow_next_grid();
}

struct RmsArgs {
    const void* x;               // forward: a block's output; backward: h
    const void* r;               // forward: the stream; backward: the stream's own gradient (either may be NULL)
    const void* dy;
    const void* weight;
    const float* rstd_in;
    void* h;
    void* y;
    uint8_t* q;
    uint8_t* q_scale;
    float* rstd;
    void* dx;
    float* part;                 // [blocks][dim]: partial dweight
    int64_t rows, dim, x_stride, y_stride, scale_cols;
    float eps;
    int warps;                   // of a group
    int take;                    // rows of a batch, up to the kernel's RB
    int block;                   // values to a scale
    int q_wide;                  // a vector's codes are stored at once
};

// 1 / sqrt(a), the approximation once corrected by what it leaves (an error of the
// row's factor moves every value of the row at once).
__device__ __forceinline__ float inverse_root(float a)
{
    const float r = rsqrtf(a), better = fmaf(0.5f * r, fmaf(-a * r, r, 1.0f), r);
    return r > 0.0f && r < INFINITY ? better : r;
}

// ---- 8-bit results ------------------------------------------------------------------------
// Codes are e4m3 (448 the largest), a block's scale 2^(e - 127) the least power of
// two that keeps its largest magnitude within 448.  A power of two scales
// exactly, so each value is rounded once.  A block with an infinity or a NaN:
// scale byte 255, NaN codes.
__device__ __forceinline__ uint32_t scale_byte(uint32_t most)
{
    // 448 = 1.75 * 2^8: a fraction above 0x600000 carries into the exponent
    const uint32_t e = (uint32_t)max((int)((most + 0x1fffffu) >> 23) - 8, 0);
    return most >= 0x7f800000u ? 255u : e;
}

// 2^(127 - e), NaN for 255.
__device__ __forceinline__ float scale_up(uint32_t e) { return __uint_as_float(e == 255u ? 0x7fffffffu : (254u - e) << 23); }

__device__ __forceinline__ uint32_t codes2(float a, float b)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t code1(float a) { return codes2(a, 0.0f) & 0xffu; }

// Two codes (bytes 8 and 24 up of w) as bfloat16 values times `scale`.  A code's seven
// low bits, moved into a bfloat16's exponent and fraction, are 2^-120 times its value,
// subnormal or not (all ones: NaN).
__device__ __forceinline__ uint32_t values2(uint32_t w, __nv_bfloat162 scale)
{
    const uint32_t size = (w >> 4) & 0x07f007f0u;
    const uint32_t bits = (w & 0x80008000u) | size | (__vcmpeq2(size, 0x07f007f0u) & 0x7fff7fffu);   // the last is NaN
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&bits), scale);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// 2^120 * 2^(e - 127), NaN for 255; above bfloat16's range `rest` is what is left.
__device__ __forceinline__ __nv_bfloat162 scale_of(uint32_t e, uint32_t& rest)
{
    const uint32_t most = 254u - 120u;                // 2^127
    rest = e == 255u ? 0u : e - min(e, most);
    const uint32_t one = e == 255u ? 0x7fffu : (min(e, most) + 120u) << 7, two = one | one << 16;
    return *reinterpret_cast<const __nv_bfloat162*>(&two);
}

// A pair of values times 2^rest.
__device__ __forceinline__ uint32_t scaled_more(uint32_t v, uint32_t rest)
{
    const uint32_t one = (rest + 127u) << 7, two = one | one << 16;
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&two));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// The largest of three magnitudes, NaN if one is.
__device__ __forceinline__ float most_of(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// a + b, rounded once to the rows' type (16-bit pairs at once: what a binary32 sum
// rounded again gives too, which is exact wherever the smaller value can matter).
template <int DT>
__device__ __forceinline__ Vals<DT> added(const Vals<DT>& a, const Vals<DT>& b)
{
    Vals<DT> r;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if constexpr (DT == kF32) {
            r.w[k] = __float_as_uint(__uint_as_float(a.w[k]) + __uint_as_float(b.w[k]));
        } else if constexpr (DT == kBF16) {
            const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a.w[k]),
                                             *reinterpret_cast<const __nv_bfloat162*>(&b.w[k]));
            r.w[k] = *reinterpret_cast<const uint32_t*>(&s);
        } else {
            const __half2 s = __hadd2(*reinterpret_cast<const __half2*>(&a.w[k]), *reinterpret_cast<const __half2*>(&b.w[k]));
            r.w[k] = *reinterpret_cast<const uint32_t*>(&s);
        }
    }
    return r;
}

// A lane's vector of the weight as it is stored, ones where there is none, 0 past the
// row's end.
template <int DT>
__device__ __forceinline__ Vals<DT> weight_held(const void* p, int64_t i, int cnt)
{
    Vals<DT> v;
    if (p && cnt == kVecOf<DT>) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (DT == kF32 ? 4 : 2));
        v.w[0] = u.x; v.w[1] = u.y; v.w[2] = u.z; v.w[3] = u.w;
    } else {
        float f[kVecOf<DT>];
#pragma unroll
        for (int k = 0; k < kVecOf<DT>; k++)
            f[k] = k < cnt ? (p ? ld1<DT>(p, i + k) : 1.0f) : 0.0f;
        v = pack<DT>(f);
    }
    return v;
}

// ---- rows on 16-byte boundaries -----------------------------------------------------------
// Dealt out as layer norm's: a group of lanes to a row, V vectors to a lane,
// `take` rows (RB at most) at a time, copied ahead into per-lane slots.  The sum
// x + r is rounded to the rows' type first (what the stream holds, and what
// backward sees), then kept in registers; its slot is free for the next copy
// before the group has its sum.  Q: values to a scale of 8-bit results, 0: none; a
// block of them is Q / VE neighbouring lanes of a warp, or a whole shorter row.
// Bound by memory: 8192 x 4096 bfloat16 with a residual 45.7 us, 5.9 TB/s (a device
// copy of the same bytes takes 43.3), issuing in 42 % of the cycles, 16
// instructions a value; into 8 bits 41.5, 22 instructions a value in 55 %.  The
// lane's weights stay in registers (read for every batch they are what a warp
// waits for after the sum: 49.2), so blocks are few and large: with three blocks of
// 256 threads an SM 49 and 47 us.
template <int DT, int L, int V, int RB, int S, int T, int BLOCKS, bool RAGGED, int Q>
__global__ void __launch_bounds__(T, BLOCKS) k_rms_forward_rows(const __grid_constant__ RmsArgs a)
{
    in_turn();
    constexpr int VE = kVecOf<DT>, E = DT == kF32 ? 4 : 2;
    constexpr bool kHold = V <= 4;
    extern __shared__ uint4 slots[];                  // [S][RB * V][x, r][T]
    __shared__ float sh[2 * (T / 32) * RB];
    const int lanes = L < 32 ? L : 32 * a.warps, gl = threadIdx.x % lanes, group = threadIdx.x / lanes;
    const int groups = blockDim.x / lanes;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    int cnt[V];
    Vals<DT> wv[kHold ? V : 1];                       // a lane's columns are the same in every batch
#pragma unroll
    for (int v = 0; v < V; v++) {
        cnt[v] = vec_count<DT>(a.dim, v, gl, lanes);
        if (kHold) wv[v] = weight_held<DT>(a.weight, (int64_t)(v * lanes + gl) * VE, cnt[v]);
    }
    const int64_t stride = (int64_t)gridDim.x * groups * a.take;
    int64_t r0 = ((int64_t)blockIdx.x * groups + group) * a.take;
    int64_t ahead = r0;
    const int64_t x_row = a.x_stride * E, y_row = a.y_stride * E;
    const int apart = lanes * 16;                     // bytes between a lane's vectors
    const char* sx = static_cast<const char*>(a.x) + r0 * x_row + gl * 16;
    const char* sr = static_cast<const char*>(a.r) + r0 * x_row + gl * 16;
    const bool add = a.r != nullptr;
    uint4* const mine = slots + threadIdx.x;
    auto fetch = [&](uint4* at) {
        const int here = rows_here(a.rows, ahead, a.take);
        const char *px = sx, *pr = sr;
#pragma unroll
        for (int b = 0; b < RB; b++, px += x_row, pr += x_row)
            if (b < here)
#pragma unroll
                for (int v = 0; v < V; v++)
                    if (cnt[v]) {
                        uint4* p = at + (b * V + v) * 2 * T;
                        vec_ahead<16>(p, px + v * apart, RAGGED ? cnt[v] * E : 16);
                        if (add) vec_ahead<16>(p + T, pr + v * apart, RAGGED ? cnt[v] * E : 16);
                    }
        copies_issued();
        ahead += stride;
        sx += stride * x_row;
        sr += stride * x_row;
    };
#pragma unroll
    for (int k = 0; k < S * RB * V * 2; k++)          // vectors past the row's end are never copied: 0
        if (cnt[k / 2 % V] == 0) mine[k * T] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < S; k++)
        fetch(mine + k * RB * V * 2 * T);
    // groups of less than a warp go round together: their sums shuffle across the warp
    const int64_t first = L < 32 ? r0 - (int64_t)((threadIdx.x & 31) / L) * a.take : r0;
    int slot = 0;
    for (int64_t rw = first; rw < a.rows; rw += stride) {
        copies_wait<S - 1>();
        uint4* const q = mine + slot * RB * V * 2 * T;    // rows past the end: whatever is there, not written
        const int here = rows_here(a.rows, r0, a.take);
        Vals<DT> h[RB][V];
        float ss[RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {
            ss[b] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) {
                h[b][v] = from_slot<DT>(q + (b * V + v) * 2 * T);
                if (add) h[b][v] = added<DT>(h[b][v], from_slot<DT>(q + ((b * V + v) * 2 + 1) * T));
                float f[VE];
                unpack<DT>(h[b][v], f);
#pragma unroll
                for (int k = 0; k < VE; k++)
                    ss[b] = fmaf(f[k], f[k], ss[b]);
            }
        }
        fetch(q);
        slot = slot == S - 1 ? 0 : slot + 1;
        if (a.h) {
            char* p = static_cast<char*>(a.h) + r0 * x_row + gl * 16;
#pragma unroll
            for (int b = 0; b < RB; b++, p += x_row)
#pragma unroll
                for (int v = 0; v < V; v++)
                    if (b < here && cnt[v]) store_vec<DT, RAGGED, 16>(p + v * apart, h[b][v], cnt[v]);
        }
        group_sum<L, RB, T>(ss, a.warps, sh, turn, [&](float t) { return inverse_root(fmaf(t, inv, a.eps)); });
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (!Q && cnt[v] == 0) continue;
            const int64_t j = (int64_t)(v * lanes + gl) * VE;
            float w[VE];                              // 0 past the row's end, where h is 0 too
            unpack<DT>(kHold ? wv[v] : weight_held<DT>(a.weight, j, cnt[v]), w);
            char* p = static_cast<char*>(a.y) + r0 * y_row + gl * 16 + v * apart;
#pragma unroll
            for (int b = 0; b < RB; b++, p += y_row) {
                float f[VE];
                unpack<DT>(h[b][v], f);
#pragma unroll
                for (int k = 0; k < VE; k++)
                    f[k] = f[k] * ss[b] * w[k];
                if (a.y && b < here && cnt[v]) store_vec<DT, RAGGED, 16>(p, pack<DT>(f), cnt[v]);
                if constexpr (Q > 0) {
                    constexpr int kSpan = Q / VE < L ? Q / VE : L;            // lanes of a block; a shorter row is one
                    float most = 0.0f;
#pragma unroll
                    for (int k = 0; k < VE; k += 2)
                        most = most_of(most, f[k], f[k + 1]);
#pragma unroll
                    for (int o = 1; o < kSpan; o <<= 1)
                        most = most_of(most, 0.0f, __shfl_xor_sync(0xffffffffu, most, o));
                    if (b < here && cnt[v]) {
                        const uint32_t e = scale_byte(__float_as_uint(most));
                        const float up = scale_up(e);
                        uint32_t c[VE / 4];
#pragma unroll
                        for (int k = 0; k < VE / 4; k++)
                            c[k] = codes2(f[4 * k] * up, f[4 * k + 1] * up) | codes2(f[4 * k + 2] * up, f[4 * k + 3] * up) << 16;
                        uint8_t* at = a.q + (r0 + b) * a.y_stride + j;
                        if (a.q_wide && (!RAGGED || cnt[v] == VE)) {
                            if constexpr (VE == 8)
                                __stcs(reinterpret_cast<uint2*>(at), make_uint2(c[0], c[1]));
                            else
                                __stcs(reinterpret_cast<uint32_t*>(at), c[0]);
                        } else {
#pragma unroll
                            for (int k = 0; k < VE; k++)
                                if (k < cnt[v]) at[k] = (uint8_t)(c[k >> 2] >> (8 * (k & 3)));
                        }
                        if ((threadIdx.x & (kSpan - 1)) == 0) a.q_scale[(r0 + b) * a.scale_cols + j / Q] = (uint8_t)e;
                    }
                }
            }
        }
        if (gl == 0 && a.rstd) {
#pragma unroll
            for (int b = 0; b < RB; b++)
                if (b < here) a.rstd[r0 + b] = ss[b];
        }
        r0 += stride;
    }
    copies_wait<0>();
}

// Backward: the stream's gradient of the rows, and the column sums of dy * xhat
// over all the rows of a lane in registers, so h and dy are read once for both.
// A block writes one partial sum per column (its groups joined in group order).
// Bound by memory: 32768 x 1600 binary16 68.2 us with the sums' join, 6.2 TB/s; 26
// instructions a value in 58 % of the cycles.  Weights read for every batch: 80.6;
// as packed pairs of binary32 operations no less (70.9); two rows a batch instead of
// four 85, one 107.
template <int DT, int L, int V, int RB, int S, int T, int BLOCKS, bool RAGGED>
__global__ void __launch_bounds__(T, BLOCKS) k_rms_backward_rows(const __grid_constant__ RmsArgs a)
{
    in_turn();
    constexpr int VE = kVecOf<DT>, E = DT == kF32 ? 4 : 2;
    extern __shared__ uint4 slots[];                  // [S][RB * V][h, dy, r][T]; at the end the groups' sums
    __shared__ float sh[2 * (T / 32) * RB];
    const int lanes = L < 32 ? L : 32 * a.warps, gl = threadIdx.x % lanes, group = threadIdx.x / lanes;
    const int groups = blockDim.x / lanes;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    int cnt[V];
    float dw[V][VE];
    float w1[VE];                                     // V = 1: a lane's columns are the same in every batch
    Vals<DT> wv[V > 1 ? V : 1];
#pragma unroll
    for (int v = 0; v < V; v++) {
        cnt[v] = vec_count<DT>(a.dim, v, gl, lanes);
        wv[v] = weight_held<DT>(a.weight, (int64_t)(v * lanes + gl) * VE, cnt[v]);
        if (V == 1) unpack<DT>(wv[v], w1);
#pragma unroll
        for (int k = 0; k < VE; k++)
            dw[v][k] = 0.0f;
    }
    const int64_t stride = (int64_t)gridDim.x * groups * a.take;
    int64_t r0 = ((int64_t)blockIdx.x * groups + group) * a.take;
    int64_t ahead = r0;
    const int64_t x_row = a.x_stride * E, y_row = a.y_stride * E;
    const int apart = lanes * 16;
    const char* sx = static_cast<const char*>(a.x) + r0 * x_row + gl * 16;
    const char* sr = static_cast<const char*>(a.r) + r0 * x_row + gl * 16;
    const char* sy = static_cast<const char*>(a.dy) + r0 * y_row + gl * 16;
    const bool add = a.r != nullptr;
    uint4* const mine = slots + threadIdx.x;
    auto fetch = [&](uint4* at) {
        const int here = rows_here(a.rows, ahead, a.take);
        const char *px = sx, *py = sy, *pr = sr;
#pragma unroll
        for (int b = 0; b < RB; b++, px += x_row, py += y_row, pr += x_row)
#pragma unroll
            for (int v = 0; v < V; v++) {
                uint4* p = at + (b * V + v) * 3 * T;
                if (b < here) {
                    if (cnt[v]) {
                        vec_ahead<16>(p, px + v * apart, RAGGED ? cnt[v] * E : 16);
                        vec_ahead<16>(p + T, py + v * apart, RAGGED ? cnt[v] * E : 16);
                        if (add) vec_ahead<16>(p + 2 * T, pr + v * apart, RAGGED ? cnt[v] * E : 16);
                    }
                } else {                              // rows past the end: all 0
                    p[0] = p[T] = make_uint4(0, 0, 0, 0);
                }
            }
        copies_issued();
        ahead += stride;
        sx += stride * x_row;
        sy += stride * y_row;
        sr += stride * x_row;
    };
    float next[RB];
    auto fetch_stats = [&](int64_t from) {
        const int here = rows_here(a.rows, from, a.take);
#pragma unroll
        for (int b = 0; b < RB; b++)
            next[b] = b < here ? a.rstd_in[from + b] : 0.0f;
    };
#pragma unroll
    for (int k = 0; k < S * RB * V * 3; k++)          // vectors past the row's end are never copied: 0
        if (cnt[k / 3 % V] == 0) mine[k * T] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < S; k++)
        fetch(mine + k * RB * V * 3 * T);
    fetch_stats(r0);
    const int64_t first = L < 32 ? r0 - (int64_t)((threadIdx.x & 31) / L) * a.take : r0;
    int slot = 0;
    for (int64_t rw = first; rw < a.rows; rw += stride) {
        copies_wait<S - 1>();
        uint4* const q = mine + slot * RB * V * 3 * T;
        float rstd[RB], c[RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {
            rstd[b] = next[b];
            c[b] = 0.0f;
        }
        fetch_stats(r0 + stride);
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (cnt[v] == 0) continue;
            float w[VE];
            if (V > 1) unpack<DT>(wv[v], w);
#pragma unroll
            for (int k = 0; k < VE; k++)
                if (V == 1) w[k] = w1[k];
#pragma unroll
            for (int b = 0; b < RB; b++) {
                float xf[VE], yf[VE];
                unpack<DT>(from_slot<DT>(q + (b * V + v) * 3 * T), xf);
                unpack<DT>(from_slot<DT>(q + ((b * V + v) * 3 + 1) * T), yf);   // 0 past the ends
#pragma unroll
                for (int k = 0; k < VE; k++) {
                    const float n = xf[k] * rstd[b];
                    dw[v][k] = fmaf(yf[k], n, dw[v][k]);
                    c[b] = fmaf(yf[k] * w[k], n, c[b]);
                }
            }
        }
        if (a.dx) {
            group_sum<L, RB, T>(c, a.warps, sh, turn, [&](float t) { return t * -inv; });
#pragma unroll
            for (int b = 0; b < RB; b++)
                c[b] *= rstd[b];
            const int here = rows_here(a.rows, r0, a.take);
#pragma unroll
            for (int v = 0; v < V; v++) {
                if (cnt[v] == 0) continue;
                float w[VE];
                if (V > 1) unpack<DT>(wv[v], w);
#pragma unroll
                for (int k = 0; k < VE; k++)
                    if (V == 1) w[k] = w1[k];
                char* p = static_cast<char*>(a.dx) + r0 * x_row + gl * 16 + v * apart;
#pragma unroll
                for (int b = 0; b < RB; b++, p += x_row) {
                    float xf[VE], yf[VE];
                    unpack<DT>(from_slot<DT>(q + (b * V + v) * 3 * T), xf);
                    unpack<DT>(from_slot<DT>(q + ((b * V + v) * 3 + 1) * T), yf);
#pragma unroll
                    for (int k = 0; k < VE; k++)
                        xf[k] = fmaf(xf[k], c[b], yf[k] * w[k]);
                    if (add) {
                        unpack<DT>(from_slot<DT>(q + ((b * V + v) * 3 + 2) * T), yf);
#pragma unroll
                        for (int k = 0; k < VE; k++)
                            xf[k] = fmaf(xf[k], rstd[b], yf[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < VE; k++)
                            xf[k] *= rstd[b];
                    }
                    if (b < here) store_vec<DT, RAGGED, 16>(p, pack<DT>(xf), cnt[v]);
                }
            }
        }
        fetch(q);
        slot = slot == S - 1 ? 0 : slot + 1;
        r0 += stride;
    }
    copies_wait<0>();
    if (!a.part) return;
    float* pw = a.part + (int64_t)blockIdx.x * a.dim;
    if (V == 1 && groups > 1) {
        float* join = reinterpret_cast<float*>(slots);            // [group][VE][lanes]: no more than the slots
        const int one = VE * lanes;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < VE; k++)
            join[group * one + k * lanes + gl] = dw[0][k];
        __syncthreads();
        for (int t = threadIdx.x; t < one; t += blockDim.x) {
            float s = 0.0f;
            for (int g = 0; g < groups; g++)
                s += join[g * one + t];
            const int k = t / lanes;
            const int64_t j = (int64_t)(t - k * lanes) * VE + k;
            if (j < a.dim) pw[j] = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; v++)
#pragma unroll
            for (int k = 0; k < VE; k++)
                if (k < cnt[v]) pw[(int64_t)(v * lanes + gl) * VE + k] = dw[v][k];
    }
}

// ---- other rows ------------------------------------------------------------------------
// One access a value.  W warps to a row (known to the compiler, so that a lane's places
// are distances from one address), each with blocks of 128 neighbouring values, four
// of a block to a lane, 32 apart: neighbouring lanes neighbouring values, and a
// block's largest magnitude stays inside the warp.  Bound by the accesses, 4 a value,
// and the instructions around them: 8192 x 4095 bfloat16 65 us, into 8 bits 70,
// backward 86, 2048 x 16383 96 (with the warps' number unknown to the compiler 114, 196 and 188).
// 16-bit rows on 4-byte boundaries gain nothing by copies of two values (8192 x
// 4094: 68 and 92 us, here 66 and 86).
template <int W>
__host__ __device__ constexpr int place(int k) { return (k >> 2) * W * 128 + (k & 3) * 32; }

constexpr int kAnyResident = 1024;                    // threads on an SM

// Values of the lane that are `left` or more places before the row's end; 0 for the rest.
template <int DT, int K, int W>
__device__ __forceinline__ void ld_places(const char* p, int left, float f[K])
{
    constexpr int E = DT == kF32 ? 4 : 2;
#pragma unroll
    for (int k = 0; k < K; k++) {
        uint32_t u = 0;
        if (place<W>(k) < left) {
            if constexpr (DT == kF32) u = *reinterpret_cast<const uint32_t*>(p + place<W>(k) * E);
            else u = *reinterpret_cast<const uint16_t*>(p + place<W>(k) * E);
        }
        f[k] = to_f32<DT>(u);
    }
}

template <int DT, int K, int W>
__device__ __forceinline__ void st_places(char* p, int left, const float f[K])
{
    constexpr int E = DT == kF32 ? 4 : 2;
#pragma unroll
    for (int k = 0; k < K; k++)
        if (place<W>(k) < left) st1<DT>(p + place<W>(k) * E, 0, f[k]);
}

// 8-bit results of a block of 128 values of which the lane's are 32 apart and `left`
// or more places before the row's end; q and q_scale: of the lane's first, and of the
// block's first scale.
template <int BLOCK>
__device__ __forceinline__ void codes_out(uint8_t* q, uint8_t* q_scale, int left, int lane, const float f[4])
{
    uint32_t most[4], e[4];
#pragma unroll
    for (int k = 0; k < 4; k++)
        most[k] = 32 * k < left ? magnitude(f[k]) : 0u;
    if (BLOCK == 128) {
        e[0] = scale_byte(__reduce_max_sync(0xffffffffu, max(max(most[0], most[1]), max(most[2], most[3]))));
        e[1] = e[2] = e[3] = e[0];
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
            e[k] = scale_byte(__reduce_max_sync(0xffffffffu, most[k]));
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if (32 * k < left) q[32 * k] = (uint8_t)code1(f[k] * scale_up(e[k]));
        if ((BLOCK == 32 || k == 0) && lane == 0 && 32 * k < left) q_scale[k] = (uint8_t)e[k];
    }
}

template <int DT, int K, int W, int RB, int T>
__global__ void __launch_bounds__(T, (K > 16 ? 512 : 1024) / T) k_rms_forward_any(const __grid_constant__ RmsArgs a)
{
    in_turn();
    constexpr int E = DT == kF32 ? 4 : 2;
    __shared__ float sh[2 * (T / 32) * RB];
    const int lane = threadIdx.x & 31, group = (int)(threadIdx.x >> 5) / W, warp = (int)(threadIdx.x >> 5) % W;
    const int groups = T / (32 * W), j0 = warp * 128 + lane, left = (int)a.dim - j0;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    float w[K];
    auto weights = [&]() {
        if (a.weight) {
            ld_places<DT, K, W>(static_cast<const char*>(a.weight) + j0 * E, left, w);
        } else {
#pragma unroll
            for (int k = 0; k < K; k++)
                w[k] = 1.0f;
        }
    };
    if (K <= 16) weights();
    const int64_t x_row = a.x_stride * E, y_row = a.y_stride * E;
    const int64_t stride = (int64_t)gridDim.x * groups * a.take;
    for (int64_t r0 = ((int64_t)blockIdx.x * groups + group) * a.take; r0 < a.rows; r0 += stride) {
        const int rows = rows_here(a.rows, r0, a.take);
        const int64_t x_at = r0 * x_row + j0 * E, y_at = r0 * y_row + j0 * E;
        float f[RB][K], ss[RB];
#pragma unroll
        for (int b = 0; b < RB; b++)                  // rows past the end: the last again, not written
            ld_places<DT, K, W>(static_cast<const char*>(a.x) + x_at + min(b, rows - 1) * x_row, left, f[b]);
        if (a.r) {
#pragma unroll
            for (int b = 0; b < RB; b++) {
                float g[K];
                ld_places<DT, K, W>(static_cast<const char*>(a.r) + x_at + min(b, rows - 1) * x_row, left, g);
#pragma unroll
                for (int k = 0; k < K; k++)
                    f[b][k] = to_f32<DT>(from_f32<DT>(f[b][k] + g[k]));
            }
        }
#pragma unroll
        for (int b = 0; b < RB; b++) {
            ss[b] = 0.0f;
#pragma unroll
            for (int k = 0; k < K; k++)
                ss[b] = fmaf(f[b][k], f[b][k], ss[b]);
            if (a.h && b < rows) st_places<DT, K, W>(static_cast<char*>(a.h) + x_at + b * x_row, left, f[b]);
        }
        group_sum<32, RB, T>(ss, W, sh, turn, [&](float t) { return inverse_root(fmaf(t, inv, a.eps)); });
        if (K > 16) weights();
#pragma unroll
        for (int b = 0; b < RB; b++) {
#pragma unroll
            for (int k = 0; k < K; k++)
                f[b][k] = f[b][k] * ss[b] * w[k];
            if (b >= rows) continue;
            if (a.y) st_places<DT, K, W>(static_cast<char*>(a.y) + y_at + b * y_row, left, f[b]);
            if (a.q) {
                uint8_t* q = a.q + (r0 + b) * a.y_stride + j0;
                uint8_t* q_scale = a.q_scale + (r0 + b) * a.scale_cols;
#pragma unroll
                for (int k = 0; k < K; k += 4) {
                    if (a.block == 128)
                        codes_out<128>(q + place<W>(k), q_scale + (k >> 2) * W + warp, left - place<W>(k), lane, f[b] + k);
                    else
                        codes_out<32>(q + place<W>(k), q_scale + 4 * ((k >> 2) * W + warp), left - place<W>(k), lane, f[b] + k);
                }
            }
            if (lane == 0 && warp == 0 && a.rstd) a.rstd[r0 + b] = ss[b];
        }
    }
}

template <int DT, int K, int W, int RB, int T>
__global__ void __launch_bounds__(T, kAnyResident / T) k_rms_backward_any(const __grid_constant__ RmsArgs a)
{
    in_turn();
    constexpr int E = DT == kF32 ? 4 : 2, kGroups = T / (32 * W);
    __shared__ float sh[2 * (T / 32) * RB];
    __shared__ float join[kGroups > 1 ? T * K : 1];   // [warp][K][32]
    const int lane = threadIdx.x & 31, group = (int)(threadIdx.x >> 5) / W, warp = (int)(threadIdx.x >> 5) % W;
    const int j0 = warp * 128 + lane, left = (int)a.dim - j0;
    const float inv = 1.0f / (float)a.dim;
    int turn = 0;
    constexpr bool kHeld = K <= 8;                    // else the weight is read for each row, and dh where it is added
    float dw[K], w[kHeld ? K : 1];
#pragma unroll
    for (int k = 0; k < K; k++) {
        dw[k] = 0.0f;
        if (kHeld) w[k] = 1.0f;
    }
    const char* weight = static_cast<const char*>(a.weight) + j0 * E;
    if constexpr (kHeld)
        if (a.weight) ld_places<DT, K, W>(weight, left, w);
    const int64_t x_row = a.x_stride * E, y_row = a.y_stride * E, stride = (int64_t)gridDim.x * kGroups * RB;
    for (int64_t r0 = ((int64_t)blockIdx.x * kGroups + group) * RB; r0 < a.rows; r0 += stride) {
        const int64_t x_at = r0 * x_row + j0 * E, y_at = r0 * y_row + j0 * E;
        float n[RB][K], g[RB][K], r[kHeld ? RB : 1][kHeld ? K : 1], rstd[RB], c[RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {                // rows past the end: none of their places is there
            const bool there = RB == 1 || r0 + b < a.rows;
            const int here = there ? left : 0;
            ld_places<DT, K, W>(static_cast<const char*>(a.x) + x_at + b * x_row, here, n[b]);
            ld_places<DT, K, W>(static_cast<const char*>(a.dy) + y_at + b * y_row, here, g[b]);
            if constexpr (kHeld)
                if (a.r) ld_places<DT, K, W>(static_cast<const char*>(a.r) + x_at + b * x_row, here, r[b]);
            rstd[b] = there ? a.rstd_in[r0 + b] : 0.0f;
        }
#pragma unroll
        for (int b = 0; b < RB; b++) {
            c[b] = 0.0f;
#pragma unroll
            for (int k = 0; k < K; k++) {
                n[b][k] *= rstd[b];                   // xhat; 0 past the end
                dw[k] = fmaf(g[b][k], n[b][k], dw[k]);
                if constexpr (kHeld) g[b][k] *= w[k];
                else if (a.weight && place<W>(k) < left) g[b][k] *= ld1<DT>(weight, place<W>(k));
                c[b] = fmaf(g[b][k], n[b][k], c[b]);
            }
        }
        if (!a.dx) continue;
        group_sum<32, RB, T>(c, W, sh, turn, [&](float t) { return t * -inv; });
#pragma unroll
        for (int b = 0; b < RB; b++) {
#pragma unroll
            for (int k = 0; k < K; k++) {
                g[b][k] = fmaf(n[b][k], c[b], g[b][k]);
                if constexpr (kHeld) {
                    g[b][k] = a.r ? fmaf(g[b][k], rstd[b], r[b][k]) : g[b][k] * rstd[b];
                } else {
                    const float d = a.r && place<W>(k) < left ? ld1<DT>(static_cast<const char*>(a.r) + x_at, place<W>(k)) : 0.0f;
                    g[b][k] = a.r ? fmaf(g[b][k], rstd[b], d) : g[b][k] * rstd[b];
                }
            }
            st_places<DT, K, W>(static_cast<char*>(a.dx) + x_at + b * x_row, RB == 1 || r0 + b < a.rows ? left : 0, g[b]);
        }
    }
    if (!a.part) return;
    float* pw = a.part + (int64_t)blockIdx.x * a.dim;
    if constexpr (kGroups > 1) {
#pragma unroll
        for (int k = 0; k < K; k++)
            join[((threadIdx.x >> 5) * K + k) * 32 + lane] = dw[k];
        __syncthreads();
        for (int t = threadIdx.x; t < W * K * 32; t += T) {
            const int of = t / (K * 32), k = t / 32 % K, j = of * 128 + place<W>(k) + t % 32;
            float s = 0.0f;
            for (int g = 0; g < kGroups; g++)
                s += join[((g * W + of) * K + k) * 32 + t % 32];
            if (j < a.dim) pw[j] = s;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; k++)
            if (place<W>(k) < left) pw[j0 + place<W>(k)] = dw[k];
    }
}

// ---- long rows -------------------------------------------------------------------------
// More than a block's registers hold (over 4096 vectors, or 16384 values off their
// boundaries; backward over 16384 values): a block per row, values read again for every
// use (from cache), bound by the latency of one access a value: 512 x 40000 bfloat16
// 53 us forward, backward 114, 42 of them for the weight (with one value of a thread
// on its way at a time 70 and 162).  Warps take blocks of 128 values in turn, K / 4
// of them before any use, so a thread reads of h what it wrote.  K = 8 for few rows
// (200 x 200000 132 us forward, 205 with 4), 4 for many (8192 x 16385 261 and
// backward 562, 297 and 687 with 8).
constexpr int kLongThreads = 512;
constexpr int64_t kLongRows = 2 * kSms;               // up to so many rows: half as many blocks an SM, twice the loads of a thread on their way

__device__ __forceinline__ float long_sum(float v, float* sh)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int k = 0; k < kLongThreads / 32; k++)
        t += sh[k];
    return t;
}

template <int DT, int K>
__global__ void __launch_bounds__(kLongThreads, 16 / K) k_rms_forward_long(const __grid_constant__ RmsArgs a)
{
    in_turn();
    constexpr int E = DT == kF32 ? 4 : 2, W = kLongThreads / 32;
    __shared__ float sh[W];
    const int lane = threadIdx.x & 31, j0 = (int)(threadIdx.x >> 5) * 128 + lane;
    const float inv = 1.0f / (float)a.dim;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t xo = r * a.x_stride, yo = r * a.y_stride;
        const char* x = static_cast<const char*>(a.x) + xo * E;
        const char* res = static_cast<const char*>(a.r) + xo * E;
        char* h = static_cast<char*>(a.h) + xo * E;
        float ss = 0.0f;
        for (int j = j0; j < a.dim; j += K * kLongThreads) {
            const int left = (int)a.dim - j;
            float f[K], g[K];
            ld_places<DT, K, W>(x + j * E, left, f);
            if (a.r) {
                ld_places<DT, K, W>(res + j * E, left, g);
#pragma unroll
                for (int k = 0; k < K; k++)
                    f[k] = to_f32<DT>(from_f32<DT>(f[k] + g[k]));
            }
            if (a.h) st_places<DT, K, W>(h + j * E, left, f);
#pragma unroll
            for (int k = 0; k < K; k++)
                ss = fmaf(f[k], f[k], ss);
        }
        const float rstd = inverse_root(fmaf(long_sum(ss, sh), inv, a.eps));
        if (a.h) x = h;
        for (int j = j0; j - lane < a.dim; j += K * kLongThreads) {            // whole warps: codes_out's maxima
            const int left = (int)a.dim - j;
            float f[K], w[K];
            ld_places<DT, K, W>(x + j * E, left, f);
            if (a.weight) ld_places<DT, K, W>(static_cast<const char*>(a.weight) + j * E, left, w);
#pragma unroll
            for (int k = 0; k < K; k++)
                f[k] = f[k] * rstd * (a.weight ? w[k] : 1.0f);
            if (a.y) st_places<DT, K, W>(static_cast<char*>(a.y) + (yo + j) * E, left, f);
            if (!a.q) continue;
            uint8_t* q = a.q + yo + j;
            uint8_t* q_scale = a.q_scale + r * a.scale_cols;
#pragma unroll
            for (int k = 0; k < K; k += 4) {
                const int at = j - lane + place<W>(k);
                if (at >= a.dim) break;
                if (a.block == 128) codes_out<128>(q + place<W>(k), q_scale + at / 128, left - place<W>(k), lane, f + k);
                else codes_out<32>(q + place<W>(k), q_scale + at / 32, left - place<W>(k), lane, f + k);
            }
        }
        if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
    }
}

template <int DT, int K>
__global__ void __launch_bounds__(kLongThreads, 16 / K) k_rms_dx_long(const __grid_constant__ RmsArgs a)
{
    in_turn();
    constexpr int E = DT == kF32 ? 4 : 2, W = kLongThreads / 32;
    __shared__ float sh[W];
    const int j0 = (int)(threadIdx.x >> 5) * 128 + (threadIdx.x & 31);
    const float inv = 1.0f / (float)a.dim;
    const char* weight = static_cast<const char*>(a.weight);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t xo = r * a.x_stride;
        const char* x = static_cast<const char*>(a.x) + xo * E;
        const char* res = static_cast<const char*>(a.r) + xo * E;
        const char* dy = static_cast<const char*>(a.dy) + r * a.y_stride * E;
        const float rstd = a.rstd_in[r];
        float n[K], g[K], w[K];
        auto load = [&](int j) {                      // xhat and dy weight
            const int left = (int)a.dim - j;
            ld_places<DT, K, W>(x + j * E, left, n);
            ld_places<DT, K, W>(dy + j * E, left, g);
            if (weight) ld_places<DT, K, W>(weight + j * E, left, w);
#pragma unroll
            for (int k = 0; k < K; k++) {
                n[k] *= rstd;
                if (weight) g[k] *= w[k];
            }
        };
        float s = 0.0f;
        for (int j = j0; j < a.dim; j += K * kLongThreads) {
            load(j);
#pragma unroll
            for (int k = 0; k < K; k++)
                s = fmaf(g[k], n[k], s);
        }
        const float c = long_sum(s, sh) * -inv;
        for (int j = j0; j < a.dim; j += K * kLongThreads) {
            const int left = (int)a.dim - j;
            float d[K];
            if (a.r) ld_places<DT, K, W>(res + j * E, left, d);
            load(j);
#pragma unroll
            for (int k = 0; k < K; k++) {
                g[k] = fmaf(n[k], c, g[k]) * rstd;
                if (a.r) g[k] += d[k];
            }
            st_places<DT, K, W>(static_cast<char*>(a.dx) + (xo + j) * E, left, g);
        }
    }
}

// Column sums over the row group blockIdx.y: one thread a column.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) k_rms_dw_part(const __grid_constant__ RmsArgs a)
{
    in_turn();
    const int64_t j = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
    if (j >= a.dim) return;
    const int64_t G = gridDim.y, per = (a.rows + G - 1) / G;
    const int64_t lo = min(blockIdx.y * per, a.rows), hi = min(lo + per, a.rows);
    constexpr int U = 8;
    float dw = 0.0f;
    for (int64_t r0 = lo; r0 < hi; r0 += U) {
        float g[U], n[U];
#pragma unroll
        for (int u = 0; u < U; u++) {                 // past the end: 0
            const int64_t r = r0 + u;
            g[u] = r < hi ? ld1<DT>(a.dy, r * a.y_stride + j) : 0.0f;
            n[u] = r < hi ? ld1<DT>(a.x, r * a.x_stride + j) * a.rstd_in[r] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; u++)
            dw = fmaf(g[u], n[u], dw);
    }
    a.part[(int64_t)blockIdx.y * a.dim + j] = dw;
}

// The blocks' partial sums: 32 columns a block, its 32 warps a part of the
// partial sums each, joined in warp order.  Bound by its own latency, 4.4 us of the
// 68.2 above.
template <int DT>
__global__ void __launch_bounds__(1024) k_rms_dw_sum(const float* part, int blocks, int64_t dim, void* dw)
{
    in_turn();
    __shared__ float sh[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (j < dim)
#pragma unroll 10
        for (int k = warp; k < blocks; k += 32)
            s += part[(int64_t)k * dim + j];
    sh[warp][lane] = s;
    __syncthreads();
    if (warp > 0 || j >= dim) return;
    for (int k = 1; k < 32; k++)
        s += sh[k][lane];
    st1<DT>(dw, j, s);
}

// ---- read-out --------------------------------------------------------------------------
// 8-bit results as bfloat16 values.  Rows that start and end on 16 codes: 16 to a
// thread at once; blockDim.x threads along a row, blockDim.y rows, and each thread
// kValuesRows of them, all read before any is written.  8192 x 4096: 19.4 us, 5.2
// TB/s, a third of the issue slots used; more warps an SM with fewer loads each on
// their way were slower (24.9 with 48 of them).  Other rows 44 us.
constexpr int kValuesRows = 4;

// Other rows: a warp 256 values of one, a code a lane at a time.
__global__ void __launch_bounds__(256) k_rms_values_any(const __grid_constant__ RmsArgs a, uint16_t* out, int64_t per)
{
    in_turn();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * 8, all = a.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < all; i += warps) {
        const int64_t row = i / per;
        const int j0 = (int)(i - row * per) * 256, left = (int)a.dim - j0 - lane;
        const uint8_t* src = a.q + row * a.y_stride + j0 + lane;
        const uint8_t* scale = a.q_scale + row * a.scale_cols + (a.block == 32 ? j0 >> 5 : j0 >> 7);
        uint16_t* dst = out + row * a.y_stride + j0 + lane;
        uint32_t c[8], e[8];
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (32 * k < left) {
                c[k] = src[32 * k];
                e[k] = scale[a.block == 32 ? k : k >> 2];
            }
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (32 * k < left) {
                uint32_t rest;
                __nv_bfloat162 up = scale_of(e[k], rest);
                uint32_t v = values2(c[k] << 8, up);
                if (rest) v = scaled_more(v, rest);
                dst[32 * k] = (uint16_t)v;
            }
    }
}

__global__ void __launch_bounds__(256) k_rms_values(const __grid_constant__ RmsArgs a, uint16_t* out)
{
    in_turn();
    const int j = (int)(blockIdx.x * blockDim.x + threadIdx.x) * 16;
    if (j >= a.dim) return;
    const int64_t step = blockDim.y, apart = step * a.y_stride, scales_apart = step * a.scale_cols;
    for (int64_t r0 = (int64_t)blockIdx.y * step * kValuesRows + threadIdx.y; r0 < a.rows; r0 += gridDim.y * step * kValuesRows) {
        const int rows = (int)min((int64_t)kValuesRows, (a.rows - r0 + step - 1) / step);
        const uint8_t* src = a.q + r0 * a.y_stride + j;
        const uint8_t* scale = a.q_scale + r0 * a.scale_cols + (j >> (a.block == 32 ? 5 : 7));
        uint16_t* dst = out + r0 * a.y_stride + j;
        uint4 c[kValuesRows];
        uint32_t e[kValuesRows];
#pragma unroll
        for (int b = 0; b < kValuesRows; b++) {
            if (b < rows) {
                e[b] = *scale;
                c[b] = __ldcs(reinterpret_cast<const uint4*>(src));
            }
            scale += scales_apart;
            src += apart;
        }
#pragma unroll
        for (int b = 0; b < kValuesRows; b++) {
            if (b >= rows) break;
            uint32_t rest;
            const __nv_bfloat162 up = scale_of(e[b], rest);
            const uint32_t q[4] = {c[b].x, c[b].y, c[b].z, c[b].w};
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; k++)
                w[k] = values2(__byte_perm(q[k >> 1], 0, k & 1 ? 0x3424 : 0x1404), up);
            if (rest)
#pragma unroll
                for (int k = 0; k < 8; k++)
                    w[k] = scaled_more(w[k], rest);
            __stcs(reinterpret_cast<uint4*>(dst), make_uint4(w[0], w[1], w[2], w[3]));
            __stcs(reinterpret_cast<uint4*>(dst) + 1, make_uint4(w[4], w[5], w[6], w[7]));
            dst += apart;
        }
    }
}

// ---- host ---------------------------------------------------------------------------------
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

zero_status_t cuda_failed(cudaError_t e, const char* what)
{
    char msg[200];
    std::snprintf(msg, sizeof msg, "%s: launch failed: %s", what, cudaGetErrorString(e));
    return set_error(ZERO_ECUDA, msg);
}

zero_status_t check_rms_plan(const zero_rms_plan_t* p)
{
    if (!p) return set_error(ZERO_EINVAL, "root-mean-square norm plan is NULL");
    zero_rms_plan_t fresh;
    const zero_status_t st = zero_rms_plan(p->rows, p->dim, p->dtype, p->x_stride, p->y_stride, p->block, &fresh);
    if (st != ZERO_OK) return st;
    if (std::memcmp(&fresh, p, sizeof fresh) != 0)
        return set_error(ZERO_EINVAL, "root-mean-square norm plan was not made by zero_rms_plan");
    return ZERO_OK;
}

// Rows of a batch: RB where there are enough to keep `most` resident blocks busy,
// else fewer, so that few rows spread over the SMs.
int rows_of_batch(int64_t rows, int64_t groups, int64_t most, int RB)
{
    const int64_t each = (rows + groups * most - 1) / (groups * most);
    return (int)(each < 1 ? 1 : each < RB ? each : RB);
}

int64_t blocks_for(int64_t rows, int64_t at_once, int64_t most)
{
    const int64_t need = (rows + at_once - 1) / at_once;
    return need < most ? need : most;
}

cudaError_t launch_rms(void (*kernel)(const RmsArgs), const RmsArgs& a, int64_t blocks, int threads, size_t smem,
                       cudaStream_t s)
{
    return launch_after(kernel, dim3((unsigned)blocks), threads, smem, s, a);
}

// A row kernel; SMEM bytes of slots.
template <void (*KERNEL)(const RmsArgs), size_t SMEM>
cudaError_t launch_slots(const RmsArgs& a, int64_t blocks, int threads, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem((const void*)KERNEL, (int)SMEM, done);
    return e == cudaSuccess ? launch_rms(KERNEL, a, blocks, threads, SMEM, s) : e;
}

template <int DT, int L, int V, int RB, int S, int T, int BLOCKS, int Q>
cudaError_t forward_shape(RmsArgs a, int64_t vecs, cudaStream_t s)
{
    const RowShape h = shape_of(vecs, L, V, T);
    a.warps = h.warps;
    const int64_t most = (int64_t)kSms * (BLOCKS * T / h.threads);            // resident at once
    a.take = rows_of_batch(a.rows, h.groups, most, RB);
    const int64_t blocks = blocks_for(a.rows, (int64_t)h.groups * a.take, most);
    constexpr size_t smem = (size_t)S * RB * V * 2 * T * 16;
    if constexpr (L == 32) {                          // fewer lanes: whole rows on 16-byte boundaries only
        if (a.dim % kVecOf<DT>)
            return launch_slots<k_rms_forward_rows<DT, L, V, RB, S, T, BLOCKS, true, Q>, smem>(a, blocks, h.threads, s);
    }
    return launch_slots<k_rms_forward_rows<DT, L, V, RB, S, T, BLOCKS, false, Q>, smem>(a, blocks, h.threads, s);
}

// The same shape with 8-bit results and without.
template <int DT, int L, int V, int RB, int S, int T, int BLOCKS>
cudaError_t forward_rows(const RmsArgs& a, int64_t vecs, cudaStream_t s)
{
    return !a.q ? forward_shape<DT, L, V, RB, S, T, BLOCKS, 0>(a, vecs, s)
           : a.block == 32 ? forward_shape<DT, L, V, RB, S, T, BLOCKS, 32>(a, vecs, s)
                           : forward_shape<DT, L, V, RB, S, T, BLOCKS, 128>(a, vecs, s);
}

template <int DT, int K, int W, int RB, int T>
cudaError_t forward_any(RmsArgs a, cudaStream_t s)
{
    constexpr int64_t groups = T / (32 * W), most = (int64_t)kSms * ((K > 16 ? 512 : 1024) / T);
    a.take = rows_of_batch(a.rows, groups, most, RB);
    return launch_rms(k_rms_forward_any<DT, K, W, RB, T>, a, blocks_for(a.rows, groups * a.take, most), T, 0, s);
}

// aligned: every row starts on 16 bytes.
template <int DT>
cudaError_t forward(const RmsArgs& a, bool aligned, cudaStream_t s)
{
    constexpr int VE = kVecOf<DT>, T = kRowThreads;
    const int64_t vecs = (a.dim + VE - 1) / VE;
    const bool whole = a.dim % VE == 0 && aligned;
    if (whole && vecs <= 8) return forward_rows<DT, 8, 1, 4, 2, T, 2>(a, vecs, s);
    if (whole && vecs <= 16) return forward_rows<DT, 16, 1, 4, 2, T, 2>(a, vecs, s);
    if (aligned) {
        if (vecs <= 256) return forward_rows<DT, 32, 1, 4, 2, T, 2>(a, vecs, s);
        // 8192 x 4096 bfloat16: 47.7 us as two vectors a lane, 49.2 as one; into 8 bits 44.1 and 41.5
        if (vecs <= 512 && !a.q) return forward_shape<DT, 32, 2, 2, 2, T, 2, 0>(a, vecs, s);
        if (vecs <= 512)
            return a.block == 32 ? forward_shape<DT, 32, 1, 4, 2, 2 * T, 1, 32>(a, vecs, s)
                                 : forward_shape<DT, 32, 1, 4, 2, 2 * T, 1, 128>(a, vecs, s);
        if (vecs <= 1024) return forward_rows<DT, 32, 2, 2, 2, 2 * T, 1>(a, vecs, s);
        if (vecs <= 2048) return forward_rows<DT, 32, 4, 1, 2, 2 * T, 1>(a, vecs, s);
        if (vecs <= 4096) return forward_rows<DT, 32, 8, 1, 1, 2 * T, 1>(a, vecs, s);
    } else {
        if (a.dim <= 128) return forward_any<DT, 4, 1, 4, T>(a, s);
        if (a.dim <= 256) return forward_any<DT, 8, 1, 2, T>(a, s);
        if (a.dim <= 512) return forward_any<DT, 8, 2, 2, T>(a, s);
        if (a.dim <= 1024) return forward_any<DT, 8, 4, 2, T>(a, s);
        if (a.dim <= 2048) return forward_any<DT, 8, 8, 2, T>(a, s);
        if (a.dim <= 4096) return forward_any<DT, 8, 16, 2, 2 * T>(a, s);
        if (a.dim <= 8192) return forward_any<DT, 16, 16, 1, 2 * T>(a, s);
        if (a.dim <= 16384) return forward_any<DT, 32, 16, 1, 2 * T>(a, s);
    }
    if (a.rows <= kLongRows) return launch_rms(k_rms_forward_long<DT, 8>, a, a.rows, kLongThreads, 0, s);
    return launch_rms(k_rms_forward_long<DT, 4>, a, std::min<int64_t>(a.rows, kSms * 4), kLongThreads, 0, s);
}

// How the backward pass deals out a row: lanes of a group, vectors of a lane,
// threads and resident blocks, rows at a time.
struct BackwardShape {
    int L, V, T, blocks, rows;
};

BackwardShape backward_shape(int64_t vecs, bool whole)
{
    const int L = whole && vecs <= 8 ? 8 : whole && vecs <= 16 ? 16 : 32;
    if (vecs <= 256) return {L, 1, kRowThreads, 2, 4};
    if (vecs <= 512) return {L, 1, 2 * kRowThreads, 1, 4};
    if (vecs <= 1024) return {L, 2, 2 * kRowThreads, 1, 2};
    return {L, 4, 2 * kRowThreads, 1, 1};
}

int64_t backward_most(const BackwardShape& b, const RowShape& h) { return (int64_t)kSms * (b.blocks * b.T / h.threads); }

template <int DT, int L, int V, int RB, int T, int BLOCKS>
cudaError_t backward_rows(RmsArgs a, int64_t vecs, int64_t blocks, cudaStream_t s)
{
    const RowShape h = shape_of(vecs, L, V, T);
    a.warps = h.warps;
    a.take = rows_of_batch(a.rows, h.groups, backward_most({L, V, T, BLOCKS, RB}, h), RB);
    constexpr int S = 2;
    constexpr size_t smem = (size_t)S * RB * V * 3 * T * 16;
    if constexpr (L == 32) {
        if (a.dim % kVecOf<DT>)
            return launch_slots<k_rms_backward_rows<DT, L, V, RB, S, T, BLOCKS, true>, smem>(a, blocks, h.threads, s);
    }
    return launch_slots<k_rms_backward_rows<DT, L, V, RB, S, T, BLOCKS, false>, smem>(a, blocks, h.threads, s);
}

// Its blocks: as many as are resident at once on 152 SMs, and no more than have rows.
int64_t backward_blocks(int64_t rows, int64_t vecs, int L)
{
    BackwardShape b = backward_shape(vecs, false);
    const RowShape h = shape_of(vecs <= 2048 ? vecs : 2048, b.L = L, b.V, b.T);
    const int64_t most = backward_most(b, h);
    return blocks_for(rows, (int64_t)h.groups * rows_of_batch(rows, h.groups, most, b.rows), most);
}

// Warps to a row in the kernel for other rows, of 8 values a lane, 16 above 8192; threads of
// its blocks, and the blocks: as many as are resident, and no more than have rows.
// (Two rows of a group at a time, with half of the warps: 8192 x 4095 123 us for 86;
// short rows are two at a time, 65536 x 67 24 us for 32.  2048 x 16383 98 us, as a
// long row's kernels 191.  Binary32 rows of 8193 to 16384 values on 16-byte
// boundaries: 2048 x 8196 70, 12288 85 and 16384 109 us, as a long row's kernels 97,
// 133 and 187, 64 x 12288 10 and 13.  The long rows' is ahead only where dx alone is
// asked for of many rows below some 10000 values, 8192 x 8196 203 us for 246; that the
// two calls' dx have the same bits counts more.)
constexpr int64_t kAnyBackward = 16384;
constexpr int64_t any_warps(int64_t dim) { return dim <= 256 ? 1 : dim <= 512 ? 2 : dim <= 1024 ? 4 : dim <= 2048 ? 8 : dim <= 4096 ? 16 : 32; }
constexpr int64_t any_threads(int64_t W) { return W <= 8 ? 256 : 32 * W; }

int64_t any_blocks(int64_t rows, int64_t dim)
{
    const int64_t W = any_warps(dim), T = any_threads(W);
    return blocks_for(rows, T / (32 * W) * (dim <= 128 ? 2 : 1), kSms * (kAnyResident / T));
}

template <int DT, int K, int W, int RB = 1>
cudaError_t backward_any(const RmsArgs& a, int64_t& blocks, cudaStream_t s)
{
    constexpr int T = (int)any_threads(W);
    blocks = any_blocks(a.rows, a.dim);
    return launch_rms(k_rms_backward_any<DT, K, W, RB, T>, a, blocks, T, 0, s);
}

// Row groups of a long row's column sums: what fills the SMs once, or groups of 256
// rows (as many as the plan allows, of three rows each: 512 x 40000 74 us for 43).
int64_t dw_groups(int64_t rows, int64_t cols)
{
    const int64_t fill = kSms * (2048 / kRowThreads) / cols, most = (rows + 255) / 256;
    return std::min(rows, std::max<int64_t>(1, std::max(fill, most)));
}

template <int DT>
cudaError_t backward(RmsArgs a, bool aligned, int64_t most, void* dw, cudaStream_t s)
{
    constexpr int VE = kVecOf<DT>, T = kRowThreads;
    const int64_t vecs = (a.dim + VE - 1) / VE;
    if (!dw) a.part = nullptr;
    cudaError_t e = cudaSuccess;
    int64_t blocks = most;                            // partial sums of the weight's gradient
    if (a.rows && vecs <= 2048 && aligned) {
        const int L = backward_shape(vecs, a.dim % VE == 0).L;
        blocks = backward_blocks(a.rows, vecs, L);
        if (L == 8) e = backward_rows<DT, 8, 1, 4, T, 2>(a, vecs, blocks, s);
        else if (L == 16) e = backward_rows<DT, 16, 1, 4, T, 2>(a, vecs, blocks, s);
        else if (vecs <= 256) e = backward_rows<DT, 32, 1, 4, T, 2>(a, vecs, blocks, s);
        else if (vecs <= 512) e = backward_rows<DT, 32, 1, 4, 2 * T, 1>(a, vecs, blocks, s);
        else if (vecs <= 1024) e = backward_rows<DT, 32, 2, 2, 2 * T, 1>(a, vecs, blocks, s);
        else e = backward_rows<DT, 32, 4, 1, 2 * T, 1>(a, vecs, blocks, s);
    } else if (a.rows && a.dim <= kAnyBackward) {     // binary32 on 16-byte boundaries above 8192 values too
        if (a.dim <= 128) e = backward_any<DT, 4, 1, 2>(a, blocks, s);
        else if (a.dim <= 256) e = backward_any<DT, 8, 1>(a, blocks, s);
        else if (a.dim <= 512) e = backward_any<DT, 8, 2>(a, blocks, s);
        else if (a.dim <= 1024) e = backward_any<DT, 8, 4>(a, blocks, s);
        else if (a.dim <= 2048) e = backward_any<DT, 8, 8>(a, blocks, s);
        else if (a.dim <= 4096) e = backward_any<DT, 8, 16>(a, blocks, s);
        else if (a.dim <= 8192) e = backward_any<DT, 8, 32>(a, blocks, s);
        else e = backward_any<DT, 16, 32>(a, blocks, s);
    } else {
        if (a.dx && a.rows)
            e = a.rows <= kLongRows ? launch_rms(k_rms_dx_long<DT, 8>, a, a.rows, kLongThreads, 0, s)
                                    : launch_rms(k_rms_dx_long<DT, 4>, a, std::min<int64_t>(a.rows, kSms * 4), kLongThreads, 0, s);
        if (e == cudaSuccess && dw && blocks) {
            const int64_t cols = (a.dim + kRowThreads - 1) / kRowThreads;
            blocks = std::min(most, dw_groups(a.rows, cols));
            e = launch_after(k_rms_dw_part<DT>, dim3((unsigned)cols, (unsigned)blocks), kRowThreads, 0, s, a);
        }
    }
    if (e == cudaSuccess && dw)
        e = launch_after(k_rms_dw_sum<DT>, dim3((unsigned)((a.dim + 31) / 32)), 1024, 0, s, a.part, (int)blocks, a.dim, dw);
    return e;
}

// Whether every row of the given arrays, and the weight, starts on 16 bytes.
bool rows_aligned(const zero_rms_plan_t& p, const void* weight, const void* const* arrays, int n)
{
    const uint64_t e = p.dtype == ZERO_FP32 ? 4 : 2;
    uint64_t any = (uint64_t)p.x_stride * e | (uint64_t)p.y_stride * e;
    for (int k = 0; k < n; k++)
        any |= (uintptr_t)arrays[k];
    return (any | (uintptr_t)weight) % 16 == 0;
}

RmsArgs args_of(const zero_rms_plan_t& p)
{
    RmsArgs a;
    std::memset(&a, 0, sizeof a);
    a.rows = p.rows; a.dim = p.dim; a.x_stride = p.x_stride; a.y_stride = p.y_stride;
    a.block = p.block; a.scale_cols = p.scale_cols;
    return a;
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

zero_status_t zero_rms_plan(int64_t rows, int64_t dim, int32_t dtype, int64_t x_stride, int64_t y_stride, int32_t block,
                            zero_rms_plan_t* out)
{
    if (!out) return set_error(ZERO_EINVAL, "zero_rms_plan: out is NULL");
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16 && dtype != ZERO_FP32)
        return set_error(ZERO_EINVAL, "zero_rms_plan: dtype unknown");
    if (rows < 0 || dim < 1) return set_error(ZERO_EINVAL, "zero_rms_plan: rows must be >= 0 and dim >= 1");
    if (block != 0 && block != 32 && block != 128)
        return set_error(ZERO_EUNSUPPORTED, "zero_rms_plan: block must be 0, 32 or 128");
    if (rows > (int64_t(1) << 40) || dim > (int64_t(1) << 20))
        return set_error(ZERO_EUNSUPPORTED, "zero_rms_plan: rows exceed 2^40 or dim exceeds 2^20");
    const int64_t xs = x_stride ? x_stride : dim, ys = y_stride ? y_stride : dim;
    if (xs < dim || ys < dim || xs > (int64_t(1) << 40) || ys > (int64_t(1) << 40))
        return set_error(ZERO_EINVAL, "zero_rms_plan: a stride is below dim or above 2^40");
    if (rows && (xs > INT64_MAX / 32 / rows || ys > INT64_MAX / 32 / rows))   // 5 * 4 bytes of each below INT64_MAX
        return set_error(ZERO_EUNSUPPORTED, "zero_rms_plan: the rows span too many bytes");
    std::memset(out, 0, sizeof *out);
    out->rows = rows;
    out->dim = dim;
    out->x_stride = xs;
    out->y_stride = ys;
    out->dtype = dtype;
    out->block = block;
    out->scale_cols = block ? (dim + block - 1) / block : 0;
    const int64_t e = dtype == ZERO_FP32 ? 4 : 2;
    // each adds up its rows' weight gradients; the most of any alignment of the pointers
    const int64_t vecs = (dim * e + 15) / 16;
    const int64_t by_vec = backward_blocks(rows, vecs, 32), by_some = backward_blocks(rows, vecs, backward_shape(vecs, dim * e % 16 == 0).L);
    const int64_t by_one = dim <= kAnyBackward ? any_blocks(rows, dim) : 0, more = by_vec > by_some ? by_vec : by_some;
    out->blocks = (int32_t)(more > by_one ? more : by_one);
    out->workspace_bytes = 16 + (int64_t)out->blocks * dim * 4;
    out->hbm_bytes_forward = rows * (3 * dim * e + 4 + (block ? dim + out->scale_cols : dim * e)) + dim * e;
    out->hbm_bytes_backward = rows * (4 * dim * e + 4) + 2 * dim * e;
    return ZERO_OK;
}

zero_status_t zero_rms_forward(const zero_rms_plan_t* plan, const void* x, const void* residual, const void* weight,
                               float eps, void* h, void* y, void* q, uint8_t* q_scale, float* rstd, void* stream)
{
    NvtxRange range("zero_rms_forward");
    const zero_status_t st = check_rms_plan(plan);
    if (st != ZERO_OK) return st;
    if (!(eps >= 0.0f)) return set_error(ZERO_EINVAL, "zero_rms_forward: eps must be >= 0");
    if (q && !plan->block) return set_error(ZERO_EINVAL, "zero_rms_forward: the plan has no block for 8-bit results");
    if (h && !residual) return set_error(ZERO_EINVAL, "zero_rms_forward: h without a residual");
    if (plan->rows == 0) return ZERO_OK;
    if (!x || (!y && !q) || (residual && !h) || (q && !q_scale))
        return set_error(ZERO_ENOMEM, "zero_rms_forward: x, both of y and q, h of a residual or q_scale of q is NULL");
    const size_t e = plan->dtype == ZERO_FP32 ? 4 : 2;
    if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(weight, e) || !aligned_to(h, e) ||
        !aligned_to(y, e) || !aligned_to(rstd, 4))
        return set_error(ZERO_EALIGN, "zero_rms_forward: a pointer is not aligned to its type");
    RmsArgs a = args_of(*plan);
    a.x = x; a.r = residual; a.weight = weight; a.h = h; a.y = y; a.rstd = rstd; a.eps = eps;
    a.q = static_cast<uint8_t*>(q);
    a.q_scale = q_scale;
    a.q_wide = aligned_to(q, 8) && plan->y_stride % 8 == 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const void* arrays[] = {x, residual, h, y};
    const bool aligned = rows_aligned(*plan, weight, arrays, 4);
    const cudaError_t err = plan->dtype == ZERO_FP32   ? forward<kF32>(a, aligned, s)
                            : plan->dtype == ZERO_BF16 ? forward<kBF16>(a, aligned, s)
                                                       : forward<kF16>(a, aligned, s);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_rms_forward");
}

zero_status_t zero_rms_values(const zero_rms_plan_t* plan, const void* q, const uint8_t* q_scale, void* values, void* stream)
{
    NvtxRange range("zero_rms_values");
    const zero_status_t st = check_rms_plan(plan);
    if (st != ZERO_OK) return st;
    if (!plan->block) return set_error(ZERO_EINVAL, "zero_rms_values: the plan has no block for 8-bit results");
    if (plan->rows == 0) return ZERO_OK;
    if (!q || !q_scale || !values) return set_error(ZERO_ENOMEM, "zero_rms_values: a buffer is NULL");
    if (!aligned_to(values, 2)) return set_error(ZERO_EALIGN, "zero_rms_values: values is not aligned to its type");
    RmsArgs a = args_of(*plan);
    a.q = static_cast<uint8_t*>(const_cast<void*>(q));
    a.q_scale = const_cast<uint8_t*>(q_scale);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err;
    const bool wide = aligned_to(q, 16) && aligned_to(values, 16) && plan->y_stride % 16 == 0 && plan->dim % 16 == 0;
    if (wide) {
        unsigned along = 1;                           // short rows share a warp
        while (along < 256 && along < plan->dim / 16) along *= 2;
        const int64_t high = (plan->rows + 256 / along * kValuesRows - 1) / (256 / along * kValuesRows);
        const dim3 block(along, 256 / along);
        const dim3 grid((unsigned)((plan->dim / 16 + along - 1) / along), (unsigned)(high < 65535 ? high : 65535));
        err = launch_after(k_rms_values, grid, block, 0, s, a, static_cast<uint16_t*>(values));
    } else {
        const int64_t per = (plan->dim + 255) / 256;
        err = launch_after(k_rms_values_any, dim3((unsigned)blocks_for(plan->rows * per, 8, kSms * 32)), 256, 0, s, a,
                          static_cast<uint16_t*>(values), per);
    }
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_rms_values");
}

zero_status_t zero_rms_backward(const zero_rms_plan_t* plan, const void* dy, const void* dh, const void* h,
                                const void* weight, const float* rstd, void* dx, void* dweight, void* workspace,
                                void* stream)
{
    NvtxRange range("zero_rms_backward");
    const zero_status_t st = check_rms_plan(plan);
    if (st != ZERO_OK) return st;
    if (plan->rows && (!dy || !h || !rstd)) return set_error(ZERO_ENOMEM, "zero_rms_backward: dy, h or rstd is NULL");
    if (dweight && !workspace) return set_error(ZERO_ENOMEM, "zero_rms_backward: workspace is NULL");
    const size_t e = plan->dtype == ZERO_FP32 ? 4 : 2;
    if (!aligned_to(dy, e) || !aligned_to(dh, e) || !aligned_to(h, e) || !aligned_to(weight, e) || !aligned_to(dx, e) ||
        !aligned_to(dweight, e) || !aligned_to(rstd, 4))
        return set_error(ZERO_EALIGN, "zero_rms_backward: a pointer is not aligned to its type");
    if (!aligned_to(workspace, 16)) return set_error(ZERO_EALIGN, "zero_rms_backward: workspace is not 16-byte aligned");
    if (!dx && !dweight) return ZERO_OK;
    RmsArgs a = args_of(*plan);
    a.x = h; a.r = dx ? dh : nullptr; a.dy = dy; a.weight = weight; a.rstd_in = rstd; a.dx = dx;
    a.part = static_cast<float*>(workspace) + 4;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const void* arrays[] = {dy, a.r, h, dx};
    const bool aligned = rows_aligned(*plan, weight, arrays, 4);
    const cudaError_t err = plan->dtype == ZERO_FP32   ? backward<kF32>(a, aligned, plan->blocks, dweight, s)
                            : plan->dtype == ZERO_BF16 ? backward<kBF16>(a, aligned, plan->blocks, dweight, s)
                                                       : backward<kF16>(a, aligned, plan->blocks, dweight, s);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_rms_backward");
}

}  // extern "C"
