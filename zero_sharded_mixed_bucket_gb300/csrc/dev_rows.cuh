// Rows of values dealt out to groups of lanes: single-value and 16-byte
// accesses, per-lane copy slots, sums over a group.  For the norm kernels.
#pragma once

#include "dev_common.cuh"
#include "dev_copy.cuh"

namespace zg {
namespace rows {

constexpr int kRowThreads = 256;
constexpr int kSms = 152;

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
    for (int k = 0; k < kRowThreads / 32; k++)
        t += sh[k];
    return t;
}

// Values of vector v of lane gl of a group of `lanes` that exist.
template <int DT>
__device__ __forceinline__ int vec_count(int64_t dim, int v, int gl, int lanes)
{
    constexpr int VE = kVecOf<DT>;
    return (int)max((int64_t)0, min((int64_t)VE, dim - (int64_t)(v * lanes + gl) * VE));
}

// Lane l gets the sum over its L lanes (L <= 32) of value l % N (N a power of
// two up to L): each step halves the values a lane still has, sending the
// others' half away.
template <int L, int N>
__device__ __forceinline__ float lane_sums(float (&x)[N])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = N / 2; h > 0; h /= 2) {
        const bool up = lane & h;
#pragma unroll
        for (int k = 0; k < h; k++) {
            const float keep = up ? x[k + h] : x[k], send = up ? x[k] : x[k + h];
            x[k] = keep + __shfl_xor_sync(0xffffffffu, send, h);
        }
    }
    float s = x[0];
#pragma unroll
    for (int o = N; o < L; o <<= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// finish(sum) over the group of N values at once, the same in every lane.  sh: room
// for [2][T / 32 warps][N] of the block; `turn` alternates, so one barrier a call.
template <int L, int N, int T = kRowThreads, typename F>
__device__ __forceinline__ void group_sum(float (&x)[N], int warps, float* sh, int& turn, F finish)
{
    const int lane = threadIdx.x & 31;
    float s = lane_sums<L, N>(x);
    if (L == 32 && warps > 1) {
        const int warp = threadIdx.x >> 5, group = warp / warps;
        float* slot = sh + (turn & 1) * (T / 32) * N;
        if (lane < N) slot[warp * N + lane] = s;
        asm volatile("bar.sync %0, %1;" :: "r"(1 + group), "r"(32 * warps) : "memory");
        // lane l: value l % N of every (32 / N)th warp; then a tree over the lanes of
        // the same value
        s = 0.0f;
        slot += group * warps * N;
#pragma unroll
        for (int q = 0; q < (T / 32 * N + 31) / 32; q++) {
            const int at = lane + 32 * q;
            if (at < warps * N) s += slot[at];
        }
#pragma unroll
        for (int o = N; o < 32; o <<= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        turn++;
    }
    s = finish(s);                                    // once, before all lanes have it
#pragma unroll
    for (int k = 0; k < N; k++)
        x[k] = __shfl_sync(0xffffffffu, s, k, L);
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

template <int DT>
__device__ __forceinline__ Vals<DT> from_slot(const uint4* slot)
{
    const uint4 u = *slot;
    Vals<DT> v;
    v.w[0] = u.x; v.w[1] = u.y; v.w[2] = u.z; v.w[3] = u.w;
    return v;
}

// 16 bytes, streaming.
__device__ __forceinline__ void store16(char* p, const uint32_t w[4])
{
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// A lane's vector out: all of it, or (RAGGED) the values that exist; rows on
// ALIGN-byte boundaries (16 or 4).
template <int DT, bool RAGGED, int ALIGN>
__device__ __forceinline__ void store_vec(char* p, const Vals<DT>& v, int cnt)
{
    if (RAGGED && cnt < kVecOf<DT>) {
        st_vals<DT>(p, 0, v, cnt);
    } else if (ALIGN == 16) {
        store16(p, v.w);
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
            __stcs(reinterpret_cast<uint32_t*>(p) + k, v.w[k]);
    }
}

// `bytes` of a lane's vector ahead, the rest of the slot 0.
template <int ALIGN>
__device__ __forceinline__ void vec_ahead(uint4* slot, const char* src, int bytes)
{
    if (ALIGN == 16) {
        copy_ahead<16>(slot, src, bytes);
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
            copy_ahead<4>(reinterpret_cast<uint32_t*>(slot) + k, 4 * k < bytes ? src + 4 * k : src,
                          max(0, min(4, bytes - 4 * k)));
    }
}

template <int DT, bool RAGGED>
__device__ __forceinline__ void weight_vec(const void* p, int64_t i, int cnt, float fill, float f[kVecOf<DT>])
{
    ld_weight<DT>(p, i, RAGGED ? cnt : kVecOf<DT>, fill, f);
}

// Rows of a group still to come, from this one on, that a batch of RB takes.
__device__ __forceinline__ int rows_here(int64_t rows, int64_t r0, int RB)
{
    return (int)max((int64_t)0, min((int64_t)RB, rows - r0));
}

// How rows of `vecs` 16-byte vectors are dealt out.
struct RowShape {
    int warps;                   // of a group
    int threads;                 // of a block
    int groups;                  // of a block
};

inline RowShape shape_of(int64_t vecs, int L, int V, int T = kRowThreads)
{
    RowShape r;
    if (L < 32) {
        r.warps = 1;
        r.threads = T;
        r.groups = T / L;
    } else {
        r.warps = (int)((vecs + 32 * V - 1) / (32 * V));
        r.groups = T / 32 / r.warps;
        r.threads = 32 * r.warps * r.groups;
    }
    return r;
}

}  // namespace rows
}  // namespace zg
