// AdamW over a list of tensors: the plan, the list's table in device memory,
// the step with binary32 or 8-bit moments, the gradients' global norm and
// clipping.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "dev_common.cuh"
#include "nvtx_ranges.h"

namespace zg {
namespace {

constexpr int kQBlock = 256;         // values per scale byte
constexpr int kChunk = 4096;         // values per block of threads: one tensor's, from a multiple of kChunk
// Threads per block, each measured: the binary32 step is bound by memory and
// likes 4 warps, the 8-bit one by instructions, and its warps keep out of step
// best as blocks of their own (4.25 ms for the 1.56e9 values of the 48-layer
// d=1600 list; 4.53 as pairs, 4.68 as fours).
constexpr int kAd32Threads = 128, kAd8Threads = 32, kStateThreads = 64;

// One tensor in the table.
struct AdRec {
    zero_adamw_tensor_t t;
    int64_t start;                   // place in the flat order
    int64_t first_chunk;
    int64_t aligned;                 // every buffer starts on a 16-byte boundary
    int64_t pad;
};
static_assert(sizeof(AdRec) == 104, "the plan sizes the table");

struct AdTable {
    const AdRec* rec;
    const int32_t* chunk_tensor;
};

int64_t chunk_map_offset(int64_t n) { return (n * (int64_t)sizeof(AdRec) + 15) / 16 * 16; }

__host__ __device__ inline AdTable table_of(const void* table, int64_t n)
{
    const unsigned char* b = static_cast<const unsigned char*>(table);
    return AdTable{reinterpret_cast<const AdRec*>(b),
                   reinterpret_cast<const int32_t*>(b + (n * (int64_t)sizeof(AdRec) + 15) / 16 * 16)};
}

// Step scalars, rounded once to binary32 on the host.
struct AdHP {
    AdamHP a;                        // lr, b1, 1-b1, b2, 1-b2, eps, bc1, bc2
    float gs;
    float step8;                     // lr / bc1
    float root8;                     // 1 / sqrt(bc2)
    uint32_t mix;                    // seed + t * constant
};

// Random bits of the 8 values from i on (a multiple of 8): hash_base once,
// then pair k = 0..3's two 16-bit numbers, low and high half.
constexpr uint32_t kHashA = 0x9E3779B1u, kHashB = 0x6A09E667u, kHashC = 0xBB67AE85u, kHashD = 0xA54FF53Bu;

__device__ __forceinline__ uint32_t hash_base(uint64_t i, uint32_t mix)
{
    const uint64_t j = i >> 1;
    return (uint32_t)j * kHashA + (uint32_t)(j >> 32) * kHashB + mix;
}

__device__ __forceinline__ uint32_t hash_pair(uint32_t base, uint32_t k)
{
    uint32_t h = base + k * kHashA;
    h = (h ^ (h >> 15)) * kHashC;
    h = (h ^ (h >> 15)) * kHashD;
    return h ^ (h >> 16);
}

// Codes.  Moved up to bits 26..19 a code is a binary32 pattern with the code's
// exponent and fraction, subnormals (E = 0) included, whose value is the
// code's times 2^-120 (m) or 2^-112 (r): one multiplication by a power of two,
// the scale with it, decodes it.  The other way the product with the inverse
// rounds to 19 bits below the code's last one (to nearest; only below the
// least normal), and the random bits decide the carry into it.
constexpr uint32_t kUpM = 120, kUpR = 112;

// 2^(e - 127) for an exponent field 1..254, 0 for 0.
__device__ __forceinline__ float pow2_field(uint32_t e) { return __uint_as_float(e << 23); }

// Factor that decodes a block with scale byte e: 2^(e - 127 + UP), 0 for e = 0;
// and its inverse, which encodes.  Scales from 2^7 (m) or 2^15 (r) on are out
// of one factor's range: `far_scale`; such a block multiplies by the rest,
// 2^(e - kFarScale), or its inverse, besides.
template <uint32_t UP>
constexpr uint32_t kFarScale = 253u - UP;

template <uint32_t UP>
__device__ __forceinline__ bool far_scale(uint32_t e) { return e > kFarScale<UP>; }

template <uint32_t UP>
__device__ __forceinline__ float dec_factor(uint32_t e) { return e ? pow2_field(min(e, kFarScale<UP>) + UP) : 0.0f; }

template <uint32_t UP>
__device__ __forceinline__ float enc_factor(uint32_t e) { return pow2_field(254u - UP - min(e, kFarScale<UP>)); }

template <uint32_t UP>
__device__ __forceinline__ float rest_factor(uint32_t e) { return pow2_field(127u + e - min(e, kFarScale<UP>)); }

template <uint32_t UP>
__device__ __forceinline__ float rest_inverse(uint32_t e) { return pow2_field(127u - e + min(e, kFarScale<UP>)); }

// Byte k of w at bits 31..24, zeros below.
template <int K>
__device__ __forceinline__ uint32_t byte_on_top(uint32_t w)
{
    return K == 0 ? w << 24 : K == 3 ? w & 0xff000000u : __byte_perm(w, 0, K == 2 ? 0x2444 : 0x1444);
}

__device__ __forceinline__ uint32_t byte_on_top(uint2 w, int k)
{
    const uint32_t x = k < 4 ? w.x : w.y;
    return (k & 3) == 0 ? byte_on_top<0>(x) : (k & 3) == 1 ? byte_on_top<1>(x) : (k & 3) == 2 ? byte_on_top<2>(x)
                                                                                             : byte_on_top<3>(x);
}

// `top`: the code in bits 31..24, zeros below; `dec`: the block's factor.
__device__ __forceinline__ float decode_m(uint32_t top, float dec)
{
    // the arithmetic shift leaves the sign in bit 31, the mask only that copy of it
    return __fmul_rn(__uint_as_float((uint32_t)((int32_t)top >> 5) & 0x83f80000u), dec);
}

__device__ __forceinline__ float decode_r(uint32_t top, float dec) { return __fmul_rn(__uint_as_float(top >> 5), dec); }

// Four codes of m in a word, from the scaled values plus the random bits (as
// bit patterns: sign, then the code from bit 19 on); no negative zero.
__device__ __forceinline__ uint32_t pack_m(const uint32_t u[4])
{
    const uint32_t mag = ((u[0] >> 19) & 0x7fu) | ((u[1] >> 11) & 0x7f00u) | ((u[2] >> 3) & 0x7f0000u) | ((u[3] << 5) & 0x7f000000u);
    const uint32_t sign = ((u[0] >> 24) & 0x80u) | ((u[1] >> 16) & 0x8000u) | ((u[2] >> 8) & 0x800000u) | (u[3] & 0x80000000u);
    return mag | (sign & (mag + 0x7f7f7f7fu));          // bit 7 of a byte of the sum: its magnitude is not 0
}

// Four codes of r; a nonzero root keeps a nonzero code.
__device__ __forceinline__ uint32_t pack_r(const uint32_t u[4], const float r[4])
{
    uint32_t w = __byte_perm(__byte_perm(u[0] >> 19, u[1] >> 19, 0x0040), __byte_perm(u[2] >> 19, u[3] >> 19, 0x0040), 0x5410);
    if ((w - 0x01010101u) & ~w & 0x80808080u)           // some byte is 0
#pragma unroll
        for (int k = 0; k < 4; k++)
            if (!(w >> (8 * k) & 0xffu) && r[k] > 0.0f) w |= 1u << (8 * k);
    return w;
}

// A block's scale byte, from the bit pattern of its largest magnitude: the
// exponent field one code step (1/16 of the binade) above it, so that the
// largest value too can round up.  Scaled by its own exponent alone, a value
// within one step of the binade's end could only be cut to the largest code:
// an average that moves by less than a step would stop there for good.
__device__ __forceinline__ uint32_t scale_field(uint32_t most) { return min((most + (1u << 19)) >> 23, 253u); }

template <int V, typename T>
__device__ __forceinline__ void ld_any(const T* p, int cnt, bool vec, T x[V])
{
    static_assert(sizeof(T) * V >= 8, "");
    if (vec && cnt == V) {
        if constexpr (sizeof(T) * V == 8) {
            *reinterpret_cast<uint2*>(x) = __ldcs(reinterpret_cast<const uint2*>(p));
        } else {
#pragma unroll
            for (int k = 0; k < (int)(sizeof(T) * V / 16); k++)
                reinterpret_cast<uint4*>(x)[k] = __ldcs(reinterpret_cast<const uint4*>(p) + k);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; j++)
            x[j] = j < cnt ? p[j] : T(0);
    }
}

template <int V, typename T>
__device__ __forceinline__ void st_any(T* p, int cnt, bool vec, const T x[V])
{
    if (vec && cnt == V) {
        if constexpr (sizeof(T) * V == 8) {
            __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(x));
        } else {
#pragma unroll
            for (int k = 0; k < (int)(sizeof(T) * V / 16); k++)
                __stcs(reinterpret_cast<uint4*>(p) + k, reinterpret_cast<const uint4*>(x)[k]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; j++)
            if (j < cnt) p[j] = x[j];
    }
}

// The block's record, in shared memory: in global memory a store might alias
// it, and every pointer would be read again after each one.
__device__ __forceinline__ const AdRec& record_of(const AdTable& tab, AdRec& held)
{
    const AdRec& r = tab.rec[tab.chunk_tensor[blockIdx.x]];
    static_assert(sizeof(AdRec) % 4 == 0 && sizeof(AdRec) / 4 <= 32, "one word a thread");
    if (threadIdx.x < sizeof(AdRec) / 4)
        reinterpret_cast<uint32_t*>(&held)[threadIdx.x] = reinterpret_cast<const uint32_t*>(&r)[threadIdx.x];
    __syncthreads();
    return held;
}

template <int DT>
using Bits = typename std::conditional<DT == kF32, uint32_t, uint16_t>::type;

// Binary32 moments: groups of 4 values, one 16-byte access per binary32 array.
// Bound by memory: 511 us for the 1.24e8 values of the 12-layer d=768 list, 28
// bytes each, 6.8 TB/s, a device copy's rate.
template <int DT>
__global__ void __launch_bounds__(kAd32Threads) k_adamw32(const AdTable tab, const __grid_constant__ AdHP hp,
                                                        const uint32_t* skip, const float* norm)
{
    wait_prev_grid();
    if (skip && *skip) return;
    const float gs = norm ? __fmul_rn(norm[1], hp.gs) : hp.gs;
    constexpr int V = 4;
    __shared__ AdRec held;
    const AdRec& r = record_of(tab, held);
    const int64_t lo = ((int64_t)blockIdx.x - r.first_chunk) * kChunk;
    const int64_t hi = min(lo + kChunk, r.t.numel);
    const bool vec = r.aligned;
    const float keep = __fmaf_rn(-hp.a.lr, r.t.weight_decay, 1.0f);
    const Bits<DT>* grad = static_cast<const Bits<DT>*>(r.t.grad);
    Bits<DT>* param = static_cast<Bits<DT>*>(r.t.param);
    float* mp = static_cast<float*>(r.t.m);
    float* vp = static_cast<float*>(r.t.v);
    for (int64_t i = lo + threadIdx.x * V; i < hi; i += kAd32Threads * V) {
        const int cnt = (int)min((int64_t)V, hi - i);
        alignas(16) Bits<DT> g[V], p[V];
        alignas(16) float w[V], m[V], v[V];
        ld_any<V>(grad + i, cnt, vec, g);
        ld_any<V>(r.t.master + i, cnt, vec, w);
        ld_any<V>(mp + i, cnt, vec, m);
        ld_any<V>(vp + i, cnt, vec, v);
#pragma unroll
        for (int j = 0; j < V; j++) {
            w[j] = __fmul_rn(w[j], keep);
            adam1(__fmul_rn(to_f32<DT>(g[j]), gs), w[j], m[j], v[j], hp.a);
            p[j] = (Bits<DT>)from_f32<DT>(w[j]);
        }
        st_any<V>(r.t.master + i, cnt, vec, w);
        st_any<V>(mp + i, cnt, vec, m);
        st_any<V>(vp + i, cnt, vec, v);
        if (param) st_any<V>(param + i, cnt, vec, p);
    }
}

// 8-bit moments: a warp takes a block of 256 values, 8 per lane, so the
// block's largest magnitudes are one warp-wide maximum each.  Instructions
// bound it, about 86 a value (a correctly rounded square root and division,
// the codes' integer work): the 30 warps of an SM issue in 74 % of the cycles.
// Copying the next block's inputs ahead into shared memory costs more
// instructions than the latency it hides (412 us against 357 for the 1.24e8
// values of the 12-layer d=768 list), packed pairs of binary32 operations more
// moves (553).
template <int DT>
__global__ void __launch_bounds__(kAd8Threads, 32) k_adamw8(const AdTable tab, const __grid_constant__ AdHP hp,
                                                           const uint32_t* skip, const float* norm)
{
    wait_prev_grid();
    if (skip && *skip) return;
    const float gs = norm ? __fmul_rn(norm[1], hp.gs) : hp.gs;
    constexpr int V = 8;
    const AdRec& r = tab.rec[tab.chunk_tensor[blockIdx.x]];
    const zero_adamw_tensor_t& t = r.t;
    const int64_t lo = ((int64_t)blockIdx.x - r.first_chunk) * kChunk;
    const int64_t hi = min(lo + kChunk, t.numel);
    const bool vec = r.aligned;
    const float keep = __fmaf_rn(-hp.a.lr, t.weight_decay, 1.0f);
    const int lane = threadIdx.x;
    for (int64_t b = lo + blockIdx.y * kQBlock; b < hi; b += gridDim.y * kQBlock) {
        const int64_t i = b + lane * V;
        const int cnt = i < hi ? (int)min((int64_t)V, hi - i) : 0;
        alignas(16) Bits<DT> g[V];
        alignas(16) float w[V];
        alignas(8) uint8_t cm8[V], cr8[V];
        ld_any<V>(static_cast<const Bits<DT>*>(t.grad) + i, cnt, vec, g);
        ld_any<V>(t.master + i, cnt, vec, w);
        ld_any<V>(static_cast<const uint8_t*>(t.m) + i, cnt, vec, cm8);
        ld_any<V>(static_cast<const uint8_t*>(t.v) + i, cnt, vec, cr8);
        const uint2 wm = *reinterpret_cast<const uint2*>(cm8), wr = *reinterpret_cast<const uint2*>(cr8);
        const uint32_t em0 = t.m_scale[b / kQBlock], er0 = t.v_scale[b / kQBlock];
        const float dm = dec_factor<kUpM>(em0), dr = dec_factor<kUpR>(er0);
        float m[V], q[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
            m[j] = decode_m(byte_on_top(wm, j), dm);
            q[j] = decode_r(byte_on_top(wr, j), dr);
        }
        if (far_scale<kUpM>(em0) || far_scale<kUpR>(er0)) {
#pragma unroll
            for (int j = 0; j < V; j++) {
                m[j] = __fmul_rn(m[j], rest_factor<kUpM>(em0));
                q[j] = __fmul_rn(q[j], rest_factor<kUpR>(er0));
            }
        }
        alignas(16) Bits<DT> p[V];
        uint32_t most_m = 0, most_r = 0;
#pragma unroll
        for (int j = 0; j < V; j++) {
            const float gj = __fmul_rn(to_f32<DT>(g[j]), gs);
            m[j] = __fadd_rn(__fmul_rn(m[j], hp.a.b1), __fmul_rn(gj, hp.a.omb1));
            q[j] = __fsqrt_rn(__fadd_rn(__fmul_rn(__fmul_rn(q[j], q[j]), hp.a.b2), __fmul_rn(__fmul_rn(gj, gj), hp.a.omb2)));
            const float d = __fadd_rn(__fmul_rn(q[j], hp.root8), hp.a.eps);
            w[j] = __fsub_rn(__fmul_rn(w[j], keep), __fdiv_rn(__fmul_rn(m[j], hp.step8), d));
            p[j] = (Bits<DT>)from_f32<DT>(w[j]);
        }
#pragma unroll
        for (int j = 0; j < V; j += 2) {               // values past cnt are 0: m = r = 0; a root has no sign
            most_m = __vimax3_u32(most_m, __float_as_uint(m[j]) & 0x7fffffffu, __float_as_uint(m[j + 1]) & 0x7fffffffu);
            most_r = __vimax3_u32(most_r, __float_as_uint(q[j]), __float_as_uint(q[j + 1]));
        }
        st_any<V>(t.master + i, cnt, vec, w);
        if (t.param) st_any<V>(static_cast<Bits<DT>*>(t.param) + i, cnt, vec, p);
        const uint32_t em = scale_field(__reduce_max_sync(0xffffffffu, most_m));
        const uint32_t er = scale_field(__reduce_max_sync(0xffffffffu, most_r));
        const float cm = enc_factor<kUpM>(em), cr = enc_factor<kUpR>(er);
        const uint32_t base = hash_base((uint64_t)(r.start + i), hp.mix);
        const bool far = far_scale<kUpM>(em) || far_scale<kUpR>(er);
        uint32_t um[V], ur[V];
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const uint32_t h = hash_pair(base, j / 2);
            const uint32_t r0 = (h << 3) & 0x7fff8u, r1 = (h >> 13) & 0x7fff8u;
            um[j] = __float_as_uint(__fmul_rn(m[j], cm)) + r0;
            um[j + 1] = __float_as_uint(__fmul_rn(m[j + 1], cm)) + r1;
            ur[j] = __float_as_uint(__fmul_rn(q[j], cr)) + r0;
            ur[j + 1] = __float_as_uint(__fmul_rn(q[j + 1], cr)) + r1;
        }
        if (far) {
            // two factors; the last scale, and what is not finite, is cut to the
            // largest code
#pragma unroll
            for (int j = 0; j < V; j++) {
                const uint32_t h = hash_pair(base, j / 2), rnd = j & 1 ? (h >> 13) & 0x7fff8u : (h << 3) & 0x7fff8u;
                const uint32_t xm = __float_as_uint(__fmul_rn(__fmul_rn(fabsf(m[j]), rest_inverse<kUpM>(em)), cm));
                const uint32_t xr = __float_as_uint(__fmul_rn(__fmul_rn(q[j], rest_inverse<kUpR>(er)), cr));
                um[j] = (min((min(xm, 0x7f800000u) + rnd) >> 19, 127u) << 19) | (m[j] < 0.0f ? 0x80000000u : 0u);
                ur[j] = min((min(xr, 0x7f800000u) + rnd) >> 19, 255u) << 19;
            }
        }
        alignas(8) uint8_t nm8[V], nr8[V];
        *reinterpret_cast<uint2*>(nm8) = make_uint2(pack_m(um), pack_m(um + 4));
        *reinterpret_cast<uint2*>(nr8) = make_uint2(pack_r(ur, q), pack_r(ur + 4, q + 4));
        st_any<V>(static_cast<uint8_t*>(t.m) + i, cnt, vec, nm8);
        st_any<V>(static_cast<uint8_t*>(t.v) + i, cnt, vec, nr8);
        if (lane == 0) {
            t.m_scale[b / kQBlock] = (uint8_t)em;
            t.v_scale[b / kQBlock] = (uint8_t)er;
        }
    }
}

// Stored 8-bit moments as bfloat16 values (5 significant bits: the upper half
// of the binary32 pattern, exact but for m of scale bytes below 4, cut to
// bfloat16's subnormals).  Bound by memory: 116 us
// for the 1.24e8 values of the 12-layer d=768 list, 6 bytes each, 6.4 TB/s.
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi)
{
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

__global__ void __launch_bounds__(kStateThreads) k_adamw_states(const AdTable tab, uint16_t* m_out, uint16_t* r_out)
{
    constexpr int V = 8;
    const AdRec& r = tab.rec[tab.chunk_tensor[blockIdx.x]];
    const zero_adamw_tensor_t t = r.t;
    const int64_t start = r.start;
    const int64_t lo = ((int64_t)blockIdx.x - r.first_chunk) * kChunk;
    const int64_t hi = min(lo + kChunk, t.numel);
    const bool vec = r.aligned;
#pragma unroll 4
    for (int64_t i = lo + threadIdx.x * V; i < hi; i += kStateThreads * V) {
        const int cnt = (int)min((int64_t)V, hi - i);
        alignas(8) uint8_t cm[V], cr[V];
        ld_any<V>(static_cast<const uint8_t*>(t.m) + i, cnt, vec, cm);
        ld_any<V>(static_cast<const uint8_t*>(t.v) + i, cnt, vec, cr);
        const uint2 wm = *reinterpret_cast<const uint2*>(cm), wr = *reinterpret_cast<const uint2*>(cr);
        const uint32_t em = t.m_scale[i / kQBlock], er = t.v_scale[i / kQBlock];
        const float dm = dec_factor<kUpM>(em), dr = dec_factor<kUpR>(er);
        alignas(16) uint32_t m[V / 2], q[V / 2];
#pragma unroll
        for (int k = 0; k < V / 2; k++) {
            float x[2], y[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                x[e] = decode_m(byte_on_top(wm, 2 * k + e), dm);
                y[e] = decode_r(byte_on_top(wr, 2 * k + e), dr);
                if (far_scale<kUpM>(em)) x[e] = __fmul_rn(x[e], rest_factor<kUpM>(em));
                if (far_scale<kUpR>(er)) y[e] = __fmul_rn(y[e], rest_factor<kUpR>(er));
            }
            m[k] = upper_halves(x[0], x[1]);
            q[k] = upper_halves(y[0], y[1]);
        }
        st_any<V>(m_out + start + i, cnt, true, reinterpret_cast<const uint16_t*>(m));
        st_any<V>(r_out + start + i, cnt, true, reinterpret_cast<const uint16_t*>(q));
    }
}

template <int DT>
__global__ void __launch_bounds__(kAd32Threads) k_adamw_check(const AdTable tab, uint32_t* flag)
{
    constexpr int V = 8;
    const AdRec& r = tab.rec[tab.chunk_tensor[blockIdx.x]];
    const int64_t lo = ((int64_t)blockIdx.x - r.first_chunk) * kChunk;
    const int64_t hi = min(lo + kChunk, r.t.numel);
    const Bits<DT>* grad = static_cast<const Bits<DT>*>(r.t.grad);
    uint32_t bad = 0;
    for (int64_t i = lo + threadIdx.x * V; i < hi; i += kAd32Threads * V) {
        const int cnt = (int)min((int64_t)V, hi - i);
        alignas(16) Bits<DT> g[V];
        ld_any<V>(grad + i, cnt, r.aligned, g);
#pragma unroll
        for (int j = 0; j < V; j++)
            bad |= nonfinite32(__float_as_uint(to_f32<DT>(g[j])));
    }
    if (__syncthreads_or((int)bad) && threadIdx.x == 0) *flag = 1u;
}

// ---- the gradients' norm --------------------------------------------------------------
// sqrt(sum of g^2) over the list.  A group of G threads takes a run of consecutive
// chunks, whose tensors' values lie side by side, so it streams; kNormUnroll 16-byte
// loads of a thread are on their way at once.  A thread adds up the squares of a batch (32
// 16-bit values, 16 of 32 bits) in binary32 and the batches in binary64: one
// binary64 operation to a batch is out of the way of memory, one to a value is not
// (GB300 has 2 of them a clock and SM, a fifth of what the values would need).  A
// batch whose binary32 sum overflows, or is so small that squares may have
// been cut off below 2^-126, is read again and summed in binary64 alone; so is one
// that holds an infinity or a NaN, which is where those are counted.  Bound by
// memory: 1.56e9 bfloat16 values 447-453 us, 6.9 TB/s; the 12-layer d=768 list 44
// before a step of 514.
constexpr int kNormThreads = 256, kNormUnroll = 4;
constexpr int64_t kNormBlocks = 152 * 8;              // all resident at once
// Up to so many chunks one block does all, a chunk to each of its warps, and needs no
// second kernel.
constexpr int kNormAlone = 32;

struct NormPart {
    double sum;
    uint64_t bad;                // a gradient is inf or NaN
};

struct NormOut {
    NormPart* part;
    float* norm;                 // {norm, factor}
    uint32_t* flag;
    double scale;                // |grad_scale|
    double max_norm;             // 0: no clipping
};

template <int DT>
__device__ __noinline__ double squares64(const Bits<DT>* p, int n, uint64_t& bad)
{
    double s = 0.0;
    for (int j = 0; j < n; j++) {
        const float g = to_f32<DT>(p[j]);
        if (nonfinite32(__float_as_uint(g))) bad = 1;
        s = fma((double)g, (double)g, s);
    }
    return s;
}

// The sum, and the factor that clips, as the sharded step has them.
__device__ __forceinline__ void norm_out(const NormOut& o, double sum, uint64_t bad)
{
    const double norm = sqrt(sum) * o.scale;
    o.norm[0] = (float)norm;
    const double c = o.max_norm / (norm + 1e-6);
    o.norm[1] = o.max_norm > 0.0 && !(c >= 1.0) ? (float)c : 1.0f;      // NaN of a NaN
    if (o.flag) *o.flag = bad != 0;
}

// Sum over the block, in a fixed order, in thread 0.
template <int T>
__device__ __forceinline__ NormPart norm_join(double sum, uint64_t bad)
{
    __shared__ double sh[T / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_down_sync(0xffffffffu, sum, o);
    if (lane == 0) sh[warp] = sum;
    const int any = __syncthreads_or(bad != 0);
    NormPart r{0.0, (uint64_t)(any != 0)};
    if (threadIdx.x == 0)
        for (int k = 0; k < T / 32; k++)
            r.sum += sh[k];
    return r;
}

template <int DT, int G, int T>
__global__ void __launch_bounds__(T, T < 1024 ? 2048 / T : 1) k_adamw_norm(const AdTable tab, int64_t n_chunks,
                                                            const __grid_constant__ NormOut out)
{
    constexpr int V = kVecOf<DT>, U = kNormUnroll, kBatch = G * V;
    wait_prev_grid();
    allow_next_grid();
    double sum = 0.0;
    uint64_t bad = 0;
    const int64_t groups = (int64_t)gridDim.x * (T / G), group = (int64_t)blockIdx.x * (T / G) + threadIdx.x / G;
    int64_t c = n_chunks * group / groups;
    const int64_t end = n_chunks * (group + 1) / groups;
    while (c < end) {
        const AdRec& r = tab.rec[tab.chunk_tensor[c]];
        const Bits<DT>* g = static_cast<const Bits<DT>*>(r.t.grad);
        const int64_t numel = r.t.numel, first = r.first_chunk;
        const int64_t stop = min(end, first + (numel + kChunk - 1) / kChunk);
        const int64_t lo = (c - first) * kChunk, hi = min((stop - first) * kChunk, numel);
        const bool vec = ((uintptr_t)g & 15u) == 0;
        c = stop;
        for (int64_t i0 = lo; i0 < hi; i0 += U * kBatch) {
            const int64_t i = i0 + threadIdx.x % G * V;
            float s = 0.0f;
            uint32_t any = 0;
            auto add = [&](const uint4& q) {
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    any |= w[k];
                    if constexpr (DT == kF32) {
                        s = fmaf(__uint_as_float(w[k]), __uint_as_float(w[k]), s);
                    } else {
                        const float2 f = to_f32x2<DT>(w[k]);
                        s = fmaf(f.x, f.x, s);
                        s = fmaf(f.y, f.y, s);
                    }
                }
            };
            if (vec && i0 + U * kBatch <= hi) {
                uint4 q[U];
#pragma unroll
                for (int u = 0; u < U; u++)
                    q[u] = *reinterpret_cast<const uint4*>(g + i + u * kBatch);
#pragma unroll
                for (int u = 0; u < U; u++)
                    add(q[u]);
            } else {
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int64_t left = hi - (i + u * kBatch);
                    alignas(16) Bits<DT> x[V];
                    const int cnt = left <= 0 ? 0 : left < V ? (int)left : V;
                    if (vec && cnt == V) {
                        *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(g + i + u * kBatch);
                    } else {
#pragma unroll
                        for (int j = 0; j < V; j++)
                            x[j] = j < cnt ? g[i + u * kBatch + j] : Bits<DT>(0);
                    }
                    add(*reinterpret_cast<const uint4*>(x));
                }
            }
            any &= DT == kF32 ? 0x7fffffffu : 0x7fff7fffu;            // zeros of either sign
            // 2^-80: what 32 squares below 2^-126 lost is nothing beside it
            if (s >= 0x1p-80f && s < INFINITY) {
                sum += (double)s;
            } else if (any) {
#pragma unroll 1
                for (int u = 0; u < U; u++) {
                    const int64_t left = hi - (i + u * kBatch);
                    if (left > 0) sum += squares64<DT>(g + i + u * kBatch, left < V ? (int)left : V, bad);
                }
            }
        }
    }
    const NormPart r = norm_join<T>(sum, bad);
    if (threadIdx.x) return;
    if (G < T)
        norm_out(out, r.sum, r.bad);
    else
        out.part[blockIdx.x] = r;
}

// One block: the blocks' sums, in a fixed order.
__global__ void __launch_bounds__(kNormThreads) k_adamw_norm_join(int parts, const __grid_constant__ NormOut out)
{
    wait_prev_grid();
    double sum = 0.0;
    uint64_t bad = 0;
    for (int k = threadIdx.x; k < parts; k += kNormThreads) {
        sum += out.part[k].sum;
        bad |= out.part[k].bad;
    }
    const NormPart r = norm_join<kNormThreads>(sum, bad);
    if (threadIdx.x == 0) norm_out(out, r.sum, r.bad);
}

// Gradients times the factor, rounded to their type; nothing to do where it is 1.
// Bound by memory, of the 12-layer d=768 list in binary16 75 us, 6.6 TB/s; with a factor of 1 18 us, its
// blocks' launch.
template <int DT>
__global__ void __launch_bounds__(kAd32Threads) k_adamw_clip(const AdTable tab, const float* norm)
{
    wait_prev_grid();
    const float factor = norm[1];
    if (factor == 1.0f) return;
    constexpr int V = kVecOf<DT>;
    const AdRec& r = tab.rec[tab.chunk_tensor[blockIdx.x]];
    const int64_t lo = ((int64_t)blockIdx.x - r.first_chunk) * kChunk;
    const int64_t hi = min(lo + kChunk, r.t.numel);
    Bits<DT>* grad = static_cast<Bits<DT>*>(const_cast<void*>(r.t.grad));
    const bool vec = ((uintptr_t)grad & 15u) == 0;
#pragma unroll 4
    for (int64_t i = lo + threadIdx.x * V; i < hi; i += kAd32Threads * V) {
        const int cnt = (int)min((int64_t)V, hi - i);
        alignas(16) Bits<DT> g[V];
        ld_any<V>(grad + i, cnt, vec, g);
#pragma unroll
        for (int j = 0; j < V; j++)
            g[j] = (Bits<DT>)from_f32<DT>(__fmul_rn(to_f32<DT>(g[j]), factor));
        st_any<V>(grad + i, cnt, vec, g);
    }
}

// One warp: the tensors' places in the flat order and in the chunk order.
__global__ void __launch_bounds__(32) k_adamw_places(AdRec* rec, int64_t n)
{
    int64_t start = 0, chunk = 0;
    const int lane = threadIdx.x;
    for (int64_t k0 = 0; k0 < n; k0 += 32) {
        const int64_t k = k0 + lane;
        const int64_t num = k < n ? rec[k].t.numel : 0;
        const int64_t len = (num + kQBlock - 1) / kQBlock * kQBlock, chunks = (num + kChunk - 1) / kChunk;
        int64_t ls = len, cs = chunks;               // inclusive sums over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t l = __shfl_up_sync(0xffffffffu, ls, o), c = __shfl_up_sync(0xffffffffu, cs, o);
            if (lane >= o) {
                ls += l;
                cs += c;
            }
        }
        if (k < n) {
            const zero_adamw_tensor_t& t = rec[k].t;
            const uintptr_t any = (uintptr_t)t.grad | (uintptr_t)t.param | (uintptr_t)t.master | (uintptr_t)t.m |
                                  (uintptr_t)t.v;
            rec[k].start = start + ls - len;
            rec[k].first_chunk = chunk + cs - chunks;
            rec[k].aligned = (any & 15u) == 0;
        }
        start += __shfl_sync(0xffffffffu, ls, 31);
        chunk += __shfl_sync(0xffffffffu, cs, 31);
    }
}

__global__ void k_adamw_chunks(const AdRec* rec, int64_t n, int32_t* chunk_tensor)
{
    for (int64_t k = blockIdx.x; k < n; k += gridDim.x) {
        const int64_t c = (rec[k].t.numel + kChunk - 1) / kChunk;
        for (int64_t j = threadIdx.x; j < c; j += blockDim.x)
            chunk_tensor[rec[k].first_chunk + j] = (int32_t)k;
    }
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

zero_status_t cuda_failed(cudaError_t e, const char* what)
{
    char msg[200];
    std::snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return set_error(ZERO_ECUDA, msg);
}

// A mark over a plan's other fields (FNV-1a by 64-bit words): the list that they
// were counted from is not at hand when a plan is used.
int64_t mark_of(const zero_adamw_plan_t& p)
{
    const uint64_t f[] = {(uint64_t)p.n_tensors,   (uint64_t)p.numel,     (uint64_t)p.flat_elems, (uint64_t)p.n_chunks,
                          (uint64_t)p.table_bytes, (uint64_t)p.hbm_bytes, (uint64_t)p.dtype,      (uint64_t)p.state_bits};
    uint64_t h = 0xcbf29ce484222325ull;
    for (uint64_t x : f)
        h = (h ^ x) * 0x100000001b3ull;
    return (int64_t)(h ^ (h >> 32));
}

zero_status_t check_adamw_plan(const zero_adamw_plan_t* p, const void* table)
{
    if (!p) return set_error(ZERO_EINVAL, "AdamW plan is NULL");
    if (p->mark != mark_of(*p))
        return set_error(ZERO_EINVAL, "AdamW plan was not made by zero_adamw_plan");
    if (p->n_chunks && !table) return set_error(ZERO_ENOMEM, "AdamW table is NULL");
    if (!aligned_to(table, 16)) return set_error(ZERO_EALIGN, "AdamW table is not 16-byte aligned");
    return ZERO_OK;
}

template <int DT>
cudaError_t launch_norm(const AdTable& tab, int64_t n_chunks, const NormOut& o, unsigned grid, cudaStream_t s)
{
    return grid == 1 ? launch_after(k_adamw_norm<DT, 32, 32 * kNormAlone>, dim3(1), 32 * kNormAlone, 0, s, tab, n_chunks, o)
                     : launch_after(k_adamw_norm<DT, kNormThreads, kNormThreads>, dim3(grid), kNormThreads, 0, s, tab, n_chunks, o);
}

// Blocks of the norm's kernel, a function of the list alone.
int64_t norm_blocks(const zero_adamw_plan_t& p)
{
    return p.n_chunks <= kNormAlone ? 1 : p.n_chunks < kNormBlocks ? p.n_chunks : kNormBlocks;
}

// The step; norm: NULL, or device memory whose second value multiplies the gradients besides.
zero_status_t adamw_step(const zero_adamw_plan_t* plan, const void* table, const zero_adamw_t* hp, const float* norm,
                         const uint32_t* skip, void* stream)
{
    const zero_status_t st = check_adamw_plan(plan, table);
    if (st != ZERO_OK) return st;
    if (!hp) return set_error(ZERO_EINVAL, "zero_adamw_step: hyper-parameters are NULL");
    if (hp->t < 1) return set_error(ZERO_EINVAL, "zero_adamw_step: t must be at least 1");
    if (!(hp->beta1 >= 0.0f && hp->beta1 < 1.0f) || !(hp->beta2 >= 0.0f && hp->beta2 < 1.0f))
        return set_error(ZERO_EINVAL, "zero_adamw_step: betas must be in [0, 1)");
    if (!(hp->eps >= 0.0f) || !std::isfinite(hp->lr) || !std::isfinite(hp->grad_scale))
        return set_error(ZERO_EINVAL, "zero_adamw_step: eps must be >= 0, lr and grad_scale finite");
    if (!aligned_to(skip, 4)) return set_error(ZERO_EALIGN, "zero_adamw_step: skip is not 4-byte aligned");
    if (plan->n_chunks == 0) return ZERO_OK;
    AdHP h;
    std::memset(&h, 0, sizeof h);
    const double bc1 = 1.0 - std::pow((double)hp->beta1, (double)hp->t);
    const double bc2 = 1.0 - std::pow((double)hp->beta2, (double)hp->t);
    h.a.lr = hp->lr;
    h.a.b1 = hp->beta1;
    h.a.omb1 = 1.0f - hp->beta1;
    h.a.b2 = hp->beta2;
    h.a.omb2 = 1.0f - hp->beta2;
    h.a.eps = hp->eps;
    h.a.bc1 = (float)bc1;
    h.a.bc2 = (float)bc2;
    h.gs = hp->grad_scale;
    h.step8 = (float)((double)hp->lr / bc1);
    h.root8 = (float)(1.0 / std::sqrt(bc2));
    h.mix = hp->seed + (uint32_t)hp->t * 0x510E527Fu;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const AdTable tab = table_of(table, plan->n_tensors);
    const unsigned grid = (unsigned)plan->n_chunks;
    const int dt = plan->dtype;
    cudaError_t err;
    if (plan->state_bits == 32) {
        const auto kernel = dt == ZERO_FP32 ? k_adamw32<kF32> : dt == ZERO_BF16 ? k_adamw32<kBF16> : k_adamw32<kF16>;
        err = launch_after(kernel, dim3(grid), kAd32Threads, 0, s, tab, h, skip, norm);
    } else {
        // a chunk's 16 blocks go to one warp, or in a short list to as many as fill
        // the 152 x 32 warps resident at once (148 tensors of up to 8894 values, step
        // and read-out: 17 us, with one warp 35; one of 1.7 million: 12 and 23)
        unsigned share = 1;
        while (share < kChunk / kQBlock && grid * share < 152u * 32u) share *= 2;
        const dim3 grid8(grid, share);
        const auto kernel = dt == ZERO_FP32 ? k_adamw8<kF32> : dt == ZERO_BF16 ? k_adamw8<kBF16> : k_adamw8<kF16>;
        err = launch_after(kernel, grid8, kAd8Threads, 0, s, tab, h, skip, norm);
    }
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_adamw_step");
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

zero_status_t zero_adamw_plan(const zero_adamw_tensor_t* tensors, int64_t n_tensors, int32_t dtype,
                              int32_t state_bits, zero_adamw_plan_t* out)
{
    if (!out) return set_error(ZERO_EINVAL, "zero_adamw_plan: out is NULL");
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16 && dtype != ZERO_FP32)
        return set_error(ZERO_EINVAL, "zero_adamw_plan: dtype unknown");
    if (state_bits != 8 && state_bits != 32)
        return set_error(ZERO_EUNSUPPORTED, "zero_adamw_plan: state_bits must be 8 or 32");
    if (n_tensors < 0 || (n_tensors && !tensors)) return set_error(ZERO_EINVAL, "zero_adamw_plan: no tensors given");
    if (n_tensors > (int64_t(1) << 20)) return set_error(ZERO_EUNSUPPORTED, "zero_adamw_plan: over 2^20 tensors");
    std::memset(out, 0, sizeof *out);
    int64_t numel = 0, flat = 0, chunks = 0;
    for (int64_t k = 0; k < n_tensors; k++) {
        const int64_t n = tensors[k].numel;
        if (n < 0) return set_error(ZERO_EINVAL, "zero_adamw_plan: a tensor has a negative numel");
        if (n > (int64_t(1) << 40) || numel + n > (int64_t(1) << 40))
            return set_error(ZERO_EUNSUPPORTED, "zero_adamw_plan: over 2^40 values");
        if (!std::isfinite(tensors[k].weight_decay))
            return set_error(ZERO_EINVAL, "zero_adamw_plan: a weight_decay is not finite");
        numel += n;
        flat += (n + kQBlock - 1) / kQBlock * kQBlock;
        chunks += (n + kChunk - 1) / kChunk;
    }
    out->n_tensors = n_tensors;
    out->numel = numel;
    out->flat_elems = flat;
    out->n_chunks = chunks;
    out->table_bytes = chunk_map_offset(n_tensors) + chunks * 4;
    out->dtype = dtype;
    out->state_bits = state_bits;
    out->hbm_bytes = numel * (2 * (dtype == ZERO_FP32 ? 4 : 2) + (state_bits == 32 ? 24 : 12));
    out->mark = mark_of(*out);
    return ZERO_OK;
}

zero_status_t zero_adamw_table_init(const zero_adamw_plan_t* plan, const zero_adamw_tensor_t* tensors, void* table,
                                    void* stream)
{
    NvtxRange range("zero_adamw_table_init");
    zero_status_t st = check_adamw_plan(plan, table);
    if (st != ZERO_OK) return st;
    zero_adamw_plan_t fresh;
    st = zero_adamw_plan(tensors, plan->n_tensors, plan->dtype, plan->state_bits, &fresh);
    if (st != ZERO_OK) return st;
    if (std::memcmp(&fresh, plan, sizeof fresh) != 0)
        return set_error(ZERO_EINVAL, "zero_adamw_table_init: the plan was made for other tensors");
    const size_t e = plan->dtype == ZERO_FP32 ? 4 : 2, se = plan->state_bits / 8;
    for (int64_t k = 0; k < plan->n_tensors; k++) {
        const zero_adamw_tensor_t& t = tensors[k];
        if (t.numel == 0) continue;
        if (!t.grad || !t.master || !t.m || !t.v || (plan->state_bits == 8 && (!t.m_scale || !t.v_scale)))
            return set_error(ZERO_ENOMEM, "zero_adamw_table_init: a tensor's buffer is NULL");
        if (!aligned_to(t.grad, e) || !aligned_to(t.param, e) || !aligned_to(t.master, 4) || !aligned_to(t.m, se) ||
            !aligned_to(t.v, se))
            return set_error(ZERO_EALIGN, "zero_adamw_table_init: a tensor's buffer is not aligned to its type");
    }
    if (plan->n_chunks == 0) return ZERO_OK;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    AdRec* rec = static_cast<AdRec*>(table);
    // the records' tensor parts, a strided copy; the rest is filled in on the device
    cudaError_t err = cudaMemcpy2DAsync(rec, sizeof(AdRec), tensors, sizeof(zero_adamw_tensor_t),
                                        sizeof(zero_adamw_tensor_t), (size_t)plan->n_tensors, cudaMemcpyHostToDevice, s);
    if (err == cudaSuccess) {
        k_adamw_places<<<1, 32, 0, s>>>(rec, plan->n_tensors);
        const unsigned grid = (unsigned)(plan->n_tensors < 1024 ? plan->n_tensors : 1024);
        k_adamw_chunks<<<grid, 256, 0, s>>>(rec, plan->n_tensors,
                                            const_cast<int32_t*>(table_of(table, plan->n_tensors).chunk_tensor));
        err = cudaGetLastError();
    }
    if (err == cudaSuccess) err = cudaStreamSynchronize(s);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_adamw_table_init");
}

zero_status_t zero_adamw_check(const zero_adamw_plan_t* plan, const void* table, uint32_t* flag, void* stream)
{
    NvtxRange range("zero_adamw_check");
    const zero_status_t st = check_adamw_plan(plan, table);
    if (st != ZERO_OK) return st;
    if (!flag) return set_error(ZERO_ENOMEM, "zero_adamw_check: flag is NULL");
    if (!aligned_to(flag, 4)) return set_error(ZERO_EALIGN, "zero_adamw_check: flag is not 4-byte aligned");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaMemsetAsync(flag, 0, 4, s);
    if (err == cudaSuccess && plan->n_chunks) {
        const AdTable tab = table_of(table, plan->n_tensors);
        const unsigned grid = (unsigned)plan->n_chunks;
        if (plan->dtype == ZERO_FP32)
            k_adamw_check<kF32><<<grid, kAd32Threads, 0, s>>>(tab, flag);
        else if (plan->dtype == ZERO_BF16)
            k_adamw_check<kBF16><<<grid, kAd32Threads, 0, s>>>(tab, flag);
        else
            k_adamw_check<kF16><<<grid, kAd32Threads, 0, s>>>(tab, flag);
        err = cudaGetLastError();
    }
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_adamw_check");
}

zero_status_t zero_adamw_step(const zero_adamw_plan_t* plan, const void* table, const zero_adamw_t* hp,
                              const uint32_t* skip, void* stream)
{
    NvtxRange range("zero_adamw_step");
    return adamw_step(plan, table, hp, nullptr, skip, stream);
}

zero_status_t zero_adamw_step_clipped(const zero_adamw_plan_t* plan, const void* table, const zero_adamw_t* hp,
                                      const float* norm, const uint32_t* skip, void* stream)
{
    NvtxRange range("zero_adamw_step_clipped");
    if (!norm) return set_error(ZERO_ENOMEM, "zero_adamw_step_clipped: norm is NULL");
    if (!aligned_to(norm, 4)) return set_error(ZERO_EALIGN, "zero_adamw_step_clipped: norm is not 4-byte aligned");
    return adamw_step(plan, table, hp, norm, skip, stream);
}

zero_status_t zero_adamw_norm_workspace(const zero_adamw_plan_t* plan, int64_t* bytes)
{
    if (!plan) return set_error(ZERO_EINVAL, "AdamW plan is NULL");
    if (!bytes) return set_error(ZERO_EINVAL, "zero_adamw_norm_workspace: bytes is NULL");
    if (plan->mark != mark_of(*plan)) return set_error(ZERO_EINVAL, "AdamW plan was not made by zero_adamw_plan");
    *bytes = norm_blocks(*plan) * (int64_t)sizeof(NormPart);
    return ZERO_OK;
}

zero_status_t zero_adamw_norm(const zero_adamw_plan_t* plan, const void* table, float grad_scale, float max_norm,
                              float* norm, uint32_t* flag, void* workspace, void* stream)
{
    NvtxRange range("zero_adamw_norm");
    const zero_status_t st = check_adamw_plan(plan, table);
    if (st != ZERO_OK) return st;
    if (!std::isfinite(grad_scale)) return set_error(ZERO_EINVAL, "zero_adamw_norm: grad_scale is not finite");
    if (std::isnan(max_norm)) return set_error(ZERO_EINVAL, "zero_adamw_norm: max_norm is NaN");
    if (!norm || !workspace) return set_error(ZERO_ENOMEM, "zero_adamw_norm: norm or workspace is NULL");
    if (!aligned_to(norm, 4) || !aligned_to(flag, 4) || !aligned_to(workspace, 16))
        return set_error(ZERO_EALIGN, "zero_adamw_norm: norm and flag must be 4-byte aligned, workspace 16-byte");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const AdTable tab = table_of(table, plan->n_tensors);
    const NormOut o{static_cast<NormPart*>(workspace), norm, flag, std::fabs((double)grad_scale),
                    max_norm > 0.0f && std::isfinite(max_norm) ? (double)max_norm : 0.0};
    const unsigned grid = (unsigned)norm_blocks(*plan);
    cudaError_t err = plan->dtype == ZERO_FP32   ? launch_norm<kF32>(tab, plan->n_chunks, o, grid, s)
                      : plan->dtype == ZERO_BF16 ? launch_norm<kBF16>(tab, plan->n_chunks, o, grid, s)
                                                 : launch_norm<kF16>(tab, plan->n_chunks, o, grid, s);
    if (err == cudaSuccess && grid > 1) err = launch_after(k_adamw_norm_join, dim3(1), kNormThreads, 0, s, (int)grid, o);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_adamw_norm");
}

zero_status_t zero_adamw_clip(const zero_adamw_plan_t* plan, const void* table, const float* norm, void* stream)
{
    NvtxRange range("zero_adamw_clip");
    const zero_status_t st = check_adamw_plan(plan, table);
    if (st != ZERO_OK) return st;
    if (!norm) return set_error(ZERO_ENOMEM, "zero_adamw_clip: norm is NULL");
    if (!aligned_to(norm, 4)) return set_error(ZERO_EALIGN, "zero_adamw_clip: norm is not 4-byte aligned");
    if (plan->n_chunks == 0) return ZERO_OK;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const AdTable tab = table_of(table, plan->n_tensors);
    const dim3 grid((unsigned)plan->n_chunks);
    const auto kernel = plan->dtype == ZERO_FP32   ? k_adamw_clip<kF32>
                        : plan->dtype == ZERO_BF16 ? k_adamw_clip<kBF16>
                                                   : k_adamw_clip<kF16>;
    const cudaError_t err = launch_after(kernel, grid, kAd32Threads, 0, s, tab, norm);
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_adamw_clip");
}

zero_status_t zero_adamw_states(const zero_adamw_plan_t* plan, const void* table, void* m, void* root_v, void* stream)
{
    NvtxRange range("zero_adamw_states");
    const zero_status_t st = check_adamw_plan(plan, table);
    if (st != ZERO_OK) return st;
    if (plan->state_bits != 8) return set_error(ZERO_EINVAL, "zero_adamw_states: the list's moments are binary32");
    if (plan->n_chunks == 0) return ZERO_OK;
    if (!m || !root_v) return set_error(ZERO_ENOMEM, "zero_adamw_states: an output is NULL");
    if (!aligned_to(m, 16) || !aligned_to(root_v, 16))
        return set_error(ZERO_EALIGN, "zero_adamw_states: an output is not 16-byte aligned");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    k_adamw_states<<<(unsigned)plan->n_chunks, kStateThreads, 0, s>>>(table_of(table, plan->n_tensors),
                                                                   static_cast<uint16_t*>(m),
                                                                   static_cast<uint16_t*>(root_v));
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? ZERO_OK : cuda_failed(err, "zero_adamw_states");
}

}  // extern "C"
