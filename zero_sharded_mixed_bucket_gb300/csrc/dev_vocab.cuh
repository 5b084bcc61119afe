// Products over a large vocabulary on the tensor cores, as cross entropy and log
// probabilities use them: logits with a softmax epilogue, G, dx, dw; their host
// side.
#pragma once

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "dev_common.cuh"
#include "dev_tc.cuh"

namespace zg {
namespace vocab {

constexpr int kBM = 256, kBN = 256, kBK = 64;         // a pair's tile, K-values per stage
constexpr int kStages = 6;
constexpr int kABytes = kBM / 2 * kBK * 2, kBBytes = kBN / 2 * kBK * 2;   // one CTA's part of a stage
constexpr int kEpiWarps = 8;
constexpr int kCeThreads = 64 + 32 * kEpiWarps;       // copying warp, issuing warp, epilogue warps
constexpr int kOutBytes = 4096;                       // an epilogue warp's box of results: 32 rows of 128 bytes
constexpr int kCeSmem = kStages * (kABytes + kBBytes) + kEpiWarps * kOutBytes + 1024;
constexpr int kStrip = kBN / 2;                       // vocabulary entries per (maximum, sum)
constexpr int kChunk = 16, kChunkFew = 8;             // K-blocks the tensor cores add up by themselves
constexpr int kGroup = 8;                             // row tiles that share the column tiles in L2
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kFewTokens = 3, kFewThreads = 256, kFewBlocks = 456;   // tokens with a kernel of their own
constexpr int kFewSmem = 64 * 1024;                   // all tokens' values, 16 bits each

// Epilogues: softmax statistics; G of cross entropy; binary32 sums; 16-bit results
// times alpha; statistics with the entropy's sum, and besides all logits, or those of
// strips that reach a bound; G of log probabilities and entropies.
enum { kEpiLse, kEpiGrad, kEpiAcc, kEpiOut, kEpiStat, kEpiKeep, kEpiSome, kEpiLpGrad };

// Workspace head.
struct CeHead {
    uint32_t err;                // a bounded wait ran out
    float alpha;                 // gradients are alpha times the products with G
    uint32_t joined;             // blocks of k_ce_join that are done
    uint32_t pad[61];
};

struct GemmArgs {
    CUtensorMap a, b;
    CUtensorMap c;               // results: G, binary32 sums or logits, or rounded gradients
    int64_t m, n;                // rows, columns of the product that exist
    int m_tiles, n_tiles;
    int k_blocks;                // K-blocks in all
    int chunk;                   // of them added up in tensor memory at one go
    int splits;                  // parts of the K-blocks, one result each (kEpiAcc), m_tiles * kBM rows apart
    int b_y0;                    // first vocabulary entry of the piece
    int accumulate;              // kEpiAcc: added to what is there
    int a_rows;                  // rows of A that a CTA copies: 128, or fewer for one row tile of few tokens (the
                                 //   others' results are not kept, so their operands may be anything)
    int withhold;                // test hook (environment ZERO_TEST_WITHHOLD_TILE): the first copy is announced but
                                 //   not made, so the waits run out
    CeHead* head;
    const int64_t* targets;
    float2* part;                // kEpiLse: [strips][m], a strip's maximum and sum
    float* target_logit;         //   [m]
    const float* lse;            // kEpiGrad
    const float* coef;           //   row factors of G, 0: no loss
    int64_t c_cols;              //   columns of G in memory
    uint16_t* out;               // kEpiOut: stored from registers, when a row's end is not on 16 bytes (else NULL)
    int64_t out_stride;
    float scale_log2e;           // log probabilities: the logits' scale times log2 e
    float* part_t;               // log probabilities' statistics: [strips][m], a strip's sum of e (z - maximum)
    const float* coef_h;         // kEpiLpGrad: row factors of the entropy's gradient (NULL: none)
    const float* entropy;        //   [m]
    const float* least;          // kEpiSome: [m], the rows' bounds
    float* logits;               //   [m][logit_stride], of this product's first entry on
    int64_t logit_stride;        //   a multiple of kStrip
};

template <int DT>
__device__ __forceinline__ void unpack8(uint4 v, float f[8])
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float2 p = to_f32x2<DT>(u[k]);
        f[2 * k] = p.x;
        f[2 * k + 1] = p.y;
    }
}

// Alternatives in their order as whole numbers: by logit, then the lower index first.
__device__ __forceinline__ uint64_t key_of(float z, uint32_t index)
{
    const uint32_t u = __float_as_uint(z + 0.0f);     // one zero
    return (uint64_t)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (0xffffffffu - index);
}

__device__ __forceinline__ float logit_of(uint64_t key)
{
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Tile {
    int split, mt, nt, kb0, kb1;
};

// Tile of a place in the order: splits outermost, then groups of kGroup row
// tiles, then column tiles, so that the tiles running at one time share rows
// of A and of B in L2.  32-bit arithmetic: with one K-block to a tile the 64-bit
// divisions of three roles were in the way.
__device__ __forceinline__ Tile tile_at(const GemmArgs& g, uint32_t t)
{
    const uint32_t per = (uint32_t)g.m_tiles * (uint32_t)g.n_tiles, grouped = kGroup * (uint32_t)g.n_tiles;
    Tile r;
    r.split = g.splits == 1 ? 0 : (int)(t / per);
    t -= (uint32_t)r.split * per;
    const uint32_t group = t / grouped, in = t - group * grouped;
    const uint32_t rows = min((uint32_t)kGroup, (uint32_t)g.m_tiles - group * kGroup);
    r.nt = (int)(in / rows);
    r.mt = (int)(group * kGroup + in - (uint32_t)r.nt * rows);
    r.kb0 = g.splits == 1 ? 0 : (int)((uint64_t)g.k_blocks * r.split / g.splits);
    r.kb1 = g.splits == 1 ? g.k_blocks : (int)((uint64_t)g.k_blocks * (r.split + 1) / g.splits);
    return r;
}

// A strip's statistics for log probabilities; its maximum.  Entropy is log S - T / S of
// S = sum e and T = sum e (z - max): neither is a difference of large numbers, so a
// likely token's keeps its digits.  Two instructions a logit more than the loss: 8192
// x 50257 x 768 384 us, the loss 382-400.
__device__ __forceinline__ float lp_statistics(const GemmArgs& g, const float (&z)[kStrip], int strip, int64_t row, bool live)
{
    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < kStrip; k++)
        m4[k & 3] = fmaxf(m4[k & 3], z[k]);
    const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    // (z - top) first: the largest term is exactly 1; held finite beside a term of 0
    const float ref = top == -INFINITY ? 0.0f : top;
    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f}, t4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kStrip; k++) {
        const float d = z[k] - ref, e = exp2_fast(d * g.scale_log2e);
        s4[k & 3] += e;
        t4[k & 3] = fmaf(e, fmaxf(d, -3e38f), t4[k & 3]);
    }
    if (live) {
        g.part[(int64_t)strip * g.m + row] = make_float2(top, (s4[0] + s4[1]) + (s4[2] + s4[3]));
        g.part_t[(int64_t)strip * g.m + row] = (t4[0] + t4[1]) + (t4[2] + t4[3]);
    }
    return top;
}

// C = A B^T for 256 x 256 tiles, a pair of CTAs per tile, each pair striding
// over the tiles.  One thread per CTA copies the CTA's half of A's rows and of
// B's through a ring of kStages stages; one thread of the pair issues the
// products, which accumulate in one of two halves of tensor memory while the
// epilogue warps read the other.  Every wait is bounded; one that runs out
// sets head->err and ends its role, and the others run out in turn.
//
// Bound by the tensor cores, and at length by the power they take: the logits
// of 8192 tokens, hidden 4096, vocabulary 50257 take 1.77 ms alone (1905
// TFLOP/s) and 1.91 ms in a loop (1766; the same bfloat16 product in a library
// sustains 1714).  256 x 256 by a pair halves what each SM reads of B and what L2
// delivers, beside 128 x 256 by one CTA with its epilogue in line (11.8 ms for
// loss and gradients, then 9.9); results through shared memory as tiled copies
// in place of 2-byte stores: 8.4 ms.  With few tokens w's bytes bound it.
//
// A chunk is the K-range that is accumulated in tensor memory at one go: the
// tensor cores cut their binary32 sums toward zero at every step, 256 steps
// along K = 4096, which is off by 1e-6 of the loss; so chunks of kChunk K-blocks
// are added in registers, rounding to nearest (2.6e-7).  In the gradients one
// chain over all of K took 8e-4 off a dw of 131072 tokens whose products have one
// sign, half a unit in binary16's last place, and left p - 1 of a confident
// token at hidden 4096 off by 1.5e-4: there z has to be the sum that lse was made
// from.  Where lse comes from k_ce_few, whose sums are another's, G's chunks
// are kChunkFew K-blocks, so that what is cut stays at 1e-5 of such a token.
// The chunks cost the backward pass 1 to 1.5 % (8192 tokens: 6.19 ms at hidden
// 4096, 6.10 in one chain; 1.23 and 1.21 at 768).
template <int EPI, int DT, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kCeThreads, 1) k_ce_gemm(const __grid_constant__ GemmArgs g)
{
    extern __shared__ unsigned char sm_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
    __shared__ uint32_t s_tmem;
    const uint32_t sm = (tc::smem_addr(sm_raw) + 1023u) & ~1023u;
    const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kStages;
    const uint32_t acc_full = full + 16 * kStages, acc_empty = acc_full + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            tc::mbar_init(full + 8 * s, 1);
            tc::mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; s++) {
            tc::mbar_init(acc_full + 8 * s, 1);
            tc::mbar_init(acc_empty + 8 * s, 2 * kEpiWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_addr(&s_tmem), 2 * kBN);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
    wait_prev_grid();                                 // set up while the kernel before drains; this call's kernels
    allow_next_grid();                                // all wait for their predecessor before they read or write
    const uint32_t tmem = s_tmem;
    const uint32_t tiles = (uint32_t)g.m_tiles * (uint32_t)g.n_tiles * (uint32_t)g.splits;   // below 2^31: see the plan
    const uint32_t first = blockIdx.x >> 1, stride = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int it = 0;
            const uint32_t lead_full = tc::in_leader(full);
            for (uint32_t t = first; t < tiles && ok; t += stride) {
                const Tile w = tile_at(g, t);
                const int m0 = w.mt * kBM + (int)rank * (kBM / 2), n0 = w.nt * kBN + (int)rank * (kBN / 2);
                for (int kb = w.kb0; kb < w.kb1; kb++, it++) {
                    const int s = it % kStages;
                    if (!tc::mbar_wait(empty + 8 * s, ((it / kStages) & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = lead_full + 8 * s;
                    const uint32_t sa = sm + s * (kABytes + kBBytes), sb = sa + kABytes;
                    const bool copies_a = rank == 0 || g.a_rows == kBM / 2;
                    if (rank == 0) {
                        const uint32_t a_bytes = g.a_rows == kBM / 2 ? 2 * kABytes : (uint32_t)g.a_rows * (kBK * 2);
                        tc::mbar_arrive_expect_tx(full + 8 * s, a_bytes + 2 * kBBytes);
                        if (g.withhold && blockIdx.x == 0 && it == 0) continue;
                    }
                    if (A_MN) {
#pragma unroll
                        for (int j = 0; j < kBM / 128; j++)
                            tc::tma_load(sa + j * tc::kBoxBytes, &g.a, m0 + 64 * j, kb * kBK, bar);
                    } else if (copies_a) {
                        tc::tma_load(sa, &g.a, kb * kBK, m0, bar);
                    }
                    if (B_MN) {
#pragma unroll
                        for (int j = 0; j < kBN / 128; j++)
                            tc::tma_load(sb + j * tc::kBoxBytes, &g.b, n0 + 64 * j, g.b_y0 + kb * kBK, bar);
                    } else {
                        tc::tma_load(sb, &g.b, kb * kBK, g.b_y0 + n0, bar);
                    }
                }
            }
            if (!ok) {
                // the copies in flight have landed before the pair exits (when
                // all went well the epilogue has seen every product done)
                atomicOr(&g.head->err, 1u);
                if (rank == 0)
                    for (int j = it - kStages < 0 ? 0 : it - kStages; j < it; j++)
                        tc::mbar_wait(full + 8 * (j % kStages), (j / kStages) & 1);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = tc::instr_desc<DT == kBF16, A_MN, B_MN>(kBM, kBN);
            int it = 0, unit = 0;
            bool ok = true;
            for (uint32_t t = first; t < tiles && ok; t += stride) {
                const Tile w = tile_at(g, t);
                for (int c0 = w.kb0; c0 < w.kb1 && ok; c0 += g.chunk, unit++) {
                    const int buf = unit & 1;
                    if (!tc::mbar_wait(acc_empty + 8 * buf, ((unit >> 1) & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const int c1 = min(w.kb1, c0 + g.chunk);
                    for (int kb = c0; kb < c1; kb++, it++) {
                        const int s = it % kStages;
                        if (!tc::mbar_wait(full + 8 * s, (it / kStages) & 1)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t sa = sm + s * (kABytes + kBBytes), sb = sa + kABytes;
                        const uint64_t da = tc::operand_desc<A_MN>(sa), db = tc::operand_desc<B_MN>(sb);
#pragma unroll
                        for (int k = 0; k < kBK / 16; k++)
                            tc::mma(tmem + buf * kBN, da + k * tc::kStep16<A_MN>, db + k * tc::kStep16<B_MN>, idesc,
                                    kb > c0 || k > 0);
                        tc::mma_commit(empty + 8 * s);
                    }
                    if (ok) tc::mma_commit(acc_full + 8 * buf);
                }
            }
            if (!ok) atomicOr(&g.head->err, 1u);
        }
    } else {
        const int band = warp & 3;                    // the warp's 32 lanes of tensor memory
        const int half = (warp - 2) >> 2;             // and its 128 columns
        const uint32_t src = tmem + ((uint32_t)(band * 32) << 16) + half * kStrip;
        const uint32_t box = sm + kStages * (kABytes + kBBytes) + (warp - 2) * kOutBytes;
        int unit = 0;
        bool ok = true;
        for (uint32_t t = first; t < tiles && ok; t += stride) {
            const Tile w = tile_at(g, t);
            const int64_t row = (int64_t)w.mt * kBM + rank * (kBM / 2) + band * 32 + lane;
            const bool live = row < g.m;
            const int64_t col0 = (int64_t)w.nt * kBN + half * kStrip;
            float cf = 0.0f, base = 0.0f;
            int tgt = -1;                                 // kEpiGrad: the strip's column that is the row's target
            if constexpr (EPI == kEpiGrad || EPI == kEpiLpGrad) {
                if (live) {
                    cf = g.coef[row];
                    base = g.lse[row] * kLog2e;
                    const int64_t at = g.targets[row] - g.b_y0 - col0;
                    if (cf != 0.0f && at >= 0 && at < kStrip) tgt = (int)at;
                }
            }
            float ch = 0.0f, ent = 0.0f;
            if constexpr (EPI == kEpiLpGrad) {
                if (live && g.coef_h) {
                    ch = g.coef_h[row];
                    if (ch != 0.0f) ent = g.entropy[row];
                }
            }
            // the warp's columns into registers, chunk after chunk, and tensor memory is
            // free again; a part of K may be empty
            float z[kStrip];
            if (w.kb0 == w.kb1) {
#pragma unroll
                for (int k = 0; k < kStrip; k++)
                    z[k] = 0.0f;
            }
            for (int c0 = w.kb0; c0 < w.kb1; c0 += g.chunk, unit++) {
                const int buf = unit & 1;
                ok = __all_sync(0xffffffffu, tc::mbar_wait(acc_full + 8 * buf, (unit >> 1) & 1));
                if (!ok) break;
                tc::fence_after_sync();
                if (c0 == w.kb0) {
#pragma unroll
                    for (int q = 0; q < kStrip / 32; q++)
                        tc::tmem_ld32(src + buf * kBN + 32 * q, reinterpret_cast<uint32_t*>(z) + 32 * q);
                    tc::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int q = 0; q < kStrip / 16; q++) {       // 16 at a time: registers
                        uint32_t r[16];
                        tc::tmem_ld16(src + buf * kBN + 16 * q, r);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; k++)
                            z[16 * q + k] += __uint_as_float(r[k]);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_leader(acc_empty + 8 * buf);
            }
            if (!ok) break;
            if constexpr (EPI == kEpiLse || EPI == kEpiStat || EPI == kEpiKeep || EPI == kEpiSome) {
                // the strip's maximum and its sum
                const int64_t left = g.n - col0;
                if (left < kStrip) {
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        if (k >= left) z[k] = -INFINITY;
                }
                const int64_t at = (live ? g.targets[row] : -1) - g.b_y0 - col0;
                const bool here = at >= 0 && at < kStrip && at < left;
                if (__any_sync(0xffffffffu, here)) {
                    float zt = 0.0f;
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        if (k == at) zt = z[k];
                    if (here) g.target_logit[row] = zt;
                }
                if constexpr (EPI == kEpiLse) {
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        m4[k & 3] = fmaxf(m4[k & 3], z[k]);
                    const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    // (z - top) first: the largest term is exactly 1
                    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        s4[k & 3] += exp2_fast((z[k] - ref) * kLog2e);
                    if (live)
                        g.part[((int64_t)w.nt * 2 + half) * g.m + row] = make_float2(top, (s4[0] + s4[1]) + (s4[2] + s4[3]));
                } else {
                    const float top = lp_statistics(g, z, w.nt * 2 + half, row, live);
                    if constexpr (EPI == kEpiSome) {
                        // a row's strip is its lane's alone, 512 bytes, which few rows have to write
                        const bool in = live && left > 0 && top >= g.least[row];
                        if (__any_sync(0xffffffffu, in)) {
                            float* dst = g.logits + row * g.logit_stride + col0;
#pragma unroll
                            for (int k = 0; k < kStrip; k += 4)
                                if (in) *reinterpret_cast<float4*>(dst + k) = make_float4(z[k], z[k + 1], z[k + 2], z[k + 3]);
                        }
                    }
                }
            }
            if constexpr (EPI != kEpiLse && EPI != kEpiStat && EPI != kEpiSome) {
                if constexpr (EPI == kEpiGrad) {
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        z[k] = exp2_fast(fmaf(z[k], kLog2e, -base));
                    if (__any_sync(0xffffffffu, tgt >= 0)) {
#pragma unroll
                        for (int k = 0; k < kStrip; k++)
                            if (k == tgt) z[k] -= 1.0f;
                    }
                    const int64_t left = g.n - col0;  // columns that exist
                    if (left < kStrip) {
#pragma unroll
                        for (int k = 0; k < kStrip; k++)
                            if (k >= left) z[k] = 0.0f;
                    }
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        z[k] *= cf;
                } else if constexpr (EPI == kEpiLpGrad) {
                    // a ([v = t] - p) - b p (log p + H); p is 0 below 2^-200, whatever its logarithm
                    if (g.coef_h) {
                        const float ca = fmaf(ch, ent, cf), cb = ch * kLn2;
#pragma unroll
                        for (int k = 0; k < kStrip; k++) {
                            const float l2 = fmaf(z[k], g.scale_log2e, -base);
                            z[k] = -exp2_fast(l2) * fmaf(cb, fmaxf(l2, -200.0f), ca);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < kStrip; k++)
                            z[k] = -exp2_fast(fmaf(z[k], g.scale_log2e, -base)) * cf;
                    }
                    if (__any_sync(0xffffffffu, tgt >= 0)) {
#pragma unroll
                        for (int k = 0; k < kStrip; k++)
                            if (k == tgt) z[k] += cf;
                    }
                    const int64_t left = g.n - col0;
                    if (left < kStrip) {
#pragma unroll
                        for (int k = 0; k < kStrip; k++)
                            if (k >= left) z[k] = 0.0f;
                    }
                } else if constexpr (EPI == kEpiOut) {
                    const float alpha = g.head->alpha;
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        z[k] *= alpha;
                }
                const uint32_t keep = (EPI == kEpiGrad || EPI == kEpiLpGrad) && cf == 0.0f && ch == 0.0f ? 0u : 0xffffffffu;   // 0 whatever the logit
                if (EPI == kEpiOut && g.out) {
                    // rows that do not end on a 16-byte unit, which is what a tiled copy writes
                    if (live)
#pragma unroll
                        for (int k = 0; k < kStrip; k++)
                            if (col0 + k < g.n) g.out[row * g.out_stride + col0 + k] = (uint16_t)from_f32<DT>(z[k]);
                    continue;
                }
                // the warp's box: 32 rows of 128 bytes with the copy's swizzle (16-byte
                // unit j of row i at j ^ (i & 7): no bank conflicts); one copy out per
                // box (a second box for a stage less: 2 % slower)
                const int row0 = w.mt * kBM + (int)rank * (kBM / 2) + band * 32;
                const int y = row0 + (EPI == kEpiAcc ? w.split * g.m_tiles * kBM : 0);
                constexpr bool kSingle = EPI == kEpiAcc || EPI == kEpiKeep;       // binary32
                constexpr int kCols = kSingle ? 32 : 64;              // columns of a box
#pragma unroll
                for (int c = 0; c < kStrip; c += kCols) {
                    if (lane == 0) tc::bulk_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const uint32_t at = box + lane * 128 + ((k ^ (lane & 7)) << 4);
                        if constexpr (kSingle) {
                            const float* p = z + c + 4 * k;
                            tc::st_shared16(at, __float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]),
                                            __float_as_uint(p[3]));
                        } else {
                            const float* p = z + c + 8 * k;
                            tc::st_shared16(at, from_f32x2<DT>(p[0], p[1]) & keep, from_f32x2<DT>(p[2], p[3]) & keep,
                                            from_f32x2<DT>(p[4], p[5]) & keep, from_f32x2<DT>(p[6], p[7]) & keep);
                        }
                    }
                    tc::fence_async_shared();
                    __syncwarp();
                    const int64_t x = col0 + c;
                    if (lane == 0 && row0 < g.m && x < (EPI == kEpiGrad || EPI == kEpiLpGrad ? g.c_cols : g.n)) {
                        if (EPI == kEpiAcc && g.accumulate)
                            tc::tma_add(&g.c, (int)x, y, box);
                        else
                            tc::tma_store(&g.c, (int)x, y, box);
                        tc::bulk_commit();
                    }
                }
            }
        }
        if (lane == 0) tc::bulk_wait_all();
        if (!ok && lane == 0) atomicOr(&g.head->err, 1u);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_free(tmem, 2 * kBN);
}

// A gradient that a timed-out product left incomplete, or did not write at all.
struct Spoiled {
    uint16_t* out;               // NULL: none
    int64_t rows, cols, stride;
};

__device__ __forceinline__ void spoil(const CeHead* head, const Spoiled& o)
{
    if (!o.out || !head->err) return;
    for (int64_t i = blockIdx.y; i < o.rows; i += gridDim.y)
        for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < o.cols; c += (int64_t)gridDim.x * 256)
            o.out[i * o.stride + c] = 0x7fff;                     // NaN in both types
}

static __global__ void __launch_bounds__(256) k_ce_spoil(const CeHead* head, const Spoiled o)
{
    wait_prev_grid();
    spoil(head, o);
}

// dx (or dw, where its product is split): alpha times the sum of the splits,
// rounded; 4 columns a thread, a row a blockIdx.y stride.  coef (and coef_h): dx's
// row factors; a row whose factors are 0 is 0, also where w holds infinities, whose
// products with G's zeros are NaN.  The last kernel of a backward pass also
// turns dw into NaN if a wait ran out (dx is by way of alpha).
template <int DT>
__global__ void __launch_bounds__(256) k_ce_sum(const CeHead* head, const float* acc, int splits, int64_t split_stride,
                                               int64_t m, int64_t n, int64_t acc_cols, const float* coef, const float* coef_h,
                                               uint16_t* out, int64_t stride, const Spoiled dw)
{
    wait_prev_grid();
    spoil(head, dw);
    const float alpha = head->err ? NAN : head->alpha;
    const int64_t c = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (c >= n) return;
    for (int64_t i = blockIdx.y; i < m; i += gridDim.y) {
        const float* src = acc + i * acc_cols + c;
        float4 s = __ldcs(reinterpret_cast<const float4*>(src));
        for (int k = 1; k < splits; k++) {
            const float4 q = __ldcs(reinterpret_cast<const float4*>(src + k * split_stride));
            s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
        }
        uint2 h = make_uint2(from_f32x2<DT>(s.x * alpha, s.y * alpha), from_f32x2<DT>(s.z * alpha, s.w * alpha));
        if (coef && coef[i] == 0.0f && (!coef_h || coef_h[i] == 0.0f) && alpha == alpha) h = make_uint2(0, 0);
        uint16_t* dst = out + i * stride + c;
        if (c + 4 <= n) {
            *reinterpret_cast<uint2*>(dst) = h;
        } else {
            dst[0] = (uint16_t)h.x;
            if (c + 1 < n) dst[1] = (uint16_t)(h.x >> 16);
            if (c + 2 < n) dst[2] = (uint16_t)h.y;
        }
    }
}

static __global__ void __launch_bounds__(256) k_ce_zero(uint16_t* p, int64_t rows, int64_t cols, int64_t stride)
{
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < rows * cols; e += (int64_t)gridDim.x * 256)
        p[e / cols * stride + e % cols] = 0;
}

// Logits of up to kFewTokens tokens, by multiply-adds: the tokens lie in shared memory
// (xs: T rows of hidden, rounded up to 8), a warp takes a row of w at a time (3
// tokens: two, which share the unpacked tokens), neighbouring warps neighbouring rows,
// U 16-byte loads of a lane on their way.  each(v, z): the tokens' logits of entry v, in all
// lanes, entry after entry of the warp's; target_logit [T]: those of the targets.
template <int DT, int T, typename EACH>
__device__ __forceinline__ void few_logits(const uint16_t* x, int64_t x_stride, const uint16_t* w, int64_t w_stride,
                                           int64_t hidden, int64_t vocab, const int64_t* targets, uint16_t* xs,
                                           float* target_logit, EACH each)
{
    constexpr int R = T <= 2 ? 1 : 2, U = 8 / R;      // rows at a time, loads in flight per row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wide = (int)((hidden + 7) / 8 * 8);
#pragma unroll
    for (int t = 0; t < T; t++)
        for (int j = threadIdx.x * 8; j < wide; j += kFewThreads * 8) {
            const uint16_t* p = x + t * x_stride + j;
            if (j + 8 <= hidden) {
                *reinterpret_cast<uint4*>(xs + t * wide + j) = *reinterpret_cast<const uint4*>(p);
            } else {
                for (int k = 0; k < 8; k++)
                    xs[t * wide + j + k] = j + k < hidden ? p[k] : (uint16_t)0;
            }
        }
    __syncthreads();
    const int64_t warps = (int64_t)gridDim.x * (kFewThreads / 32), me = (int64_t)blockIdx.x * (kFewThreads / 32) + warp;
    for (int64_t v = me * R; v < vocab; v += warps * R) {
        const uint16_t* row[R];
        float acc[R][T];
#pragma unroll
        for (int q = 0; q < R; q++) {
            row[q] = w + min(v + q, vocab - 1) * w_stride;
#pragma unroll
            for (int t = 0; t < T; t++)
                acc[q][t] = 0.0f;
        }
        auto add = [&](const uint4 r[R], int j) {
            float wv[R][8];
#pragma unroll
            for (int q = 0; q < R; q++)
                unpack8<DT>(r[q], wv[q]);
#pragma unroll
            for (int t = 0; t < T; t++) {
                float xv[8];
                unpack8<DT>(*reinterpret_cast<const uint4*>(xs + t * wide + j), xv);
#pragma unroll
                for (int q = 0; q < R; q++)
#pragma unroll
                    for (int k = 0; k < 8; k++)
                        acc[q][t] = fmaf(wv[q][k], xv[k], acc[q][t]);
            }
        };
        int j = lane * 8;
        for (; j + 8 <= hidden; j += 256 * U) {
            uint4 r[U][R];                            // all loads before any use; 0 past the row's end
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int q = 0; q < R; q++)
                    r[u][q] = j + 256 * u + 8 <= hidden ? __ldcs(reinterpret_cast<const uint4*>(row[q] + j + 256 * u))
                                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; u++)
                if (j + 256 * u + 8 <= hidden) add(r[u], j + 256 * u);
        }
        if (lane == (hidden / 8) % 32 && hidden % 8) {    // the rows' ragged end
            const int e = (int)(hidden / 8 * 8);
            uint4 r[R];
#pragma unroll
            for (int q = 0; q < R; q++) {
                uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < 8; k++)
                    if (e + k < hidden) u[k >> 1] |= (uint32_t)row[q][e + k] << ((k & 1) * 16);
                r[q] = make_uint4(u[0], u[1], u[2], u[3]);
            }
            add(r, e);
        }
#pragma unroll
        for (int q = 0; q < R; q++) {
            if (v + q >= vocab) break;
            float z[T];
#pragma unroll
            for (int t = 0; t < T; t++) {
                z[t] = acc[q][t];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    z[t] += __shfl_xor_sync(0xffffffffu, z[t], o);
                if (lane == 0 && v + q == targets[t]) target_logit[t] = z[t];
            }
            each(v + q, z);
        }
    }
}

// ---- host -------------------------------------------------------------------------
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up256(int64_t a) { return (a + 255) / 256 * 256; }

// The forward pass of few tokens has its own kernel.
inline bool few_tokens(const zero_ce_plan_t& p)
{
    return p.tokens <= kFewTokens && p.tokens * ((p.hidden + 7) / 8 * 8) * 2 <= kFewSmem;
}

// Its blocks: three to an SM of 152, and no more than give every warp a row.
inline int64_t few_blocks(const zero_ce_plan_t& p)
{
    const int64_t most = ceil_div(p.vocab, kFewThreads / 32);
    return most < kFewBlocks ? most : kFewBlocks;
}

// Parts of K, each at least 8 K-blocks, that a product of `tiles` tiles is summed
// in until its tiles fill the 76 pairs of SMs.
inline int64_t parts_of(int64_t tiles, int64_t blocks)
{
    int64_t best = 1;
    double cost = 1e30;
    for (int64_t s = 1; s <= 32 && s * 8 <= blocks; s++) {
        const double c = (double)ceil_div(tiles * s, 76) / (double)s * (1.0 + 0.01 * (double)s);
        if (c < cost * 0.97) {
            cost = c;
            best = s;
        }
    }
    return best;
}

// dw's, whose K are the tokens: in parts where half of the pairs would idle, so
// with a small vocabulary (16384 tokens, hidden 768, vocabulary 256: the backward
// pass takes 70 us, 138 in one part; 4096 tokens, hidden 512, vocabulary 1000: 44
// and 58); else its tiles are rounded where they are.
inline int64_t dw_parts(const zero_ce_plan_t& p)
{
    const int64_t tiles = ceil_div(p.piece, kBM) * ceil_div(p.hidden, kBN);
    return tiles <= 38 ? parts_of(tiles, ceil_div(p.tokens, kBK)) : 1;
}

// Byte offsets in the workspace.
struct CeLayout {
    int64_t coef, target_logit, block_total, part, g, acc, acc_w, end;
    int64_t acc_rows, acc_cols;                       // of one split's binary32 sums
};

inline CeLayout layout_of(const zero_ce_plan_t& p)
{
    CeLayout l;
    l.coef = sizeof(CeHead);
    l.target_logit = l.coef + up256(p.tokens * 4);
    l.block_total = l.target_logit + up256(p.tokens * 4);
    l.part = l.block_total + up256(ceil_div(p.tokens, 32) * 8);
    l.g = l.part;                                     // the two passes do not meet
    l.acc = l.g + up256(p.tokens * p.piece * 2);
    const int64_t fwd = l.part + (few_tokens(p) ? few_blocks(p) : ceil_div(p.vocab, kBN) * 2) * p.tokens * 8;
    l.acc_rows = ceil_div(p.tokens, kBM) * kBM;
    l.acc_cols = (p.hidden + 3) / 4 * 4;
    l.acc_w = l.acc + up256(p.splits * l.acc_rows * l.acc_cols * 4);
    const int64_t parts = dw_parts(p), bwd = l.acc_w + (parts > 1 ? parts * p.piece * l.acc_cols * 4 : 0);
    l.end = up256(fwd > bwd ? fwd : bwd);
    return l;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn()
{
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// rows x cols values, `stride` values between rows; boxes of 128 bytes of
// columns x box_rows rows, 128-byte swizzle; zeros outside.
inline bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t rows, int64_t cols, int64_t stride,
              int box_rows)
{
    const int e = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * e};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / e), (cuuint32_t)box_rows}, step[2] = {1, 1};
    return encode_fn()(map, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline CUtensorMapDataType map_type(int dtype)
{
    return dtype == ZERO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// GemmArgs::a_rows where the rows of A are tokens.
inline int a_rows_of(int64_t tokens) { return tokens >= kBM / 2 ? kBM / 2 : (int)((tokens + 7) / 8 * 8); }

inline int sm_count()
{
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 1 ? n : 152;
}

// Test hook: which product's first copy is withheld: 0 none, 1 the logits', 2 dw's.
inline int withheld_product()
{
    const char* v = std::getenv("ZERO_TEST_WITHHOLD_TILE");
    return !v ? 0 : v[0] == '2' ? 2 : 1;
}

template <int EPI, int DT, bool A_MN, bool B_MN>
cudaError_t launch_gemm(const GemmArgs& g, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem((const void*)k_ce_gemm<EPI, DT, A_MN, B_MN>, kCeSmem, done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)g.m_tiles * g.n_tiles * g.splits;
    const int64_t pairs = sm_count() / 2;
    return launch_after(k_ce_gemm<EPI, DT, A_MN, B_MN>, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), kCeThreads,
                        kCeSmem, s, g);
}

inline cudaError_t launch_sum(int dtype, const CeHead* head, const float* acc, int splits, int64_t apart, int64_t rows, int64_t cols,
                       int64_t acc_cols, const float* coef, const float* coef_h, uint16_t* out, int64_t stride, const Spoiled& dw, cudaStream_t s)
{
    const dim3 grid((unsigned)ceil_div(acc_cols, 1024), (unsigned)(rows < 4096 ? rows : 4096));
    return launch_after(dtype == ZERO_BF16 ? k_ce_sum<kBF16> : k_ce_sum<kF16>, grid, 256, 0, s, head, acc, splits, apart, rows,
                        cols, acc_cols, coef, coef_h, out, stride, dw);
}

template <int EPI, bool A_MN, bool B_MN>
cudaError_t gemm(int dtype, const GemmArgs& g, cudaStream_t s)
{
    return dtype == ZERO_BF16 ? launch_gemm<EPI, kBF16, A_MN, B_MN>(g, s) : launch_gemm<EPI, kF16, A_MN, B_MN>(g, s);
}

// The gradients' products, a piece of the vocabulary at a time: G (its epilogue EPI,
// whose fields base has), dx += G w, dw = G^T x; then dx rounded, and dw turned
// into NaN if a wait ran out.  ok: false if a tensor map was refused.
template <int EPI>
cudaError_t launch_gradients(const zero_ce_plan_t& p, const CeLayout& l, const GemmArgs& base, const void* x, const void* w,
                             void* dx, void* dw, unsigned char* ws, cudaStream_t s, bool& ok)
{
    uint16_t* G = reinterpret_cast<uint16_t*>(ws + l.g);
    float* acc = reinterpret_cast<float*>(ws + l.acc);
    const CUtensorMapDataType type = map_type(p.dtype);
    const int withheld = withheld_product();
    cudaError_t e = cudaSuccess;
    for (int64_t v0 = 0; v0 < p.vocab && e == cudaSuccess; v0 += p.piece) {
        const int64_t nv = p.vocab - v0 < p.piece ? p.vocab - v0 : p.piece;
        GemmArgs g = base;                           // G of the piece
        g.a_rows = a_rows_of(p.tokens);
        ok = make_map(&g.a, type, x, p.tokens, p.hidden, p.x_stride, g.a_rows) &&
                  make_map(&g.b, type, w, p.vocab, p.hidden, p.w_stride, kBN / 2) &&
                  make_map(&g.c, type, G, p.tokens, p.piece, p.piece, 32);
        g.m = p.tokens;
        g.n = nv;
        g.c_cols = p.piece;
        g.m_tiles = (int)ceil_div(p.tokens, kBM);
        g.n_tiles = (int)ceil_div(nv, kBN);
        g.k_blocks = (int)ceil_div(p.hidden, kBK);
        g.chunk = few_tokens(p) ? kChunkFew : kChunk;
        g.splits = 1;
        g.b_y0 = (int)v0;
        g.withhold = v0 == 0 && withheld == 1;
        if (ok) e = gemm<EPI, false, false>(p.dtype, g, s);
        g.n = p.hidden;
        g.n_tiles = (int)ceil_div(p.hidden, kBN);
        g.chunk = kChunk;
        g.withhold = 0;
        if (ok && dx && e == cudaSuccess) {          // dx += G w
            ok = make_map(&g.a, type, G, p.tokens, p.piece, p.piece, g.a_rows) &&
                 make_map(&g.b, type, w, p.vocab, p.hidden, p.w_stride, 64) &&
                 make_map(&g.c, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, acc, p.splits * l.acc_rows, l.acc_cols, l.acc_cols, 32);
            g.k_blocks = (int)ceil_div(nv, kBK);
            g.splits = p.splits;
            g.accumulate = v0 > 0;
            if (ok) e = gemm<kEpiAcc, false, true>(p.dtype, g, s);
        }
        if (ok && dw && e == cudaSuccess) {          // dw = G^T x
            ok = make_map(&g.a, type, G, p.tokens, p.piece, p.piece, 64) &&
                 make_map(&g.b, type, x, p.tokens, p.hidden, p.x_stride, 64);
            uint16_t* out = static_cast<uint16_t*>(dw) + v0 * p.w_stride;
            g.b_y0 = 0;
            g.a_rows = kBM / 2;
            g.m = nv;
            g.m_tiles = (int)ceil_div(nv, kBM);
            g.k_blocks = (int)ceil_div(p.tokens, kBK);
            g.splits = (int)dw_parts(p);
            g.withhold = v0 == 0 && withheld == 2;
            g.accumulate = 0;
            if (g.splits > 1) {
                float* sums = reinterpret_cast<float*>(ws + l.acc_w);
                const int64_t rows = (int64_t)g.m_tiles * kBM;
                ok = ok && make_map(&g.c, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, sums, g.splits * rows, l.acc_cols, l.acc_cols, 32);
                if (ok) e = gemm<kEpiAcc, true, true>(p.dtype, g, s);
                if (ok && e == cudaSuccess)
                    e = launch_sum(p.dtype, base.head, sums, g.splits, rows * l.acc_cols, nv, p.hidden, l.acc_cols,
                                   nullptr, nullptr, out, p.w_stride, Spoiled{}, s);
            } else {
                ok = ok && make_map(&g.c, type, out, nv, p.hidden, p.w_stride, 32);
                if (p.hidden % 8) {
                    g.out = out;
                    g.out_stride = p.w_stride;
                }
                if (ok) e = gemm<kEpiOut, true, true>(p.dtype, g, s);
            }
        }
        if (!ok) return e;
    }
    const Spoiled all{static_cast<uint16_t*>(dw), p.vocab, p.hidden, p.w_stride};
    if (dx && e == cudaSuccess)
        e = launch_sum(p.dtype, base.head, acc, p.splits, l.acc_rows * l.acc_cols, p.tokens, p.hidden, l.acc_cols, base.coef,
                       base.coef_h, static_cast<uint16_t*>(dx), p.x_stride, all, s);
    else if (e == cudaSuccess)
        e = launch_after(k_ce_spoil, dim3(1, 608), 256, 0, s, static_cast<const CeHead*>(base.head), all);
    return e;
}

}  // namespace vocab
}  // namespace zg
