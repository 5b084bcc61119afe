// Softmax cross entropy over a large vocabulary without stored logits: the
// plan, the three products (logits with a softmax epilogue, dx, dw) on the
// tensor cores, and the small kernels around them.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "dev_common.cuh"
#include "dev_tc.cuh"
#include "nvtx_ranges.h"

namespace zg {
namespace {

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
constexpr float kLog2e = 1.4426950408889634f;

// Epilogues: softmax statistics; G; binary32 sums; 16-bit results times alpha.
enum { kEpiLse, kEpiGrad, kEpiAcc, kEpiOut };

// Workspace head.
struct CeHead {
    uint32_t err;                // a bounded wait ran out
    float alpha;                 // gradients are alpha times the products with G
    uint32_t joined;             // blocks of k_ce_join that are done
    uint32_t pad[61];
};

struct GemmArgs {
    CUtensorMap a, b;
    CUtensorMap c;               // results: G, binary32 sums or rounded gradients
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
};

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
            if constexpr (EPI == kEpiGrad) {
                if (live) {
                    cf = g.coef[row];
                    base = g.lse[row] * kLog2e;
                    const int64_t at = g.targets[row] - g.b_y0 - col0;
                    if (cf != 0.0f && at >= 0 && at < kStrip) tgt = (int)at;
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
            if constexpr (EPI == kEpiLse) {
                // the strip's maximum and its sum
                const int64_t left = g.n - col0;
                if (left < kStrip) {
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        if (k >= left) z[k] = -INFINITY;
                }
                const int64_t at = (live ? g.targets[row] : -1) - col0;
                const bool here = at >= 0 && at < kStrip && at < left;
                if (__any_sync(0xffffffffu, here)) {
                    float zt = 0.0f;
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        if (k == at) zt = z[k];
                    if (here) g.target_logit[row] = zt;
                }
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
                } else if constexpr (EPI == kEpiOut) {
                    const float alpha = g.head->alpha;
#pragma unroll
                    for (int k = 0; k < kStrip; k++)
                        z[k] *= alpha;
                }
                const uint32_t keep = EPI == kEpiGrad && cf == 0.0f ? 0u : 0xffffffffu;   // 0 whatever the logit
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
                constexpr int kCols = EPI == kEpiAcc ? 32 : 64;       // columns of a box
#pragma unroll
                for (int c = 0; c < kStrip; c += kCols) {
                    if (lane == 0) tc::bulk_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const uint32_t at = box + lane * 128 + ((k ^ (lane & 7)) << 4);
                        if constexpr (EPI == kEpiAcc) {
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
                    if (lane == 0 && row0 < g.m && x < (EPI == kEpiGrad ? g.c_cols : g.n)) {
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

// The head cleared, before a forward pass.
__global__ void k_ce_clear(CeHead* head)
{
    allow_next_grid();
    wait_prev_grid();
    head->err = 0;
    head->joined = 0;
}

// Join of (maximum, sum) pairs.
__device__ __forceinline__ void merge(float& mx, float& sum, float2 q)
{
    const float top = fmaxf(mx, q.x), ref = top == -INFINITY ? 0.0f : top;
    sum = fmaf(sum, exp2f((mx - ref) * kLog2e), q.y * exp2f((q.x - ref) * kLog2e));
    mx = top;
}

struct JoinArgs {
    CeHead* head;
    const float2* part;          // [strips][n]
    int strips;
    int64_t n;
    const int64_t* targets;
    int64_t vocab;
    const float* target_logit;
    float* loss;
    float* lse;
    float2* block_total;
    float* total;
};

// lse and loss of token i from its joined maximum and sum.
__device__ __forceinline__ float2 finish_token(const JoinArgs& a, int64_t i, float mx, float sum)
{
    float l = (mx == -INFINITY ? 0.0f : mx) + logf(sum), li = 0.0f, ci = 0.0f;
    if (a.head->err) l = NAN;
    a.lse[i] = l;
    const int64_t t = a.targets[i];
    if (t >= 0 && t < a.vocab) {
        li = l - __ldcg(a.target_logit + i);
        ci = 1.0f;
    }
    a.loss[i] = li;
    return make_float2(li, ci);
}

// Per token: the strips' maxima and sums joined, in a fixed order (32 parts of
// the strips, then a tree over the parts); the loss.  The last block to finish
// adds the blocks' losses and counts, in block order.  8 us for 1023 tokens and
// 393 strips, all of it latency.
__global__ void __launch_bounds__(1024) k_ce_join(const __grid_constant__ JoinArgs a)
{
    wait_prev_grid();
    __shared__ float2 sh[32][33];
    __shared__ uint32_t last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    {
        const int64_t i = (int64_t)blockIdx.x * 32 + lane;        // the warp's part of 32 tokens
        float mx = -INFINITY, sum = 0.0f;
        if (i < a.n)
            for (int s = warp; s < a.strips; s += 128) {
                float2 q[4];
#pragma unroll
                for (int k = 0; k < 4; k++)
                    q[k] = s + 32 * k < a.strips ? a.part[(int64_t)(s + 32 * k) * a.n + i] : make_float2(-INFINITY, 0.0f);
                const float top = fmaxf(fmaxf(fmaxf(q[0].x, q[1].x), fmaxf(q[2].x, q[3].x)), mx);
                const float ref = top == -INFINITY ? 0.0f : top;
                sum *= exp2f((mx - ref) * kLog2e);
#pragma unroll
                for (int k = 0; k < 4; k++)
                    sum = fmaf(q[k].y, exp2f((q[k].x - ref) * kLog2e), sum);
                mx = top;
            }
        sh[warp][lane] = make_float2(mx, sum);
    }
    __syncthreads();
    const int64_t i = (int64_t)blockIdx.x * 32 + warp;            // the warp's token
    float2 r = sh[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float2 q = make_float2(__shfl_xor_sync(0xffffffffu, r.x, o), __shfl_xor_sync(0xffffffffu, r.y, o));
        merge(r.x, r.y, q);
    }
    r = lane == 0 && i < a.n ? finish_token(a, i, r.x, r.y) : make_float2(0.0f, 0.0f);
    __syncthreads();
    if (lane == 0) sh[0][warp] = r;
    __syncthreads();
    if (warp == 0) {
        r = sh[0][lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            r.x += __shfl_down_sync(0xffffffffu, r.x, o);
            r.y += __shfl_down_sync(0xffffffffu, r.y, o);
        }
        if (lane == 0) {
            a.block_total[blockIdx.x] = r;
            __threadfence();
            last = atomicAdd(&a.head->joined, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last || !a.total) return;
    __threadfence();
    float s = 0.0f, c = 0.0f;
    for (unsigned k = threadIdx.x; k < gridDim.x; k += 1024) {
        const float2 q = __ldcg(a.block_total + k);
        s += q.x;
        c += q.y;                                     // at most 2^24 tokens: exact
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_down_sync(0xffffffffu, s, o);
        c += __shfl_down_sync(0xffffffffu, c, o);
    }
    if (lane == 0) sh[0][warp] = make_float2(s, c);
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < 32; k++) {
            s += sh[0][k].x;
            c += sh[0][k].y;
        }
        a.total[0] = c > 0.0f ? s / c : 0.0f;
        a.total[1] = c;
    }
}

// ---- few tokens -------------------------------------------------------------------
// Up to kFewTokens tokens: w is read once and that is the time (411 MB at
// vocabulary 50257, hidden 4096: 61 us at the copy bandwidth), so no tensor
// cores: the tokens lie in shared memory, a warp takes a row of w at a time (3
// tokens: two, which share the unpacked tokens), neighbouring warps
// neighbouring rows, each lane with 128 bytes in flight, 24 warps to an SM.
// Each lane keeps one row's logit; 32 of them at a time go into the warp's
// running maximum and sum.  The last block joins the blocks' pairs.  Products
// and sums are binary32 multiply-adds.  At 4 tokens the multiply-adds bound it
// (90 us at hidden 4096; the tensor cores' path takes 83).
constexpr int kFewTokens = 3, kFewThreads = 256, kFewBlocks = 456;
constexpr int kFewSmem = 64 * 1024;                   // all tokens' values, 16 bits each

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

template <int DT, int T>
__global__ void __launch_bounds__(kFewThreads, 3) k_ce_few(const uint16_t* x, int64_t x_stride, const uint16_t* w,
                                                           int64_t w_stride, int64_t hidden, float2* part,
                                                           float* target_logit, const __grid_constant__ JoinArgs a)
{
    constexpr int R = T <= 2 ? 1 : 2, U = 8 / R;      // rows at a time, loads in flight per row
    wait_prev_grid();
    extern __shared__ __align__(16) uint16_t xs[];    // [T][wide]
    __shared__ float2 sh[kFewThreads / 32][T];
    __shared__ uint32_t last;
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
    float mx[T], sum[T], held[T];                     // held: the logit of row `lane` of the 32 under way
#pragma unroll
    for (int t = 0; t < T; t++) {
        mx[t] = held[t] = -INFINITY;
        sum[t] = 0.0f;
    }
    auto flush = [&]() {
#pragma unroll
        for (int t = 0; t < T; t++) {
            float top = held[t];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = fmaxf(top, mx[t]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float s = exp2f((held[t] - ref) * kLog2e);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            sum[t] = fmaf(sum[t], exp2f((mx[t] - ref) * kLog2e), s);
            mx[t] = top;
            held[t] = -INFINITY;
        }
    };
    const int64_t warps = (int64_t)gridDim.x * (kFewThreads / 32), me = (int64_t)blockIdx.x * (kFewThreads / 32) + warp;
    int have = 0;
    for (int64_t v = me * R; v < a.vocab; v += warps * R) {
        const uint16_t* row[R];
        float acc[R][T];
#pragma unroll
        for (int q = 0; q < R; q++) {
            row[q] = w + min(v + q, a.vocab - 1) * w_stride;
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
            if (v + q >= a.vocab) break;
#pragma unroll
            for (int t = 0; t < T; t++) {
                float z = acc[q][t];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    z += __shfl_xor_sync(0xffffffffu, z, o);
                if (lane == have) held[t] = z;
                if (lane == 0 && v + q == a.targets[t]) target_logit[t] = z;
            }
            if (++have == 32) {
                flush();
                have = 0;
            }
        }
    }
    if (have) flush();
    if (lane == 0)
#pragma unroll
        for (int t = 0; t < T; t++)
            sh[warp][t] = make_float2(mx[t], sum[t]);
    __syncthreads();
    if (threadIdx.x < T) {
        float m = -INFINITY, s = 0.0f;
        for (int k = 0; k < kFewThreads / 32; k++)
            merge(m, s, sh[k][threadIdx.x]);
        part[(int64_t)blockIdx.x * T + threadIdx.x] = make_float2(m, s);
    }
    __threadfence();                                  // pairs and target logits, before the count
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&a.head->joined, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (warp < T) {                                   // one warp a token: 32 parts, then a tree
        float m = -INFINITY, s = 0.0f;
        for (unsigned k = lane; k < gridDim.x; k += 32)
            merge(m, s, __ldcg(part + (int64_t)k * T + warp));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float2 q = make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
            merge(m, s, q);
        }
        if (lane == 0) sh[0][warp] = finish_token(a, warp, m, s);
    }
    __syncthreads();
    if (threadIdx.x == 0 && a.total) {
        float s = 0.0f, c = 0.0f;
        for (int t = 0; t < T; t++) {
            s += sh[0][t].x;
            c += sh[0][t].y;
        }
        a.total[0] = c > 0.0f ? s / c : 0.0f;
        a.total[1] = c;
    }
}

// One block: the row factors of G and what the products are multiplied by.
// Row factor = s_i / max |s| (times 2^14 in binary16, which keeps small
// probabilities out of its subnormals), so that equal factors are exactly 1.
// s_i = dloss[i] * scale; one that is not finite is no one's maximum, and its
// own row's factor is NaN.
__global__ void __launch_bounds__(1024) k_ce_factors(CeHead* head, const int64_t* targets, int64_t n, int64_t vocab,
                                                     const float* dloss, float scale, float up, float* coef)
{
    allow_next_grid();
    __shared__ float sm[1024];
    __shared__ int64_t sc[1024];
    float most = 0.0f;
    int64_t c = 0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) {
        const int64_t t = targets[i];
        if (t >= 0 && t < vocab) {
            c++;
            const float d = dloss ? fabsf(dloss[i] * scale) : 1.0f;
            if (d < INFINITY) most = fmaxf(most, d);
        }
    }
    sm[threadIdx.x] = most;
    sc[threadIdx.x] = c;
    __syncthreads();
    for (int o = 512; o > 0; o >>= 1) {
        if (threadIdx.x < o) {
            sm[threadIdx.x] = fmaxf(sm[threadIdx.x], sm[threadIdx.x + o]);
            sc[threadIdx.x] += sc[threadIdx.x + o];
        }
        __syncthreads();
    }
    most = sm[0];
    if (most > 0.0f) most = fmaxf(most, 0x1p-120f);          // its inverse stays finite
    const float inv = most > 0.0f ? 1.0f / most : 0.0f;
    if (threadIdx.x == 0) {
        head->err = 0;
        head->alpha = (dloss ? most : (sc[0] ? scale / (float)sc[0] : 0.0f)) / up;
    }
    for (int64_t i = threadIdx.x; i < n; i += 1024) {
        const int64_t t = targets[i];
        float c = 0.0f;
        if (t >= 0 && t < vocab) {
            const float d = dloss ? dloss[i] * scale : 1.0f;
            c = !dloss ? up : fabsf(d) < INFINITY ? d * inv * up : NAN;
        }
        coef[i] = c;
    }
}

// A gradient that a timed-out product left incomplete, or did not write at all.
struct Spoiled {
    uint16_t* out;               // NULL: none
    int64_t rows, cols, stride;
};

__device__ void spoil(const CeHead* head, const Spoiled& o)
{
    if (!o.out || !head->err) return;
    for (int64_t i = blockIdx.y; i < o.rows; i += gridDim.y)
        for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < o.cols; c += (int64_t)gridDim.x * 256)
            o.out[i * o.stride + c] = 0x7fff;                     // NaN in both types
}

__global__ void __launch_bounds__(256) k_ce_spoil(const CeHead* head, const Spoiled o)
{
    wait_prev_grid();
    spoil(head, o);
}

// dx (or dw, where its product is split): alpha times the sum of the splits,
// rounded; 4 columns a thread, a row a blockIdx.y stride.  coef: dx's row
// factors; a row whose factor is 0 is 0, also where w holds infinities, whose
// products with G's zeros are NaN.  The last kernel of a backward pass also
// turns dw into NaN if a wait ran out (dx is by way of alpha).
template <int DT>
__global__ void __launch_bounds__(256) k_ce_sum(const CeHead* head, const float* acc, int splits, int64_t split_stride,
                                               int64_t m, int64_t n, int64_t acc_cols, const float* coef, uint16_t* out,
                                               int64_t stride, const Spoiled dw)
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
        if (coef && coef[i] == 0.0f && alpha == alpha) h = make_uint2(0, 0);
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

__global__ void __launch_bounds__(256) k_ce_zero(uint16_t* p, int64_t rows, int64_t cols, int64_t stride)
{
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < rows * cols; e += (int64_t)gridDim.x * 256)
        p[e / cols * stride + e % cols] = 0;
}

// ---- host -------------------------------------------------------------------------
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up256(int64_t a) { return (a + 255) / 256 * 256; }

zero_status_t cuda_failed(cudaError_t e, const char* what)
{
    char msg[200];
    std::snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return set_error(ZERO_ECUDA, msg);
}

// The forward pass of few tokens has its own kernel.
bool few_tokens(const zero_ce_plan_t& p)
{
    return p.tokens <= kFewTokens && p.tokens * ((p.hidden + 7) / 8 * 8) * 2 <= kFewSmem;
}

// Its blocks: three to an SM of 152, and no more than give every warp a row.
int64_t few_blocks(const zero_ce_plan_t& p)
{
    const int64_t most = ceil_div(p.vocab, kFewThreads / 32);
    return most < kFewBlocks ? most : kFewBlocks;
}

// Parts of K, each at least 8 K-blocks, that a product of `tiles` tiles is summed
// in until its tiles fill the 76 pairs of SMs.
int64_t parts_of(int64_t tiles, int64_t blocks)
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
int64_t dw_parts(const zero_ce_plan_t& p)
{
    const int64_t tiles = ceil_div(p.piece, kBM) * ceil_div(p.hidden, kBN);
    return tiles <= 38 ? parts_of(tiles, ceil_div(p.tokens, kBK)) : 1;
}

// Byte offsets in the workspace.
struct CeLayout {
    int64_t coef, target_logit, block_total, part, g, acc, acc_w, end;
    int64_t acc_rows, acc_cols;                       // of one split's binary32 sums
};

CeLayout layout_of(const zero_ce_plan_t& p)
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

zero_status_t check_ce_plan(const zero_ce_plan_t* p)
{
    if (!p) return set_error(ZERO_EINVAL, "cross entropy plan is NULL");
    zero_ce_plan_t fresh;
    const zero_status_t st = zero_ce_plan(p->tokens, p->vocab, p->hidden, p->dtype, p->x_stride, p->w_stride, p->piece,
                                          &fresh);
    if (st != ZERO_OK) return st;
    if (std::memcmp(&fresh, p, sizeof fresh) != 0)
        return set_error(ZERO_EINVAL, "cross entropy plan was not made by zero_ce_plan");
    return ZERO_OK;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
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
bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t rows, int64_t cols, int64_t stride,
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

CUtensorMapDataType map_type(int dtype)
{
    return dtype == ZERO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// GemmArgs::a_rows where the rows of A are tokens.
int a_rows_of(int64_t tokens) { return tokens >= kBM / 2 ? kBM / 2 : (int)((tokens + 7) / 8 * 8); }

// A launch that may begin while the stream's kernel before it drains.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

int sm_count()
{
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 1 ? n : 152;
}

// Test hook: which product's first copy is withheld: 0 none, 1 the logits', 2 dw's.
int withheld_product()
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

template <int DT, int T>
cudaError_t launch_few_t(const zero_ce_plan_t& p, const void* x, const void* w, unsigned char* ws, const CeLayout& l,
                         const JoinArgs& j, cudaStream_t s)
{
    const size_t bytes = (size_t)(T * ((p.hidden + 7) / 8 * 8) * 2);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem((const void*)k_ce_few<DT, T>, kFewSmem, done);
    if (e != cudaSuccess) return e;
    return launch_after(k_ce_few<DT, T>, dim3((unsigned)few_blocks(p)), kFewThreads, bytes, s, static_cast<const uint16_t*>(x),
                        p.x_stride, static_cast<const uint16_t*>(w), p.w_stride, p.hidden,
                        reinterpret_cast<float2*>(ws + l.part), reinterpret_cast<float*>(ws + l.target_logit), j);
}

template <int DT>
cudaError_t launch_few(const zero_ce_plan_t& p, const void* x, const void* w, unsigned char* ws, const CeLayout& l,
                       const JoinArgs& j, cudaStream_t s)
{
    switch (p.tokens) {
    case 1: return launch_few_t<DT, 1>(p, x, w, ws, l, j, s);
    case 2: return launch_few_t<DT, 2>(p, x, w, ws, l, j, s);
    default: return launch_few_t<DT, 3>(p, x, w, ws, l, j, s);
    }
}

cudaError_t launch_sum(int dtype, const CeHead* head, const float* acc, int splits, int64_t apart, int64_t rows, int64_t cols,
                       int64_t acc_cols, const float* coef, uint16_t* out, int64_t stride, const Spoiled& dw, cudaStream_t s)
{
    const dim3 grid((unsigned)ceil_div(acc_cols, 1024), (unsigned)(rows < 4096 ? rows : 4096));
    return launch_after(dtype == ZERO_BF16 ? k_ce_sum<kBF16> : k_ce_sum<kF16>, grid, 256, 0, s, head, acc, splits, apart, rows,
                        cols, acc_cols, coef, out, stride, dw);
}

template <int EPI, bool A_MN, bool B_MN>
cudaError_t gemm(int dtype, const GemmArgs& g, cudaStream_t s)
{
    return dtype == ZERO_BF16 ? launch_gemm<EPI, kBF16, A_MN, B_MN>(g, s) : launch_gemm<EPI, kF16, A_MN, B_MN>(g, s);
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

zero_status_t zero_ce_plan(int64_t tokens, int64_t vocab, int64_t hidden, int32_t dtype, int64_t x_stride,
                           int64_t w_stride, int64_t piece, zero_ce_plan_t* out)
{
    if (!out) return set_error(ZERO_EINVAL, "zero_ce_plan: out is NULL");
    if (dtype == ZERO_FP32) return set_error(ZERO_EUNSUPPORTED, "zero_ce_plan: 16-bit types only");
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16) return set_error(ZERO_EINVAL, "zero_ce_plan: dtype unknown");
    if (tokens < 0 || vocab < 1 || hidden < 1)
        return set_error(ZERO_EINVAL, "zero_ce_plan: tokens must be >= 0, vocab and hidden >= 1");
    if (tokens > (int64_t(1) << 24) || vocab > (int64_t(1) << 24) || hidden > (int64_t(1) << 20))
        return set_error(ZERO_EUNSUPPORTED, "zero_ce_plan: tokens or vocab exceed 2^24, or hidden 2^20");
    const int64_t xs = x_stride ? x_stride : hidden, ws = w_stride ? w_stride : hidden;
    if (xs < hidden || ws < hidden || piece < 0)
        return set_error(ZERO_EINVAL, "zero_ce_plan: a stride is below hidden, or piece below 0");
    if (xs % 8 || ws % 8) return set_error(ZERO_EALIGN, "zero_ce_plan: row strides must be multiples of 8 values");
    if (xs >= (int64_t(1) << 38) || ws >= (int64_t(1) << 38))
        return set_error(ZERO_EUNSUPPORTED, "zero_ce_plan: a stride is 2^38 or more");
    if (ceil_div(tokens, kBM) * ceil_div(vocab, kBN) > (int64_t(1) << 30) || ceil_div(vocab, kBM) * ceil_div(hidden, kBN) > (int64_t(1) << 30))
        return set_error(ZERO_EUNSUPPORTED, "zero_ce_plan: over 2^30 tiles");
    // a pair's count of K-blocks stays far inside an int, and 6 tokens vocab hidden inside int64_t
    if (ceil_div(tokens, kBM) * ceil_div(vocab, kBM) * ceil_div(hidden, kBK) > (int64_t(1) << 36) ||
        ceil_div(tokens, kBM) * ceil_div(hidden, kBN) * ceil_div(vocab, kBK) > (int64_t(1) << 36) ||
        ceil_div(vocab, kBM) * ceil_div(hidden, kBN) * ceil_div(tokens, kBK) > (int64_t(1) << 36))
        return set_error(ZERO_EUNSUPPORTED, "zero_ce_plan: tokens * vocab * hidden is about 2^58 or more");
    std::memset(out, 0, sizeof *out);
    out->tokens = tokens;
    out->vocab = vocab;
    out->hidden = hidden;
    out->x_stride = xs;
    out->w_stride = ws;
    out->dtype = dtype;
    const int64_t all = up256(vocab);
    if (piece) {
        out->piece = piece < all ? up256(piece) : all;
    } else {
        // about 512 MiB of G, in pieces of about the same size: fewer pieces pass
        // dx's sums through memory less often.  Backward pass of 8192 tokens,
        // hidden 768, vocabulary 50257: 1475 us with 105 MB of G, 1333 with 210,
        // 1283 with 415, 1250 with all of it (824)
        const int64_t most = tokens ? (int64_t(1) << 28) / tokens / 256 * 256 : all;
        const int64_t fit = most < 256 ? 256 : (most < all ? most : all);
        out->piece = up256(ceil_div(vocab, ceil_div(all, fit)));
    }
    // dx has few tiles when there are few tokens; its K is the piece
    out->splits = (int32_t)parts_of(ceil_div(tokens, kBM) * ceil_div(hidden, kBN), ceil_div(out->piece, kBK));
    out->workspace_bytes = layout_of(*out).end;
    out->flops_forward = 2 * tokens * vocab * hidden;
    out->flops_backward = 3 * out->flops_forward;
    return ZERO_OK;
}

zero_status_t zero_ce_forward(const zero_ce_plan_t* plan, const void* x, const void* w, const int64_t* targets,
                              float* loss, float* lse, float* total, void* workspace, void* stream)
{
    NvtxRange range("zero_ce_forward");
    const zero_status_t st = check_ce_plan(plan);
    if (st != ZERO_OK) return st;
    const zero_ce_plan_t& p = *plan;
    if (!workspace) return set_error(ZERO_ENOMEM, "zero_ce_forward: workspace is NULL");
    if (p.tokens && (!x || !w || !targets || !loss || !lse))
        return set_error(ZERO_ENOMEM, "zero_ce_forward: a buffer is NULL");
    if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(workspace, 16) || !aligned_to(targets, 8) ||
        !aligned_to(loss, 4) || !aligned_to(lse, 4) || !aligned_to(total, 4))
        return set_error(ZERO_EALIGN, "zero_ce_forward: x, w and workspace must be 16-byte aligned, the others to their type");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    k_ce_clear<<<1, 1, 0, s>>>(reinterpret_cast<CeHead*>(ws));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_failed(e, "zero_ce_forward");
    if (p.tokens) {
        if (!encode_fn()) return set_error(ZERO_ECUDA, "zero_ce_forward: the driver has no cuTensorMapEncodeTiled");
        const CeLayout l = layout_of(p);
        JoinArgs j;
        j.head = reinterpret_cast<CeHead*>(ws);
        j.part = reinterpret_cast<float2*>(ws + l.part);
        j.strips = 2 * (int)ceil_div(p.vocab, kBN);
        j.n = p.tokens;
        j.targets = targets;
        j.vocab = p.vocab;
        j.target_logit = reinterpret_cast<float*>(ws + l.target_logit);
        j.loss = loss;
        j.lse = lse;
        j.block_total = reinterpret_cast<float2*>(ws + l.block_total);
        j.total = total;
        if (few_tokens(p)) {
            e = p.dtype == ZERO_BF16 ? launch_few<kBF16>(p, x, w, ws, l, j, s) : launch_few<kF16>(p, x, w, ws, l, j, s);
            return e == cudaSuccess ? ZERO_OK : cuda_failed(e, "zero_ce_forward");
        }
        const CUtensorMapDataType type = map_type(p.dtype);
        GemmArgs g;
        std::memset(&g, 0, sizeof g);
        g.a_rows = a_rows_of(p.tokens);
        if (!make_map(&g.a, type, x, p.tokens, p.hidden, p.x_stride, g.a_rows) ||
            !make_map(&g.b, type, w, p.vocab, p.hidden, p.w_stride, kBN / 2))
            return set_error(ZERO_ECUDA, "zero_ce_forward: cuTensorMapEncodeTiled refused a buffer");
        g.m = p.tokens;
        g.n = p.vocab;
        g.m_tiles = (int)ceil_div(p.tokens, kBM);
        g.n_tiles = (int)ceil_div(p.vocab, kBN);
        g.k_blocks = (int)ceil_div(p.hidden, kBK);
        g.chunk = kChunk;
        g.splits = 1;
        g.head = reinterpret_cast<CeHead*>(ws);
        g.targets = targets;
        g.part = reinterpret_cast<float2*>(ws + l.part);
        g.target_logit = reinterpret_cast<float*>(ws + l.target_logit);
        g.withhold = withheld_product() > 0;
        e = gemm<kEpiLse, false, false>(p.dtype, g, s);
        if (e == cudaSuccess) {
            e = launch_after(k_ce_join, dim3((unsigned)ceil_div(p.tokens, 32)), 1024, 0, s, j);
        }
    } else if (total) {
        e = cudaMemsetAsync(total, 0, 8, s);
    }
    return e == cudaSuccess ? ZERO_OK : cuda_failed(e, "zero_ce_forward");
}

zero_status_t zero_ce_backward(const zero_ce_plan_t* plan, const void* x, const void* w, const int64_t* targets,
                               const float* lse, const float* dloss, float grad_scale, void* dx, void* dw,
                               void* workspace, void* stream)
{
    NvtxRange range("zero_ce_backward");
    const zero_status_t st = check_ce_plan(plan);
    if (st != ZERO_OK) return st;
    const zero_ce_plan_t& p = *plan;
    if (!std::isfinite(grad_scale)) return set_error(ZERO_EINVAL, "zero_ce_backward: grad_scale is not finite");
    if (!workspace) return set_error(ZERO_ENOMEM, "zero_ce_backward: workspace is NULL");
    if (p.tokens && (!x || !w || !targets || !lse)) return set_error(ZERO_ENOMEM, "zero_ce_backward: a buffer is NULL");
    if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(dx, 16) || !aligned_to(dw, 16) ||
        !aligned_to(workspace, 16) || !aligned_to(targets, 8) || !aligned_to(lse, 4) || !aligned_to(dloss, 4))
        return set_error(ZERO_EALIGN, "zero_ce_backward: x, w, dx, dw and workspace must be 16-byte aligned, the others to their type");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!p.tokens) {
        if (dw) k_ce_zero<<<1024, 256, 0, s>>>(static_cast<uint16_t*>(dw), p.vocab, p.hidden, p.w_stride);
        cudaError_t e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, sizeof(CeHead), s);
        return e == cudaSuccess ? ZERO_OK : cuda_failed(e, "zero_ce_backward");
    }
    if (!dx && !dw) return ZERO_OK;
    if (!encode_fn()) return set_error(ZERO_ECUDA, "zero_ce_backward: the driver has no cuTensorMapEncodeTiled");
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    const CeLayout l = layout_of(p);
    CeHead* head = reinterpret_cast<CeHead*>(ws);
    float* coef = reinterpret_cast<float*>(ws + l.coef);
    uint16_t* G = reinterpret_cast<uint16_t*>(ws + l.g);
    float* acc = reinterpret_cast<float*>(ws + l.acc);
    const CUtensorMapDataType type = map_type(p.dtype);
    const int withheld = withheld_product();
    const float up = p.dtype == ZERO_FP16 ? 16384.0f : 1.0f;
    k_ce_factors<<<1, 1024, 0, s>>>(head, targets, p.tokens, p.vocab, dloss, grad_scale, up, coef);
    cudaError_t e = cudaGetLastError();
    for (int64_t v0 = 0; v0 < p.vocab && e == cudaSuccess; v0 += p.piece) {
        const int64_t nv = p.vocab - v0 < p.piece ? p.vocab - v0 : p.piece;
        GemmArgs g;                                  // G of the piece
        std::memset(&g, 0, sizeof g);
        g.a_rows = a_rows_of(p.tokens);
        bool ok = make_map(&g.a, type, x, p.tokens, p.hidden, p.x_stride, g.a_rows) &&
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
        g.head = head;
        g.targets = targets;
        g.lse = lse;
        g.coef = coef;
        g.withhold = v0 == 0 && withheld == 1;
        if (ok) e = gemm<kEpiGrad, false, false>(p.dtype, g, s);
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
                    e = launch_sum(p.dtype, head, sums, g.splits, rows * l.acc_cols, nv, p.hidden, l.acc_cols,
                                   nullptr, out, p.w_stride, Spoiled{}, s);
            } else {
                ok = ok && make_map(&g.c, type, out, nv, p.hidden, p.w_stride, 32);
                if (p.hidden % 8) {
                    g.out = out;
                    g.out_stride = p.w_stride;
                }
                if (ok) e = gemm<kEpiOut, true, true>(p.dtype, g, s);
            }
        }
        if (!ok) return set_error(ZERO_ECUDA, "zero_ce_backward: cuTensorMapEncodeTiled refused a buffer");
    }
    const Spoiled all{static_cast<uint16_t*>(dw), p.vocab, p.hidden, p.w_stride};
    if (dx && e == cudaSuccess)
        e = launch_sum(p.dtype, head, acc, p.splits, l.acc_rows * l.acc_cols, p.tokens, p.hidden, l.acc_cols, coef,
                       static_cast<uint16_t*>(dx), p.x_stride, all, s);
    else if (e == cudaSuccess)
        e = launch_after(k_ce_spoil, dim3(1, 608), 256, 0, s, head, all);
    return e == cudaSuccess ? ZERO_OK : cuda_failed(e, "zero_ce_backward");
}

zero_status_t zero_ce_status(const zero_ce_plan_t* plan, const void* workspace, void* stream)
{
    const zero_status_t st = check_ce_plan(plan);
    if (st != ZERO_OK) return st;
    if (!workspace) return set_error(ZERO_ENOMEM, "zero_ce_status: workspace is NULL");
    if (!aligned_to(workspace, 16)) return set_error(ZERO_EALIGN, "zero_ce_status: workspace is not 16-byte aligned");
    uint32_t err = 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(&err, workspace, 4, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_failed(e, "zero_ce_status");
    return err ? set_error(ZERO_ETIMEOUT, "a bounded wait inside the cross entropy kernels ran out") : ZERO_OK;
}

}  // extern "C"
