// Log probabilities of given tokens over a large vocabulary, entropies, the most
// likely alternatives, and the gradients of the first two, without stored
// logits: the plan and the small kernels around the products that cross entropy
// uses too.
#include "dev_vocab.cuh"
#include "nvtx_ranges.h"

namespace zg {

using namespace vocab;

namespace {

constexpr int kMostTop = 32;                          // alternatives: a warp's lanes
constexpr int64_t kSample = 8192;                     // entries that give the rows their bounds
constexpr unsigned kAll = 0xffffffffu;

struct LpArgs {
    CeHead* head;
    const int64_t* targets;
    int64_t n, vocab;            // rows here
    float scale;
    const float2* part;          // [strips][n] maximum, sum
    const float* part_t;         // [strips][n]
    int strips;
    const float* target_logit;   // [n]
    float* logp;
    float* lse;
    float* entropy;              // may be NULL
    float2* stat;                // [n] maximum, log of the sum
    int top;
    const float* logits;         // [n][logit_stride]: all, or those of the sample and of strips that reach `least`
    int64_t logit_stride;
    float* least;                // [n]: the last alternative of the row's sample (NULL: all logits are kept)
    uint64_t* cand;              // few rows: [n][blocks][top]
    float* top_logp;
    int64_t* top_index;
};

// The head cleared, before a forward pass.  The caller's kernels have ended before the
// next may start: a product takes its tensor memory before it waits.
__global__ void k_lp_clear(CeHead* head)
{
    wait_prev_grid();
    allow_next_grid();
    head->err = 0;
    head->joined = 0;
}

// Maximum, sum of e = exp((z - maximum) scale), sum of e (z - maximum), of some
// logits of a row.
struct Stat {
    float mx, sum, t;
};

__device__ __forceinline__ Stat none() { return {-INFINITY, 0.0f, 0.0f}; }

// The same over two sets.  One that adds nothing adds nothing to t either, however
// far off (or minus infinity) its maximum is; a NaN is in the sum.
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float scale_log2e)
{
    Stat r;
    r.mx = fmaxf(a.mx, b.mx);
    const float ref = r.mx == -INFINITY ? 0.0f : r.mx;
    const float da = a.mx - ref, db = b.mx - ref;
    const float fa = exp2f(da * scale_log2e), fb = exp2f(db * scale_log2e);
    r.sum = fmaf(a.sum, fa, b.sum * fb);
    r.t = (fa > 0.0f ? fa * fmaf(da, a.sum, a.t) : 0.0f) + (fb > 0.0f ? fb * fmaf(db, b.sum, b.t) : 0.0f);
    return r;
}

// b added to a, whose maximum is no less.
__device__ __forceinline__ void add(Stat& a, const Stat& b, float scale_log2e)
{
    const float d = b.mx - (a.mx == -INFINITY ? 0.0f : a.mx), f = exp2_fast(d * scale_log2e);
    a.sum = fmaf(b.sum, f, a.sum);
    a.t += f > 0.0f ? f * fmaf(d, b.sum, b.t) : 0.0f;
}

__device__ __forceinline__ Stat shuffled(const Stat& a, int o)
{
    return {__shfl_xor_sync(kAll, a.mx, o), __shfl_xor_sync(kAll, a.sum, o), __shfl_xor_sync(kAll, a.t, o)};
}

__device__ __forceinline__ Stat warp_join(Stat a, float scale_log2e)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = join(a, shuffled(a, o), scale_log2e);
    return a;
}

// (z - maximum) scale - log sum, rather than z scale - lse: a likely token's log
// probability keeps its digits.
__device__ __forceinline__ float logp_of(float z, float2 stat, float scale) { return fmaf(z - stat.x, scale, -stat.y); }

__device__ __forceinline__ float2 finish_row(const LpArgs& a, int64_t i, const Stat& r)
{
    float2 st = make_float2(r.mx, logf(r.sum));
    if (a.head->err) st.y = NAN;
    a.lse[i] = fmaf(r.mx, a.scale, st.y);
    if (a.entropy) a.entropy[i] = fmaf(-a.scale, r.t / r.sum, st.y);
    const int64_t t = a.targets[i];
    a.logp[i] = t >= 0 && t < a.vocab ? logp_of(__ldcg(a.target_logit + i), st, a.scale) : 0.0f;
    return st;
}

// Per row: the strips' statistics joined, in a fixed order: kJoinParts parts of the
// strips, a thread each, kJoinRows rows side by side, then a tree over the parts.
// Latency for few rows (6 us for 1023 of 393 strips; 32 rows to a block of 1024
// threads took 10), exponentials for many.
constexpr int kJoinRows = 8, kJoinParts = 64, kJoinThreads = kJoinRows * kJoinParts, kJoinAhead = 8;

__global__ void __launch_bounds__(kJoinThreads) k_lp_join(const __grid_constant__ LpArgs a)
{
    wait_prev_grid();
    __shared__ Stat sh[kJoinThreads / 32][kJoinRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = threadIdx.x / kJoinRows;
    const float c = a.scale * kLog2e;
    const int64_t i = (int64_t)blockIdx.x * kJoinRows + threadIdx.x % kJoinRows;
    Stat r = none();
    if (i < a.n)
        for (int s = part; s < a.strips; s += kJoinParts * kJoinAhead) {
            Stat q[kJoinAhead];
            float top = r.mx;
#pragma unroll
            for (int k = 0; k < kJoinAhead; k++) {
                const int at = s + k * kJoinParts;
                q[k] = none();
                if (at < a.strips) {
                    const float2 p = a.part[(int64_t)at * a.n + i];
                    q[k] = {p.x, p.y, a.part_t[(int64_t)at * a.n + i]};
                }
                top = fmaxf(top, q[k].mx);
            }
            r = join(r, Stat{top, 0.0f, 0.0f}, c);    // to the new maximum
#pragma unroll
            for (int k = 0; k < kJoinAhead; k++)
                add(r, q[k], c);
        }
    r = join(r, shuffled(r, 8), c);
    r = join(r, shuffled(r, 16), c);
    if (lane < kJoinRows) sh[warp][lane] = r;
    __syncthreads();
    if (warp < kJoinRows / 2) {                       // a warp two rows, 16 lanes each
        r = sh[lane & 15][2 * warp + (lane >> 4)];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            r = join(r, shuffled(r, o), c);
        const int64_t at = (int64_t)blockIdx.x * kJoinRows + 2 * warp + (lane >> 4);
        if ((lane & 15) == 0 && at < a.n) a.stat[at] = finish_row(a, at, r);
    }
}

// ---- alternatives ---------------------------------------------------------------------
// A warp's list: lane j has the jth largest key, 0 where there are fewer.
__device__ __forceinline__ uint64_t key_max(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t key_min(uint64_t a, uint64_t b) { return a > b ? b : a; }

// Falling order over the lanes of what rises and then falls, or the other way.
__device__ __forceinline__ uint64_t sorted_bitonic(uint64_t x, int lane)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t y = __shfl_xor_sync(kAll, x, o);
        x = lane & o ? key_min(x, y) : key_max(x, y);
    }
    return x;
}

// The 32 largest of two lists.
__device__ __forceinline__ uint64_t lists_merged(uint64_t a, uint64_t b, int lane)
{
    return sorted_bitonic(key_max(a, __shfl_sync(kAll, b, 31 - lane)), lane);
}

__device__ __forceinline__ uint64_t sorted(uint64_t x, int lane)
{
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
        for (int o = n >> 1; o > 0; o >>= 1) {
            const uint64_t y = __shfl_xor_sync(kAll, x, o);
            const bool low = !(lane & o), falls = n == 32 || !(lane & n);
            x = low == falls ? key_max(x, y) : key_min(x, y);
        }
    return x;
}

// Keys on their way into a warp's list, gathered so that 32 at a time are sorted;
// those below a bound that the row is known to have `top` of are dropped.
struct Gather {
    uint64_t* held;              // [64] of the warp, shared memory
    int n;                       // so many are held
    int top;
    uint64_t bound;
    float least;                 // the bound's logit
    uint64_t list;

    __device__ __forceinline__ void raise(uint64_t b)
    {
        bound = key_max(bound, b);
        least = logit_of(bound);
    }

    __device__ __forceinline__ void sort(uint64_t key, int lane)
    {
        list = lists_merged(list, sorted(key, lane), lane);
        raise(__shfl_sync(kAll, list, top - 1));
    }

    // A key of each lane with `in`.
    __device__ __forceinline__ void add(bool in, uint64_t key, int lane)
    {
        in = in && key >= bound;
        const unsigned b = __ballot_sync(kAll, in);
        if (!b) return;
        if (in) held[n + __popc(b & ((1u << lane) - 1))] = key;
        n += __popc(b);
        __syncwarp();
        if (n < 32) return;
        sort(held[lane], lane);
        n -= 32;
        const uint64_t rest = held[32 + lane];
        __syncwarp();
        held[lane] = rest;
        __syncwarp();
    }

    __device__ __forceinline__ uint64_t all(int lane)
    {
        if (n) sort(lane < n ? held[lane] : 0, lane);
        return list;
    }
};

// An empty list; -infinity is no alternative, and NaN none.
__device__ __forceinline__ Gather gather(uint64_t* held, int top)
{
    return {held, 0, top, key_of(-3.4028235e38f, 0xffffffffu), -3.4028235e38f, 0};
}

// The lists of a block's 8 warps, in warp 0.
__device__ __forceinline__ uint64_t block_merged(uint64_t list, uint64_t (*sh)[32], int warp, int lane)
{
    __syncthreads();
    sh[warp][lane] = list;
    for (int o = 4; o > 0; o >>= 1) {
        __syncthreads();
        if (warp < o) sh[warp][lane] = list = lists_merged(list, sh[warp + o][lane], lane);
    }
    return list;
}

__device__ __forceinline__ void write_top(const LpArgs& a, int64_t i, uint64_t list, float2 stat, int lane)
{
    if (lane >= a.top) return;
    const bool failed = a.head->err;
    a.top_logp[i * a.top + lane] = failed ? NAN : list ? logp_of(logit_of(list), stat, a.scale) : -INFINITY;
    a.top_index[i * a.top + lane] = list && !failed ? (int64_t)(0xffffffffu - (uint32_t)list) : -1;
}

// Per row: the first `top` of its logits, by W warps.  Of the strips' maxima, two
// sets to a lane, the top-th largest set's is a bound that the row is known to have
// `top` logits of; only strips whose maximum is no less are read, 9 of 393 for 8
// alternatives, 22 for 20 or 45 for 32, and have about as many logits to sort.
// FINAL: written out; else only the sample's are there, and their last becomes the
// row's `least`.  Latency: 1023 rows of 50257 12 us beside the products' 105 and what
// keeping 206 MB of logits adds to them, 13.  (Reading all logits, 25 us for 4096 of
// each row; lists of each strip's largest made in the products' epilogue, 40 us a
// tile for 20 alternatives.)
template <int W, bool FINAL>
__global__ void __launch_bounds__(256) k_lp_top(const __grid_constant__ LpArgs a)
{
    constexpr int U = 8;                              // maxima, or strips, on their way
    wait_prev_grid();
    if constexpr (!FINAL) allow_next_grid();
    __shared__ uint64_t sh[8][32], held[8][64];
    __shared__ int chosen[8][32 * U];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = W == 1 ? (int64_t)blockIdx.x * 8 + warp : blockIdx.x;
    if (W == 1 && i >= a.n) return;
    const float2* part = a.part + i;
    const int strips = FINAL ? a.strips : (int)(kSample / kStrip);
    const int first = (W == 1 ? 0 : warp * 32) + lane;            // strips first, first + 32 W, ...
    float most[2] = {-INFINITY, -INFINITY};
    for (int s0 = first - lane; s0 < strips; s0 += 32 * W * U) {
        float m[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int s = s0 + lane + 32 * W * u;
            m[u] = s < strips ? part[(int64_t)s * a.n].x : -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < U; u++)
            most[u & 1] = fmaxf(most[u & 1], m[u]);
    }
    uint64_t bound = lists_merged(sorted(key_of(most[0], 0), lane), sorted(key_of(most[1], 0), lane), lane);
    if constexpr (W > 1) {
        bound = block_merged(bound, sh, warp, lane);
        if (warp == 0) sh[0][lane] = bound;
        __syncthreads();
        bound = sh[0][lane];
    }
    Gather g = gather(held[warp], a.top);
    g.raise(__shfl_sync(kAll, bound, a.top - 1) & ~0xffffffffull);            // of whatever index
    if (FINAL && a.least) g.raise(key_of(fmaxf(a.least[i], -3.4028235e38f), 0xffffffffu));       // others are not there
    const float* z = a.logits + i * a.logit_stride;
    int* mine = chosen[warp];
    for (int s0 = first - lane; s0 < strips; s0 += 32 * W * U) {
        int n = 0;                                    // strips to look at
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int s = s0 + lane + 32 * W * u;
            const bool in = s < strips && part[(int64_t)s * a.n].x >= g.least;
            const unsigned b = __ballot_sync(kAll, in);
            if (in) mine[n + __popc(b & ((1u << lane) - 1))] = s;
            n += __popc(b);
        }
        __syncwarp();
        for (int k0 = 0; k0 < n; k0 += U) {
            int at[U];
            float4 q[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                at[u] = k0 + u < n ? mine[k0 + u] * kStrip + 4 * lane : 0;
                if (k0 + u < n) q[u] = *reinterpret_cast<const float4*>(z + at[u]);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (k0 + u >= n) break;
                const float f[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                // a lane seldom has two: the next of all lanes that have one, again and again
                unsigned in = 0;
#pragma unroll
                for (int k = 0; k < 4; k++)
                    if (at[u] + k < a.vocab && f[k] >= g.least) in |= 1u << k;
                while (__any_sync(kAll, in)) {
                    const int k = in ? __ffs(in) - 1 : 0;
                    const float v = k == 0 ? f[0] : k == 1 ? f[1] : k == 2 ? f[2] : f[3];
                    g.add(in, key_of(v, (uint32_t)(at[u] + k)), lane);
                    in &= in - 1;
                }
            }
        }
        __syncwarp();
    }
    uint64_t list = g.all(lane);
    if constexpr (W > 1) {
        list = block_merged(list, sh, warp, lane);
        if (warp) return;
    }
    if constexpr (FINAL) {
        write_top(a, i, list, a.stat[i], lane);
    } else {
        if (lane == a.top - 1) a.least[i] = list ? logit_of(list) : -INFINITY;
    }
}

// ---- few rows -------------------------------------------------------------------------
__device__ __forceinline__ uint64_t load_key(const uint64_t* p)
{
    return __ldcg(reinterpret_cast<const unsigned long long*>(p));
}

// Up to kFewTokens rows, as cross entropy's: w is read once and that is the time.
// Each lane keeps one row's logit; 32 of them at a time go into the warp's
// statistics and list.  The last block joins the blocks'.  One row of 50257 x 4096
// with 8 alternatives 70 us, 5.9 TB/s, without 66.5; two 79, three 89 (four, by the
// tensor cores, 91).
template <int DT, int T>
__global__ void __launch_bounds__(kFewThreads, 3) k_lp_few(const uint16_t* x, int64_t x_stride, const uint16_t* w,
                                                           int64_t w_stride, int64_t hidden, Stat* part, float* target_logit,
                                                           const __grid_constant__ LpArgs a)
{
    constexpr int kWarps = kFewThreads / 32;
    wait_prev_grid();
    extern __shared__ __align__(16) uint16_t xs[];    // [T][wide]
    constexpr int kPer = T == 1 ? 8 : T == 2 ? 4 : 2; // warps to a row, at the end
    __shared__ Stat sh[kWarps][T];
    __shared__ uint64_t lists[kWarps][T][32], joined[kWarps][32], least[T];
    __shared__ uint32_t last;
    __shared__ int chosen[T], which[T][kFewBlocks];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float c = a.scale * kLog2e;
    Stat st[T];
    float held[T];                                    // the logit of row `lane` of the 32 under way
    uint64_t list[T];
#pragma unroll
    for (int t = 0; t < T; t++) {
        st[t] = none();
        held[t] = -INFINITY;
        list[t] = 0;
    }
    int have = 0;
    int64_t holds = 0;                                // the vocabulary entry that the lane holds
    auto flush = [&]() {
#pragma unroll
        for (int t = 0; t < T; t++) {
            const bool any = lane < have;
            // one logit; a NaN is in the sum, a maximum would drop it
            const Stat one = any && held[t] != -INFINITY ? Stat{held[t], held[t] == held[t] ? 1.0f : held[t], 0.0f} : none();
            st[t] = join(st[t], warp_join(one, c), c);
            if (a.top)
                list[t] = lists_merged(list[t], sorted(any && held[t] > -INFINITY ? key_of(held[t], (uint32_t)holds) : 0, lane), lane);
        }
        have = 0;
    };
    few_logits<DT, T>(x, x_stride, w, w_stride, hidden, a.vocab, a.targets, xs, target_logit, [&](int64_t v, const float (&z)[T]) {
#pragma unroll
        for (int t = 0; t < T; t++)
            if (lane == have) held[t] = z[t];
        if (lane == have) holds = v;
        if (++have == 32) flush();
    });
    if (have) flush();
#pragma unroll
    for (int t = 0; t < T; t++) {
        if (lane == 0) sh[warp][t] = st[t];
        lists[warp][t][lane] = list[t];
    }
    // the warps' statistics and lists: kPer warps to a row
    const int t = warp / kPer, wi = warp % kPer;
    const bool on = t < T;
    auto merged = [&](uint64_t x) {                   // of a row's warps, in its first
        __syncthreads();
        joined[warp][lane] = x;
        for (int o = kPer / 2; o > 0; o >>= 1) {
            __syncthreads();
            if (wi < o) joined[warp][lane] = x = lists_merged(x, joined[warp + o][lane], lane);
        }
        return x;
    };
    __syncthreads();
    if (on && wi == 0) {
        const Stat r = warp_join(lane < kWarps ? sh[lane][t] : none(), c);
        if (lane == 0) part[(int64_t)t * gridDim.x + blockIdx.x] = r;
    }
    if (a.top) {
        uint64_t best = 0;
        if (on)
            for (int k = wi; k < kWarps; k += kPer)
                best = lists_merged(best, lists[k][t][lane], lane);
        best = merged(best);
        if (on && wi == 0 && lane < a.top) a.cand[((int64_t)t * gridDim.x + blockIdx.x) * a.top + lane] = best;
    }
    __threadfence();                                  // statistics, keys and target logits, before the count
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&a.head->joined, 1u) == gridDim.x - 1;
    if (threadIdx.x < T) chosen[threadIdx.x] = 0;
    __syncthreads();
    if (!last) return;
    __threadfence();
    // the blocks' statistics, kEach to a lane, in a fixed order; of their lists, those
    // that start no lower than the top-th of the lanes' best
    constexpr int kEach = (kFewBlocks + 32 * kPer - 1) / (32 * kPer);
    const int blocks = (int)gridDim.x;
    Stat r = none();
    uint64_t best[kEach], most = 0;
#pragma unroll
    for (int u = 0; u < kEach; u++) {
        const int k = wi * 32 + lane + u * 32 * kPer;
        best[u] = 0;
        if (!on || k >= blocks) continue;
        const Stat* p = part + (int64_t)t * blocks + k;
        if (a.top) best[u] = load_key(a.cand + ((int64_t)t * blocks + k) * a.top);
        r = join(r, Stat{__ldcg(&p->mx), __ldcg(&p->sum), __ldcg(&p->t)}, c);
        most = key_max(most, best[u]);
    }
    r = warp_join(r, c);
    if (lane == 0) sh[warp][0] = r;
    __syncthreads();
    float2 done = make_float2(0.0f, 0.0f);
    if (on && wi == 0) {
        r = warp_join(lane < kPer ? sh[warp + lane][0] : none(), c);
        if (lane == 0) done = finish_row(a, t, r);
        done.x = __shfl_sync(kAll, done.x, 0);
        done.y = __shfl_sync(kAll, done.y, 0);
    }
    if (!a.top) return;
    const uint64_t bound = merged(sorted(most, lane));
    if (on && wi == 0 && lane == a.top - 1) least[t] = bound;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kEach; u++)                   // 0: the block has none
        if (best[u] && best[u] >= least[t]) which[t][atomicAdd(&chosen[t], 1)] = wi * 32 + lane + u * 32 * kPer;
    __syncthreads();
    uint64_t mine = 0;
    if (on)
        for (int k = wi; k < chosen[t]; k += kPer)
            mine = lists_merged(mine, lane < a.top ? load_key(a.cand + ((int64_t)t * blocks + which[t][k]) * a.top + lane) : 0, lane);
    mine = merged(mine);
    if (on && wi == 0) write_top(a, t, mine, done, lane);
}

// One block: the row factors of G and what the products are multiplied by.  G =
// a ([v = t] - p) - b p (log p + H) in 16 bits; |p (log p + H)| is below 5 for up
// to 2^24 entries, so rows are scaled by the largest |a| + 4 |b| (binary16: to 2^14
// instead of 1, which keeps small probabilities out of its subnormals; 1.25 times
// that is in its range).  A factor that is not finite is no one's maximum, and its
// own row's are NaN.  Every factor's size 2^-120 at least, so that its inverse is finite.
// Why 16 bits: the tensor cores take both operands of dx and dw in x's and w's type, and
// G as the sum of two such numbers would make those products 8TVd instead of 4.  What it
// costs, 8192 x 50257 x 768 bfloat16, of the gradients' norm: G's rounding alone 1.67e-3,
// as much as the results' own (1.66e-3, which G in binary32 leaves too), both 2.36e-3;
// G rounded and all else in 64 bits gives the kernels' results within 7e-5.
__global__ void __launch_bounds__(1024) k_lp_factors(CeHead* head, const int64_t* targets, int64_t n, int64_t vocab,
                                                     const float* dlogp, const float* dentropy, float scale, float up,
                                                     float* coef, float* coef_h)
{
    wait_prev_grid();
    allow_next_grid();                                // as in k_lp_clear
    __shared__ float sm[32];
    auto factor = [&](int64_t i, float& b) {
        const int64_t t = targets[i];
        b = dentropy ? dentropy[i] * scale : 0.0f;
        return dlogp && t >= 0 && t < vocab ? dlogp[i] * scale : 0.0f;
    };
    float most = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += 1024) {
        float b;
        const float a = factor(i, b), d = fabsf(a) + 4.0f * fabsf(b);
        if (d < INFINITY) most = fmaxf(most, d);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = most;
    __syncthreads();
    most = sm[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
    if (most > 0.0f) most = fmaxf(most, 0x1p-120f);
    const float inv = most > 0.0f ? 1.0f / most : 0.0f;
    if (threadIdx.x == 0) {
        head->err = 0;
        head->alpha = most / up;
    }
    for (int64_t i = threadIdx.x; i < n; i += 1024) {
        float b;
        const float a = factor(i, b);
        const bool fine = fabsf(a) + 4.0f * fabsf(b) < INFINITY;
        coef[i] = fine ? a * inv * up : NAN;
        if (dentropy) coef_h[i] = fine ? b * inv * up : 0.0f;
    }
}

// ---- host ---------------------------------------------------------------------------------
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

zero_status_t cuda_failed(cudaError_t e, const char* what)
{
    char msg[200];
    std::snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return set_error(ZERO_ECUDA, msg);
}

int64_t strips_of(int64_t vocab) { return ceil_div(vocab, kBN) * 2; }

// Whether all logits are kept in memory for the alternatives, or where a sample would
// be most of them; else those of a sample, which gives every row a bound, and of the
// strips that reach it.  Kept logits cost their writes; a sample costs a product and a
// search of its own and, the more alternatives, the more strips that reach the bound.
// us, bfloat16, kept / by sample:
//   hidden 768:  700 x 50257 with 8 76 / 82;  1023 with 8 98 / 93, 16 101 / 102, 32 112 / 132;
//     1400 with 8 131 / 123, 20 137 / 140, 32 145 / 164;  2048 with 8 171 / 150, 20 177 / 172,
//     32 186 / 202;  2670 with 32 248 / 253;  4096 with 20 342 / 309, 32 362 / 362;
//     4096 x 32000 with 16 227 / 211, 32 248 / 265;  1000 x 128000 with 8 222 / 177, 32 235 / 233
//   hidden 1024: 1400 x 50257 with 1 126 / 131, 32 143 / 181;  4096 with 1 311 / 326, 32 357 / 417
//   hidden 1600: 1023 with 20 139 / 153;  4096 with 1 468 / 468, 32 502 / 558;  8192 with 8 967 / 936
//   hidden 4096: 2048 with 8 518 / 557;  2670 with 8 762 / 751, 32 731 / 785;  8192 with 8 2186 / 2149
// So from 1024 hidden values on, where the writes hide behind the product, up to 3 x 2^26
// logits; below it 2^22 logits for each alternative, ten at least.  (A sample of 4096
// entries, 2048 x 768 with 32: 247, of 2048 entries 291.)
bool all_kept(const zero_lp_plan_t& p)
{
    const int64_t most = p.hidden >= 1024 ? int64_t(3) << 26 : int64_t(p.top > 10 ? p.top : 10) << 22;
    return p.vocab <= kSample + kSample / 4 || p.tokens * p.vocab <= most;
}

int64_t logit_stride(int64_t vocab) { return ceil_div(vocab, kStrip) * kStrip; }

// Rows at a time of a forward pass: what the strips leave, 12 bytes each, takes about
// 512 MiB, or with alternatives that and the logits 2 GiB.
int64_t rows_at_once(int64_t vocab, int64_t top)
{
    const int64_t per = strips_of(vocab) * 12 + (top ? 4 * logit_stride(vocab) : 0);
    const int64_t fit = (int64_t(1) << (top ? 31 : 29)) / per / kBM * kBM;
    return fit < kBM ? kBM : fit;
}

// Byte offsets of a forward pass in the workspace.
struct LpLayout {
    int64_t target_logit, stat, least, part, part_t, logits, cand, end;
};

LpLayout lp_layout(const zero_lp_plan_t& p, bool few)
{
    LpLayout l;
    const int64_t rows = p.rows < p.tokens ? p.rows : p.tokens, strips = strips_of(p.vocab);
    l.target_logit = sizeof(CeHead);
    l.stat = l.target_logit + up256(rows * 4);
    l.least = l.stat + up256(rows * 8);
    l.part = l.least + up256(rows * 4);
    l.part_t = l.part + up256(few ? kFewBlocks * rows * (int64_t)sizeof(Stat) : strips * rows * 8);
    l.logits = l.part_t + (few ? 0 : up256(strips * rows * 4));
    l.cand = l.logits + (few || !p.top ? 0 : up256(rows * logit_stride(p.vocab) * 4));
    l.end = l.cand + (few ? up256(kFewBlocks * rows * p.top * 8) : 0);
    return l;
}

zero_status_t products_plan(const zero_lp_plan_t& p, zero_ce_plan_t* out)
{
    return zero_ce_plan(p.tokens, p.vocab, p.hidden, p.dtype, p.x_stride, p.w_stride, p.piece, out);
}

zero_status_t check_lp_plan(const zero_lp_plan_t* p, zero_ce_plan_t* products)
{
    if (!p) return set_error(ZERO_EINVAL, "log probabilities' plan is NULL");
    zero_lp_plan_t fresh;
    const zero_status_t st = zero_lp_plan(p->tokens, p->vocab, p->hidden, p->dtype, p->x_stride, p->w_stride, p->piece, p->top,
                                          &fresh);
    if (st != ZERO_OK) return st;
    if (std::memcmp(&fresh, p, sizeof fresh) != 0)
        return set_error(ZERO_EINVAL, "log probabilities' plan was not made by zero_lp_plan");
    return products_plan(fresh, products);
}

template <int DT, int T>
cudaError_t launch_few_t(const zero_lp_plan_t& p, int64_t blocks, const void* x, const void* w, unsigned char* ws,
                         const LpLayout& l, const LpArgs& a, cudaStream_t s)
{
    const size_t bytes = (size_t)(T * ((p.hidden + 7) / 8 * 8) * 2);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem((const void*)k_lp_few<DT, T>, kFewSmem, done);
    if (e != cudaSuccess) return e;
    return launch_after(k_lp_few<DT, T>, dim3((unsigned)blocks), kFewThreads, bytes, s, static_cast<const uint16_t*>(x),
                        p.x_stride, static_cast<const uint16_t*>(w), p.w_stride, p.hidden, reinterpret_cast<Stat*>(ws + l.part),
                        reinterpret_cast<float*>(ws + l.target_logit), a);
}

template <int DT>
cudaError_t launch_few(const zero_lp_plan_t& p, int64_t blocks, const void* x, const void* w, unsigned char* ws,
                       const LpLayout& l, const LpArgs& a, cudaStream_t s)
{
    switch (p.tokens) {
    case 1: return launch_few_t<DT, 1>(p, blocks, x, w, ws, l, a, s);
    case 2: return launch_few_t<DT, 2>(p, blocks, x, w, ws, l, a, s);
    default: return launch_few_t<DT, 3>(p, blocks, x, w, ws, l, a, s);
    }
}

// Warps to a row: 8 where there are few rows and more than a sample's strips.
template <bool FINAL>
cudaError_t launch_top(const LpArgs& a, cudaStream_t s)
{
    if (a.n > 2 * 152 || !FINAL || a.strips <= 64)
        return launch_after(k_lp_top<1, FINAL>, dim3((unsigned)ceil_div(a.n, 8)), 256, 0, s, a);
    return launch_after(k_lp_top<8, FINAL>, dim3((unsigned)a.n), 256, 0, s, a);
}

// The forward pass of rows [r0, r0 + a.n).
cudaError_t forward_rows(const zero_lp_plan_t& p, const void* x, const void* w, unsigned char* ws, const LpLayout& l, LpArgs a,
                         int64_t r0, bool first, cudaStream_t s, bool& ok)
{
    const CUtensorMapDataType type = map_type(p.dtype);
    const void* xr = static_cast<const uint16_t*>(x) + r0 * p.x_stride;
    GemmArgs g;
    std::memset(&g, 0, sizeof g);
    g.a_rows = a_rows_of(a.n);
    ok = make_map(&g.a, type, xr, a.n, p.hidden, p.x_stride, g.a_rows) &&
         make_map(&g.b, type, w, p.vocab, p.hidden, p.w_stride, kBN / 2) &&
         (!a.top || make_map(&g.c, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.logits, a.n, p.vocab, a.logit_stride, 32));
    if (!ok) return cudaSuccess;
    g.m = a.n;
    g.m_tiles = (int)ceil_div(a.n, kBM);
    g.k_blocks = (int)ceil_div(p.hidden, kBK);
    g.chunk = kChunk;
    g.splits = 1;
    g.head = a.head;
    g.targets = a.targets;
    g.target_logit = reinterpret_cast<float*>(ws + l.target_logit);
    g.scale_log2e = a.scale * kLog2e;
    g.least = a.least;
    g.logit_stride = a.logit_stride;
    auto product = [&](int64_t v0, int64_t v1) {
        const int64_t s0 = v0 / kStrip;
        g.b_y0 = (int)v0;
        g.n = v1 - v0;
        g.n_tiles = (int)ceil_div(g.n, kBN);
        g.part = const_cast<float2*>(a.part) + s0 * a.n;
        g.part_t = const_cast<float*>(a.part_t) + s0 * a.n;
        g.logits = const_cast<float*>(a.logits) + v0;
        g.withhold = first && v0 == 0 && withheld_product() > 0;
        return !a.top ? gemm<kEpiStat, false, false>(p.dtype, g, s)
               : v0 == 0 ? gemm<kEpiKeep, false, false>(p.dtype, g, s) : gemm<kEpiSome, false, false>(p.dtype, g, s);
    };
    cudaError_t e = product(0, a.least ? kSample : p.vocab);
    if (a.least) {
        if (e == cudaSuccess) e = launch_top<false>(a, s);
        if (e == cudaSuccess) e = product(kSample, p.vocab);
    }
    if (e == cudaSuccess) e = launch_after(k_lp_join, dim3((unsigned)ceil_div(a.n, kJoinRows)), kJoinThreads, 0, s, a);
    if (e == cudaSuccess && a.top) e = launch_top<true>(a, s);
    return e;
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" {

zero_status_t zero_lp_plan(int64_t tokens, int64_t vocab, int64_t hidden, int32_t dtype, int64_t x_stride, int64_t w_stride,
                           int64_t piece, int32_t top, zero_lp_plan_t* out)
{
    if (!out) return set_error(ZERO_EINVAL, "zero_lp_plan: out is NULL");
    if (top < 0) return set_error(ZERO_EINVAL, "zero_lp_plan: top must be >= 0");
    if (top > kMostTop) return set_error(ZERO_EUNSUPPORTED, "zero_lp_plan: top exceeds 32");
    zero_ce_plan_t c;
    const zero_status_t st = zero_ce_plan(tokens, vocab, hidden, dtype, x_stride, w_stride, piece, &c);
    if (st != ZERO_OK) return st;
    std::memset(out, 0, sizeof *out);
    out->tokens = tokens;
    out->vocab = vocab;
    out->hidden = hidden;
    out->x_stride = c.x_stride;
    out->w_stride = c.w_stride;
    out->piece = c.piece;
    out->dtype = dtype;
    out->splits = c.splits;
    out->top = top;
    out->rows = rows_at_once(vocab, top);
    const int64_t forward = lp_layout(*out, few_tokens(c)).end;
    out->workspace_bytes = forward > c.workspace_bytes ? forward : c.workspace_bytes;
    out->flops_forward = c.flops_forward;
    out->flops_backward = c.flops_backward;
    return ZERO_OK;
}

zero_status_t zero_lp_forward(const zero_lp_plan_t* plan, const void* x, const void* w, const int64_t* targets, float scale,
                              float* logp, float* lse, float* entropy, float* top_logp, int64_t* top_index, void* workspace,
                              void* stream)
{
    NvtxRange range("zero_lp_forward");
    zero_ce_plan_t c;
    const zero_status_t st = check_lp_plan(plan, &c);
    if (st != ZERO_OK) return st;
    const zero_lp_plan_t& p = *plan;
    if (!(scale > 0.0f) || !std::isfinite(scale * kLog2e))
        return set_error(ZERO_EINVAL, "zero_lp_forward: scale must be positive and finite");
    if (!workspace) return set_error(ZERO_ENOMEM, "zero_lp_forward: workspace is NULL");
    if (p.tokens && (!x || !w || !targets || !logp || !lse || (p.top && (!top_logp || !top_index))))
        return set_error(ZERO_ENOMEM, "zero_lp_forward: a buffer is NULL");
    if (!p.top && (top_logp || top_index))
        return set_error(ZERO_EINVAL, "zero_lp_forward: the plan has no alternatives");
    if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(workspace, 16) || !aligned_to(targets, 8) ||
        !aligned_to(logp, 4) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(top_logp, 4) ||
        !aligned_to(top_index, 8))
        return set_error(ZERO_EALIGN, "zero_lp_forward: x, w and workspace must be 16-byte aligned, the others to their type");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    cudaError_t e = launch_after(k_lp_clear, dim3(1), 1, 0, s, reinterpret_cast<CeHead*>(ws));
    const bool few = few_tokens(c);
    const LpLayout l = lp_layout(p, few);
    for (int64_t r0 = 0; r0 < p.tokens && e == cudaSuccess; r0 += p.rows) {
        LpArgs a;
        std::memset(&a, 0, sizeof a);
        a.head = reinterpret_cast<CeHead*>(ws);
        a.targets = targets + r0;
        a.n = p.tokens - r0 < p.rows ? p.tokens - r0 : p.rows;
        a.vocab = p.vocab;
        a.scale = scale;
        a.part = reinterpret_cast<float2*>(ws + l.part);
        a.part_t = reinterpret_cast<float*>(ws + l.part_t);
        a.strips = (int)strips_of(p.vocab);
        a.target_logit = reinterpret_cast<float*>(ws + l.target_logit);
        a.logp = logp + r0;
        a.lse = lse + r0;
        a.entropy = entropy ? entropy + r0 : nullptr;
        a.stat = reinterpret_cast<float2*>(ws + l.stat);
        a.top = p.top;
        a.logits = reinterpret_cast<const float*>(ws + l.logits);
        a.logit_stride = logit_stride(p.vocab);
        a.cand = reinterpret_cast<uint64_t*>(ws + l.cand);
        a.least = p.top && !all_kept(p) ? reinterpret_cast<float*>(ws + l.least) : nullptr;
        a.top_logp = top_logp + r0 * p.top;
        a.top_index = top_index + r0 * p.top;
        if (few) {
            const int64_t blocks = few_blocks(c);
            e = p.dtype == ZERO_BF16 ? launch_few<kBF16>(p, blocks, x, w, ws, l, a, s) : launch_few<kF16>(p, blocks, x, w, ws, l, a, s);
            break;
        }
        if (!encode_fn()) return set_error(ZERO_ECUDA, "zero_lp_forward: the driver has no cuTensorMapEncodeTiled");
        bool ok = true;
        e = forward_rows(p, x, w, ws, l, a, r0, r0 == 0, s, ok);
        if (!ok) return set_error(ZERO_ECUDA, "zero_lp_forward: cuTensorMapEncodeTiled refused a buffer");
    }
    return e == cudaSuccess ? ZERO_OK : cuda_failed(e, "zero_lp_forward");
}

zero_status_t zero_lp_backward(const zero_lp_plan_t* plan, const void* x, const void* w, const int64_t* targets, float scale,
                               const float* lse, const float* entropy, const float* dlogp, const float* dentropy,
                               float grad_scale, void* dx, void* dw, void* workspace, void* stream)
{
    NvtxRange range("zero_lp_backward");
    zero_ce_plan_t p;
    const zero_status_t st = check_lp_plan(plan, &p);
    if (st != ZERO_OK) return st;
    if (!(scale > 0.0f) || !std::isfinite(scale * kLog2e))
        return set_error(ZERO_EINVAL, "zero_lp_backward: scale must be positive and finite");
    if (!std::isfinite(grad_scale * scale)) return set_error(ZERO_EINVAL, "zero_lp_backward: grad_scale is not finite");
    if (!workspace) return set_error(ZERO_ENOMEM, "zero_lp_backward: workspace is NULL");
    if (p.tokens && (!x || !w || !targets || !lse || (dentropy && !entropy)))
        return set_error(ZERO_ENOMEM, "zero_lp_backward: a buffer is NULL");
    if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(dx, 16) || !aligned_to(dw, 16) || !aligned_to(workspace, 16) ||
        !aligned_to(targets, 8) || !aligned_to(lse, 4) || !aligned_to(entropy, 4) || !aligned_to(dlogp, 4) ||
        !aligned_to(dentropy, 4))
        return set_error(ZERO_EALIGN, "zero_lp_backward: x, w, dx, dw and workspace must be 16-byte aligned, the others to their type");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!p.tokens || (!dx && !dw)) {                  // no products; the workspace has no error of this call
        if (dw) k_ce_zero<<<1024, 256, 0, s>>>(static_cast<uint16_t*>(dw), p.vocab, p.hidden, p.w_stride);
        cudaError_t e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, sizeof(CeHead), s);
        return e == cudaSuccess ? ZERO_OK : cuda_failed(e, "zero_lp_backward");
    }
    if (!encode_fn()) return set_error(ZERO_ECUDA, "zero_lp_backward: the driver has no cuTensorMapEncodeTiled");
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    const CeLayout l = layout_of(p);
    CeHead* head = reinterpret_cast<CeHead*>(ws);
    float* coef = reinterpret_cast<float*>(ws + l.coef);
    float* coef_h = reinterpret_cast<float*>(ws + l.target_logit);   // free in a backward pass
    const float up = p.dtype == ZERO_FP16 ? 16384.0f : 1.0f;
    cudaError_t e = launch_after(k_lp_factors, dim3(1), 1024, 0, s, head, targets, p.tokens, p.vocab, dlogp, dentropy,
                                 grad_scale * scale, up, coef, coef_h);
    GemmArgs base;
    std::memset(&base, 0, sizeof base);
    base.head = head;
    base.targets = targets;
    base.lse = lse;
    base.coef = coef;
    base.coef_h = dentropy ? coef_h : nullptr;
    base.entropy = entropy;
    base.scale_log2e = scale * kLog2e;
    bool ok = true;
    if (e == cudaSuccess) e = launch_gradients<kEpiLpGrad>(p, l, base, x, w, dx, dw, ws, s, ok);
    if (!ok) return set_error(ZERO_ECUDA, "zero_lp_backward: cuTensorMapEncodeTiled refused a buffer");
    return e == cudaSuccess ? ZERO_OK : cuda_failed(e, "zero_lp_backward");
}

zero_status_t zero_lp_status(const zero_lp_plan_t* plan, const void* workspace, void* stream)
{
    zero_ce_plan_t c;
    const zero_status_t st = check_lp_plan(plan, &c);
    if (st != ZERO_OK) return st;
    if (!workspace) return set_error(ZERO_ENOMEM, "zero_lp_status: workspace is NULL");
    if (!aligned_to(workspace, 16)) return set_error(ZERO_EALIGN, "zero_lp_status: workspace is not 16-byte aligned");
    uint32_t err = 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(&err, workspace, 4, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_failed(e, "zero_lp_status");
    return err ? set_error(ZERO_ETIMEOUT, "a bounded wait inside the log probabilities' kernels ran out") : ZERO_OK;
}

}  // extern "C"
