// Softmax cross entropy over a large vocabulary without stored logits: the
// plan and the small kernels around its three products on the tensor cores.
#include "dev_vocab.cuh"
#include "nvtx_ranges.h"

namespace zg {

using namespace vocab;

namespace {

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
template <int DT, int T>
__global__ void __launch_bounds__(kFewThreads, 3) k_ce_few(const uint16_t* x, int64_t x_stride, const uint16_t* w,
                                                           int64_t w_stride, int64_t hidden, float2* part,
                                                           float* target_logit, const __grid_constant__ JoinArgs a)
{
    wait_prev_grid();
    extern __shared__ __align__(16) uint16_t xs[];    // [T][wide]
    __shared__ float2 sh[kFewThreads / 32][T];
    __shared__ uint32_t last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    int have = 0;
    few_logits<DT, T>(x, x_stride, w, w_stride, hidden, a.vocab, a.targets, xs, target_logit, [&](int64_t, const float (&z)[T]) {
#pragma unroll
        for (int t = 0; t < T; t++)
            if (lane == have) held[t] = z[t];
        if (++have == 32) {
            flush();
            have = 0;
        }
    });
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

// ---- host -------------------------------------------------------------------------
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
zero_status_t cuda_failed(cudaError_t e, const char* what)
{
    char msg[200];
    std::snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return set_error(ZERO_ECUDA, msg);
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
    if (!p.tokens || (!dx && !dw)) {                  // no products; the workspace has no error of this call
        if (dw) k_ce_zero<<<1024, 256, 0, s>>>(static_cast<uint16_t*>(dw), p.vocab, p.hidden, p.w_stride);
        cudaError_t e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, sizeof(CeHead), s);
        return e == cudaSuccess ? ZERO_OK : cuda_failed(e, "zero_ce_backward");
    }
    if (!encode_fn()) return set_error(ZERO_ECUDA, "zero_ce_backward: the driver has no cuTensorMapEncodeTiled");
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    const CeLayout l = layout_of(p);
    CeHead* head = reinterpret_cast<CeHead*>(ws);
    float* coef = reinterpret_cast<float*>(ws + l.coef);
    const float up = p.dtype == ZERO_FP16 ? 16384.0f : 1.0f;
    k_ce_factors<<<1, 1024, 0, s>>>(head, targets, p.tokens, p.vocab, dloss, grad_scale, up, coef);
    cudaError_t e = cudaGetLastError();
    GemmArgs base;
    std::memset(&base, 0, sizeof base);
    base.head = head;
    base.targets = targets;
    base.lse = lse;
    base.coef = coef;
    bool ok = true;
    if (e == cudaSuccess) e = launch_gradients<kEpiGrad>(p, l, base, x, w, dx, dw, ws, s, ok);
    if (!ok) return set_error(ZERO_ECUDA, "zero_ce_backward: cuTensorMapEncodeTiled refused a buffer");
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
