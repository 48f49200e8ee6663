// The small kernels around the post-training operators' row kernels: the teacher's normalisers and
// the responses' token counts (distill), and the pairs' losses and coefficients (pref).
#include <algorithm>

#include "post.cuh"

namespace rlk {

namespace {

constexpr int kPrepThreads = 256;

// The token range of response i, clamped into [0, T]; raises RL_ERR_SEQLENS where it is malformed.
__device__ __forceinline__ int2 seq_range(const int32_t *cu, int S, int T, int i, uint32_t *status) {
    int b = __ldg(cu + i), e = __ldg(cu + i + 1);
    if ((b < 0) || (e < b) || (e > T) || (i == 0 && b != 0) || (i == S - 1 && e != T)) {
        if (threadIdx.x == 0) post_raise(status, RL_ERR_SEQLENS);
        b = min(max(b, 0), T);
        e = min(max(e, b), T);
    }
    return make_int2(b, e);
}

// Adds e^v, v <= 88, to a sum.
__device__ __forceinline__ void add_exp(Sum2 &sum, float v) {
    if (v < -87.f) return;  // below 2e-38
    float hi, lo;
    exp_parts(v, hi, lo);
    sum.add(hi, lo);
}

// Blocks [0, S) count the mask=1 tokens of one response each; the others take eight rows each, a
// warp per row: ln of the teacher's normaliser, its remaining mass and its total mass less 1. A teacher
// given by log-probs keeps them (m = ln sum = 0) and its remaining mass is 1 - sum q, the sum held in two
// parts: with most of the mass in the entries, fp32 would leave it no digits. 6000 rows of 128 entries:
// 6.7 us, a launch and two dependent loads (6 MB would take 1); the rows' launch begins as it ends.
__global__ void __launch_bounds__(kPrepThreads) distill_prep_kernel(DistillPrepParams p) {
    __shared__ int s_i[32];
    if (blockIdx.x == 0)
        for (int k = threadIdx.x; k < p.n_counters; k += kPrepThreads) p.counters[k] = 0;
    if ((int)blockIdx.x < p.S) {
        const int i = blockIdx.x;
        const int2 r = seq_range(p.cu_seqlens, p.S, p.T, i, p.status);
        int n = 0;
#pragma unroll 4
        for (int t = r.x + threadIdx.x; t < r.y; t += kPrepThreads) n += __ldg(p.mask + t) ? 1 : 0;
        n = block_sum_i32(n, s_i);
        if (threadIdx.x == 0) {
            p.seq_n[i] = n;
            if (n == 0) post_raise(p.status, RL_ERR_EMPTY_SEQ);
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t t = ((int64_t)blockIdx.x - p.S) * (kPrepThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.T || !__ldg(p.mask + t)) return;
    const int32_t *ids = p.ids + t * p.ldk;
    const float *vals = p.vals + t * p.ldk;
    float4 rec = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.tail) {
        Sum2 q{0.f, 0.f};
        bool nan = false;
#pragma unroll 4
        for (int k = lane; k < p.K; k += 32) {
            const float v = __ldg(vals + k);
            if (__ldg(ids + k) < 0) continue;
            nan |= isnan(v);
            add_exp(q, v);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, q.hi, off), l = __shfl_xor_sync(0xffffffffu, q.lo, off);
            q.add(h, l);
        }
        const float rest = fmaxf((1.f - q.hi) - q.lo, p.floor);
        nan = __any_sync(0xffffffffu, nan);
        rec.z = nan ? __int_as_float(0x7fc00000) : rest;
        rec.w = ((q.hi - 1.f) + q.lo) + rest;
    } else {
        float m = -INFINITY;
        bool nan = false;
        for (int k = lane; k < p.K; k += 32) {
            if (__ldg(ids + k) < 0) continue;
            const float v = __ldg(vals + k);
            nan |= isnan(v);
            m = fmaxf(m, v);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        nan = __any_sync(0xffffffffu, nan);
        float s = 0.f;
        if (m > -INFINITY)
            for (int k = lane; k < p.K; k += 32)
                if (__ldg(ids + k) >= 0) s += expf(__ldg(vals + k) - m);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
        rec.x = m;
        rec.y = logf(s);
        rec.w = nan ? __int_as_float(0x7fc00000) : m > -INFINITY ? 0.f : -1.f;  // no entry with mass: Q = 0
    }
    if (lane == 0) p.rec[t] = rec;
}

// One block per pair (responses 2j and 2j + 1), half of its warps on each: the log ratios in token order
// per thread and a fixed tree, held in two fp32 parts (tens of thousands of log-probs near -10 sum to
// differences near 1), the pair's loss and the coefficients dL/dlogp of its tokens. The last block sums the
// losses in pair order. The loss itself needs fp32 only: the device's fp64 exponentials and logarithms took
// 14 us of a launch.
__global__ void __launch_bounds__(kPrepThreads) pref_pairs_kernel(PrefPairParams p) {
    constexpr int kHalf = kPrepThreads / 2, kHalfWarps = kHalf / 32;
    __shared__ Sum2 s_ratio[2][kHalfWarps], s_lp[2][kHalfWarps];
    __shared__ int s_n[2][kHalfWarps];
    __shared__ Sum2 s_loss[kPrepThreads / 32];
    __shared__ int s_last;
    const int j = blockIdx.x, P = p.S / 2;
    grid_dependency_wait();  // the log-probs
    if (j == 0 && threadIdx.x < 8) p.tickets[threadIdx.x] = 0;
    const int h = threadIdx.x / kHalf, lane = threadIdx.x & 31, warp = (threadIdx.x % kHalf) / 32;
    {
        int b = __ldg(p.cu_seqlens + 2 * j + h), e = __ldg(p.cu_seqlens + 2 * j + h + 1);
        const int i = 2 * j + h;
        if ((b < 0) || (e < b) || (e > p.T) || (i == 0 && b != 0) || (i == p.S - 1 && e != p.T)) {
            if (threadIdx.x % kHalf == 0) post_raise(p.status, RL_ERR_SEQLENS);
            b = min(max(b, 0), p.T);
            e = min(max(e, b), p.T);
        }
        Sum2 ratio{0.f, 0.f}, lp{0.f, 0.f};
        int n = 0;
#pragma unroll 4
        for (int t = b + threadIdx.x % kHalf; t < e; t += kHalf) {
            const float x = p.logp[t], ref = p.logp_ref ? __ldg(p.logp_ref + t) : 0.f;
            if (!__ldg(p.mask + t)) continue;
            n += 1;
            if ((uint32_t)__ldg(p.targets + t) >= (uint32_t)p.V) continue;  // the token is excluded
            ratio.add(x, 0.f);
            ratio.add(-ref, 0.f);
            lp.add(x, 0.f);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float a = __shfl_xor_sync(0xffffffffu, ratio.hi, off), c = __shfl_xor_sync(0xffffffffu, ratio.lo, off);
            const float d = __shfl_xor_sync(0xffffffffu, lp.hi, off), f = __shfl_xor_sync(0xffffffffu, lp.lo, off);
            n += __shfl_xor_sync(0xffffffffu, n, off);
            ratio.add(a, c);
            lp.add(d, f);
        }
        if (lane == 0) {
            s_ratio[h][warp] = ratio;
            s_lp[h][warp] = lp;
            s_n[h][warp] = n;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        Sum2 r[2], lp{0.f, 0.f};
        int n[2];
        float per[2];
        for (int k = 0; k < 2; ++k) {
            r[k] = Sum2{0.f, 0.f};
            n[k] = 0;
            for (int w = 0; w < kHalfWarps; ++w) {
                r[k].add(s_ratio[k][w].hi, s_ratio[k][w].lo);
                if (k == 0) lp.add(s_lp[k][w].hi, s_lp[k][w].lo);
                n[k] += s_n[k][w];
            }
            per[k] = p.mean ? (n[k] > 0 ? 1.f / (float)n[k] : 0.f) : 1.f;
            if (p.mean && n[k] > 0) {  // the quotient of a two-part number: of its parts, with the first one's remainder
                const float q = r[k].hi / (float)n[k];
                r[k] = Sum2{q, fabsf(q) < INFINITY ? (fmaf(-q, (float)n[k], r[k].hi) + r[k].lo) / (float)n[k] : 0.f};
            }
        }
        if (n[0] == 0 || n[1] == 0) post_raise(p.status, RL_ERR_EMPTY_SEQ);
        Sum2 diff = r[0];
        diff.add(-r[1].hi, -r[1].lo);
        const float D = diff.hi + diff.lo, beta = p.beta, eps = p.smoothing;
        // D is infinite where a token of probability 0 was sampled: each kind's limit, and no 0 times infinity
        float loss, slope;  // of the pair's loss in D
        if (p.kind == RL_PREF_SIGMOID) {
            const float x = fmaf(beta, D, -p.margin);
            const float soft = log1pf(expf(-fabsf(x)));  // -ln sigma(|x|)
            loss = (1.f - eps) * (soft + fmaxf(-x, 0.f)) + (eps != 0.f ? eps * (soft + fmaxf(x, 0.f)) : 0.f);
            slope = beta * (eps / (1.f + expf(-x)) - (1.f - eps) / (1.f + expf(x)));
        } else if (p.kind == RL_PREF_HINGE) {
            const float x = fmaf(beta, D, -p.margin);
            loss = isnan(x) ? x : fmaxf(1.f - x, 0.f);
            slope = x < 1.f ? -beta : 0.f;
        } else {
            const float d = D - 0.5f / beta;
            loss = d * d;
            slope = 2.f * d;
        }
        if (isnan(D)) loss = slope = D;  // a row that is not finite: max() would hide it
        const float like = n[0] > 0 ? -(lp.hi + lp.lo) / (float)n[0] : 0.f;
        if (p.nll != 0.f) loss = fmaf(p.nll, like, loss);
        const float inv_p = 1.f / (float)P;
        p.coef[2 * j] = (slope * per[0] - (n[0] > 0 ? p.nll / (float)n[0] : 0.f)) * inv_p;
        p.coef[2 * j + 1] = -slope * per[1] * inv_p;
        p.pair32[j] = loss;
        if (p.pair_loss) p.pair_loss[j] = loss;
        if (p.seq_logratio) {
            p.seq_logratio[2 * j] = r[0].hi + r[0].lo;
            p.seq_logratio[2 * j + 1] = r[1].hi + r[1].lo;
        }
        __threadfence();
        s_last = atomicAdd(p.pairs_done, 1u) == (uint32_t)P - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    Sum2 L{0.f, 0.f};
    for (int k = threadIdx.x; k < P; k += kPrepThreads) L.add(p.pair32[k], 0.f);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, L.hi, off), c = __shfl_xor_sync(0xffffffffu, L.lo, off);
        L.add(a, c);
    }
    if (lane == 0) s_loss[threadIdx.x / 32] = L;
    __syncthreads();
    if (threadIdx.x == 0) {
        L = s_loss[0];
        for (int w = 1; w < kPrepThreads / 32; ++w) L.add(s_loss[w].hi, s_loss[w].lo);
        const double total = ((double)L.hi + (double)L.lo) / P;
        p.loss[0] = (float)total;
        if (p.loss_f64) p.loss_f64[0] = total;
        if (!isfinite(total)) post_raise(p.status, RL_ERR_NONFINITE);
    }
}

}  // namespace

cudaError_t launch_distill_prep(const DistillPrepParams &p, cudaStream_t stream) {
    const int rows_per = kPrepThreads / 32;
    distill_prep_kernel<<<p.S + (p.T + rows_per - 1) / rows_per, kPrepThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_pref_pairs(const PrefPairParams &p, cudaStream_t stream) {
    // begins while the log-prob pass of the same call ends
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.S / 2));
    cfg.blockDim = dim3(kPrepThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pref_pairs_kernel, p);
}

}  // namespace rlk
