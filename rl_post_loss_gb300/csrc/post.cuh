// The vocabulary-wide post-training operators: parameters and per-row mathematics shared by their
// kernels (sm_103a).
//
//   logp     logp_t = z_y - log sum_v exp z_v and the entropy, forward only
//   policy   Eq. (1) (or DIS) plus a KL term to a reference policy
//   distill  KL between a teacher known by its top entries and the student softmax(z / tau)
//   pref     a preference loss over pairs of responses
//
// Every gradient row is one coefficient times the row's exponentials, plus a few entries of its own
// (the sampled token, or the teacher's entries). Exponentials are taken in base 2 against the row's
// own maximum, 2^{c (z_v - m)} with c = log2(e) / tau and m = max z_v, and the sum S is kept apart
// from m: ln p_v = (z_v - m) / tau - ln S has no large term to cancel, so a log-prob near 0
// keeps its digits, and p_v = 2^{c (z_v - m)} / S costs one multiplication by a per-row constant.
// The difference is taken before the factor c: it is exact for entries near the maximum, and 0 at
// it, whatever the size of the logits.
#pragma once

#include <cfloat>

#include "common.cuh"

namespace rlk {

// ---------------------------------------------------------------- pairs of fp32

// Two fp32 values in a 64-bit register pair: one instruction adds or multiplies both.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ---------------------------------------------------------------- sums in two parts

// A sum held as two fp32 values, |lo| a rounding of hi at most: about 48 bits at fp32's speed (the
// device's fp64 units are some sixty times slower). An infinite term makes an infinite sum.
struct Sum2 {
    float hi, lo;
    __device__ __forceinline__ void add(float h, float l) {
        const float s = __fadd_rn(hi, h), b = __fsub_rn(s, hi);
        const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(h, b));  // Knuth's exact error of hi + h
        l = __fadd_rn(__fadd_rn(lo, l), err);
        const float t = __fadd_rn(s, l);
        const bool fin = fabsf(t) < INFINITY;  // else err is inf - inf where s is infinite: s itself is the sum
        lo = fin ? __fsub_rn(l, __fsub_rn(t, s)) : 0.f;
        hi = fin ? t : s;
    }
};

// e^v = hi + lo for |v| < 88, within 1.3e-8 relative (2e-9 rms): v = n ln 2 + r in Cody and Waite's two parts of
// ln 2 (the first has 10 bits, so that n times it is exact), then e^r = 1 + r + the rest of Taylor's series,
// of which only the rest, below 0.07, is rounded to fp32.
__device__ __forceinline__ void exp_parts(float v, float &hi, float &lo) {
    const float n = rintf(v * kLog2e);
    const float a = fmaf(-n, 0.693359375f, v), b = n * 2.12194440e-4f;
    const float r = __fadd_rn(a, b), rl = __fsub_rn(b, __fsub_rn(r, a));
    float q = 1.f / 40320.f;
    q = fmaf(r, q, 1.f / 5040.f);
    q = fmaf(r, q, 1.f / 720.f);
    q = fmaf(r, q, 1.f / 120.f);
    q = fmaf(r, q, 1.f / 24.f);
    q = fmaf(r, q, 1.f / 6.f);
    q = fmaf(r, q, 0.5f);
    const float one = __fadd_rn(1.f, r), ol = __fsub_rn(r, __fsub_rn(one, 1.f));
    const float scale = ex2_approx(n);  // a power of two: exact
    hi = one * scale;
    lo = (fmaf(r * r, q, rl) + ol) * scale;
}

// What rounding left of ln(x + x_lo), l = ln x in fp32: Newton's step (x + x_lo) e^{-l} - 1, to 1.3e-8 (half a
// step of l itself is 2.4e-7 from 4 to 8).
__device__ __forceinline__ float log_rest(float x, float x_lo, float l) {
    float hi, lo;
    exp_parts(-l, hi, lo);
    return fmaf(x_lo, hi, fmaf(x, lo, fmaf(x, hi, -1.f)));
}

// The rounding error of s = a - b (Knuth), for finite values.
__device__ __forceinline__ float diff_rest(float a, float b, float s) {
    const float t = __fsub_rn(s, a);
    return __fsub_rn(__fsub_rn(a, __fsub_rn(s, t)), __fadd_rn(b, t));
}

// (a + lo) - b, rounded once where it is finite.
__device__ __forceinline__ float diff_of(float a, float lo, float b) {
    const float s = __fsub_rn(a, b);
    return fabsf(s) < INFINITY ? __fadd_rn(s, __fadd_rn(diff_rest(a, b, s), lo)) : s;
}

// ---------------------------------------------------------------- logits of either type

template <typename T>
struct PostVec;

template <>
struct PostVec<float> {
    static constexpr int kElems = 4;
    using Tag = uint32_t;
    static constexpr Tag kNegInf = 0xff800000u;
    // a group of -inf
    __device__ __forceinline__ static uint4 none() { return make_uint4(kNegInf, kNegInf, kNegInf, kNegInf); }
    __device__ __forceinline__ static void decode(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    static constexpr int kPairs = 2;
    __device__ __forceinline__ static void pairs(const uint4 &v, f32x2 (&x)[2]) {
        x[0] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ __forceinline__ static uint4 from_pairs(const f32x2 (&x)[2]) {
        float a, b, c, d;
        unpack2(x[0], a, b);
        unpack2(x[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
    // The largest of the group (NaN counts as missing).
    __device__ __forceinline__ static float max_of(const uint4 &v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    __device__ __forceinline__ static uint4 encode(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    __device__ __forceinline__ static float load1(const void *p, int64_t v) { return reinterpret_cast<const float *>(p)[v]; }
    __device__ __forceinline__ static void store1(void *p, int64_t v, float x) { reinterpret_cast<float *>(p)[v] = x; }
};

template <>
struct PostVec<__nv_bfloat16> {
    static constexpr int kElems = 8;
    using Tag = uint16_t;
    static constexpr Tag kNegInf = 0xff80u;
    __device__ __forceinline__ static uint4 none() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    __device__ __forceinline__ static void decode(const uint4 &v, float (&x)[8]) {
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
    }
    static constexpr int kPairs = 4;
    __device__ __forceinline__ static void pairs(const uint4 &v, f32x2 (&x)[4]) {
        x[0] = pack2(bf16_lo(v.x), bf16_hi(v.x));
        x[1] = pack2(bf16_lo(v.y), bf16_hi(v.y));
        x[2] = pack2(bf16_lo(v.z), bf16_hi(v.z));
        x[3] = pack2(bf16_lo(v.w), bf16_hi(v.w));
    }
    __device__ __forceinline__ static uint32_t from_pair(f32x2 x) {
        float a, b;
        unpack2(x, a, b);
        return pack_bf16x2(a, b);
    }
    __device__ __forceinline__ static uint4 from_pairs(const f32x2 (&x)[4]) {
        return make_uint4(from_pair(x[0]), from_pair(x[1]), from_pair(x[2]), from_pair(x[3]));
    }
    __device__ __forceinline__ static float max_of(const uint4 &v) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ static uint4 encode(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    __device__ __forceinline__ static float load1(const void *p, int64_t v) {
        return __uint_as_float((uint32_t) reinterpret_cast<const unsigned short *>(p)[v] << 16);
    }
    __device__ __forceinline__ static void store1(void *p, int64_t v, float x) {
        reinterpret_cast<__nv_bfloat16 *>(p)[v] = __float2bfloat16_rn(x);
    }
};

// ---------------------------------------------------------------- running statistics

// Running softmax statistics of part of a row: the reference m (its maximum), s = sum 2^d and
// u = sum 2^d d with d = c (z - m). They start from a finite reference point, so that a -inf logit
// is 2^-inf = 0 against it; merging a start that saw nothing scales its zero sums by 0.
struct PostStats {
    float m, s, u;
};
constexpr PostStats kPostStart{-FLT_MAX, 0.f, 0.f};

// Where d is below this, 2^d is 0 in fp32: products 2^d d hold d here, so that they are 0 and not
// 0 times infinity.
constexpr float kNoWeight = -1024.f;

// Moves partial statistics to the reference M >= st.m. ex2.approx truncates (its results are 5e-8
// low on average), which a chain of merges would add up: the factor of a merge is exp2f's.
template <bool kEnt, bool kExact = true>
__device__ __forceinline__ void post_rescale(PostStats &st, float M, float c) {
    const float dm = __fmul_rn(__fsub_rn(st.m, M), c);
    const float f = kExact ? exp2f(dm) : ex2_approx(dm);
    if (kEnt) st.u = __fmul_rn(f, __fadd_rn(st.u, __fmul_rn(fmaxf(dm, kNoWeight), st.s)));
    st.s = __fmul_rn(st.s, f);
    st.m = M;
}

// The sum of a group, in pairs.
template <int N>
__device__ __forceinline__ float group_sum(float (&e)[N]) {
#pragma unroll
    for (int h = N / 2; h > 0; h >>= 1)
#pragma unroll
        for (int k = 0; k < h; ++k) e[k] += e[k + h];
    return e[0];
}

// Adds the terms of a group to the statistics; no entry exceeds st.m. A logit of -inf adds 0 to u
// (0 log 0 = 0), while e comes from d itself, so that a NaN reaches s.
template <bool kEnt, int N>
__device__ __forceinline__ void post_add(PostStats &st, const float (&x)[N], float c) {
    float e[N], u[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float d = (x[k] - st.m) * c;
        e[k] = ex2_approx(d);
        if (kEnt) u[k] = e[k] * fmaxf(d, kNoWeight);
    }
    // the group is summed by itself: single terms below half a step of s would all be lost
    st.s += group_sum(e);
    if (kEnt) st.u += group_sum(u);
}

// Folds a group of logits into the statistics (one rescale at most).
template <bool kEnt, int N>
__device__ __forceinline__ void post_fold(PostStats &st, const float (&x)[N], float c) {
    float mv = x[0];
#pragma unroll
    for (int k = 1; k < N; ++k) mv = fmaxf(mv, x[k]);
    if (mv > st.m) post_rescale<kEnt, false>(st, mv, c);
    post_add<kEnt>(st, x, c);
}

// A thread's running statistics with the sums held as two halves (even and odd entries).
struct PostAcc {
    float m;
    f32x2 s, u;
    __device__ __forceinline__ PostStats stats() const {
        float a, b, x, y;
        unpack2(s, a, b);
        unpack2(u, x, y);
        return PostStats{m, a + b, x + y};
    }
};
__device__ __forceinline__ PostAcc post_acc() { return PostAcc{-FLT_MAX, 0ull, 0ull}; }

// Folds M 16-byte groups: one comparison with the reference for all of them, so that their
// exponentials overlap, and one addition to the running sums.
template <typename T, bool kEnt, int M>
__device__ __forceinline__ void post_fold_groups(PostAcc &st, const uint4 (&v)[M], float c) {
    using VT = PostVec<T>;
    constexpr int P = VT::kPairs;
    float mv = VT::max_of(v[0]);
#pragma unroll
    for (int i = 1; i < M; ++i) mv = fmaxf(mv, VT::max_of(v[i]));
    if (mv > st.m) {
        const float dm = (st.m - mv) * c;
        const float f = ex2_approx(dm);
        if (kEnt) {
            const float h = fmaxf(dm, kNoWeight);
            st.u = mul2(pack2(f, f), add2(st.u, mul2(pack2(h, h), st.s)));
        }
        st.s = mul2(st.s, pack2(f, f));
        st.m = mv;
    }
    const f32x2 nm = pack2(-st.m, -st.m), cc = pack2(c, c);
    f32x2 es = 0ull, us = 0ull;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        f32x2 x[P], u[P];
        VT::pairs(v[i], x);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            float a, b;
            unpack2(mul2(add2(x[k], nm), cc), a, b);
            x[k] = pack2(ex2_approx(a), ex2_approx(b));
            if (kEnt) u[k] = mul2(x[k], pack2(fmaxf(a, kNoWeight), fmaxf(b, kNoWeight)));
        }
#pragma unroll
        for (int h = P / 2; h > 0; h >>= 1)
#pragma unroll
            for (int k = 0; k < h; ++k) {
                x[k] = add2(x[k], x[k + h]);
                if (kEnt) u[k] = add2(u[k], u[k + h]);
            }
        es = i == 0 ? x[0] : add2(es, x[0]);
        if (kEnt) us = i == 0 ? u[0] : add2(us, u[0]);
    }
    st.s = add2(st.s, es);
    if (kEnt) st.u = add2(st.u, us);
}

// dz of a 16-byte group: a 2^{c (z - m)}.
template <typename T>
__device__ __forceinline__ uint4 post_grad_group(const uint4 &v, float a, float m, float c) {
    using VT = PostVec<T>;
    constexpr int P = VT::kPairs;
    const f32x2 nm = pack2(-m, -m), cc = pack2(c, c), aa = pack2(a, a);
    f32x2 x[P];
    VT::pairs(v, x);
#pragma unroll
    for (int k = 0; k < P; ++k) {
        float p, q;
        unpack2(mul2(add2(x[k], nm), cc), p, q);
        x[k] = mul2(pack2(ex2_approx(p), ex2_approx(q)), aa);
    }
    return VT::from_pairs(x);
}

// Merges two partial statistics.
template <bool kEnt>
__device__ __forceinline__ PostStats post_merge(PostStats a, PostStats b, float c) {
    const float M = fmaxf(a.m, b.m);
    post_rescale<kEnt>(a, M, c);
    post_rescale<kEnt>(b, M, c);
    return PostStats{M, __fadd_rn(a.s, b.s), kEnt ? __fadd_rn(a.u, b.u) : 0.f};
}

// Merges the lanes' statistics: their maximum first, so that each is rescaled once; sums in a
// butterfly, which leaves the same bits in every lane. (kLanes: within groups of so many lanes.)
template <bool kEnt, int kLanes = 32>
__device__ __forceinline__ PostStats post_warp_merge(PostStats r, float c) {
    float M = r.m;
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    post_rescale<kEnt>(r, M, c);
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) {
        r.s = __fadd_rn(r.s, __shfl_xor_sync(0xffffffffu, r.s, off));
        if (kEnt) r.u = __fadd_rn(r.u, __shfl_xor_sync(0xffffffffu, r.u, off));
    }
    return r;
}

__device__ __forceinline__ void post_raise(uint32_t *status, rl_status code) {
    if (status) raise_status(status, code);  // the status word is optional for the entry points without a handle
}

// Waits for the launches before this one where it began while they ran.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------- parameters

// What a row adds to the batch's sums, written by whichever block took the row, and sums of them: over
// chunks of kSumRows consecutive rows, each by the block that finishes its last row, then over the chunks
// by the block that finishes the last one. Rows go to blocks as these come for them; the order of the
// additions depends on the sizes alone. (Short rows, a warp each: see line_sums.)
struct alignas(16) PostTerm {
    float loss, loss_lo, ent, kl;
};
constexpr int kSumRows = 256;
struct PostPartial {
    Sum2 loss, ent, kl;
    int32_t n, popped, clipped, masked;
};

// Words of PostRows::counters.
enum PostCount {
    kCountTickets = 0,   // rows handed out; for the pref gradient one for each part of the rows
    kCountDone = 8,      // chunks summed
    kCountChunks = 16    // from here: finished rows of each chunk
};
inline size_t post_chunks(int64_t T) { return (size_t)((T + kSumRows - 1) / kSumRows); }
inline size_t post_counters(int64_t T) { return (size_t)kCountChunks + post_chunks(T); }

struct PostRows {
    const void *logits;
    int64_t ld;
    void *dlogits;
    int64_t ldd;
    int32_t T, V, S;
    const int32_t *targets;
    const uint8_t *mask;         // may be null (logp): every row counts
    const int32_t *cu_seqlens;
    float *logp;                 // optional for policy and pref
    float *entropy;              // optional
    uint32_t *status;            // optional
    // sums of the batch: a term per row, a partial sum per chunk, and counters, all zero at
    // the launch (PostCount)
    PostTerm *terms;
    uint32_t *term_flags;        // [T] flags of the rows (policy; else null)
    PostPartial *partials;
    uint32_t *counters;
    float *loss;
    double *loss_f64;
};

// pref: the statistics of every row (m, S), kept from the log-prob pass for the gradient pass
struct LogpParams {
    PostRows r;
    float2 *stats;               // optional [T]
    uint32_t *zero;              // optional: a word this launch sets to 0 for the next one
};

struct KlTerm {
    const float *logp_ref;       // [T]
    float coef;
    int32_t estimator;           // rl_kl_estimator
    float *kl;                   // optional [T]
    float *mean_kl;              // optional [1]
};

struct PolicyParams {
    PostRows r;
    LossConsts c;
    const float *logp_old, *logp_infer;
    const float *token_adv;      // RL_ADV_PER_TOKEN, else null
    const float *teacher;        // RL_ADV_TEACHER_LOGP, else null
    const float *seq_adv, *seq_w;
    const double *seq_w64;
    const int32_t *seq_n;
    uint8_t *flags;              // optional
    int32_t *counts;             // optional
    float *mean_entropy;         // optional
    int32_t read_masked;         // the log-probs or entropies of masked tokens are wanted
    KlTerm kl;
};

struct DistillParams {
    PostRows r;
    const int32_t *ids;          // [T, ldk]
    const float *vals;           // [T, ldk]
    int64_t ldk;
    int32_t K, tail, reverse, per_token;
    float c;                     // log2(e) / tau
    float inv_tau, scale;
    const float4 *rec;           // [T] {m, ln sum, q_rest, Q} of the teacher's row (distill_prep)
    const int32_t *seq_n;        // [S]
    float *kl;                   // optional [T]
};

struct DistillPrepParams {
    const int32_t *ids;
    const float *vals;
    int64_t ldk;
    int32_t K, T, S, tail;
    float floor;
    const uint8_t *mask;
    const int32_t *cu_seqlens;
    float4 *rec;
    int32_t *seq_n;
    uint32_t *counters;          // PostRows::counters, set to 0
    int32_t n_counters;
    uint32_t *status;
};

struct PrefPairParams {
    int32_t T, S, V;
    const int32_t *targets;
    const uint8_t *mask;
    const int32_t *cu_seqlens;
    const float *logp, *logp_ref;
    int32_t kind, mean;
    float beta, smoothing, margin, nll;
    float *coef;                 // [S] dL/dlogp of the response's tokens
    float *pair32;               // [S/2]
    float *seq_logratio, *pair_loss;  // optional
    uint32_t *pairs_done;
    uint32_t *tickets;           // [8], set to 0 for the gradient's launch
    float *loss;
    double *loss_f64;
    uint32_t *status;
};

struct ScaleParams {
    PostRows r;  // counters: zeroed by the pairs' kernel
    const float2 *stats;         // [T] (m, S)
    const float *coef;           // [S]
};

cudaError_t launch_post_logp(const LogpParams &p, int dtype, cudaStream_t stream);
// launch_seg_prep that also sets the words of `zero` (the loss's counters) to 0.
cudaError_t launch_seg_prep(const SeqPrepParams &p, uint32_t *zero, int n_zero, cudaStream_t stream);
cudaError_t launch_post_policy(const PolicyParams &p, int dtype, cudaStream_t stream);
cudaError_t launch_distill_prep(const DistillPrepParams &p, cudaStream_t stream);
cudaError_t launch_post_distill(const DistillParams &p, int dtype, cudaStream_t stream);
cudaError_t launch_pref_pairs(const PrefPairParams &p, cudaStream_t stream);
cudaError_t launch_post_scale(const ScaleParams &p, int dtype, cudaStream_t stream);

constexpr int kDistillMaxK = 1024;    // the teacher's entries of a row stay in shared memory

// ---------------------------------------------------------------- the sampled token

// The statistics of a row are finite: no NaN or +inf logit, and not every logit -inf.
__device__ __forceinline__ bool post_finite(PostStats st) { return st.s > 0.f && st.s < INFINITY && fabsf(st.m) < INFINITY; }

// The row's statistics leave the sampled entry out: `rest` are those of the others, zy its logit.
// With x = sum_{v != y} 2^d 2^{c (m_rest - z_y)} = (1 - p_y) / p_y, ln p_y = -log1p(x) keeps its
// relative accuracy as p_y nears 1, which 1 + x has lost, and so does 1 - p_y = (the others' sum) / S.
struct PostToken {
    PostStats all;   // the whole row
    float others;    // the others' sum against the whole row's reference
    float logp;      // ln p_y (NaN where the row is not finite)
    float logp_lo;   // what rounding left of it: the loss takes its differences from near values
};
template <bool kEnt>
__device__ __forceinline__ PostToken post_target(PostStats rest, float zy) {
    PostToken r;
    if (zy >= rest.m) {
        const float dm = (rest.m - zy) * kLog2e, f = exp2f(dm);
        r.others = rest.s * f;
        r.all = PostStats{zy, r.others + ((zy - zy) + 1.f), 0.f};  // 1, or NaN for an infinite logit
        if (kEnt) r.all.u = f * fmaf(fmaxf(dm, kNoWeight), rest.s, rest.u);
        const float l = log1pf(r.others), s = r.all.s;
        r.logp = -l;
        // below 1/8 log1pf's own error is the smaller one
        r.logp_lo = r.others > 0.125f ? -log_rest(s, diff_rest(1.f, -r.others, s), l) : 0.f;
    } else {
        const float d = (zy - rest.m) * kLog2e, e = exp2f(d);
        r.others = rest.s;
        r.all = PostStats{rest.m, rest.s + e, 0.f};
        if (kEnt) r.all.u = fmaf(e, fmaxf(d, kNoWeight), rest.u);
        const float l = logf(r.all.s), dz = zy - rest.m;
        r.logp = dz - l;
        r.logp_lo = diff_rest(zy, rest.m, dz) + diff_rest(dz, l, r.logp) -
                    log_rest(r.all.s, diff_rest(rest.s, -e, r.all.s), l);
    }
    if (!post_finite(r.all)) r.logp = __int_as_float(0x7fc00000);
    if (!(fabsf(r.logp) < INFINITY)) r.logp_lo = 0.f;
    return r;
}

__device__ __forceinline__ float post_entropy(PostStats st) { return logf(st.s) - st.u / st.s * kLn2; }

// e^{-d} - 1 + d >= 0. Its terms cancel near 0, where its series is summed instead (|d| < 1:
// 1/2 - d/6 + ... times d^2, the first term left out is below 2 d / 13! of it). Both are worked out, without a
// branch, so that calls for several entries overlap.
__device__ __forceinline__ float post_k3(float d) {
    float q = 1.f / 479001600.f;
    q = fmaf(-d, q, 1.f / 39916800.f);
    q = fmaf(-d, q, 1.f / 3628800.f);
    q = fmaf(-d, q, 1.f / 362880.f);
    q = fmaf(-d, q, 1.f / 40320.f);
    q = fmaf(-d, q, 1.f / 5040.f);
    q = fmaf(-d, q, 1.f / 720.f);
    q = fmaf(-d, q, 1.f / 120.f);
    q = fmaf(-d, q, 1.f / 24.f);
    q = fmaf(-d, q, 1.f / 6.f);
    q = fmaf(-d, q, 0.5f);
    const float e = expf(-d), far = e < INFINITY ? (e - 1.f) + d : e;  // d = -inf: inf, not inf - inf
    return fabsf(d) < 1.f ? d * d * q : far;
}

// h k3(d), d = ln(h / o). Its part h e^{-d} is o: taken as such where h is 0, and where e^{-d} nears fp32's end,
// beyond which a subnormal h times infinity would stand for a term of at most o.
__device__ __forceinline__ float post_k3_term(float h, float o, float d) {
    const float near = h * post_k3(d), far = o + h * (d - 1.f);
    return h != 0.f ? (d > -80.f ? near : far) : o;  // (a NaN too)
}

// Estimators of KL(pi || pi_ref) from the sampled token, d = logp - logp_ref, and their derivative
// in logp: d; d^2 / 2; e^{-d} - 1 + d.
__device__ __forceinline__ void post_kl(int estimator, float d, float &kl, float &grad) {
    if (estimator == RL_KL_K1) {
        kl = d;
        grad = 1.f;
    } else if (estimator == RL_KL_K2) {
        kl = 0.5f * d * d;
        grad = d;
    } else {
        kl = post_k3(d);
        grad = -expm1f(-d);
    }
}

// What pass 2 of a row needs: dz_v = a 2^{c (z_v - m)}, and dz_y = gy at the sampled token.
struct RowGrad {
    float a, m, gy;
    int32_t y;  // -1: no entry of its own
};

// From kept statistics (pref): 1 - p_y from the log-prob.
__device__ __forceinline__ RowGrad post_row_grad(float g, PostStats st, float logp, int y) {
    return RowGrad{-g / st.s, st.m, -g * expm1f(logp), y};
}

// Everything a policy row needs besides its logits: what of the objective does not depend on the row's
// softmax is worked out with the record, as in the token records of the loss without a KL term.
struct PolicyTok {
    int32_t seq, y;        // seq < 0: outside every response
    int32_t m, ok;         // loss mask; the target is in the vocabulary
    uint32_t pre;          // flags and the advantage's sign
    float w, w_lo;         // weight, and what its rounding left of it
    float lref;            // logp_old, or the rollout log-prob (DIS)
    float cf, wcf;         // m pop A (m pop with the distillation advantage, m A for DIS), times w
    float ref, teacher;
};

__device__ __forceinline__ PolicyTok policy_load(const PolicyParams &p, int t, int i) {
    PolicyTok k;
    k.seq = i;
    k.y = __ldg(p.r.targets + t);
    k.ok = k.y >= 0 && k.y < p.r.V;
    k.m = i >= 0 && __ldg(p.r.mask + t) != 0;
    const float A = p.token_adv ? __ldg(p.token_adv + t) : (i >= 0 ? p.seq_adv[i] : 0.f);
    k.w = i >= 0 ? p.seq_w[i] : 0.f;
    k.w_lo = i >= 0 ? (float)(p.seq_w64[i] - (double)k.w) : 0.f;
    const float lo = __ldg(p.logp_old + t), li = __ldg(p.logp_infer + t);
    k.ref = __ldg(p.kl.logp_ref + t);
    k.teacher = p.teacher ? __ldg(p.teacher + t) : 0.f;
    k.pre = (k.m ? 0u : RL_FLAG_MASKED) | (k.ok ? 0u : RL_FLAG_BAD_TARGET) | (A > 0.f ? kPreAPos : 0u) | (A < 0.f ? kPreANeg : 0u);
    const bool in = k.m && k.ok;
    if (p.c.objective == RL_OBJ_DIS) {
        k.lref = li;
        k.cf = in ? A : 0.f;
    } else {
        const float d = __fsub_rn(lo, li);  // ln rho, one fp32 subtraction
        const bool in_bounds = (-p.c.ln_beta <= d) && (d <= p.c.ln_beta);
        k.pre |= in_bounds ? RL_FLAG_POP_IN_BOUNDS : 0u;
        k.lref = lo;
        const float pop = in && in_bounds ? (p.c.pop_indicator ? 1.f : expf(d)) : 0.f;
        k.cf = p.c.adv_teacher || pop == 0.f ? pop : pop * A;  // what a token left out has for an advantage does not matter
    }
    k.wcf = k.w * k.cf;
    return k;
}

// The token objective of Eq. (1) or DIS with its KL term, and the row's gradient.
struct PolicyRow {
    float logp, obj, kl;
    uint32_t flags;
    RowGrad grad;
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyParams &p, const PolicyTok &k, const PostToken &tok, bool read) {
    PolicyRow r;
    const LossConsts &c = p.c;
    // ln r: the branches go by one fp32 subtraction, its exponential by the difference before the log-prob was rounded
    const float logp = tok.logp, e = __fsub_rn(logp, k.lref), ln_r = diff_of(logp, tok.logp_lo, k.lref);
    const bool ok = k.ok && read;
    float g = 0.f;
    r.logp = logp;
    r.obj = 0.f;
    r.kl = 0.f;
    if (c.objective == RL_OBJ_DIS) {
        const bool gate = ok && e > c.clip_lo && e < c.clip_hi;
        r.flags = (k.pre & (RL_FLAG_MASKED | RL_FLAG_BAD_TARGET)) | (gate ? RL_FLAG_POP_IN_BOUNDS : 0u);
        if (gate && k.cf != 0.f) {
            const float ratio = expf(ln_r);
            r.obj = k.cf * ratio * logp;
            g = c.dis_stopgrad ? -k.wcf * ratio : -k.wcf * ratio * (1.f + logp);
        }
    } else {
        uint32_t pre = k.pre;
        float A = 1.f;  // cf and wcf carry it, unless it comes from the teacher
        if (c.adv_teacher) {
            A = ok ? __fsub_rn(k.teacher, logp) : 0.f;
            pre = (pre & ~(kPreAPos | kPreANeg)) | (A > 0.f ? kPreAPos : 0u) | (A < 0.f ? kPreANeg : 0u);
        }
        const bool clip = ok && (((pre & kPreAPos) && e > c.clip_hi) || ((pre & kPreANeg) && e < c.clip_lo));
        r.flags = (pre & kPreOut) | (clip ? RL_FLAG_CLIP_ACTIVE : 0u);
        if (k.cf != 0.f && A != 0.f) {
            const float ratio = expf(ln_r);
            r.obj = k.cf * A * (clip ? ((pre & kPreAPos) ? c.one_plus_eps_high : c.one_minus_eps_low) : ratio);
            g = clip ? 0.f : -k.wcf * A * ratio;
        }
    }
    if (k.m && k.ok) {
        float dkl;
        post_kl(p.kl.estimator, diff_of(logp, tok.logp_lo, k.ref), r.kl, dkl);
        if (p.kl.coef != 0.f) g = fmaf(k.w * p.kl.coef, dkl, g);  // no 0 times infinity
    }
    const float inv = 1.f / tok.all.s;
    r.grad = g == 0.f ? RowGrad{0.f, 0.f, 0.f, -1} : RowGrad{-g * inv, tok.all.m, g * (tok.others * inv), k.y};
    return r;
}

// Every per-token output of a policy row; returns what it adds to the sums.
template <bool kEnt>
__device__ __forceinline__ PostTerm policy_write(const PolicyParams &p, int t, const PolicyTok &k, const PostToken &tok, const PolicyRow &r,
                                                 bool read) {
    const bool ok = k.ok, m = k.m;
    const float nan = __int_as_float(0x7fc00000);
    const float H = kEnt && read ? post_entropy(tok.all) : 0.f;
    if (k.seq < 0) post_raise(p.r.status, RL_ERR_SEQLENS);
    if (!ok) post_raise(p.r.status, RL_ERR_TARGET_RANGE);
    if (read && !post_finite(tok.all)) post_raise(p.r.status, RL_ERR_NONFINITE);
    if (p.r.logp) p.r.logp[t] = ok ? r.logp : nan;
    if (p.r.entropy) p.r.entropy[t] = H;
    if (p.flags) p.flags[t] = (uint8_t)r.flags;
    if (p.kl.kl) p.kl.kl[t] = m && !ok ? nan : r.kl;
    // x = coef k - obj and w x in two parts each: a loss of centred advantages is a small difference of large sums,
    // and the same weight for a whole response, rounded, would not average out
    const float ck = p.kl.coef != 0.f ? p.kl.coef * r.kl : 0.f, x = ck - r.obj, wx = k.w * x;
    const float x_lo = diff_rest(ck, r.obj, x) + fmaf(p.kl.coef, r.kl, -ck);
    const float lo = fabsf(wx) < INFINITY ? fmaf(k.w_lo, x, fmaf(k.w, x, -wx)) + k.w * x_lo : 0.f;
    p.r.term_flags[t] = r.flags;
    return PostTerm{wx, lo, m ? H : 0.f, m ? r.kl : 0.f};
}

// ---------------------------------------------------------------- the teacher's entries

// One row of distillation after its statistics: dz_v = ct 2^{c (z_v - m)} outside the teacher's
// entries, and distill_entry() at them.
struct DistillRow {
    float ct, m;           // tail: coefficient and reference
    float M, ls, inv_s;    // the whole row: reference, ln S and 1 / S
    float po, lpo;         // the student's mass outside the teacher's entries, and its logarithm
    float kl, w;           // the row's divergence (reverse); its weight * scale / tau
    float Q;               // total mass of the teacher's distribution
    bool rest;             // there are entries outside
};

// What a row's entries give before the rest of the row is known, by one warp.
struct DistillEntries {
    float m, s;            // the student's statistics over the teacher's entries
    float shift;           // reverse: ln of the mass that they are taken to have, see distill_reverse
    float f, mass, a;      // reverse: sums of p k3(x), p and p x at that mass
    float lqo;             // ln q_o
};

// s_z[k] holds the student's logit at entry k (-inf where the entry is padding), s_lq[k] the teacher's log-prob.
__device__ __forceinline__ DistillEntries distill_entries(const DistillParams &p, const float *s_z, const float *s_lq, float4 rec) {
    const int lane = threadIdx.x & 31, K = p.K;
    DistillEntries e{};
    float m = -FLT_MAX;
#pragma unroll 4
    for (int k = lane; k < K; k += 32) m = fmaxf(m, s_z[k]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float s = 0.f;
#pragma unroll 4
    for (int k = lane; k < K; k += 32) s += ex2_approx((s_z[k] - m) * p.c);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    e.m = m;
    e.s = s;
    if (!p.reverse) return e;
    e.lqo = logf(rec.z);
    e.mass = s != 0.f ? fmaxf(1.f + rec.w - rec.z, 1e-6f) : 0.f;
    e.shift = s != 0.f ? logf(e.mass) : 0.f;
    const float ls = logf(s) - e.shift, r = e.mass / s;
    float f = 0.f, a = 0.f;
#pragma unroll 4
    for (int k = lane; k < K; k += 32) {
        const float d = s_z[k] - m, lq = s_lq[k], pk = s != 0.f ? ex2_approx(d * p.c) * r : 0.f;
        const float x = (d * p.inv_tau - ls) - lq, px = pk * x;
        f += post_k3_term(pk, expf(lq), x);
        a += pk != 0.f ? px : 0.f;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        f = __fadd_rn(f, __shfl_xor_sync(0xffffffffu, f, off));
        a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, a, off));
    }
    e.f = f;
    e.a = a;
    return e;
}

// The row's divergence: its terms h ln(h / o) (h the distribution the mean is over, o the other one) nearly
// cancel for a student near its teacher. With the masses added and taken away,
//   sum h ln(h / o) = sum [h ln(h / o) - h + o] + sum h - sum o = sum h k3(ln(h / o)) + sum h - sum o,
// k3(d) = e^{-d} - 1 + d: no term is negative, and an error e of a logarithm enters as h (1 - o / h) e
// and not as h e; a common one cancels. The difference of the masses is Q - 1, known to 1e-8 (distill_prep).

// Forward, by one warp.
__device__ __forceinline__ float distill_forward(const DistillParams &p, const DistillRow &r, const float *s_z, const float *s_lq,
                                                 float4 rec) {
    const int lane = threadIdx.x & 31;
    float sum = 0.f;
#pragma unroll 4
    for (int k = lane; k < p.K; k += 32) {
        const float d = s_z[k] - r.M, lq = s_lq[k], q = expf(lq);
        sum += post_k3_term(q, ex2_approx(d * p.c) * r.inv_s, lq - (d * p.inv_tau - r.ls));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, off));
    float gap = rec.w;  // sum q - sum p
    if (p.tail && r.rest) {
        sum += post_k3_term(rec.z, r.po, logf(rec.z) - r.lpo);
    } else if (p.tail) {
        gap -= rec.z;  // the entries are the whole vocabulary: there is no further outcome
    } else {
        sum += r.po;   // outside, q = 0
    }
    return sum + gap;
}

// Reverse, which the gradient waits for. The sum over the entries is made before the rest of the row is known,
// as if the student gave them the mass that the teacher does, p' (x' = ln(p' / q)). With their true mass
// p = p' e^{-y}, x = x' - y:
//   sum p k3(x) = sum p' k3(x') + (sum p') (y (1 - e^{-y}) - k3(y)) - (sum p' x') (1 - e^{-y}).
// y is near 0 where the student is near its teacher, so there the two last terms are small of second order, as
// the first one is. in, out: the student's sums over the entries and outside, to one reference.
__device__ __forceinline__ float distill_reverse(const DistillRow &r, const DistillEntries &e, float in, float out, float4 rec) {
    float sum;
    const float y = e.shift + log1pf(out / in);
    if (in == 0.f || y > 80.f) {  // e^{-y} = 0
        sum = e.f + e.mass - e.a;
    } else {
        const float u = -expm1f(-y);
        sum = e.f + (e.mass * (y * u - post_k3(y)) - e.a * u);
    }
    float gap = rec.w;
    if (r.rest) sum += post_k3_term(r.po, rec.z, r.lpo - e.lqo);
    else gap -= rec.z;
    return sum - gap;
}

// The row's coefficients, by one warp. `tail` are the statistics of the vocabulary outside the
// teacher's entries, e what the entries give, rec of distill_prep, w the row's weight * scale / tau, n_rest the number of
// vocabulary entries outside the teacher's.
//
// With q_o = rec.z the teacher's remaining mass, p_o the student's and Q = sum q + q_o (forward, the
// remaining mass being one more outcome):
//   KL = sum_k q_k ln(q_k / p_k) + q_o ln(q_o / p_o),  dKL/dz'_v = Q p_v - q_v  (an entry),
//                                                                  Q p_v - q_o p_v / p_o  (outside)
// renormalised: q_o = 0, Q = 1. Reverse:
//   KL = sum_k p_k a_k + p_o a_o,  a = ln(p / q),  dKL/dz'_v = p_v (a_v - KL), a_v = a_o outside.
// p_o is the sum of the entries outside, not 1 - sum_k p_k, which would cancel.
__device__ __forceinline__ DistillRow distill_finish(const DistillParams &p, PostStats tail, const DistillEntries &e, float4 rec,
                                                     float w, int n_rest) {
    DistillRow r;
    r.w = w;
    r.Q = 1.f + rec.w;
    r.m = tail.m;
    r.M = fmaxf(e.m, tail.m);
    const float ft = exp2f((tail.m - r.M) * p.c);
    const float in = __fmul_rn(e.s, exp2f((e.m - r.M) * p.c)), out = __fmul_rn(tail.s, ft), S = __fadd_rn(in, out);
    r.inv_s = 1.f / S;
    r.ls = logf(S);
    r.rest = n_rest > 0;
    r.po = tail.s * ft * r.inv_s;
    // a tail far below the row's maximum keeps its logarithm by its own reference
    r.lpo = (tail.m - r.M) * p.inv_tau + (logf(tail.s) - r.ls);
    r.kl = 0.f;
    const bool bucket = p.tail && r.rest;
    if (p.reverse) {  // the gradient needs the divergence
        r.kl = distill_reverse(r, e, in, out, rec);
        const float a = bucket ? r.lpo - e.lqo : 0.f;
        r.ct = tail.s > 0.f ? (a - r.kl) * ft * r.inv_s : 0.f;
    } else {
        r.ct = r.Q * ft * r.inv_s;
        if (bucket) r.ct = tail.s > 0.f ? r.ct - rec.z / tail.s : 0.f;
    }
    r.ct *= w;
    return r;
}

// dL/dz of one of the teacher's entries.
__device__ __forceinline__ float distill_entry(const DistillParams &p, const DistillRow &r, float z, float lq) {
    const float pk = ex2_approx((z - r.M) * p.c) * r.inv_s;
    if (!p.reverse) return r.w * fmaf(r.Q, pk, -expf(lq));
    return pk == 0.f ? 0.f : r.w * pk * (((z - r.M) * p.inv_tau - r.ls) - lq - r.kl);
}

}  // namespace rlk
