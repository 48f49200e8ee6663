// C ABI of the post-training operators that need no handle (declared in include/rl_loss.h): argument
// checks, workspace layout and launches.
#include <cmath>

#include "handle.cuh"
#include "post.cuh"

namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The checks every operator makes of its logits: type, vocabulary, rows and strides.
rl_status check_rows(int32_t dtype, int32_t T, int32_t V, const void *logits, int64_t ld, const void *dlogits,
                     int64_t ldd, bool grad) {
    if (dtype != RL_F32 && dtype != RL_BF16) return RL_ERR_DTYPE;
    if (T < 0 || V < 1 || V >= rlk::kMaxVocab) return RL_ERR_SHAPE;
    if (T == 0) return RL_OK;
    if (!logits || (grad && !dlogits)) return RL_ERR_INVALID_ARG;
    if (ld < V || (grad && ldd < V)) return RL_ERR_SHAPE;
    const int64_t es = dtype == RL_F32 ? 4 : 2;
    if (!aligned(logits, 16) || (ld * es) % 16 != 0) return RL_ERR_ALIGNMENT;
    if (grad && (!aligned(dlogits, 16) || (ldd * es) % 16 != 0)) return RL_ERR_ALIGNMENT;
    if (grad && logits == dlogits && ld != ldd) return RL_ERR_INVALID_ARG;
    return RL_OK;
}

struct Carve {
    char *base;
    size_t off = 0;
    template <typename X>
    X *take(size_t n) {
        off = align_up(off, 256);
        X *p = base ? reinterpret_cast<X *>(base + off) : nullptr;
        off += n * sizeof(X);
        return p;
    }
};

struct DistillWork {
    rlk::PostPartial *partials;
    rlk::PostTerm *terms;
    uint32_t *counters;
    int32_t *seq_n;
    float4 *rec;
};
size_t distill_layout(int32_t T, int32_t S, void *base, DistillWork &w) {
    Carve c{static_cast<char *>(base)};
    w.counters = c.take<uint32_t>(rlk::post_counters(T));
    w.partials = c.take<rlk::PostPartial>(rlk::post_chunks(T) + 1);
    w.terms = c.take<rlk::PostTerm>((size_t)T);
    w.seq_n = c.take<int32_t>((size_t)S);
    w.rec = c.take<float4>((size_t)T);
    return align_up(c.off, 256);
}

struct PrefWork {
    uint32_t *done;
    uint32_t *counters;
    float *logp;
    float2 *stats;
    float *coef;
    float *pair32;
};
size_t pref_layout(int32_t T, int32_t S, void *base, PrefWork &w) {
    Carve c{static_cast<char *>(base)};
    w.done = c.take<uint32_t>(1);
    w.counters = c.take<uint32_t>(rlk::kCountChunks);
    w.logp = c.take<float>((size_t)T);
    w.stats = c.take<float2>((size_t)T);
    w.coef = c.take<float>((size_t)S);
    w.pair32 = c.take<float>((size_t)S / 2);
    return align_up(c.off, 256);
}

}  // namespace

extern "C" {

RL_LOSS_API rl_status rl_loss_token_logp(int32_t dtype, int32_t T, int32_t V, const void *logits, int64_t ld,
                                         const int32_t *targets, const uint8_t *mask, float *logp, float *entropy,
                                         uint32_t *device_status, void *stream) {
    const rl_status st = check_rows(dtype, T, V, logits, ld, nullptr, 0, false);
    if (st != RL_OK) return st;
    if (T == 0) return RL_OK;
    if (!targets || !logp) return RL_ERR_INVALID_ARG;
    if (!aligned(targets, 4) || !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(device_status, 4))
        return RL_ERR_ALIGNMENT;
    rlk::LogpParams p{};
    p.r.logits = logits;
    p.r.ld = ld;
    p.r.T = T;
    p.r.V = V;
    p.r.targets = targets;
    p.r.mask = mask;
    p.r.logp = logp;
    p.r.entropy = entropy;
    p.r.status = device_status;
    return rlk::launch_post_logp(p, dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

RL_LOSS_API int32_t rl_loss_distill_max_k(void) { return rlk::kDistillMaxK; }

RL_LOSS_API size_t rl_loss_distill_workspace_bytes(int32_t num_tokens, int32_t num_seqs) {
    DistillWork w;
    return distill_layout(num_tokens < 0 ? 0 : num_tokens, num_seqs < 0 ? 0 : num_seqs, nullptr, w);
}

RL_LOSS_API rl_status rl_loss_distill(const rl_loss_distill_config *config, int32_t T, int32_t S, const void *logits,
                                      int64_t ld, const int32_t *ids, const float *vals, int64_t ldk,
                                      const uint8_t *mask, const int32_t *cu_seqlens, float *loss, double *loss_f64,
                                      void *dlogits, int64_t ldd, float *kl, void *workspace, size_t workspace_bytes,
                                      uint32_t *device_status, void *stream_ptr) {
    if (!config) return RL_ERR_INVALID_ARG;
    const rl_loss_distill_config &c = *config;
    const rl_status st = check_rows(c.logits_dtype, T, c.vocab_size, logits, ld, dlogits, ldd, true);
    if (st != RL_OK) return st;
    if (S < 1) return RL_ERR_SHAPE;
    if (c.mode != RL_DISTILL_RENORM && c.mode != RL_DISTILL_TAIL) return RL_ERR_INVALID_ARG;
    if (c.reverse != 0 && c.reverse != 1) return RL_ERR_INVALID_ARG;
    if (c.loss_norm != RL_NORM_PER_RESPONSE && c.loss_norm != RL_NORM_PER_TOKEN) return RL_ERR_INVALID_ARG;
    if (!(c.temperature > 0.f) || !std::isfinite(c.temperature) || !std::isfinite(c.scale)) return RL_ERR_INVALID_ARG;
    if (!(c.tail_floor >= 0.f && c.tail_floor < 1.f)) return RL_ERR_INVALID_ARG;
    if (c.k < 1 || c.k > rlk::kDistillMaxK || (c.reverse && c.mode != RL_DISTILL_TAIL)) return RL_ERR_UNSUPPORTED;
    if (!loss || !cu_seqlens || !workspace || (T > 0 && (!ids || !vals || !mask))) return RL_ERR_INVALID_ARG;
    if (T > 0 && ldk < c.k) return RL_ERR_SHAPE;
    if (!aligned(workspace, 256) || !aligned(ids, 4) || !aligned(vals, 4) || !aligned(kl, 4) || !aligned(loss, 4) ||
        !aligned(loss_f64, 8) || !aligned(cu_seqlens, 4) || !aligned(device_status, 4))
        return RL_ERR_ALIGNMENT;
    DistillWork w;
    if (workspace_bytes < distill_layout(T, S, workspace, w)) return RL_ERR_CAPACITY;

    rlk::DistillPrepParams q{};
    q.ids = ids;
    q.vals = vals;
    q.ldk = ldk;
    q.K = c.k;
    q.T = T;
    q.S = S;
    q.tail = c.mode == RL_DISTILL_TAIL;
    q.floor = c.tail_floor;
    q.mask = mask;
    q.cu_seqlens = cu_seqlens;
    q.rec = w.rec;
    q.seq_n = w.seq_n;
    q.counters = w.counters;
    q.n_counters = (int32_t)rlk::post_counters(T);
    q.status = device_status;

    rlk::DistillParams p{};
    p.r.logits = logits;
    p.r.ld = ld;
    p.r.dlogits = dlogits;
    p.r.ldd = ldd;
    p.r.T = T;
    p.r.V = c.vocab_size;
    p.r.S = S;
    p.r.mask = mask;
    p.r.cu_seqlens = cu_seqlens;
    p.r.status = device_status;
    p.r.terms = w.terms;
    p.r.partials = w.partials;
    p.r.counters = w.counters;
    p.r.loss = loss;
    p.r.loss_f64 = loss_f64;
    p.ids = ids;
    p.vals = vals;
    p.ldk = ldk;
    p.K = c.k;
    p.tail = q.tail;
    p.reverse = c.reverse;
    p.per_token = c.loss_norm == RL_NORM_PER_TOKEN;
    p.c = (float)(1.4426950408889634 / (double)c.temperature);
    p.inv_tau = (float)(1.0 / (double)c.temperature);
    p.scale = c.scale;
    p.rec = w.rec;
    p.seq_n = w.seq_n;
    p.kl = kl;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_ptr);
    if (rlk::launch_distill_prep(q, stream) != cudaSuccess) return RL_ERR_CUDA;
    return rlk::launch_post_distill(p, c.logits_dtype, stream) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

RL_LOSS_API size_t rl_loss_preference_workspace_bytes(int32_t num_tokens, int32_t num_seqs) {
    PrefWork w;
    return pref_layout(num_tokens < 0 ? 0 : num_tokens, num_seqs < 0 ? 0 : num_seqs, nullptr, w);
}

RL_LOSS_API rl_status rl_loss_preference(const rl_loss_pref_config *config, int32_t T, int32_t S, const void *logits,
                                         int64_t ld, const int32_t *targets, const float *logp_ref,
                                         const uint8_t *mask, const int32_t *cu_seqlens, float *loss,
                                         double *loss_f64, void *dlogits, int64_t ldd, float *logp,
                                         float *seq_logratio, float *pair_loss, void *workspace,
                                         size_t workspace_bytes, uint32_t *device_status, void *stream_ptr) {
    if (!config) return RL_ERR_INVALID_ARG;
    const rl_loss_pref_config &c = *config;
    const rl_status st = check_rows(c.logits_dtype, T, c.vocab_size, logits, ld, dlogits, ldd, true);
    if (st != RL_OK) return st;
    if (S < 2 || S % 2 != 0) return RL_ERR_SHAPE;
    if (c.loss_type < RL_PREF_SIGMOID || c.loss_type > RL_PREF_IPO) return RL_ERR_INVALID_ARG;
    if (c.length_norm != 0 && c.length_norm != 1) return RL_ERR_INVALID_ARG;
    if (!(c.beta > 0.f) || !std::isfinite(c.beta) || !std::isfinite(c.margin)) return RL_ERR_INVALID_ARG;
    if (!(c.label_smoothing >= 0.f && c.label_smoothing < 0.5f)) return RL_ERR_INVALID_ARG;
    if (!(c.nll_coef >= 0.f) || !std::isfinite(c.nll_coef)) return RL_ERR_INVALID_ARG;
    if (!loss || !cu_seqlens || !workspace || (T > 0 && (!targets || !mask))) return RL_ERR_INVALID_ARG;
    if (!aligned(workspace, 256) || !aligned(targets, 4) || !aligned(logp_ref, 4) || !aligned(logp, 4) ||
        !aligned(seq_logratio, 4) || !aligned(pair_loss, 4) || !aligned(loss, 4) || !aligned(loss_f64, 8) ||
        !aligned(cu_seqlens, 4) || !aligned(device_status, 4))
        return RL_ERR_ALIGNMENT;
    PrefWork w;
    if (workspace_bytes < pref_layout(T, S, workspace, w)) return RL_ERR_CAPACITY;

    rlk::LogpParams q{};
    q.r.logits = logits;
    q.r.ld = ld;
    q.r.dlogits = dlogits;
    q.r.ldd = ldd;
    q.r.T = T;
    q.r.V = c.vocab_size;
    q.r.S = S;
    q.r.targets = targets;
    q.r.mask = mask;
    q.r.cu_seqlens = cu_seqlens;
    q.r.logp = logp ? logp : w.logp;
    q.r.status = device_status;
    q.stats = w.stats;
    q.zero = w.done;

    rlk::PrefPairParams b{};
    b.T = T;
    b.S = S;
    b.V = c.vocab_size;
    b.targets = targets;
    b.mask = mask;
    b.cu_seqlens = cu_seqlens;
    b.logp = q.r.logp;
    b.logp_ref = logp_ref;
    b.kind = c.loss_type;
    b.mean = c.length_norm;
    b.beta = c.beta;
    b.smoothing = c.label_smoothing;
    b.margin = c.margin;
    b.nll = c.nll_coef;
    b.coef = w.coef;
    b.pair32 = w.pair32;
    b.seq_logratio = seq_logratio;
    b.pair_loss = pair_loss;
    b.pairs_done = w.done;
    b.tickets = w.counters + rlk::kCountTickets;
    b.loss = loss;
    b.loss_f64 = loss_f64;
    b.status = device_status;

    rlk::ScaleParams g{};
    g.r = q.r;
    g.r.counters = w.counters;
    g.stats = w.stats;
    g.coef = w.coef;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_ptr);
    cudaError_t e = rlk::launch_post_logp(q, c.logits_dtype, stream);
    if (e == cudaSuccess) e = rlk::launch_pref_pairs(b, stream);
    if (e == cudaSuccess) e = rlk::launch_post_scale(g, c.logits_dtype, stream);
    return e == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

}  // extern "C"
