// Row kernels of the vocabulary-wide post-training operators (post.cuh has their mathematics).
//
// A row is cut over the CTAs of a cluster (one to eight), and a CTA's slice over its consumer warps. In
// each CTA
//  - a producer warp copies every consumer warp's segments of the next rows into a ring of that warp's
//    own (bulk copies completing on mbarriers) and gathers what a row needs besides its logits: the
//    token's record, for 32 rows at a time, or the teacher's entries;
//  - each consumer warp folds its segment into softmax statistics (A) and later walks it, still in shared
//    memory, for the gradient (B): each logit is read from memory once. Warps wait for their own copies
//    alone, never for one another;
//  - a finisher warp merges the warps' statistics, exchanges them with the other CTAs through distributed
//    shared memory and works out the row's results.
// Three CTAs on an SM fill each other's waits for the finisher; where a ring holds two slices the warps
// also fold row r + 1 before they write row r.
//
// Short rows (up to 24 KB) are a warp's each (line_rows_kernel). Rows too long for the rings of a cluster (above
// about 1.8 MB with eight CTAs) take the block-per-row kernels at the end, which read a row twice.
//
// Bounds: HBM for long rows. 6000 x 151552 bf16: the loss with a KL term 570 us, 94% of the copy rate; log-probs
// of 16000 rows 102-107%; distillation (128 entries) 681 us, 79%, bounded by a row's stay in the rings (9.4 us, of
// which 4.4 copy and write).
#include <algorithm>
#include <cstddef>
#include <mutex>

#include "post.cuh"
#include "ptx.cuh"

namespace rlk {

namespace {

// ---------------------------------------------------------------- sums of the batch

__device__ __forceinline__ void add_partial(PostPartial &a, const PostPartial &q) {
    a.loss.add(q.loss.hi, q.loss.lo);
    a.ent.add(q.ent.hi, q.ent.lo);
    a.kl.add(q.kl.hi, q.kl.lo);
    a.n += q.n;
    a.popped += q.popped;
    a.clipped += q.clipped;
    a.masked += q.masked;
}

// A row's term, with its flags.
__device__ __forceinline__ void add_row(PostPartial &a, const PostTerm &v, uint32_t f) {
    const bool m = !(f & RL_FLAG_MASKED);
    a.loss.add(v.loss, v.loss_lo);
    a.ent.add(v.ent, 0.f);
    a.kl.add(v.kl, 0.f);
    a.n += m;
    a.masked += !m;
    a.popped += m && !(f & RL_FLAG_POP_IN_BOUNDS);
    a.clipped += m && (f & RL_FLAG_CLIP_ACTIVE);
}

__device__ __forceinline__ Sum2 shfl_xor(const Sum2 &s, int off) {
    return Sum2{__shfl_xor_sync(0xffffffffu, s.hi, off), __shfl_xor_sync(0xffffffffu, s.lo, off)};
}
__device__ __forceinline__ PostPartial warp_sum(PostPartial a) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        PostPartial q;
        q.loss = shfl_xor(a.loss, off);
        q.ent = shfl_xor(a.ent, off);
        q.kl = shfl_xor(a.kl, off);
        q.n = __shfl_xor_sync(0xffffffffu, a.n, off);
        q.popped = __shfl_xor_sync(0xffffffffu, a.popped, off);
        q.clipped = __shfl_xor_sync(0xffffffffu, a.clipped, off);
        q.masked = __shfl_xor_sync(0xffffffffu, a.masked, off);
        add_partial(a, q);
    }
    return a;
}

// The batch's results from its sums, by one warp.
__device__ __forceinline__ void write_sums(const PolicyParams &p, const PostPartial &a) {
    const int lane = threadIdx.x & 31;
    int empty = 0;
    for (int i = lane; i < p.r.S; i += 32) empty += p.seq_n[i] == 0;
    empty = warp_sum_i32(empty);
    if (lane != 0) return;
    if (p.counts) {
        p.counts[0] = a.popped;
        p.counts[1] = a.clipped;
        p.counts[2] = a.masked;
        p.counts[3] = empty;
    }
    if (p.mean_entropy) p.mean_entropy[0] = a.n > 0 ? (a.ent.hi + a.ent.lo) / (float)a.n : 0.f;
    if (p.kl.mean_kl) p.kl.mean_kl[0] = a.n > 0 ? (a.kl.hi + a.kl.lo) / (float)a.n : 0.f;
}
__device__ __forceinline__ void write_sums(const DistillParams &, const PostPartial &) {}

template <typename P>
__device__ __forceinline__ void write_loss(const P &p, const PostPartial &a) {
    write_sums(p, a);
    if ((threadIdx.x & 31) == 0) {
        const float loss = a.loss.hi + a.loss.lo;
        p.r.loss[0] = loss;
        if (p.r.loss_f64) p.r.loss_f64[0] = (double)a.loss.hi + (double)a.loss.lo;
        if (!isfinite(loss)) post_raise(p.r.status, RL_ERR_NONFINITE);
    }
}

// Sums a chunk whose terms are all written. The warp that sums the last chunk writes the batch's results.
template <typename P>
__device__ __forceinline__ void sum_chunk(const P &p, int chunk) {
    const int lane = threadIdx.x & 31, T = p.r.T;
    const int c0 = chunk * kSumRows, c1 = min(T, c0 + kSumRows), chunks = (T + kSumRows - 1) / kSumRows;
    int last = 0;
    __threadfence();
    PostPartial a{};
#pragma unroll
    for (int i = 0; i < kSumRows / 32; ++i) {
        const int k = c0 + lane + 32 * i;
        if (k >= c1) continue;
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.r.terms + k));
        const uint32_t f = p.r.term_flags ? __ldcg(p.r.term_flags + k) : RL_FLAG_MASKED;
        add_row(a, PostTerm{v.x, v.y, v.z, v.w}, f);
    }
    a = warp_sum(a);
    if (lane == 0) {
        p.r.partials[chunk] = a;
        __threadfence();
        last = atomicAdd(p.r.counters + kCountDone, 1u) == (uint32_t)chunks - 1;
    }
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    __threadfence();
    a = PostPartial{};
    for (int k = lane; k < chunks; k += 32) {
        const volatile PostPartial &q = p.r.partials[k];
        add_partial(a, PostPartial{{q.loss.hi, q.loss.lo}, {q.ent.hi, q.ent.lo}, {q.kl.hi, q.kl.lo}, q.n, q.popped, q.clipped, q.masked});
    }
    write_loss(p, warp_sum(a));
}

// Counts `n` rows of a chunk whose terms this warp has written; the warp that counts a chunk's last row sums it.
template <typename P>
__device__ __forceinline__ void count_rows(const P &p, int chunk, int n) {
    const int rows = min(p.r.T, (chunk + 1) * kSumRows) - chunk * kSumRows;
    int last = 0;
    if ((threadIdx.x & 31) == 0) {
        __threadfence();
        last = atomicAdd(p.r.counters + kCountChunks + chunk, (uint32_t)n) == (uint32_t)(rows - n);
    }
    if (__shfl_sync(0xffffffffu, last, 0)) sum_chunk(p, chunk);
}

// The rows of one chunk that a warp has written and not yet counted: counting takes a fence and an atomic,
// once for the rows of a ticket.
struct PendingRows {
    int chunk = 0, n = 0;
};
template <typename P>
__device__ __forceinline__ void add_term(const P &p, PendingRows &pend, int t, const PostTerm &term) {
    const int chunk = t / kSumRows;
    if (pend.n > 0 && chunk != pend.chunk) {
        count_rows(p, pend.chunk, pend.n);
        pend.n = 0;
    }
    if ((threadIdx.x & 31) == 0) p.r.terms[t] = term;
    pend.chunk = chunk;
    pend.n += 1;
}
template <typename P>
__device__ __forceinline__ void flush_rows(const P &p, PendingRows &pend) {
    if (pend.n > 0) count_rows(p, pend.chunk, pend.n);
    pend.n = 0;
}

template <typename P>
__device__ __forceinline__ void one_term(const P &p, int t, const PostTerm &term) {
    PendingRows pend;
    add_term(p, pend, t, term);
    flush_rows(p, pend);
}

template <typename T>
__device__ __forceinline__ const char *row_in(const PostRows &r, int t) {
    return reinterpret_cast<const char *>(r.logits) + (size_t)t * r.ld * sizeof(T);
}
template <typename T>
__device__ __forceinline__ char *row_out(const PostRows &r, int t) {
    return reinterpret_cast<char *>(r.dlogits) + (size_t)t * r.ldd * sizeof(T);
}

// ---------------------------------------------------------------- the ring kernel

enum RowOp { kOpLogp, kOpPolicy, kOpDistill, kOpScale };

constexpr int kWarps = 8;                      // consumer warps
constexpr int kRowThreads = 32 * (kWarps + 2); // and the producer and the finisher
constexpr int kRowBlocks = 3;                  // CTAs on an SM
constexpr int kMaxCluster = 8;
constexpr int kMaxDepth = 4;
constexpr int kBatch = 4;                      // 16-byte groups a lane takes at once
constexpr int kTickets = 4;                    // tickets of a cluster in flight

// Rows whose records are held. A ring of one slice has use for the next row's record alone; a distilled
// row's record takes two dependent loads to gather and starts a row earlier; the others have room.
constexpr int kMetaOf(int op) { return op == kOpPolicy ? 2 : op == kOpDistill ? 3 : 4; }

// How a launch cuts its rows.
struct RowPlan {
    int32_t cluster;    // CTAs per row
    int32_t slice;      // 16-byte groups per CTA
    int32_t parts;      // segments of a warp's share of the slice
    int32_t seg;        // 16-byte groups per segment
    int32_t depth;      // segments in a warp's ring
    int32_t rows;       // consecutive rows per ticket (at most 32)
    int32_t lag;        // rows folded ahead of the row that is written: 1 where the ring holds two slices, else 0
};

template <int OP>
struct RowMeta;
template <>
struct RowMeta<kOpLogp> {
    int32_t t;             // the row, -1: there are no more
    int32_t last;          // of its ticket
    int32_t read;          // the row's logits are needed (and copied)
    int32_t y;             // the sampled entry, -1: none
    float zy;
};
template <>
struct RowMeta<kOpPolicy> {
    int32_t t;             // the row, -1: there are no more
    int32_t last;          // of its ticket
    int32_t read, y;
    float zy;
    PolicyTok tok;
};
template <>
struct RowMeta<kOpDistill> {
    int32_t t;             // the row, -1: there are no more
    int32_t last;          // of its ticket
    int32_t read, copied;  // its logits are needed; they were copied (its entries then turned out bad)
    int32_t bad, have;     // an id outside the vocabulary; entries that are not padding
    float4 rec;
    float w;               // the row's weight
};
template <>
struct RowMeta<kOpScale> {
    int32_t t;             // the row, -1: there are no more
    int32_t last;          // of its ticket
    int32_t read;
    RowGrad grad;
};

// The results of row t of the log-prob pass, by one thread.
template <bool kEnt>
__device__ __forceinline__ void logp_write(const LogpParams &p, const RowMeta<kOpLogp> &meta, PostStats st, int t) {
    float logp = 0.f, ent = 0.f;
    if (meta.read) {
        logp = __int_as_float(0x7fc00000);
        if (meta.y >= 0) {
            const PostToken tok = post_target<kEnt>(st, meta.zy);
            st = tok.all;
            logp = tok.logp;
        } else {
            post_raise(p.r.status, RL_ERR_TARGET_RANGE);
        }
        if (!post_finite(st)) post_raise(p.r.status, RL_ERR_NONFINITE);
        if (kEnt) ent = post_entropy(st);
    }
    p.r.logp[t] = logp;
    if (kEnt) p.r.entropy[t] = ent;
    if (p.stats) p.stats[t] = make_float2(st.m, st.s);
}

// The teacher gives the row no mass: it contributes nothing, once its ids have been looked at like any row's.
constexpr float kNoMass = -1.f;  // Q - 1 of such a row (distill_prep)
__device__ __forceinline__ bool no_mass(const RowMeta<kOpDistill> &m) { return m.rec.w == kNoMass; }

// The results of a distilled row t, by one warp, and its term of the loss.
__device__ __forceinline__ PostTerm distill_write(const DistillParams &p, const RowMeta<kOpDistill> &meta, int t, bool live, bool dup,
                                                  const DistillRow &row, float kl) {
    if ((threadIdx.x & 31) == 0) {
        const bool bad = meta.bad || dup;
        if (bad) post_raise(p.r.status, RL_ERR_TARGET_RANGE);
        if (live && !isfinite(row.ls)) post_raise(p.r.status, RL_ERR_NONFINITE);
        if (p.kl) p.kl[t] = bad ? __int_as_float(0x7fc00000) : kl;
    }
    __syncwarp();
    return PostTerm{live ? meta.w * p.scale * kl : 0.f, 0.f, 0.f, 0.f};
}

struct alignas(16) RowMsg {  // sent by one 16-byte store
    float m, s, u;
    int32_t bad;
};

// What a row's finisher publishes.
struct RowFin {
    RowGrad grad;
};

template <int OP>
struct RowShared {
    static constexpr int kMeta = kMetaOf(OP);
    uint64_t mfull[kMeta], mempty[kMeta];         // records: gathered; no longer needed
    uint64_t part_full[kMeta];                    // the warps' statistics of a row
    uint64_t fin_full[kMeta];                     // a row's results
    uint64_t written[kMeta];                      // distill: the warps have written the row
    uint64_t tbar[kTickets], tfree[kTickets];     // the cluster's tickets: come; taken by every CTA (the first CTA's count)
    uint64_t xbar[2];  // the cluster's statistics: two in turn, as another CTA's next ones may come before the last of these
    RowMsg xmsg[2][kMaxCluster];
    RowMsg part[kMeta][kWarps];
    RowMeta<OP> meta[kMeta];
    RowFin fin[kMeta];
    int32_t ticket[kTickets];
    int32_t dead;                                 // a wait ran out: nothing waits any more
};
static_assert(offsetof(RowShared<kOpLogp>, xmsg) % 16 == 0 && offsetof(RowShared<kOpPolicy>, xmsg) % 16 == 0 &&
              offsetof(RowShared<kOpDistill>, xmsg) % 16 == 0 && sizeof(RowMsg) == 16, "st.async takes 16-byte boundaries");

// A bounded wait that gives up for good once any wait of the block has.
template <int OP>
__device__ __forceinline__ void row_wait(RowShared<OP> &sh, uint64_t *bar, uint32_t parity, uint32_t *status) {
    const uint32_t b = ptx::smem_u32(bar);
    if (ptx::mbar_try_wait(b, parity)) return;
    if (*reinterpret_cast<volatile int32_t *>(&sh.dead)) return;
    if (!ptx::mbar_wait(b, parity)) {
        *reinterpret_cast<volatile int32_t *>(&sh.dead) = 1;
        post_raise(status, RL_ERR_TIMEOUT);
    }
}

template <int OP>
__device__ __forceinline__ bool any_dead(RowShared<OP> &sh) {
    return __any_sync(0xffffffffu, *reinterpret_cast<volatile int32_t *>(&sh.dead) != 0);
}

// A bounded wait for one barrier per lane (null: none): `act` runs for a lane as soon as its barrier is
// through.
template <int OP, typename Act>
__device__ __forceinline__ void lanes_wait(RowShared<OP> &sh, bool mine, uint64_t *bar, uint32_t parity, uint32_t *status, Act act) {
    uint64_t t0 = 0;
    bool pending = mine;
    while (true) {
        if (pending && (bar == nullptr || ptx::mbar_try_wait(ptx::smem_u32(bar), parity))) {
            act();
            pending = false;
        }
        if (!__any_sync(0xffffffffu, pending)) return;
        if (any_dead(sh)) return;
        uint64_t now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (t0 == 0) t0 = now;
        if (now - t0 > 2000000000ull) {
            *reinterpret_cast<volatile int32_t *>(&sh.dead) = 1;
            post_raise(status, RL_ERR_TIMEOUT);
        }
    }
}

// 16 bytes into the shared memory of a CTA of the cluster, counted on its mbarrier.
__device__ __forceinline__ void st_async16(uint32_t dst, uint32_t bar, const RowMsg &v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "r"(__float_as_uint(v.m)), "r"(__float_as_uint(v.s)), "r"(__float_as_uint(v.u)), "r"(v.bad), "r"(bar)
                 : "memory");
}

// 4 bytes likewise.
__device__ __forceinline__ void st_async4(uint32_t dst, uint32_t bar, int v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst), "r"(v), "r"(bar)
                 : "memory");
}

template <int OP>
struct OpParams;
template <>
struct OpParams<kOpLogp> { using type = LogpParams; };
template <>
struct OpParams<kOpPolicy> { using type = PolicyParams; };
template <>
struct OpParams<kOpDistill> { using type = DistillParams; };
template <>
struct OpParams<kOpScale> { using type = ScaleParams; };

// The record of row t, by one lane (the producer's lanes gather those of 32 rows at once).
template <typename T, int OP>
__device__ __forceinline__ RowMeta<OP> load_meta(const typename OpParams<OP>::type &p, int t, int N) {
    using VT = PostVec<T>;
    RowMeta<OP> m{};
    m.t = t;
    const char *z = row_in<T>(p.r, t);
    if constexpr (OP == kOpLogp) {
        const int y = __ldg(p.r.targets + t);
        m.read = !p.r.mask || __ldg(p.r.mask + t);
        m.y = y >= 0 && y < p.r.V ? y : -1;
        m.zy = m.read && m.y >= 0 ? VT::load1(z, y) : 0.f;
    } else if constexpr (OP == kOpPolicy) {
        m.tok = policy_load(p, t, find_seq(p.r.cu_seqlens, p.r.S, t));
        m.read = m.tok.m || p.read_masked;
        m.y = m.tok.ok ? m.tok.y : -1;
        m.zy = m.read && m.tok.ok ? VT::load1(z, m.tok.y) : 0.f;
    } else if constexpr (OP == kOpScale) {
        const int i = find_seq(p.r.cu_seqlens, p.r.S, t);
        const int y = __ldg(p.r.targets + t);
        m.grad = RowGrad{0.f, 0.f, 0.f, -1};
        if (i >= 0 && __ldg(p.r.mask + t) && y >= 0 && y < p.r.V) {
            const float2 st = p.stats[t];
            const float g = p.coef[i];
            if (g != 0.f) m.grad = post_row_grad(g, PostStats{st.x, st.y, 0.f}, p.r.logp[t], y);
        }
        m.read = m.grad.y >= 0;
    } else {
        const int i = find_seq(p.r.cu_seqlens, p.r.S, t);
        m.read = i >= 0 && __ldg(p.r.mask + t);
        if (m.read) {
            m.rec = p.rec[t];
            m.w = 1.f / (p.per_token ? (float)N : (float)p.r.S * (float)p.seq_n[i]);
        }
        m.copied = m.read;
    }
    return m;
}

// distill: a row's first entries in registers, loaded while the row before is gathered: the ids and the logits
// there are two dependent loads.
struct NextEntries {
    static constexpr int kLane = 4;
    int id[kLane];
    float val[kLane];
};
__device__ __forceinline__ void next_entries(const DistillParams &p, int t, NextEntries &e) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NextEntries::kLane; ++i) {
        const int k = lane + 32 * i;
        e.id[i] = k < p.K ? __ldg(p.ids + (int64_t)t * p.ldk + k) : -1;
        e.val[i] = k < p.K ? __ldg(p.vals + (int64_t)t * p.ldk + k) : 0.f;
    }
}

// distill: the teacher's entries of row t and the student's logits there, by the producer warp.
template <typename T>
__device__ __forceinline__ void load_entries(const DistillParams &p, int t, const NextEntries &e, RowMeta<kOpDistill> &m, float *s_z,
                                             float *s_lq, int *s_id) {
    using VT = PostVec<T>;
    constexpr int U = NextEntries::kLane;
    const int lane = threadIdx.x & 31;
    const char *z = row_in<T>(p.r, t);
    const float4 rec = m.rec;
    int bad = 0, have = 0;
    auto put = [&](int k, int id, float val, float zk) {
        const bool real = id >= 0 && id < p.r.V;
        bad |= id < -1 || id >= p.r.V;
        have += real;
        s_id[k] = real ? id : -1;
        s_z[k] = zk;
        s_lq[k] = real ? (val - rec.x) - rec.y : -INFINITY;
    };
    auto logit = [&](int id) { return id >= 0 && id < p.r.V ? VT::load1(z, id) : -INFINITY; };
    float zk[U];
#pragma unroll
    for (int i = 0; i < U; ++i) zk[i] = logit(e.id[i]);
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (lane + 32 * i < p.K) put(lane + 32 * i, e.id[i], e.val[i], zk[i]);
#pragma unroll 4
    for (int k = lane + 32 * U; k < p.K; k += 32) {
        const int id = __ldg(p.ids + (int64_t)t * p.ldk + k);
        put(k, id, __ldg(p.vals + (int64_t)t * p.ldk + k), logit(id));
    }
    have = warp_sum_i32(have);
    bad = __any_sync(0xffffffffu, bad);
    __syncwarp();
    if (lane == 0) {
        m.bad = bad;
        m.have = have;
        if (bad || have == 0) m.read = 0;
    }
    __syncwarp();
}

// Takes the teacher's entries out of a warp's segment (groups v0 .. v0 + g of the row), by that warp: each
// becomes -inf, so that the fold leaves it out. It first gets its index as a tag: an entry listed twice
// finds another's tag, or -inf, in its place. `tail` receives the entries among the row's last V mod VEC
// where `tail0` >= 0 is the first of them. Returns whether an entry is listed twice.
template <typename T>
__device__ __forceinline__ bool mark_entries(uint4 *seg, int v0, int g, int tail0, const int *s_id, int K, uint32_t &tail) {
    using VT = PostVec<T>;
    using Tag = typename VT::Tag;
    constexpr int VEC = VT::kElems;
    const int lane = threadIdx.x & 31;
    Tag *at = reinterpret_cast<Tag *>(seg);
    const int lo = v0 * VEC, hi = (v0 + g) * VEC;
    constexpr int U = 4;  // entries of a lane at once: their loads and stores go out together
    // the places of this lane's entries k, k + 32, ... in the segment, -1: none
    auto places = [&](int k, int (&at_k)[U]) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int id = k + 32 * i < K ? s_id[k + 32 * i] : -1;
            at_k[i] = id >= lo && id < hi ? id - lo : -1;
        }
    };
    bool dup = false, any = false;
    uint32_t mine = 0;
    for (int k = lane; k < K; k += 32 * U) {
        int at_k[U];
        places(k, at_k);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (at_k[i] >= 0) {
                at[at_k[i]] = (Tag)(k + 32 * i);
                any = true;
            }
    }
    tail = 0;
    if (tail0 >= 0) {
        for (int k = lane; k < K; k += 32) {
            const int id = s_id[k];
            if (id < tail0) continue;
            const uint32_t bit = 1u << (id - tail0);
            dup |= (mine & bit) != 0;
            mine |= bit;
        }  // a bit that two lanes hold was listed twice
#pragma unroll
        for (int b = 0; b < VEC - 1; ++b) {
            const uint32_t who = __ballot_sync(0xffffffffu, (mine >> b) & 1);
            dup |= __popc(who) > 1;
            tail |= who ? 1u << b : 0u;
        }
    }
    if (__any_sync(0xffffffffu, any)) {
        __syncwarp();
        for (int k = lane; k < K; k += 32 * U) {
            int at_k[U];
            bool lost[U];
            places(k, at_k);
#pragma unroll
            for (int i = 0; i < U; ++i) lost[i] = at_k[i] >= 0 && at[at_k[i]] != (Tag)(k + 32 * i);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (at_k[i] >= 0 && !lost[i]) at[at_k[i]] = VT::kNegInf;
                dup |= lost[i];
            }
        }
        __syncwarp();
    }
    return __any_sync(0xffffffffu, dup);
}

template <typename T, int OP, bool kEnt>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks)
ring_rows_kernel(const __grid_constant__ typename OpParams<OP>::type p, const __grid_constant__ RowPlan plan, int nclusters) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    constexpr int kMeta = kMetaOf(OP);
    constexpr bool kStats = OP != kOpScale;   // a row is folded
    constexpr bool kGrad = OP != kOpLogp;     // a row is written
    extern __shared__ __align__(128) uint4 s_ring[];  // [depth][kWarps][seg]
    __shared__ RowShared<OP> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = plan.cluster;
    const int rank = (int)blockIdx.x % C, q = (int)blockIdx.x / C;
    const int T_ = p.r.T, V = p.r.V, nvec = V / VEC;
    const int v0 = min(nvec, rank * plan.slice), v1 = min(nvec, v0 + plan.slice);  // this CTA's 16-byte groups
    const bool last_rank = rank == C - 1;    // has the last V mod VEC entries too
    float c = kLog2e;
    int K = 0, N = 0;
    if constexpr (OP == kOpDistill) {
        c = p.c;
        K = p.K;
    }
    // after the ring: the segments' barriers (copied; free again), [depth][kWarps] each, and the teacher's
    // entries, [kMeta][3][K]
    uint64_t *s_full = reinterpret_cast<uint64_t *>(s_ring + (size_t)plan.depth * kWarps * plan.seg);
    uint64_t *s_empty = s_full + plan.depth * kWarps;
    float *s_meta = reinterpret_cast<float *>(s_empty + plan.depth * kWarps);
    auto use = [](int r) { return (uint32_t)(r / kMeta) & 1u; };  // the phase of row r's record
    // groups of part j of warp w's share
    auto seg_groups = [&](int w, int j) { return max(0, min(plan.seg, v1 - v0 - (j * kWarps + w) * plan.seg)); };

    if (tid == 0) {
        for (int s = 0; s < plan.depth * kWarps; ++s) {
            ptx::mbar_init(ptx::smem_u32(&s_full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&s_empty[s]), 1);
        }
        for (int s = 0; s < kMeta; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.mfull[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.mempty[s]), kWarps + (kStats ? 1 : 0));
            ptx::mbar_init(ptx::smem_u32(&sh.part_full[s]), kWarps);
            ptx::mbar_init(ptx::smem_u32(&sh.fin_full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.written[s]), kWarps);
        }
        for (int s = 0; s < 2; ++s) ptx::mbar_init(ptx::smem_u32(&sh.xbar[s]), 1);
        for (int s = 0; s < kTickets; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.tbar[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.tfree[s]), C);
        }
        ptx::fence_mbar_init();
        sh.dead = 0;
    }
    grid_dependency_wait();  // what follows reads what the launches before this one wrote
    if constexpr (OP == kOpLogp)
        if (p.zero && blockIdx.x == 0 && tid == 0) *p.zero = 0;
    if constexpr (OP == kOpDistill) {
        if (p.per_token) {
            for (int i = tid; i < p.r.S; i += kRowThreads) N += p.seq_n[i];
            N = block_sum_i32(N, reinterpret_cast<int *>(s_ring));
            ptx::fence_proxy_async_smem();  // the ring's first copies come after this use of its memory
        }
    }
    __syncthreads();
    if (kStats && C > 1) ptx::cluster_sync();  // every CTA's mbarriers are ready
    if (warp == kWarps) {
        // ------------------------------------------------ producer
        int n = 0, d = 0;      // segments issued for each warp; their next place
        uint32_t phase = 0;
        const uint64_t pol = ptx::l2_evict_first_policy();
        // The next rows: those of the log-prob pass go round the clusters in turn; the others are handed out
        // by a counter, as the SMs do not run alike (the slowest clusters took 9% longer than the middle
        // ones). The first CTA of a cluster asks, one ticket ahead, and tells the others.
        constexpr bool kDynamic = OP != kOpLogp;
        const bool shared = kStats && C > 1;
        uint32_t *counter = p.r.counters + kCountTickets + (kStats ? 0 : rank);
        int ahead = 0, n_tickets = -1;
        auto take = [&]() -> int {
            if (!kDynamic) return ahead++;
            int v = ahead;
            if (!shared || rank == 0)
                if (lane == 0) ahead = nclusters + (int)atomicAdd(counter, 1u);
            if (n_tickets < 0) {  // the first one is the cluster's own number
                n_tickets = 0;
                return q;
            }
            if (shared) {
                const int s = n_tickets % kTickets;
                const uint32_t phase_t = (uint32_t)(n_tickets / kTickets) & 1u;
                const uint32_t bar = ptx::smem_u32(&sh.tbar[s]), at = ptx::smem_u32(&sh.ticket[s]);
                if (rank == 0) {
                    if (n_tickets >= kTickets) row_wait(sh, &sh.tfree[s], phase_t ^ 1, p.r.status);
                    v = __shfl_sync(0xffffffffu, v, 0);
                    if (lane < C) st_async4(ptx::mapa_shared(at, lane), ptx::mapa_shared(bar, lane), v);
                }
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, 4);
                __syncwarp();
                row_wait(sh, &sh.tbar[s], phase_t, p.r.status);
                v = *reinterpret_cast<volatile int32_t *>(&sh.ticket[s]);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&sh.tfree[s]), 0));
                ++n_tickets;
            }
            return __shfl_sync(0xffffffffu, v, 0);
        };
        const int n_rows = kDynamic ? T_ : q < T_ ? (T_ - 1 - q) / nclusters + 1 : 0;
        // the k-th row; scale: from the last row backwards, the rows read last being the likeliest in L2
        auto row_of = [&](int k) { return OP == kOpScale ? T_ - 1 - k : kDynamic ? k : q + k * nclusters; };
        RowMeta<OP> mine{};  // the record of the ticket's row `lane`
        int row0 = 0, left = 0, at = 0;
        NextEntries entries;
        auto entries_ahead = [&] {  // of the ticket's next row
            if constexpr (OP == kOpDistill)
                if (at < left) next_entries(p, row_of(row0 + at), entries);
        };
        auto fetch = [&] {
            const int64_t first = (int64_t)take() * plan.rows;
            left = first < n_rows ? min(plan.rows, n_rows - (int)first) : 0;
            row0 = (int)first;
            at = 0;
            entries_ahead();
            if (lane < left) mine = load_meta<T, OP>(p, row_of(row0 + lane), N);
        };
        fetch();
        for (int r = 0;; ++r) {
            const int ms = r % kMeta;
            if (left == 0 || any_dead(sh)) {  // the end
                if (r >= kMeta) row_wait(sh, &sh.mempty[ms], use(r) ^ 1, p.r.status);
                if (lane == 0) {
                    sh.meta[ms].t = -1;
                    ptx::mbar_arrive(ptx::smem_u32(&sh.mfull[ms]));
                }
                break;
            }
            const int i = at++, t = row_of(row0 + i);
            const int read = __shfl_sync(0xffffffffu, mine.read, i);
            const char *src = row_in<T>(p.r, t) + (size_t)v0 * 16;
            float *mz = s_meta + (size_t)ms * 3 * K;
            int *s_id = reinterpret_cast<int *>(mz + 2 * K);
            // the record goes out before the row's copies, which wait for segments
            if (r >= kMeta) row_wait(sh, &sh.mempty[ms], use(r) ^ 1, p.r.status);
            if (lane == i) sh.meta[ms] = mine;
            __syncwarp();
            if (lane == 0) sh.meta[ms].last = at == left;
            if constexpr (OP == kOpDistill) {
                __syncwarp();
                if (read) load_entries<T>(p, t, entries, sh.meta[ms], mz, mz + K, s_id);
                entries_ahead();
            }
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.mfull[ms]));
            const bool more = at == left;
            if (!read) {
                if (more) fetch();
                continue;
            }
            for (int j = 0; j < plan.parts; ++j) {
                const int w = lane % kWarps;
                const int g = seg_groups(w, j);
                uint64_t *bar = n >= plan.depth ? &s_empty[d * kWarps + w] : nullptr;
                lanes_wait(sh, lane < kWarps, bar, phase ^ 1, p.r.status, [&] {
                    const uint32_t full = ptx::smem_u32(&s_full[d * kWarps + w]);
                    if (g == 0) {
                        ptx::mbar_arrive(full);
                        return;
                    }
                    ptx::mbar_arrive_expect_tx(full, (uint32_t)g * 16);
                    const uint32_t dst = ptx::smem_u32(s_ring + ((size_t)d * kWarps + w) * plan.seg);
                    const char *from = src + ((size_t)j * kWarps + w) * plan.seg * 16;
                    if (OP == kOpLogp && p.r.dlogits) ptx::bulk_g2s(dst, from, (uint32_t)g * 16, full);  // read again
                    else ptx::bulk_g2s_hint(dst, from, (uint32_t)g * 16, full, pol);
                });
                ++n;
                if (++d == plan.depth) d = 0, phase ^= 1;
                // the next ticket and its rows' records, a chain of dependent loads, come behind the copies that
                // need not wait for segments of this row
                if (more && j == min(plan.parts, plan.depth) - 1) fetch();
                if (any_dead(sh)) break;
            }
        }
        if (*reinterpret_cast<volatile int32_t *>(&sh.dead) && lane < kWarps) {
            // a wait ran out: no copy may be in flight when the block exits
            for (int k = max(0, n - plan.depth); k < n; ++k)
                ptx::mbar_wait(ptx::smem_u32(&s_full[(k % plan.depth) * kWarps + lane]), (k / plan.depth) & 1, 100000000ull);
        }
    } else if (warp > kWarps) {
        // ------------------------------------------------ finisher
        int exchanges = 0;
        DistillRow last{};      // distill: the row before this one, whose entries are still to be written
        bool last_live = false;
        int last_t = 0;
        PendingRows pend;
        // The entries are written after the rest of the row, whose value they replace, and after the next
        // row's results are out: nobody waits for them.
        auto write_entries = [&](int r) {
            if constexpr (OP == kOpDistill) {
                const int ms = r % kMeta;
                const float *s_z = s_meta + (size_t)ms * 3 * K, *s_lq = s_z + K;
                const int *s_id = reinterpret_cast<const int *>(s_z + 2 * K);
                row_wait(sh, &sh.written[ms], use(r), p.r.status);
                if (last_live) {
                    char *dz = row_out<T>(p.r, last_t);
                    for (int k = lane; k < K; k += 32) {
                        const int id = s_id[k];
                        if ((id >= v0 * VEC && id < v1 * VEC) || (last_rank && id >= nvec * VEC))
                            VT::store1(dz, id, distill_entry(p, last, s_z[k], s_lq[k]));
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.mempty[ms]));
            }
        };
        int r = 0;
        for (; kStats; ++r) {
            const int ms = r % kMeta;
            const bool writes = r % C == rank;  // the CTAs take turns in writing the rows' results
            row_wait(sh, &sh.mfull[ms], use(r), p.r.status);
            const RowMeta<OP> &meta = sh.meta[ms];
            const int t = meta.t;
            if (t < 0 || any_dead(sh)) break;
            RowFin &fin = sh.fin[ms];
            const bool read = meta.read;
            const float *s_z = s_meta + (size_t)ms * 3 * K, *s_lq = s_z + K;
            DistillEntries entries{};
            if constexpr (OP == kOpDistill)
                if (read) entries = distill_entries(p, s_z, s_lq, meta.rec);
            row_wait(sh, &sh.part_full[ms], use(r), p.r.status);
            PostStats st{0.f, 1.f, 0.f};
            int dup = 0;
            if (read) {
                static_assert(kWarps == 8 && kMaxCluster == 8, "the merges go over groups of eight lanes");
                RowMsg w = sh.part[ms][lane & 7];
                dup = __any_sync(0xffffffffu, w.bad);
                st = post_warp_merge<kEnt, 8>(PostStats{w.m, w.s, w.u}, c);
                if (C > 1) {
                    const int x = exchanges & 1;
                    const uint32_t bar = ptx::smem_u32(&sh.xbar[x]);
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(C * sizeof(RowMsg)));
                    __syncwarp();
                    if (lane < C)
                        st_async16(ptx::mapa_shared(ptx::smem_u32(&sh.xmsg[x][rank]), lane), ptx::mapa_shared(bar, lane),
                                   RowMsg{st.m, st.s, st.u, dup});
                    row_wait(sh, &sh.xbar[x], (exchanges >> 1) & 1, p.r.status);
                    const bool in = (lane & 7) < C;
                    w = sh.xmsg[x][in ? lane & 7 : 0];
                    ++exchanges;
                    dup = __any_sync(0xffffffffu, w.bad);
                    st = post_warp_merge<kEnt, 8>(in ? PostStats{w.m, w.s, w.u} : kPostStart, c);
                }
            }
            if constexpr (OP == kOpLogp) {
                if (lane == 0 && writes) logp_write<kEnt>(p, meta, st, t);
            } else if constexpr (OP == kOpPolicy) {
                PostTerm term{};
                if (lane == 0) {
                    PostToken tok{st, 0.f, 0.f};
                    if (read && meta.y >= 0) tok = post_target<kEnt>(st, meta.zy);
                    const PolicyRow row = policy_row(p, meta.tok, tok, read);
                    fin.grad = row.grad;
                    ptx::mbar_arrive(ptx::smem_u32(&sh.fin_full[ms]));
                    if (writes) term = policy_write<kEnt>(p, t, meta.tok, tok, row, read);
                }
                __syncwarp();
                if (writes) add_term(p, pend, t, term);
                if (meta.last) flush_rows(p, pend);
            } else if constexpr (OP == kOpDistill) {
                const bool live = read && !dup && !no_mass(meta);
                DistillRow row{};
                if (live) row = distill_finish(p, st, entries, meta.rec, meta.w * p.scale * p.inv_tau, V - meta.have);
                if (lane == 0) {
                    fin.grad = RowGrad{live ? row.ct : 0.f, row.m, 0.f, live ? 0 : -1};
                    ptx::mbar_arrive(ptx::smem_u32(&sh.fin_full[ms]));
                }
                if (writes) {
                    const float kl = !live ? 0.f : p.reverse ? row.kl : distill_forward(p, row, s_z, s_lq, meta.rec);
                    add_term(p, pend, t, distill_write(p, meta, t, live, dup, row, kl));
                }
                if (meta.last) flush_rows(p, pend);
                if (r > 0) write_entries(r - 1);
                last = row;
                last_live = live;
                last_t = t;
            }
            if constexpr (OP != kOpDistill) {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.mempty[ms]));
            }
        }
        if (r > 0) write_entries(r - 1);
    } else {
        // ------------------------------------------------ consumers
        const int tail_v = nvec * VEC + tid;     // this thread's entry of the last V mod VEC
        const bool has_tail = last_rank && tail_v < V;
        // asked for before the waits of a fold or a write, which its latency would lengthen
        auto tail_of = [&](int t) { return has_tail ? VT::load1(row_in<T>(p.r, t), tail_v) : 0.f; };
        int da = 0, db = 0;                      // the next segments of the fold and of the write
        uint32_t phase_a = 0, phase_b = 0;
        auto next = [&](int &d, uint32_t &phase) {
            if (++d == plan.depth) d = 0, phase ^= 1;
        };
        auto copied = [&](const RowMeta<OP> &m) {  // whether the row is in the ring
            if constexpr (OP == kOpDistill) return m.copied != 0;
            else return m.read != 0;
        };
        // A: the statistics of row r; false where there are no more rows
        auto fold = [&](int r) -> bool {
            const int ms = r % kMeta;
            row_wait(sh, &sh.mfull[ms], use(r), p.r.status);
            const RowMeta<OP> &meta = sh.meta[ms];
            if (meta.t < 0 || any_dead(sh)) return false;
            if (meta.read) {
                int y = -1;
                uint32_t marks = 0;
                bool dup = false;
                if constexpr (OP == kOpLogp || OP == kOpPolicy) y = meta.y;
                const int ky = y >= 0 && y < nvec * VEC ? y / VEC - v0 : -1;  // the sampled entry's group
                const float tail_z = tail_of(meta.t);
                PostAcc acc = post_acc();
                for (int j = 0; j < plan.parts; ++j) {
                    row_wait(sh, &s_full[da * kWarps + warp], phase_a, p.r.status);
                    uint4 *seg = s_ring + ((size_t)da * kWarps + warp) * plan.seg;
                    const int g = seg_groups(warp, j);
                    if constexpr (OP != kOpDistill) {
                        // the lane that folds the sampled entry's group takes the entry out of it
                        const int ks = ky - (j * kWarps + warp) * plan.seg;
                        if (ky >= 0 && ks >= 0 && ks < g && (ks & 31) == lane) {
                            reinterpret_cast<volatile typename VT::Tag *>(seg + ks)[y % VEC] = VT::kNegInf;
                            if (!kGrad) ptx::fence_proxy_async_smem();  // the next copy into the segment comes after this
                        }
                    }
                    if constexpr (OP == kOpDistill)
                        dup = mark_entries<T>(seg, v0 + warp * plan.seg, g, last_rank && warp == 0 && nvec * VEC < V ? nvec * VEC : -1,
                                              reinterpret_cast<const int *>(s_meta + (size_t)ms * 3 * K + 2 * K), K, marks);
                    int k = lane;
                    for (; k - lane + 32 * kBatch <= g; k += 32 * kBatch) {
                        uint4 v[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) v[i] = seg[k + 32 * i];
                        post_fold_groups<T, kEnt>(acc, v, c);
                    }
                    if (k - lane < g) {  // the rest of the segment, filled up with -inf
                        uint4 v[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) v[i] = k + 32 * i < g ? seg[k + 32 * i] : VT::none();
                        post_fold_groups<T, kEnt>(acc, v, c);
                    }
                    if (!kGrad) {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&s_empty[da * kWarps + warp]));
                    }
                    next(da, phase_a);
                }
                PostStats st = acc.stats();
                if (has_tail && tail_v != y && !((marks >> tid) & 1)) {
                    const float x[1] = {tail_z};
                    post_fold<kEnt>(st, x, c);
                }
                st = post_warp_merge<kEnt>(st, c);
                if (lane == 0) sh.part[ms][warp] = RowMsg{st.m, st.s, st.u, dup};
            } else if (copied(meta)) {
                for (int j = 0; j < plan.parts; ++j) next(da, phase_a);
            }
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(ptx::smem_u32(&sh.part_full[ms]));
                if (!kGrad) ptx::mbar_arrive(ptx::smem_u32(&sh.mempty[ms]));
            }
            return true;
        };
        // B: the gradient of row r
        auto write = [&](int r) -> bool {
            const int ms = r % kMeta;
            RowGrad gr;
            float tail_z;
            if constexpr (OP == kOpScale) {
                row_wait(sh, &sh.mfull[ms], use(r), p.r.status);
                if (sh.meta[ms].t < 0 || any_dead(sh)) return false;
                gr = sh.meta[ms].grad;
                tail_z = tail_of(sh.meta[ms].t);
            } else {
                tail_z = tail_of(sh.meta[ms].t);
                row_wait(sh, &sh.fin_full[ms], use(r), p.r.status);
                gr = sh.fin[ms].grad;
            }
            const int t = sh.meta[ms].t;
            const bool in_ring = copied(sh.meta[ms]), zero = gr.y < 0;
            char *dz = row_out<T>(p.r, t);
            const int ky = OP == kOpDistill || zero || gr.y >= nvec * VEC ? -1 : gr.y / VEC - v0;
            for (int j = 0; j < plan.parts; ++j) {
                const int g = seg_groups(warp, j), at = (j * kWarps + warp) * plan.seg;
                uint4 *to = reinterpret_cast<uint4 *>(dz) + v0 + at;
                if (in_ring) row_wait(sh, &s_full[db * kWarps + warp], phase_b, p.r.status);  // a row that was not folded
                if (zero) {
                    for (int k = lane; k < g; k += 32) __stcs(to + k, make_uint4(0, 0, 0, 0));
                } else {
                    const uint4 *seg = s_ring + ((size_t)db * kWarps + warp) * plan.seg;
                    int k = lane;
                    for (; k - lane + 32 * kBatch <= g; k += 32 * kBatch) {
                        uint4 v[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) v[i] = seg[k + 32 * i];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) __stcs(to + k + 32 * i, post_grad_group<T>(v[i], gr.a, gr.m, c));
                    }
                    for (; k < g; k += 32) __stcs(to + k, post_grad_group<T>(seg[k], gr.a, gr.m, c));
                    // by the lane that wrote the group, after it
                    const int ks = ky - at;
                    if (OP != kOpDistill && ky >= 0 && ks >= 0 && ks < g && (ks & 31) == lane) VT::store1(dz, gr.y, gr.gy);
                }
                if (in_ring) {
                    if (kStats) ptx::fence_proxy_async_smem();  // the next copy comes after the fold's marks in the segment
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&s_empty[db * kWarps + warp]));
                    next(db, phase_b);
                }
            }
            if (has_tail) {
                const float e = zero ? 0.f : gr.a * ex2_approx((tail_z - gr.m) * c);
                VT::store1(dz, tail_v, OP != kOpDistill && !zero && tail_v == gr.y ? gr.gy : e);
            }
            __syncwarp();
            if (lane == 0) {
                if (OP == kOpDistill) ptx::mbar_arrive(ptx::smem_u32(&sh.written[ms]));
                ptx::mbar_arrive(ptx::smem_u32(&sh.mempty[ms]));
            }
            return true;
        };
        int r = 0;
        if constexpr (!kGrad) {
            while (fold(r)) ++r;
        } else if constexpr (!kStats) {
            while (write(r)) ++r;
        } else {
            for (; fold(r); ++r)
                if (r >= plan.lag) write(r - plan.lag);
            for (int k = max(0, r - plan.lag); k < r && !any_dead(sh); ++k) write(k);
        }
    }
    if constexpr (OP == kOpPolicy || OP == kOpDistill) {
        // an empty batch: there is no row whose term could be the last
        if (T_ == 0 && blockIdx.x == 0 && warp == 0) write_loss(p, PostPartial{});
    }
    if (kStats && C > 1) ptx::cluster_sync();  // no CTA leaves while another may still write to it
}

// ---------------------------------------------------------------- short rows

constexpr int kLineWarps = 4;                   // rows of a block at once
constexpr int kLineBlocks = 6;                  // blocks on an SM
constexpr int kLineBytes = 24576;               // the longest row that takes this way

// The batch's sums from those of the warps: of a block's in their order, then of the blocks' by the block that
// comes last. The order of the additions goes by how many blocks the launch has, which is by the sizes and by how many
// the device holds at once. A block's takes the place of three rows' terms, of which there are as many. (Chunks of rows as in
// the ring kernel would each be summed by the warp that comes last there: one slow warp, for all its rows. They
// took 45 us of 140.)
template <typename P>
__device__ __forceinline__ void line_sums(const P &p, const PostPartial &mine) {
    __shared__ PostPartial s_sum[kLineWarps];
    __shared__ int s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = gridDim.x;
    static_assert(sizeof(PostPartial) <= 3 * sizeof(PostTerm), "");
    auto block_total = [&](const PostPartial &a) {  // in the first thread
        if (lane == 0) s_sum[warp] = a;
        __syncthreads();
        PostPartial b{};
        if (threadIdx.x == 0)
            for (int w = 0; w < kLineWarps; ++w) add_partial(b, s_sum[w]);
        return b;
    };
    PostPartial a = block_total(mine);
    if (blocks > 1) {
        auto place = [&](int b) { return reinterpret_cast<PostPartial *>(p.r.terms + 3 * (size_t)b); };
        if (threadIdx.x == 0) {
            *place(blockIdx.x) = a;
            __threadfence();
            s_last = atomicAdd(p.r.counters + kCountDone, 1u) == (uint32_t)blocks - 1;
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        a = PostPartial{};
        for (int b = threadIdx.x; b < blocks; b += 32 * kLineWarps) {
            const volatile PostPartial &q = *place(b);
            add_partial(a, PostPartial{{q.loss.hi, q.loss.lo}, {q.ent.hi, q.ent.lo}, {q.kl.hi, q.kl.lo}, q.n, q.popped, q.clipped, q.masked});
        }
        a = block_total(warp_sum(a));
    }
    if (warp == 0) write_loss(p, a);
}

// A row per warp, in shared memory: for short rows the steps between a row's warps, its finisher and its
// producer take longer than its bytes. The warps on an SM cover one another's copies and chains: 24 of them for rows
// up to 9 KB (distillation of 128 entries at 8 KB: 20), 8 at 24 KB. Bytes of a row here and on the rings, rows of bf16
// (us): 8 KB, 30000 rows: the loss 106 and 261, distillation (K = 128) 171 and 443, log-probs 44 and 116; 24 KB, 15000:
// 142 and 189, 226 and 271, 69 and 80; 32 KB, 15000: 234 and 206, 346 and 289, 115 and 81.
template <typename T, int OP, bool kEnt>
__global__ void __launch_bounds__(32 * kLineWarps, kLineBlocks)
line_rows_kernel(const __grid_constant__ typename OpParams<OP>::type p, int stride) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    constexpr bool kGrad = OP != kOpLogp, kFold = OP != kOpScale;
    extern __shared__ __align__(128) uint4 s_lines[];  // [kLineWarps][stride]: a row, then the teacher's entries, [3][K]
    __shared__ uint64_t s_bar[kLineWarps];
    __shared__ RowMeta<OP> s_meta[kLineWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int T_ = p.r.T, V = p.r.V, nvec = V / VEC;
    float c = kLog2e;
    int K = 0, N = 0;
    if constexpr (OP == kOpDistill) {
        c = p.c;
        K = p.K;
    }
    uint4 *line = s_lines + (size_t)warp * stride;
    float *s_z = reinterpret_cast<float *>(line + nvec), *s_lq = s_z + K;
    int *s_id = reinterpret_cast<int *>(s_z + 2 * K);
    const uint32_t bar = ptx::smem_u32(&s_bar[warp]);
    if (lane == 0) {
        ptx::mbar_init(bar, 1);
        ptx::fence_mbar_init();
    }
    __syncwarp();
    grid_dependency_wait();
    if constexpr (OP == kOpLogp)
        if (p.zero && blockIdx.x == 0 && threadIdx.x == 0) *p.zero = 0;
    if constexpr (OP == kOpDistill) {
        if (p.per_token) {
            for (int i = lane; i < p.r.S; i += 32) N += p.seq_n[i];
            N = warp_sum_i32(N);
        }
    }
    // Rows go to the warps in turn; the lanes hold the records of a warp's next 32.
    const int W = gridDim.x * kLineWarps;
    int64_t first = (int64_t)warp * gridDim.x + blockIdx.x;
    auto row_of = [&](int i) { return (int)(OP == kOpScale ? T_ - 1 - (first + (int64_t)i * W) : first + (int64_t)i * W); };
    auto count_of = [&] { return first < T_ ? (int)min((int64_t)32, (T_ - 1 - first) / W + 1) : 0; };
    int n = count_of();
    RowMeta<OP> mine{};
    if (lane < n) mine = load_meta<T, OP>(p, row_of(lane), N);
    NextEntries entries;
    const uint64_t pol = ptx::l2_evict_first_policy();
    auto start = [&](int i) {
        const int t = row_of(i);
        if constexpr (OP == kOpDistill) next_entries(p, t, entries);
        if (nvec > 0 && __shfl_sync(0xffffffffu, mine.read, i) && lane == 0) {
            ptx::mbar_arrive_expect_tx(bar, (uint32_t)nvec * 16);
            if (OP == kOpLogp && p.r.dlogits) ptx::bulk_g2s(ptx::smem_u32(line), row_in<T>(p.r, t), (uint32_t)nvec * 16, bar);  // read again
            else ptx::bulk_g2s_hint(ptx::smem_u32(line), row_in<T>(p.r, t), (uint32_t)nvec * 16, bar, pol);
        }
    };
    const int tail_v = nvec * VEC + lane;  // this lane's entry of the last V mod VEC
    const bool has_tail = tail_v < V;
    PostPartial sum{};  // of this warp's rows
    uint32_t phase = 0;
    int i = 0;
    if (n > 0) start(0);
    while (n > 0) {
        const int t = row_of(i), in_line = __shfl_sync(0xffffffffu, mine.read, i);
        RowMeta<OP> &meta = s_meta[warp];
        if (lane == i) meta = mine;
        __syncwarp();
        DistillEntries de{};
        if constexpr (OP == kOpDistill) {
            if (meta.read) load_entries<T>(p, t, entries, meta, s_z, s_lq, s_id);
            if (meta.read) de = distill_entries(p, s_z, s_lq, meta.rec);
        }
        const bool read = meta.read;
        const float tail_z = has_tail && in_line ? VT::load1(row_in<T>(p.r, t), tail_v) : 0.f;  // before the wait
        if (in_line && nvec > 0) {
            const bool there = ptx::mbar_wait(bar, phase);
            phase ^= 1;
            if (!__all_sync(0xffffffffu, there)) {
                if (lane == 0) {
                    post_raise(p.r.status, RL_ERR_TIMEOUT);
                    ptx::mbar_wait(bar, phase ^ 1);  // no copy may be in flight when the warp leaves
                }
                break;
            }
        }
        // the statistics
        PostStats st{0.f, 1.f, 0.f};
        bool dup = false;
        uint32_t marks = 0;
        int y = -1;
        if constexpr (OP == kOpLogp || OP == kOpPolicy) y = meta.y;
        if (kFold && read) {
            const int ky = y >= 0 && y < nvec * VEC ? y / VEC : -1;
            if (ky >= 0 && (ky & 31) == lane)  // the lane that folds the sampled entry's group takes the entry out of it
                reinterpret_cast<volatile typename VT::Tag *>(line + ky)[y % VEC] = VT::kNegInf;
            if constexpr (OP == kOpDistill) dup = mark_entries<T>(line, 0, nvec, nvec * VEC < V ? nvec * VEC : -1, s_id, K, marks);
            PostAcc acc = post_acc();
            for (int k = lane; k - lane < nvec; k += 32 * kBatch) {
                uint4 v[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) v[b] = k + 32 * b < nvec ? line[k + 32 * b] : VT::none();
                post_fold_groups<T, kEnt>(acc, v, c);
            }
            st = acc.stats();
            if (has_tail && tail_v != y && !((marks >> lane) & 1)) {
                const float x[1] = {tail_z};
                post_fold<kEnt>(st, x, c);
            }
            st = post_warp_merge<kEnt>(st, c);
        }
        // the row's results
        RowGrad gr{0.f, 0.f, 0.f, -1};
        DistillRow row{};
        bool live = read && !dup;
        if constexpr (OP == kOpDistill) live = live && !no_mass(meta);
        if constexpr (OP == kOpLogp) {
            if (lane == 0) logp_write<kEnt>(p, meta, st, t);
        } else if constexpr (OP == kOpPolicy) {
            PostToken tok{st, 0.f, 0.f};
            if (read && y >= 0) tok = post_target<kEnt>(st, meta.zy);
            const PolicyRow pr = policy_row(p, meta.tok, tok, read);
            gr = pr.grad;
            if (lane == 0) add_row(sum, policy_write<kEnt>(p, t, meta.tok, tok, pr, read), pr.flags);
        } else if constexpr (OP == kOpDistill) {
            if (live) row = distill_finish(p, st, de, meta.rec, meta.w * p.scale * p.inv_tau, V - meta.have);
            gr = RowGrad{live ? row.ct : 0.f, row.m, 0.f, live ? 0 : -1};
            const float kl = !live ? 0.f : p.reverse ? row.kl : distill_forward(p, row, s_z, s_lq, meta.rec);
            const PostTerm term = distill_write(p, meta, t, live, dup, row, kl);
            if (lane == 0) add_row(sum, term, 0);
        } else {
            gr = meta.grad;
        }
        // the gradient
        if (kGrad) {
            char *dz = row_out<T>(p.r, t);
            uint4 *to = reinterpret_cast<uint4 *>(dz);
            const bool zero = gr.y < 0;
            if (zero) {
                for (int k = lane; k < nvec; k += 32) __stcs(to + k, make_uint4(0, 0, 0, 0));
            } else {
                int k = lane;
                for (; k - lane + 32 * kBatch <= nvec; k += 32 * kBatch) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) v[b] = line[k + 32 * b];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) __stcs(to + k + 32 * b, post_grad_group<T>(v[b], gr.a, gr.m, c));
                }
                for (; k < nvec; k += 32) __stcs(to + k, post_grad_group<T>(line[k], gr.a, gr.m, c));
                if (OP != kOpDistill && gr.y < nvec * VEC && ((gr.y / VEC) & 31) == lane) VT::store1(dz, gr.y, gr.gy);
            }
            if (has_tail) {
                const float e = zero ? 0.f : gr.a * ex2_approx((tail_z - gr.m) * c);
                VT::store1(dz, tail_v, OP != kOpDistill && !zero && tail_v == gr.y ? gr.gy : e);
            }
            if constexpr (OP == kOpDistill) {
                __syncwarp();  // the entries replace what the row's other lanes have written there
                if (live)
                    for (int k = lane; k < K; k += 32)
                        if (s_id[k] >= 0) VT::store1(dz, s_id[k], distill_entry(p, row, s_z[k], s_lq[k]));
            }
        }
        ptx::fence_proxy_async_smem();  // the next copy comes after the marks
        __syncwarp();
        if (++i == n) {
            i = 0;
            first += (int64_t)32 * W;
            n = count_of();
            if (lane < n) mine = load_meta<T, OP>(p, row_of(lane), N);
        }
        if (n > 0) start(i);
    }
    if constexpr (OP == kOpPolicy || OP == kOpDistill) line_sums(p, sum);
}

// ---------------------------------------------------------------- rows too long for the rings

constexpr int kThreads = 512;
constexpr int kMarkBits = 1 << 16;  // vocabulary entries whose marks are held at once (distill)

template <bool kEnt>
__device__ __forceinline__ PostStats block_merge(PostStats st, PostStats *s_warp, float c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    st = post_warp_merge<kEnt>(st, c);
    __syncthreads();
    if (lane == 0) s_warp[warp] = st;
    __syncthreads();
    st = lane < kThreads / 32 ? s_warp[lane] : kPostStart;
    return post_warp_merge<kEnt>(st, c);
}

// Statistics of a row without its entry y (y < 0: of the whole row).
template <typename T, bool kEnt>
__device__ __forceinline__ PostStats row_stats(const char *z, int V, float c, int y) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    const int nvec = V / VEC;
    PostStats st = kPostStart;
#pragma unroll 4
    for (int k = threadIdx.x; k < nvec; k += kThreads) {
        float x[VEC];
        VT::decode(*reinterpret_cast<const uint4 *>(z + (size_t)k * 16), x);
        if (y >= 0 && k == y / VEC) {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (j == y % VEC) x[j] = -INFINITY;
        }
        post_fold<kEnt>(st, x, c);
    }
    const int v = nvec * VEC + threadIdx.x;
    if (v < V && v != y) {
        float x[1] = {VT::load1(z, v)};
        post_fold<kEnt>(st, x, c);
    }
    return st;
}

// dz_v = a 2^{c (z_v - m)}, except dz_y = gy (y < 0: no such entry). a == 0 writes zeros without reading.
template <typename T>
__device__ __forceinline__ void write_row(const char *z, char *dz, int V, float c, RowGrad gr) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    const int nvec = V / VEC;
    const bool zero = gr.a == 0.f && gr.y < 0;
#pragma unroll 4
    for (int k = threadIdx.x; k < nvec; k += kThreads) {
        float x[VEC];
        if (zero) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[j] = 0.f;
        } else {
            VT::decode(*reinterpret_cast<const uint4 *>(z + (size_t)k * 16), x);
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[j] = gr.a * ex2_approx((x[j] - gr.m) * c);
            if (k == gr.y / VEC && gr.y >= 0) {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (j == gr.y % VEC) x[j] = gr.gy;
            }
        }
        __stcs(reinterpret_cast<uint4 *>(dz + (size_t)k * 16), VT::encode(x));
    }
    const int v = nvec * VEC + threadIdx.x;
    if (v < V) VT::store1(dz, v, zero ? 0.f : v == gr.y ? gr.gy : gr.a * ex2_approx((VT::load1(z, v) - gr.m) * c));
}

template <typename T, bool kEnt>
__global__ void __launch_bounds__(kThreads) long_policy_kernel(PolicyParams p) {
    __shared__ PostStats s_warp[kThreads / 32];
    __shared__ RowGrad s_grad;
    __shared__ PostTerm s_term;
    for (int t = blockIdx.x; t < p.r.T; t += gridDim.x) {
        const char *z = row_in<T>(p.r, t);
        const bool read = p.read_masked || __ldg(p.r.mask + t);
        const int y = __ldg(p.r.targets + t);
        const bool ok = y >= 0 && y < p.r.V;
        PostStats st{0.f, 1.f, 0.f};
        if (read) st = block_merge<kEnt>(row_stats<T, kEnt>(z, p.r.V, kLog2e, ok ? y : -1), s_warp, kLog2e);
        if (threadIdx.x == 0) {
            PostToken tok{st, 0.f, 0.f};
            if (ok && read) tok = post_target<kEnt>(st, PostVec<T>::load1(z, y));
            const PolicyTok k = policy_load(p, t, find_seq(p.r.cu_seqlens, p.r.S, t));
            const PolicyRow row = policy_row(p, k, tok, read);
            s_term = policy_write<kEnt>(p, t, k, tok, row, read);
            s_grad = row.grad;
        }
        __syncthreads();
        if (threadIdx.x < 32) one_term(p, t, s_term);
        const RowGrad gr = s_grad;
        write_row<T>(z, row_out<T>(p.r, t), p.r.V, kLog2e, gr);
        __syncthreads();
    }
    if (p.r.T == 0 && threadIdx.x < 32) write_loss(p, PostPartial{});
}

template <typename T>
__global__ void __launch_bounds__(kThreads) long_distill_kernel(DistillParams p) {
    using VT = PostVec<T>;
    constexpr int VEC = VT::kElems;
    extern __shared__ float s_dyn[];
    float *s_z = s_dyn, *s_lq = s_dyn + p.K;
    int *s_id = reinterpret_cast<int *>(s_dyn + 2 * p.K);
    __shared__ uint32_t s_mark[kMarkBits / 32];
    __shared__ PostStats s_warp[kThreads / 32];
    __shared__ DistillRow s_row;
    __shared__ int s_int[32];
    const int V = p.r.V, nvec = V / VEC;
    int N = 0;
    if (p.per_token) {
        for (int i = threadIdx.x; i < p.r.S; i += kThreads) N += p.seq_n[i];
        N = block_sum_i32(N, s_int);
    }
    for (int t = blockIdx.x; t < p.r.T; t += gridDim.x) {
        const char *z = row_in<T>(p.r, t);
        char *dz = row_out<T>(p.r, t);
        const int i = find_seq(p.r.cu_seqlens, p.r.S, t);
        const bool on = i >= 0 && __ldg(p.r.mask + t);
        if (!on) {
            if (threadIdx.x == 0 && p.kl) p.kl[t] = 0.f;
            if (threadIdx.x < 32) one_term(p, t, PostTerm{});
            write_row<T>(z, dz, V, p.c, RowGrad{0.f, 0.f, 0.f, -1});
            continue;
        }
        const float4 rec = p.rec[t];
        // the teacher's entries
        int bad = 0, have = 0;
        for (int k = threadIdx.x; k < p.K; k += kThreads) {
            const int id = __ldg(p.ids + (int64_t)t * p.ldk + k);
            const bool real = id >= 0 && id < V;
            bad |= id < -1 || id >= V;
            have += real;
            s_id[k] = real ? id : -1;
            s_z[k] = real ? VT::load1(z, id) : -INFINITY;
            s_lq[k] = real ? (__ldg(p.vals + (int64_t)t * p.ldk + k) - rec.x) - rec.y : -INFINITY;
        }
        have = block_sum_i32(have, s_int);
        // the statistics outside them: marked entries count as -inf
        PostStats st = kPostStart;
        for (int64_t base = 0; base < V; base += kMarkBits) {
            for (int w = threadIdx.x; w < kMarkBits / 32; w += kThreads) s_mark[w] = 0;
            __syncthreads();
            for (int k = threadIdx.x; k < p.K; k += kThreads) {
                const int64_t at = (int64_t)s_id[k] - base;
                if (s_id[k] >= 0 && at >= 0 && at < kMarkBits)
                    bad |= (atomicOr(&s_mark[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1;  // listed twice
            }
            __syncthreads();
            const int k1 = (int)min((int64_t)nvec, (base + kMarkBits) / VEC);
            for (int k = (int)(base / VEC) + threadIdx.x; k < k1; k += kThreads) {
                float x[VEC];
                VT::decode(*reinterpret_cast<const uint4 *>(z + (size_t)k * 16), x);
                const int at = (int)((int64_t)k * VEC - base);
                const uint32_t mark = s_mark[at >> 5] >> (at & 31);
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if ((mark >> j) & 1) x[j] = -INFINITY;
                post_fold<false>(st, x, p.c);
            }
            if (base + kMarkBits >= V && nvec * VEC + (int)threadIdx.x < V) {
                const int v = nvec * VEC + threadIdx.x, at = (int)(v - base);
                if (at >= 0) {  // the last entries lie in the last chunk
                    float x[1] = {(s_mark[at >> 5] >> (at & 31)) & 1 ? -INFINITY : VT::load1(z, v)};
                    post_fold<false>(st, x, p.c);
                }
            }
            __syncthreads();
        }
        bad = __syncthreads_or(bad);
        st = block_merge<false>(st, s_warp, p.c);
        const int n_i = p.seq_n[i];
        const float w = 1.f / (p.per_token ? (float)N : (float)p.r.S * (float)n_i);
        const bool none = have == 0 || rec.w == kNoMass;
        if (bad || none) {  // excluded: contributes nothing
            if (threadIdx.x == 0) {
                if (bad) post_raise(p.r.status, RL_ERR_TARGET_RANGE);
                if (p.kl) p.kl[t] = bad ? __int_as_float(0x7fc00000) : 0.f;
            }
            if (threadIdx.x < 32) one_term(p, t, PostTerm{});
            write_row<T>(z, dz, V, p.c, RowGrad{0.f, 0.f, 0.f, -1});
            __syncthreads();
            continue;
        }
        if (threadIdx.x < 32) {
            const DistillRow r = distill_finish(p, st, distill_entries(p, s_z, s_lq, rec), rec, w * p.scale * p.inv_tau, V - have);
            const float kl = p.reverse ? r.kl : distill_forward(p, r, s_z, s_lq, rec);
            if (threadIdx.x == 0) {
                s_row = r;
                if (!isfinite(r.ls)) post_raise(p.r.status, RL_ERR_NONFINITE);
                if (p.kl) p.kl[t] = kl;
            }
            __syncwarp();
            one_term(p, t, PostTerm{w * p.scale * kl, 0.f, 0.f, 0.f});
        }
        __syncthreads();
        const DistillRow r = s_row;
        // the teacher's entries are written after the rest of the row, whose value they replace
        write_row<T>(z, dz, V, p.c, RowGrad{r.ct, r.m, 0.f, -1});
        __syncthreads();
        for (int k = threadIdx.x; k < p.K; k += kThreads)
            if (s_id[k] >= 0) VT::store1(dz, s_id[k], distill_entry(p, r, s_z[k], s_lq[k]));
        __syncthreads();
    }
    if (p.r.T == 0 && threadIdx.x < 32) write_loss(p, PostPartial{});
}

// ---------------------------------------------------------------- launches

// Shared memory of a CTA: what three CTAs (two, one) on an SM leave each of its 228 KB, less the 1 KB that
// the system takes per CTA.
constexpr size_t kCtaBytes[3] = {76800, 115712, 231424};

// A GB300's SMs. A cut goes by this number and not by the device's, as the order of a row's additions goes by its cut.
constexpr int kSms = 152;

// How many clusters of this launch are resident at once; sets the kernel's shared-memory limit on its
// first use on a device and size. Remembered for the last sizes asked for.
cudaError_t resident_clusters(const void *kernel, const cudaLaunchConfig_t &cfg, int C, int max_dynamic, int *out) {
    struct Entry {
        const void *kernel = nullptr;
        int dev = -1, C = 0;
        size_t smem = 0;
        int resident = 0;
    };
    constexpr int kEntries = 64;
    static std::mutex mu;
    static Entry known[kEntries];
    static int next = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry &k : known)
        if (k.kernel == kernel && k.dev == dev && k.C == C && k.smem == cfg.dynamicSmemBytes) {
            *out = k.resident;
            return cudaSuccess;
        }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, max_dynamic);
    int resident = 0;
    if (e == cudaSuccess && cfg.numAttrs > 1) {
        e = cudaOccupancyMaxActiveClusters(&resident, kernel, &cfg);
    } else if (e == cudaSuccess) {
        int sms = 0, per = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, (int)cfg.blockDim.x, cfg.dynamicSmemBytes);
        resident = sms * per / C;
    }
    if (e != cudaSuccess) return e;
    *out = std::max(1, resident);
    known[next] = Entry{kernel, dev, C, cfg.dynamicSmemBytes, *out};
    next = (next + 1) % kEntries;
    return cudaSuccess;
}

template <typename T, int OP, bool kEnt>
cudaError_t launch_lines(const typename OpParams<OP>::type &p, int K, bool after_own, cudaStream_t stream) {
    auto kernel = line_rows_kernel<T, OP, kEnt>;
    const int stride = p.r.V / PostVec<T>::kElems + (3 * K + 3) / 4;  // 16-byte groups of a warp
    constexpr size_t kStatic = kLineWarps * (sizeof(RowMeta<OP>) + 16);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(32 * kLineWarps);
    cfg.dynamicSmemBytes = (size_t)kLineWarps * stride * 16;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = after_own ? 1 : 0;
    int resident = 0;
    const cudaError_t e = resident_clusters(reinterpret_cast<const void *>(kernel), cfg, 1, (int)(kCtaBytes[2] - kStatic), &resident);
    if (e != cudaSuccess) return e;
    // blocks without a row to spare, and no more than their sums have room for
    cfg.gridDim = dim3((unsigned)std::max(1, std::min(resident, p.r.T / kLineWarps)));
    return cudaLaunchKernelEx(&cfg, kernel, p, stride);
}

template <typename T, int OP, bool kEnt>
cudaError_t launch_ring(const typename OpParams<OP>::type &p, int K, bool after_own, cudaStream_t stream, bool &fits) {
    auto kernel = ring_rows_kernel<T, OP, kEnt>;
    constexpr bool kStats = OP != kOpScale, kKeep = OP == kOpPolicy || OP == kOpDistill;
    const int nvec = p.r.V / PostVec<T>::kElems;
    constexpr size_t kMaxDynamic = kCtaBytes[2] - sizeof(RowShared<OP>);
    fits = true;
    if (p.r.T > 0 && nvec <= kLineBytes / 16) return launch_lines<T, OP, kEnt>(p, K, after_own, stream);
    const size_t fixed = sizeof(RowShared<OP>) + (size_t)kMetaOf(OP) * 12 * K;
    RowPlan plan{};
    fits = false;
    // enough CTAs per row that the rows there are fill the SMs
    const int least = std::max(1, std::min({(int)kMaxCluster, kRowBlocks * kSms / std::max(1, p.r.T), nvec / 256}));
    if (kKeep) {
        // A row's stay in the rings is set by its chain of steps, so the rate goes by the bytes that an SM's rings
        // hold, a slice for each CTA: the plan that holds most, and of those within 5% with two or three CTAs on an SM
        // the one with the fewest per row. (50257 bf16: one a row, two on an SM, 201 KB, 82% of the copy rate; two and three,
        // 151 KB, 73%. 128256 bf16: four and three, 192 KB, 84%; three and two, 171 KB, 77%; seven and three
        // with two slices each, 73%. 100000 bf16: two and two, 200 KB, 89%; one and one, 200 KB, 80%.)
        int64_t best = 0;
        for (int occ = 0; occ < 3; ++occ) {
            const int room = (int)((kCtaBytes[occ] - fixed) / (16 * kWarps));  // groups in a warp's ring
            for (int C = least; C <= kMaxCluster; ++C) {
                const int slice = std::max(1, (nvec + C - 1) / C), share = (slice + kWarps - 1) / kWarps;
                // a segment's two barriers take one group's room
                const int depth = std::min(kMaxDepth, room / (share + 1));
                if (depth < 1) continue;
                const int64_t held = (int64_t)(3 - occ) * slice;
                if (fits && !(held * 20 > best * 21 || (occ < 2 && held * 20 >= best * 19 && C < plan.cluster))) continue;
                best = held;
                plan = RowPlan{C, slice, 1, share, depth, 1, depth >= 2};
                fits = true;
            }
        }
        if (!fits) return cudaSuccess;
    } else {  // two segments of whole batches in a warp's ring, or more shorter ones
        const int room = (int)((kCtaBytes[0] - fixed) / (16 * kWarps)), batch = 32 * kBatch;
        const int slice = std::max(1, (nvec + least - 1) / least), share = (slice + kWarps - 1) / kWarps;
        const int seg = std::min(share, std::max(batch, (room / 2 - 1) / batch * batch));
        plan = RowPlan{least, slice, (share + seg - 1) / seg, seg, std::min(kMaxDepth, room / (seg + 1)), 1, 0};
        fits = true;
    }
    const int C = plan.cluster;
    const size_t smem = std::max<size_t>((size_t)plan.depth * kWarps * (plan.seg + 1) * 16 + (size_t)kMetaOf(OP) * 12 * K, 1024);

    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = kStats && C > 1 ? 2 : 1;
    int resident = 0;
    cudaError_t e = resident_clusters(reinterpret_cast<const void *>(kernel), cfg, C, (int)kMaxDynamic, &resident);
    if (e != cudaSuccess) return e;
    // a ticket's rows: 128 KB of a CTA's share, so that the dozen dependent loads behind a ticket are spread
    // over rows that take long enough, where that leaves every cluster four tickets
    plan.rows = OP == kOpLogp ? 32 : std::max(1, std::min({32, 8192 / plan.slice, p.r.T / (4 * resident)}));
    const int nclusters = std::max(1, std::min(p.r.T, resident));
    cfg.gridDim = dim3((unsigned)(nclusters * C));
    // the launch may begin while the one before it ends (it waits before it reads anything of that one's)
    if (!after_own) cfg.attrs = attr + 1, cfg.numAttrs -= 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, plan, nclusters);
}

template <typename T>
cudaError_t launch_logp(const LogpParams &p, cudaStream_t stream) {
    bool fits;
    return p.r.entropy ? launch_ring<T, kOpLogp, true>(p, 0, false, stream, fits) : launch_ring<T, kOpLogp, false>(p, 0, false, stream, fits);
}

int long_grid(int T) { return std::max(1, std::min(T, 608)); }

template <typename T>
cudaError_t launch_policy(const PolicyParams &p, cudaStream_t stream) {
    const bool ent = p.r.entropy || p.mean_entropy;
    bool fits;
    const cudaError_t e = ent ? launch_ring<T, kOpPolicy, true>(p, 0, true, stream, fits) : launch_ring<T, kOpPolicy, false>(p, 0, true, stream, fits);
    if (fits) return e;
    if (ent) long_policy_kernel<T, true><<<long_grid(p.r.T), kThreads, 0, stream>>>(p);
    else long_policy_kernel<T, false><<<long_grid(p.r.T), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_distill(const DistillParams &p, cudaStream_t stream) {
    bool fits;
    const cudaError_t e = launch_ring<T, kOpDistill, false>(p, p.K, true, stream, fits);
    if (fits) return e;
    long_distill_kernel<T><<<long_grid(p.r.T), kThreads, (size_t)p.K * 12, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_scale(const ScaleParams &p, cudaStream_t stream) {
    bool fits;
    return launch_ring<T, kOpScale, false>(p, 0, true, stream, fits);
}

}  // namespace

cudaError_t launch_post_logp(const LogpParams &p, int dtype, cudaStream_t stream) {
    if (p.r.T == 0 && !p.zero) return cudaSuccess;
    return dtype == RL_F32 ? launch_logp<float>(p, stream) : launch_logp<__nv_bfloat16>(p, stream);
}

cudaError_t launch_post_policy(const PolicyParams &p, int dtype, cudaStream_t stream) {
    return dtype == RL_F32 ? launch_policy<float>(p, stream) : launch_policy<__nv_bfloat16>(p, stream);
}

cudaError_t launch_post_distill(const DistillParams &p, int dtype, cudaStream_t stream) {
    return dtype == RL_F32 ? launch_distill<float>(p, stream) : launch_distill<__nv_bfloat16>(p, stream);
}

cudaError_t launch_post_scale(const ScaleParams &p, int dtype, cudaStream_t stream) {
    if (p.r.T == 0) return cudaSuccess;
    return dtype == RL_F32 ? launch_scale<float>(p, stream) : launch_scale<__nv_bfloat16>(p, stream);
}

}  // namespace rlk
