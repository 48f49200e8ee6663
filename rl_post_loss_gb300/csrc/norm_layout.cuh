// How the norms lay rows over blocks and shared memory: arithmetic on the host alone (plain C++, no CUDA), so that
// every access that a kernel makes of its shared memory can be checked against the allocation for all widths and types.
//
// A row's room in a stage is that of its whole vectors of eight columns, as the last one is read whole (what lies past the
// row's end is then set to 0): for fp32 up to 16 bytes more than a copy brings.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace rlk {

constexpr int kNormMaxCols = 16384;
constexpr int kNormSMs = 152;
constexpr int kNormVec = 8;        // columns of a vector
constexpr int kNormWarps = 16;     // of an SM in the backward pass: 128 registers a thread
constexpr int kForwardWarps = 16;  // and in the forward pass
constexpr int kShortWarps = 24;    // of a block of the forward pass of short rows: 80 registers a thread
constexpr int kShortCols = 512;    // rows of norm_short.cuh, at most
constexpr int kNormDepth = 8;      // rows (of short ones: batches) of a ring, at most
constexpr size_t kNormRingSmem = 225 * 1024;  // of a block, beside its barriers and sums
constexpr size_t kSmemOfSM = 228 * 1024;
// what a block takes beside its rows
constexpr size_t kForwardExtra = 1024 + 1024, kBackwardExtra = 1024 + 512;

enum RowMode { kBlockRow, kWarpRow, kAnyRow, kShiftRow };  // norm_rows.cuh
constexpr bool starts_anywhere(int mode) { return mode == kAnyRow || mode == kShiftRow; }

struct NormTeams {
    int mode;                         // RowMode
    int warps, vecs, blocks_per_sm;   // of a row; vectors of eight columns of a thread
    int blocks;                       // of the forward pass
    int depth;                        // rows' room of a team in shared memory
    int w_in_smem;                    // the weight beside them, where registers have no room for it
    int copy_bytes[3];                // what a copy brings of a row of each matrix (where rows start anywhere: `window`)
    int at_dy, at_ds, stage_bytes;    // of a row
    size_t smem;
};

// What the layout depends on. `es`: bytes of an element, 0 where there is no such matrix.
struct NormForwardShape {
    int rows, cols;
    int x_es, residual_es;
    bool rms, bias, masked, codes;
};
struct NormBackwardShape {
    int rows, cols;
    int h_es, dy_es, dsummed_es;  // h_es 1: from a checkpoint
    bool rms, want_db;
};

inline int norm_vectors(int cols) { return (cols + kNormVec - 1) / kNormVec; }
inline int norm_copy_bytes(int cols, int es) { return (cols * es + 15) / 16 * 16; }
inline int norm_room(int cols, int es, int mode) {
    return starts_anywhere(mode) ? norm_copy_bytes(cols, es) + 32 : (norm_vectors(cols) * kNormVec * es + 15) / 16 * 16;
}

// ---------------------------------------------------------------- forward

// Two rows of a block in its ring: with as many as fit, reads far ahead of the writes cost the memory's rate. (65536 x 6144
// bf16, RMS: 246 us, with eight 281; 32768 x 16384: 317, 367.)
constexpr int kForwardDepth = 2;

// The mean or a bias are part of the work (they always are where rows start anywhere).
inline bool forward_full(const NormForwardShape &p, int mode) { return starts_anywhere(mode) || !p.rms || p.bias; }

inline RowMode norm_forward_mode(const NormForwardShape &p, bool fast) {
    // The pieces shifted into place, where 8-bit codes are made or a thread would hold more than two vectors' single columns,
    // whose weights have no room in registers: 16000 x 3001 bf16 layer norm to int8 94 us (single columns 199), 8920 x 9118 bf16
    // with a residual 182 (270), 8192 x 6145 layer norm 95 (99); but 8192 x 4095 61 (52), 30000 x 1031 fp32 with a residual 115 (88).
    if (!fast) return p.codes || p.cols > 4096 ? kShiftRow : kAnyRow;
    // a warp per row where there are rows for all
    return p.cols <= (forward_full(p, kBlockRow) ? 768 : 1024) && p.rows >= kNormSMs * kForwardWarps ? kWarpRow : kBlockRow;
}

// The blocks that run at once, or, for as many bytes to write as to read, blocks of eight rows for a warp or block, which
// start when others end: they do not read and write all in step, and a slow SM takes fewer. Where the weights' way into shared memory
// or arithmetic is what a block waits for, their starts cost more, and masked rows break the step too. (RMS with a
// residual, us: 65536 x 6144 bf16 with an int8 checkpoint 599 -> 525, 32768 x 6144 fp32 527 -> 471, 8192 x 6144 bf16 72 -> 65; layer norm
// so 534 -> 466; but with an e4m3 checkpoint 65536 x 5120 489 -> 576, without a residual 16384 x 6144 79 -> 88, with a mask 125 -> 132.)
inline int forward_blocks(const NormForwardShape &p, int mode, const NormTeams &n, int teams) {
    const bool full = forward_full(p, mode);
    const int at_once = std::min(p.rows, kNormSMs * n.blocks_per_sm), short_ones = p.rows / (8 * teams);
    const bool apart = p.residual_es && !p.masked && !starts_anywhere(mode) && (!full || (mode == kBlockRow && n.vecs < 4 && !p.codes));
    return apart && short_ones >= 3 * at_once ? short_ones : at_once;
}

// A block per row, 16 warps on an SM: of the numbers of vectors a thread, the one whose blocks take all rows soonest, by a
// row's time of its vectors and two or three more for its exchanges of sums and what else is done once a row. (16384 x
// 8192 bf16: layer norm with two, three, four vectors 141, 147, 125 us, RMS with a residual 180, 174, 181 (without blocks of eight rows); 20000 x 5120: 156, 92,
// 102 us; so layer norm with four, whose weights are read from shared memory, counts as 9.8.)
inline NormTeams norm_forward_teams(const NormForwardShape &p, RowMode mode) {
    const int vecs = norm_vectors(p.cols);
    const bool full = forward_full(p, mode);
    NormTeams n{};
    n.mode = mode;
    n.copy_bytes[0] = norm_copy_bytes(p.cols, p.x_es);
    n.copy_bytes[1] = p.residual_es ? n.copy_bytes[0] : 0;
    n.at_dy = norm_room(p.cols, p.x_es, mode);
    n.stage_bytes = n.at_dy * (p.residual_es ? 2 : 1);
    if (mode == kWarpRow) {
        n.warps = 1;
        n.vecs = vecs > 96 ? 4 : 3;
        n.blocks_per_sm = 1;
        n.depth = (int)std::min<size_t>(kNormDepth, kNormRingSmem / (kForwardWarps * n.stage_bytes));
        n.smem = (size_t)(kForwardWarps) * n.depth * n.stage_bytes;
        n.blocks = forward_blocks(p, mode, n, kForwardWarps);
        return n;
    }
    double best = 0;
    for (int v = 1; v <= 4; ++v) {
        const int warps = (vecs + 32 * v - 1) / (32 * v);
        if (warps > kForwardWarps || (v - 1) * warps * 32 >= vecs) continue;
        if (n.warps && mode == kAnyRow && v > 2) continue;  // (registers)
        // layer norm with four vectors a thread: weight and bias in shared memory, as registers have no room
        size_t params = mode != kAnyRow && full && v == 4 ? (size_t)2 * v * warps * 32 * kNormVec * 4 : 0;
        int blocks = kForwardWarps / warps;
        while (blocks > 1 && blocks * (kForwardExtra + params + 2 * n.stage_bytes) > kSmemOfSM) --blocks;
        const double time = (double)(((int64_t)p.rows + blocks * kNormSMs - 1) / (blocks * kNormSMs)) * (v + (p.rms ? 2 : v == 4 ? 5.8 : 3));
        if (n.warps && time >= best) continue;
        best = time;
        const size_t room = std::min(kNormRingSmem, kSmemOfSM / blocks - kForwardExtra);
        n.w_in_smem = params + n.stage_bytes <= room;
        if (!n.w_in_smem) params = 0;
        n.warps = warps, n.vecs = v, n.blocks_per_sm = blocks;
        n.depth = (int)std::min<size_t>(kForwardDepth, (room - params) / n.stage_bytes);
        n.smem = (size_t)n.depth * n.stage_bytes + params;
    }
    n.blocks = forward_blocks(p, mode, n, 1);
    return n;
}

// ---------------------------------------------------------------- backward

// Three rows of a block in its ring, of which the last one is filled again a row late. (65536 x 6144 bf16, RMS: 389 us, with four
// 410, with two 419; layer norm 16384 x 8192 164, 164 and 205.)
constexpr int kBackwardDepth = 3;

inline bool backward_full(const NormBackwardShape &p, int mode) { return !p.rms || p.want_db || starts_anywhere(mode); }

inline RowMode norm_backward_mode(const NormBackwardShape &p, bool fast) {
    // bf16 rows with an fp32 dy, a pair that only kAnyRow is built for, go by single columns wherever they start (16384 x 6144
    // layer norm 232 us, 51% of the measured copy rate; with a bf16 dy 105 us)
    if (!fast || (p.h_es == 2 && p.dy_es == 4)) return p.h_es == 1 ? kShiftRow : kAnyRow;
    // a warp per row where there are rows for all warps
    return p.cols <= (backward_full(p, kBlockRow) ? 768 : 1024) && p.rows >= kNormSMs * kNormWarps ? kWarpRow : kBlockRow;
}

// A block per row, 128 registers a thread, so 16 warps on an SM: of the numbers of vectors a thread, the one whose
// blocks take all rows soonest, by a row's time of its vectors and two more for the exchange of sums. Both sums with
// four vectors a thread (kAnyRow: with three) do not fit the registers, and are taken for the
// longest rows alone.
inline NormTeams norm_backward_teams(const NormBackwardShape &p, RowMode mode) {
    const bool full = backward_full(p, mode);
    const int vecs = norm_vectors(p.cols), es[3] = {p.h_es, p.dy_es, p.dsummed_es};
    NormTeams n{};
    n.mode = mode;
    for (int k = 0; k < 3; ++k) n.copy_bytes[k] = norm_copy_bytes(p.cols, es[k]);
    n.at_dy = norm_room(p.cols, p.h_es, mode);
    n.at_ds = n.at_dy + norm_room(p.cols, p.dy_es, mode);
    n.stage_bytes = n.at_ds + (p.dsummed_es ? norm_room(p.cols, p.dsummed_es, mode) : 0);
    if (mode == kWarpRow) {
        n.warps = 1;
        n.vecs = vecs > 96 ? 4 : 3;
        n.blocks_per_sm = 1;
        n.depth = (int)std::min<size_t>(kNormDepth, kNormRingSmem / (kNormWarps * n.stage_bytes));
        n.smem = std::max((size_t)kNormWarps * n.depth * n.stage_bytes, (size_t)kNormWarps * n.vecs * 32 * kNormVec * 4);
        return n;
    }
    double best = 0;
    for (int v = 1; v <= 4; ++v) {
        const int warps = (vecs + 32 * v - 1) / (32 * v);
        if ((v - 1) * warps * 32 >= vecs) continue;  // fewer vectors a thread do
        if (warps > kNormWarps || (v >= (mode == kAnyRow ? 3 : 4) && full && n.warps)) continue;
        const bool regs = mode == kAnyRow ? v == 1 : v <= (mode == kShiftRow ? 2 : 3) || !full;
        size_t w_bytes = regs ? 0 : (size_t)v * warps * 32 * kNormVec * 4;
        int blocks = kNormWarps / warps;
        while (blocks > 1 && blocks * (kBackwardExtra + w_bytes + 2 * n.stage_bytes) > kSmemOfSM) --blocks;
        const double time = (double)(((int64_t)p.rows + blocks * kNormSMs - 1) / (blocks * kNormSMs)) * (v + (v == 4 ? 3.5 : 2));
        if (n.warps && time >= best) continue;
        best = time;
        const size_t room = std::min(kNormRingSmem, kSmemOfSM / blocks - kBackwardExtra);
        n.w_in_smem = w_bytes + n.stage_bytes <= room;
        if (!n.w_in_smem) w_bytes = 0;
        n.warps = warps, n.vecs = v, n.blocks_per_sm = blocks;
        n.depth = (int)std::min<size_t>(kBackwardDepth, (room - w_bytes) / n.stage_bytes);
        n.smem = (size_t)n.depth * n.stage_bytes + w_bytes;
    }
    return n;
}

// The backward pass's blocks, which leave a partial sum each.
inline int norm_backward_blocks(const NormBackwardShape &p, const NormTeams &n) { return std::min(p.rows, kNormSMs * n.blocks_per_sm); }

// As many blocks as run at once, at most: one of 16 warps on an SM for rows that warps take, else of the warps that four
// vectors a thread need.
inline int norm_backward_parts(int rows, int cols) {
    const int warps = (norm_vectors(cols) + 127) / 128;
    return (int)std::min<int64_t>(rows, kNormSMs * (kNormWarps / warps));
}

// ---------------------------------------------------------------- short rows (norm_short.cuh)

// Up to three matrices whose rows come together.
struct NormShort {
    int lanes, vecs, depth;
    int row_bytes[3];  // of a matrix's row in shared memory, 0: no such matrix
    int at[3];         // where a matrix's rows begin in a stage
    int whole[3];      // a batch is one copy
    int stage_bytes;
    size_t smem;
};

inline int norm_short_vecs(int cols) { return cols <= 64 ? 2 : 4; }
inline int norm_short_lanes(int cols) { return cols <= 128 ? 4 : cols <= 256 ? 8 : 16; }
inline int norm_short_width(int cols) { return norm_short_vecs(cols) * norm_short_lanes(cols) * kNormVec; }

// `es` and `ld` of the matrices; `fixed` bytes of a block's shared memory for something else, after the rings. (A row's room
// is what its copy brings, as neighbouring rows come in one copy: the last vector of an fp32 row may be read up to 16 bytes past it,
// into the next row or into those `fixed` bytes, and what it reads there is set to 0.)
inline NormShort norm_short(int cols, const int *es, const int64_t *ld, int count, bool masked, int warps, size_t fixed, size_t least) {
    NormShort n{};
    n.vecs = norm_short_vecs(cols);
    n.lanes = norm_short_lanes(cols);
    for (int k = 0; k < count; ++k) {
        if (!es[k]) continue;
        n.row_bytes[k] = norm_copy_bytes(cols, es[k]);
        n.whole[k] = !masked && ld[k] * es[k] == n.row_bytes[k];
        n.at[k] = n.stage_bytes;
        n.stage_bytes += 32 / n.lanes * n.row_bytes[k];
    }
    n.depth = (int)((kNormRingSmem - fixed) / ((size_t)warps * n.stage_bytes));
    n.depth = n.depth > kNormDepth ? kNormDepth : n.depth;
    n.smem = (size_t)warps * n.depth * n.stage_bytes;
    n.smem = (n.smem > least ? n.smem : least) + fixed;
    return n;
}

}  // namespace rlk
