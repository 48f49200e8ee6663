"""Where the norms' kernels read and write shared memory, against what their launches allocate: all widths, types and row
counts that decide a layout, on the CPU (csrc/norm_layout.cuh is plain C++)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHECK = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "norm_layout.cuh"
using namespace rlk;

static long cases = 0;
#define NEED(cond)                                                                                                                \
    do {                                                                                                                          \
        if (!(cond)) {                                                                                                            \
            std::printf("%s: cols %d rows %d es %d %d %d full %d mode %d: depth %d stage %d smem %zu\n", #cond, cols, rows, es[0], \
                        es[1], es[2], (int)full, (int)mode, n.depth, n.stage_bytes, n.smem);                                      \
            std::exit(1);                                                                                                         \
        }                                                                                                                         \
    } while (0)

static int up16(int x) { return (x + 15) / 16 * 16; }

// The furthest byte behind a row's start in shared memory that a kernel reads. Vectors are read whole (16 bytes of bf16, 32
// of fp32, 8 codes); in kShiftRow a vector's pieces and the one behind them, of codes the words from `shift` on; in kAnyRow
// single columns behind a shift of up to 15 bytes.
static int furthest(int cols, int es, int mode) {
    const int vecs = (cols + 7) / 8;
    if (mode == kAnyRow) return 15 / es * es + cols * es;
    if (mode == kShiftRow) return es == 1 ? 12 + vecs * 8 + 4 : vecs * 8 * es + 16;
    return vecs * 8 * es;
}

template <typename Teams>
static void check(const Teams &n, int cols, int rows, const int (&es)[3], bool full, int mode, int warps_of_block, bool backward) {
    ++cases;
    const int at[4] = {0, n.at_dy, es[2] || backward ? n.at_ds : n.stage_bytes, n.stage_bytes}, vecs = (cols + 7) / 8;
    const int teams = mode == kWarpRow ? warps_of_block : 1, T = mode == kWarpRow ? 32 : n.warps * 32;
    const size_t rings = (size_t)teams * n.depth * n.stage_bytes;
    NEED(n.depth >= 1 && n.depth <= kNormDepth && n.smem <= kNormRingSmem && rings <= n.smem);
    NEED(n.warps >= 1 && n.warps <= 16 && n.vecs >= 1 && n.vecs <= 4 && n.blocks_per_sm >= 1);
    // every vector belongs to a thread, and only the last ones may be missing
    NEED(T * n.vecs >= vecs && T * (n.vecs - 1) < vecs);
    for (int k = 0; k < 3; ++k) {
        if (!es[k]) continue;
        NEED(at[k] % 16 == 0 && at[k + 1] <= n.stage_bytes);
        NEED(at[k] + furthest(cols, es[k], mode) <= at[k + 1]);
        const int copied = starts_anywhere(mode) ? up16(15 / es[k] * es[k] + cols * es[k]) : n.copy_bytes[k];
        NEED(copied % 16 == 0 && copied >= cols * es[k] && at[k] + copied <= at[k + 1]);
        // nothing is copied from behind the row's last 16 bytes
        NEED(starts_anywhere(mode) || copied < cols * es[k] + 16);
    }
    if (n.w_in_smem && mode != kWarpRow) {
        const int params = backward ? 1 : full && n.vecs == 4 ? 2 : 0;
        NEED(rings + (size_t)params * n.vecs * T * 8 * 4 <= n.smem || (backward && n.vecs <= (mode == kAnyRow ? 1 : mode == kShiftRow ? 2 : full ? 3 : 4)));
    }
    if (backward && mode == kWarpRow) NEED((size_t)teams * n.vecs * 32 * 8 * 4 <= n.smem);  // the warps' sums
    // blocks that are said to share an SM do
    const size_t barriers = (size_t)teams * kNormDepth * 8 + 256;
    NEED(n.blocks_per_sm * (n.smem + barriers + 1024) <= kSmemOfSM);
}

static void forward(int cols, int rows) {
    for (int xe : {2, 4})
        for (int res : {0, 1})
            for (int rms : {0, 1})
                for (int bias : {0, 1})
                    for (int codes : {0, 1})
                        for (int masked : {0, 1})
                            for (int fast : {0, 1}) {
                                if (fast && cols <= kShortCols) continue;
                                const NormForwardShape p{rows, cols, xe, res ? xe : 0, rms != 0, bias != 0, masked != 0, codes != 0};
                                const RowMode mode = norm_forward_mode(p, fast != 0);
                                const NormTeams n = norm_forward_teams(p, mode);
                                const int es[3] = {xe, res ? xe : 0, 0};
                                const bool full = forward_full(p, mode);
                                check(n, cols, rows, es, full, mode, kForwardWarps, false);
                                NEED(n.blocks >= 1 && n.blocks <= rows);
                                NEED(mode != kAnyRow || n.vecs <= 2);  // the widest kernel of that kind
                                NEED(mode != kWarpRow || n.vecs == (full || cols <= 768 ? 3 : 4));
                            }
}

static void backward(int cols, int rows) {
    for (int he : {1, 2, 4})
        for (int dye : {2, 4})
            for (int dse : {0, 2, 4})
                for (int rms : {0, 1})
                    for (int db : {0, 1})
                        for (int fast : {0, 1}) {
                            if (fast && cols <= kShortCols) continue;
                            if (he != 1 && dse && dse != he) continue;
                            const NormBackwardShape p{rows, cols, he, dye, dse, rms != 0, db != 0};
                            const RowMode mode = norm_backward_mode(p, fast != 0);
                            const NormTeams n = norm_backward_teams(p, mode);
                            const int es[3] = {he, dye, dse};
                            const bool full = backward_full(p, mode);
                            check(n, cols, rows, es, full, mode, kNormWarps, true);
                            const int blocks = norm_backward_blocks(p, n);
                            NEED(blocks >= 1 && blocks <= norm_backward_parts(rows, cols));
                            NEED(mode != kWarpRow || n.vecs == (full || cols <= 768 ? 3 : 4));
                        }
}

// The last vector of an fp32 row may be read into the next row or behind the rings, never past the block's memory.
static void shorts(int cols) {
    const int rows = 0, mode = -1;
    const bool full = false;
    const int width = norm_short_width(cols), vecs = (cols + 7) / 8;
    for (int back : {0, 1})
        for (int a : {1, 2, 4})
            for (int b : {0, 2, 4})
                for (int c : {0, 2, 4})
                    for (int masked : {0, 1})
                        for (int gap : {0, 16}) {
                            if (!back && (a == 1 || c || (b && a != b))) continue;
                            if (back && !b) continue;
                            const int es[3] = {a, b, c};
                            int64_t ld[3];
                            for (int k = 0; k < 3; ++k) ld[k] = es[k] ? (up16(cols * es[k]) + gap) / es[k] : 0;
                            const int warps = back ? kNormWarps : kShortWarps;
                            const size_t fixed = (size_t)width * (back ? 4 : 8), least = back ? (size_t)kNormWarps * width * 4 : 0;
                            const NormShort n = norm_short(cols, es, ld, back ? 3 : 2, masked != 0, warps, fixed, least);
                            ++cases;
                            NEED(n.depth >= 1 && n.depth <= kNormDepth && n.smem <= kNormRingSmem);
                            NEED(n.lanes * n.vecs >= vecs && width == n.lanes * n.vecs * 8 && 32 % n.lanes == 0 && n.lanes % 4 == 0);
                            const size_t rings = (size_t)warps * n.depth * n.stage_bytes;
                            NEED(rings + fixed <= n.smem && least <= n.smem);
                            for (int k = 0; k < 3; ++k) {
                                if (!es[k]) continue;
                                const int per = 32 / n.lanes, end = k < 2 && es[k + 1] ? n.at[k + 1] : k < 1 && es[2] ? n.at[2] : n.stage_bytes;
                                NEED(n.at[k] % 16 == 0 && n.at[k] + per * n.row_bytes[k] <= end);
                                NEED(!n.whole[k] || (!masked && !gap));
                                NEED(rings - n.stage_bytes + n.at[k] + (per - 1) * n.row_bytes[k] + vecs * 8 * es[k] <= n.smem);
                            }
                        }
}

int main() {
    static const int kRows[] = {ROWS};
    for (int cols = 1; cols <= kShortCols; ++cols) shorts(cols);
    for (int cols = 1; cols <= kNormMaxCols; ++cols)
        for (int rows : kRows) {
            forward(cols, rows);
            backward(cols, rows);
        }
    std::printf("%ld\n", cases);
}
"""


def run(tmp_path, rows, *flags):
    """Compiles and runs the check of these row counts; how many layouts it saw."""
    src, exe = tmp_path / "layout.cpp", tmp_path / "layout"
    src.write_text(CHECK.replace("ROWS", ", ".join(map(str, rows))))
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", *flags, "-I", os.path.join(ROOT, "rl_post_loss_gb300", "csrc"), str(src), "-o", str(exe)])
    done = subprocess.run([str(exe)], stdout=subprocess.PIPE, timeout=300)
    assert done.returncode == 0, done.stdout.decode()
    return int(done.stdout)


@pytest.mark.parametrize("rows", [(1, 37, 2431), (2432, 20000), (1 << 20,)], ids=str)
def test_every_access_is_inside_the_allocation(tmp_path, rows):
    assert run(tmp_path, rows) > 1000000


def test_the_most_rows_do_not_overflow(tmp_path):
    """The arithmetic of a layout in range up to 2^31 - 1 rows (an overflow ends the program)."""
    assert run(tmp_path, [2 ** 31 - 1, 2 ** 31 - 200], "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error") > 1000000
