// C ABI of the norms and of 8-bit activation checkpoints (declared in include/rl_loss.h): argument checks and launches.
#include <cmath>

#include "handle.cuh"
#include "norm.cuh"

namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool known(int32_t dtype) { return dtype == RL_F32 || dtype == RL_BF16; }

rlk::RowMat mat(const void *p, int64_t ld, int32_t dtype) {
    const int64_t es = dtype == RL_F32 ? 4 : 2;
    const auto rows_on = [&](int64_t to) { return aligned(p, (uintptr_t)to) && (ld * es) % to == 0; };
    return rlk::RowMat{const_cast<void *>(p), ld, dtype == RL_BF16, rows_on(32) ? 2 : rows_on(16) ? 1 : 0};
}
rlk::Act8Mat act8(const rl_act8 &a) {
    return rlk::Act8Mat{static_cast<uint8_t *>(a.codes), static_cast<uint8_t *>(a.scales), a.ld_codes, a.ld_scales,
                        a.format == RL_ACT8_E4M3, aligned(a.codes, 16) && a.ld_codes % 16 == 0};
}

rl_status check_mat(const void *p, int64_t ld, int32_t dtype, int32_t cols) {
    if (ld < cols) return RL_ERR_SHAPE;
    return aligned(p, dtype == RL_F32 ? 4 : 2) ? RL_OK : RL_ERR_ALIGNMENT;
}
rl_status check_act8(const rl_act8 &a, int32_t cols) {
    if (!a.codes || !a.scales || (a.format != RL_ACT8_INT8 && a.format != RL_ACT8_E4M3)) return RL_ERR_INVALID_ARG;
    return a.ld_codes < cols || a.ld_scales < (cols + rlk::kAct8Block - 1) / rlk::kAct8Block ? RL_ERR_SHAPE : RL_OK;
}

// Two matrices that start at one place are one matrix.
bool clash(const void *a, int64_t lda, int32_t ta, const void *b, int64_t ldb, int32_t tb) {
    return a && a == b && (lda != ldb || ta != tb);
}

rl_status check_norm(const rl_ln_config *c, int32_t rows) {
    if (!c) return RL_ERR_INVALID_ARG;
    if (!known(c->x_dtype) || !known(c->y_dtype) || !known(c->param_dtype)) return RL_ERR_DTYPE;
    if (rows < 0 || c->cols < 1) return RL_ERR_SHAPE;
    if (c->cols > rlk::kNormMaxCols) return RL_ERR_UNSUPPORTED;
    if (c->kind != RL_LN_LAYER && c->kind != RL_LN_RMS) return RL_ERR_INVALID_ARG;
    return RL_OK;
}

int64_t part_stride(int32_t cols) { return (cols + 63) / 64 * 64; }

#define RLK_TRY(expr)                         \
    do {                                      \
        const rl_status st_ = (expr);         \
        if (st_ != RL_OK) return st_;         \
    } while (0)

}  // namespace

extern "C" {

RL_LOSS_API int32_t rl_loss_layer_norm_max_cols(void) { return rlk::kNormMaxCols; }

RL_LOSS_API rl_status rl_loss_layer_norm(const rl_ln_config *config, int32_t rows, const void *x, int64_t ld_x,
                                         const void *residual, int64_t ld_residual, const void *weight,
                                         const void *bias, const uint8_t *mask, void *y, int64_t ld_y, void *summed,
                                         int64_t ld_summed, const rl_act8 *checkpoint, float *mean, float *rstd,
                                         uint32_t *device_status, void *stream) {
    RLK_TRY(check_norm(config, rows));
    const rl_ln_config &c = *config;
    if (!(c.eps > 0.f) || !std::isfinite(c.eps)) return RL_ERR_INVALID_ARG;
    if (rows == 0) return RL_OK;
    if (!x || !y) return RL_ERR_INVALID_ARG;
    RLK_TRY(check_mat(x, ld_x, c.x_dtype, c.cols));
    RLK_TRY(check_mat(y, ld_y, c.y_dtype, c.cols));
    if (residual) RLK_TRY(check_mat(residual, ld_residual, c.x_dtype, c.cols));
    if (summed) RLK_TRY(check_mat(summed, ld_summed, c.x_dtype, c.cols));
    if (checkpoint) RLK_TRY(check_act8(*checkpoint, c.cols));
    if (clash(x, ld_x, c.x_dtype, y, ld_y, c.y_dtype) || clash(residual, ld_residual, c.x_dtype, y, ld_y, c.y_dtype) ||
        clash(x, ld_x, c.x_dtype, summed, ld_summed, c.x_dtype) ||
        clash(residual, ld_residual, c.x_dtype, summed, ld_summed, c.x_dtype) || y == summed)
        return RL_ERR_INVALID_ARG;
    const uintptr_t ps = c.param_dtype == RL_F32 ? 4 : 2;
    if (!aligned(weight, ps) || !aligned(bias, ps) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(device_status, 4))
        return RL_ERR_ALIGNMENT;

    rlk::NormForwardParams p{};
    p.x = mat(x, ld_x, c.x_dtype);
    p.residual = mat(residual, ld_residual, c.x_dtype);
    p.y = mat(y, ld_y, c.y_dtype);
    p.h = mat(summed, ld_summed, c.x_dtype);
    if (checkpoint) p.ckpt = act8(*checkpoint);
    p.w = weight;
    p.b = bias;
    p.params_bf16 = c.param_dtype == RL_BF16;
    p.params_fast = aligned(weight, 16) && aligned(bias, 16);
    p.mask = mask;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.cols = c.cols;
    p.rms = c.kind == RL_LN_RMS;
    p.eps = c.eps;
    p.inv_cols = (float)(1.0 / c.cols);
    p.status = device_status;
    return rlk::launch_norm_forward(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

RL_LOSS_API size_t rl_loss_layer_norm_workspace_bytes(int32_t rows, int32_t cols) {
    if (rows < 1 || cols < 1 || cols > rlk::kNormMaxCols) return 256;
    return align_up((size_t)rlk::norm_backward_parts(rows, cols) * 2 * part_stride(cols) * sizeof(float), 256);
}

RL_LOSS_API rl_status rl_loss_layer_norm_backward(const rl_ln_config *config, int32_t rows, const void *dy,
                                                  int64_t ld_dy, const void *x, int64_t ld_x,
                                                  const rl_act8 *checkpoint, const void *weight, const void *bias,
                                                  const uint8_t *mask, const float *mean, const float *rstd,
                                                  const void *dsummed, int64_t ld_dsummed, void *dx, int64_t ld_dx,
                                                  float *dweight, float *dbias, int32_t accumulate, void *y,
                                                  int64_t ld_y, void *workspace, size_t workspace_bytes,
                                                  uint32_t *device_status, void *stream_ptr) {
    RLK_TRY(check_norm(config, rows));
    const rl_ln_config &c = *config;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_ptr);
    if (accumulate != 0 && accumulate != 1) return RL_ERR_INVALID_ARG;
    if (!aligned(dweight, 4) || !aligned(dbias, 4) || (dweight && dweight == dbias))
        return dweight == dbias ? RL_ERR_INVALID_ARG : RL_ERR_ALIGNMENT;
    if (rows == 0) {  // sums over no rows
        if (accumulate) return RL_OK;
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)c.cols * 4, stream);
        if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)c.cols * 4, stream);
        return e == cudaSuccess ? RL_OK : RL_ERR_CUDA;
    }
    if (!dy || !dx || !rstd || (c.kind == RL_LN_LAYER && !mean) || !x == !checkpoint) return RL_ERR_INVALID_ARG;
    RLK_TRY(check_mat(dy, ld_dy, c.y_dtype, c.cols));
    RLK_TRY(check_mat(dx, ld_dx, c.x_dtype, c.cols));
    if (x) RLK_TRY(check_mat(x, ld_x, c.x_dtype, c.cols));
    if (checkpoint) RLK_TRY(check_act8(*checkpoint, c.cols));
    if (dsummed) RLK_TRY(check_mat(dsummed, ld_dsummed, c.x_dtype, c.cols));
    if (y) RLK_TRY(check_mat(y, ld_y, c.y_dtype, c.cols));
    if (clash(dy, ld_dy, c.y_dtype, dx, ld_dx, c.x_dtype) || clash(x, ld_x, c.x_dtype, dx, ld_dx, c.x_dtype) ||
        clash(dsummed, ld_dsummed, c.x_dtype, dx, ld_dx, c.x_dtype) || clash(dy, ld_dy, c.y_dtype, y, ld_y, c.y_dtype) ||
        clash(x, ld_x, c.x_dtype, y, ld_y, c.y_dtype) || (dsummed && dsummed == y) || dx == y)
        return RL_ERR_INVALID_ARG;
    const uintptr_t ps = c.param_dtype == RL_F32 ? 4 : 2;
    if (!aligned(weight, ps) || !aligned(bias, ps) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(device_status, 4))
        return RL_ERR_ALIGNMENT;
    if (dweight || dbias) {
        if (!workspace) return RL_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return RL_ERR_ALIGNMENT;
        if (workspace_bytes < rl_loss_layer_norm_workspace_bytes(rows, c.cols)) return RL_ERR_CAPACITY;
    }

    rlk::NormBackwardParams p{};
    p.dy = mat(dy, ld_dy, c.y_dtype);
    p.x = mat(x, ld_x, c.x_dtype);
    p.dsummed = mat(dsummed, ld_dsummed, c.x_dtype);
    p.dx = mat(dx, ld_dx, c.x_dtype);
    p.y = mat(y, ld_y, c.y_dtype);
    if (checkpoint) p.ckpt = act8(*checkpoint);
    p.w = weight;
    p.b = bias;
    p.params_bf16 = c.param_dtype == RL_BF16;
    p.params_fast = aligned(weight, 16) && aligned(bias, 16);
    p.mask = mask;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.cols = c.cols;
    p.rms = c.kind == RL_LN_RMS;
    p.inv_cols = (float)(1.0 / c.cols);
    p.partials = static_cast<float *>(workspace);
    p.ld_part = part_stride(c.cols);
    p.want_dw = dweight != nullptr;
    p.want_db = dbias != nullptr;
    p.dw = dweight;
    p.db = dbias;
    p.accumulate = accumulate;
    p.status = device_status;
    return rlk::launch_norm_backward(p, stream) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

RL_LOSS_API rl_status rl_loss_act8_pack(int32_t x_dtype, int32_t rows, int32_t cols, const void *x, int64_t ld_x,
                                        const rl_act8 *out, void *stream) {
    if (!known(x_dtype)) return RL_ERR_DTYPE;
    if (!out) return RL_ERR_INVALID_ARG;
    if (rows < 0 || cols < 1 || cols > (1 << 30)) return RL_ERR_SHAPE;
    if (rows == 0) return RL_OK;
    if (!x) return RL_ERR_INVALID_ARG;
    RLK_TRY(check_mat(x, ld_x, x_dtype, cols));
    RLK_TRY(check_act8(*out, cols));
    rlk::Act8Params p{};
    p.x = mat(x, ld_x, x_dtype);
    p.a = act8(*out);
    p.rows = rows;
    p.cols = cols;
    return rlk::launch_act8_pack(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

RL_LOSS_API rl_status rl_loss_act8_unpack(int32_t x_dtype, int32_t rows, int32_t cols, const rl_act8 *in, void *x,
                                          int64_t ld_x, void *stream) {
    if (!known(x_dtype)) return RL_ERR_DTYPE;
    if (!in) return RL_ERR_INVALID_ARG;
    if (rows < 0 || cols < 1 || cols > (1 << 30)) return RL_ERR_SHAPE;
    if (rows == 0) return RL_OK;
    if (!x) return RL_ERR_INVALID_ARG;
    RLK_TRY(check_mat(x, ld_x, x_dtype, cols));
    RLK_TRY(check_act8(*in, cols));
    rlk::Act8Params p{};
    p.x = mat(x, ld_x, x_dtype);
    p.a = act8(*in);
    p.rows = rows;
    p.cols = cols;
    return rlk::launch_act8_unpack(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

}  // extern "C"
