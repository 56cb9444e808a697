// Root-mean-square norm with the residual's addition and 8-bit rows, and its gradients.
//
//   h = bf16(x + residual), rstd = 1 / sqrt(mean h^2 + eps), y = h rstd w; y in bf16 and in 8 bits with
//   a scale for each row or for each block of 1 x 128
//   dx = rstd (g - xh mean(g xh)) + dh,  dw = sum over rows of dy xh,  g = dy w, xh = h rstd
//
// Bound: HBM.
#include "common.hpp"

namespace fp8q {

constexpr int NB = 128;  // elements of a block with one factor

struct NormArgs {
    const uint16_t* x;
    int64_t cols, ld_x;
    const uint16_t* residual;
    int64_t ld_res;
    const void* w;
    uint16_t* h;
    int64_t ld_h;
    uint16_t* y;
    int64_t ld_y;
    uint8_t* q;
    int64_t ld_q;
    float* scales;
    int64_t ld_s;
    float* rstd;
    float eps;
    bool w32;      // the weight is fp32
    int scaling;   // fp8q_norm_scaling_t
};

__device__ __forceinline__ float bf16_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t bf16_rn(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);  // NaN stays NaN
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}
__device__ __forceinline__ float weight_at(const void* w, bool w32, int64_t c) {
    return w32 ? static_cast<const float*>(w)[c] : bf16_f(static_cast<const uint16_t*>(w)[c]);
}

// Sum and maximum over a block of 4 waves, the same in all threads.  red: 4 floats; a barrier stands
// before its next use.
__device__ __forceinline__ float block_sum4(float v, float* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (red[0] + red[1]) + (red[2] + red[3]);
    __syncthreads();
    return v;
}
__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

constexpr float kShrink = 8.271806125530277e-25f;  // 2^-80

__device__ __forceinline__ float rstd_of(float sum, float cols, float eps) { return 1.0f / sqrtf(sum / cols + eps); }
// Where the sum of squares has overflowed: from the squares' sum of h * 2^-80; eps is far below them.
__device__ __forceinline__ float rstd_of_shrunk(float sum, float cols) { return kShrink / sqrtf(sum / cols); }

// Any size and alignment: a block of 4 waves per row, a wave takes blocks of 128 columns in turn, a lane
// two of each; the row is read again (from cache) for the maximum and for the bytes.  A thread reads
// only what it wrote of h, so h may be x or the residual.
template <int FMT>
__global__ __launch_bounds__(256) void norm_generic_kernel(const NormArgs p) {
    __shared__ float red[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    const uint16_t* x = p.x + row * p.ld_x;
    const uint16_t* res = p.residual ? p.residual + row * p.ld_res : nullptr;
    uint16_t* h = p.h ? p.h + row * p.ld_h : nullptr;
    float sum = 0.0f;
    for (int64_t b = wave * NB; b < p.cols; b += 4 * NB)
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int64_t c = b + 2 * lane + i;
            if (c < p.cols) {
                float v = bf16_f(x[c]);
                if (res) {
                    const uint16_t s = bf16_rn(v + bf16_f(res[c]));
                    h[c] = s;
                    v = bf16_f(s);
                }
                sum += v * v;
            }
        }
    sum = block_sum4(sum, red);
    const uint16_t* src = res ? h : x;
    float rstd;
    if (sum == INFINITY) {
        float small = 0.0f;
        for (int64_t b = wave * NB; b < p.cols; b += 4 * NB)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int64_t c = b + 2 * lane + i;
                const float v = c < p.cols ? bf16_f(src[c]) * kShrink : 0.0f;
                small += v * v;
            }
        rstd = rstd_of_shrunk(block_sum4(small, red), (float)p.cols);
    } else {
        rstd = rstd_of(sum, (float)p.cols, p.eps);
    }
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    float s = 0.0f;
    if (p.scaling == FP8Q_NORM_ROW) {
        float m = 0.0f;
        for (int64_t b = wave * NB; b < p.cols; b += 4 * NB)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int64_t c = b + 2 * lane + i;
                if (c < p.cols) m = fmaxf(m, fabsf(bf16_f(src[c]) * rstd * weight_at(p.w, p.w32, c)));
            }
        m = wave_max_f(m);
        if (lane == 0) red[wave] = m;
        __syncthreads();
        s = scale_from_amax<FMT>(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        if (threadIdx.x == 0) p.scales[row] = s;
    }
    for (int64_t b = wave * NB; b < p.cols; b += 4 * NB) {
        float y[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int64_t c = b + 2 * lane + i;
            y[i] = c < p.cols ? bf16_f(src[c]) * rstd * weight_at(p.w, p.w32, c) : 0.0f;
            if (p.y && c < p.cols) p.y[row * p.ld_y + c] = bf16_rn(y[i]);
        }
        if (p.scaling == FP8Q_NORM_NONE) continue;
        if (p.scaling == FP8Q_NORM_BLOCK) {
            s = scale_from_amax<FMT>(wave_max_f(fmaxf(fabsf(y[0]), fabsf(y[1]))));
            if (lane == 0) p.scales[b / NB * p.ld_s + row] = 1.0f / s;
        }
        const float sm = s * Fmt<FMT>::mult;
        const uint32_t e = enc4<FMT>(y[0] * sm, y[1] * sm, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int64_t c = b + 2 * lane + i;
            if (c < p.cols) p.q[row * p.ld_q + c] = (uint8_t)(e >> (8 * i));
        }
    }
}

// ------------------------------------------------------------------------------------ gradients

struct NormBackArgs {
    const void *dy, *dh;
    int64_t ld_dy, ld_dh;
    const uint16_t* h;
    int64_t rows, cols, ld_h;
    const float* rstd;
    const void* w;
    void* dx;
    int64_t ld_dx;
    float* part;   // [blocks][cols] sums of dy xh
    bool w32;
};

template <bool G32>
__device__ __forceinline__ float grad_at(const void* g, int64_t i) {
    return G32 ? static_cast<const float*>(g)[i] : bf16_f(static_cast<const uint16_t*>(g)[i]);
}

// Any size and alignment: blocks take rows in turn, a thread the same columns of each; its columns' sums
// for dw are kept in the block's own piece of the workspace.
template <bool G32>
__global__ __launch_bounds__(256) void norm_back_generic_kernel(const NormBackArgs p) {
    __shared__ float red[4];
    float* part = p.part + (int64_t)blockIdx.x * p.cols;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const uint16_t* h = p.h + row * p.ld_h;
        const float rstd = p.rstd[row];
        float sum = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += 256)
            sum += grad_at<G32>(p.dy, row * p.ld_dy + c) * weight_at(p.w, p.w32, c) * (bf16_f(h[c]) * rstd);
        const float mean = block_sum4(sum, red) / (float)p.cols;
        for (int64_t c = threadIdx.x; c < p.cols; c += 256) {
            const float xh = bf16_f(h[c]) * rstd, dy = grad_at<G32>(p.dy, row * p.ld_dy + c);
            float dx = rstd * (dy * weight_at(p.w, p.w32, c) - xh * mean);
            if (p.dh) dx += grad_at<G32>(p.dh, row * p.ld_dh + c);
            if (G32) static_cast<float*>(p.dx)[row * p.ld_dx + c] = dx;
            else static_cast<uint16_t*>(p.dx)[row * p.ld_dx + c] = bf16_rn(dx);
            part[c] = first ? dy * xh : part[c] + dy * xh;
        }
        first = false;
    }
}

// dw from the blocks' sums: a block takes 32 columns, 8 threads a column's parts in turn.
__global__ __launch_bounds__(256) void norm_back_join_kernel(const float* part, int parts, int64_t cols, float* dw) {
    __shared__ float red[8][32];
    const int i = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + i;
    float s = 0.0f;
    if (c < cols)
        for (int b = k; b < parts; b += 8) s += part[(int64_t)b * cols + c];
    red[k][i] = s;
    __syncthreads();
    if (k == 0 && c < cols) {
#pragma unroll
        for (int j = 1; j < 8; j++) s += red[j][i];
        dw[c] = s;
    }
}

static inline int64_t norm_back_parts(int64_t rows) { return rows < 512 ? rows : 512; }

static inline bool dtype_ok(int d) { return d == FP8Q_OUT_BF16 || d == FP8Q_OUT_FP32; }

}  // namespace fp8q

extern "C" fp8q_status_t fp8_rms_norm(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                      const uint16_t* residual, int64_t ld_res, const void* weight,
                                      fp8q_out_t weight_dtype, float eps, uint16_t* h, int64_t ld_h, uint16_t* y,
                                      int64_t ld_y, fp8q_norm_scaling_t scaling, fp8q_format_t fmt, uint8_t* q,
                                      int64_t ld_q, float* scales, int64_t ld_s, float* rstd, hipStream_t stream) {
    using namespace fp8q;
    const bool quant = scaling != FP8Q_NORM_NONE;
    if (rows < 0 || cols < 0 || ld_x < cols || (residual && (ld_res < cols || ld_h < cols)) || (y && ld_y < cols) ||
        (quant && ld_q < cols) || !fp8q_fmt_ok(fmt) || !dtype_ok(weight_dtype) || !(eps > 0.0f))
        return FP8Q_ERR_INVALID_ARG;
    if (scaling != FP8Q_NORM_NONE && scaling != FP8Q_NORM_ROW && scaling != FP8Q_NORM_BLOCK) return FP8Q_ERR_INVALID_ARG;
    if (scaling == FP8Q_NORM_BLOCK && (fmt != FP8Q_E4M3FN || ld_s < rows)) return FP8Q_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!x || !weight || (residual != nullptr) != (h != nullptr) || (quant && (!q || !scales)) || (!quant && (q || scales || !y)))
        return FP8Q_ERR_INVALID_ARG;
    // in place: every element where it was
    if (h && ((h == x && ld_h != ld_x) || (h == residual && ld_h != ld_res))) return FP8Q_ERR_INVALID_ARG;
    if (rows > 0x7FFFFFFFLL) return FP8Q_ERR_UNSUPPORTED;
    NormArgs p{};
    p.x = x; p.cols = cols; p.ld_x = ld_x; p.residual = residual; p.ld_res = ld_res; p.w = weight; p.h = h; p.ld_h = ld_h;
    p.y = y; p.ld_y = ld_y; p.q = q; p.ld_q = ld_q; p.scales = scales; p.ld_s = ld_s; p.rstd = rstd; p.eps = eps;
    p.w32 = weight_dtype == FP8Q_OUT_FP32; p.scaling = scaling;
    if (fmt == FP8Q_E4M3FN) norm_generic_kernel<FP8Q_E4M3FN><<<dim3((unsigned)rows), dim3(256), 0, stream>>>(p);
    else norm_generic_kernel<FP8Q_E4M3FNUZ><<<dim3((unsigned)rows), dim3(256), 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

extern "C" size_t fp8_rms_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0) return 256;
    return (size_t)fp8q::norm_back_parts(rows) * (size_t)cols * 4;
}

extern "C" fp8q_status_t fp8_rms_norm_backward(const void* dy, int64_t ld_dy, const void* dh, int64_t ld_dh,
                                               fp8q_out_t grad_dtype, const uint16_t* h, int64_t rows, int64_t cols,
                                               int64_t ld_h, const float* rstd, const void* weight,
                                               fp8q_out_t weight_dtype, void* dx, int64_t ld_dx, float* dweight,
                                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace fp8q;
    if (rows < 0 || cols < 0 || ld_dy < cols || (dh && ld_dh < cols) || ld_h < cols || ld_dx < cols || !dtype_ok(grad_dtype) ||
        !dtype_ok(weight_dtype))
        return FP8Q_ERR_INVALID_ARG;
    if (cols == 0) return FP8Q_OK;
    if (!dweight || (rows > 0 && (!dy || !h || !rstd || !weight || !dx))) return FP8Q_ERR_INVALID_ARG;
    if (rows > 0 && ((dx == dy && ld_dx != ld_dy) || (dx == dh && ld_dx != ld_dh))) return FP8Q_ERR_INVALID_ARG;
    if (rows > 0x7FFFFFFFLL || cols > 0x7FFFFFFFLL) return FP8Q_ERR_UNSUPPORTED;
    if (rows > 0 && (!workspace || workspace_bytes < fp8_rms_norm_backward_workspace_size(rows, cols))) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 16)) return FP8Q_ERR_INVALID_ARG;
    NormBackArgs p{};
    p.dy = dy; p.ld_dy = ld_dy; p.dh = dh; p.ld_dh = ld_dh; p.h = h; p.rows = rows; p.cols = cols; p.ld_h = ld_h;
    p.rstd = rstd; p.w = weight; p.dx = dx; p.ld_dx = ld_dx; p.part = static_cast<float*>(workspace);
    p.w32 = weight_dtype == FP8Q_OUT_FP32;
    const int64_t parts = norm_back_parts(rows);
    if (rows > 0) {
        if (grad_dtype == FP8Q_OUT_FP32) norm_back_generic_kernel<true><<<dim3((unsigned)parts), dim3(256), 0, stream>>>(p);
        else norm_back_generic_kernel<false><<<dim3((unsigned)parts), dim3(256), 0, stream>>>(p);
        FP8Q_CHECK_LAUNCH();
    }
    norm_back_join_kernel<<<dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, stream>>>(p.part, (int)parts, cols, dweight);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}
