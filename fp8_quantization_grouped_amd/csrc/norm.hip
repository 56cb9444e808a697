// Root-mean-square norm with the residual's addition and 8-bit rows, and its gradients.
//
//   h = bf16(x + residual), rstd = 1 / sqrt(mean h^2 + eps), y = h rstd w; y in bf16 and in 8 bits with
//   a scale for each row or for each block of 1 x 128
//   dx = rstd (g - xh mean(g xh)) + dh,  dw = sum over rows of dy xh,  g = dy w, xh = h rstd
//
// Bound: HBM.  Each byte is moved once, but for partial lines of the block factors: the row stays in registers
// between its sum, its maximum and its bytes (a block that reads it again: 508 us where this takes 185).
// 16384 x 7168 with residual, bf16 and block factors 185 us (5.7 TB/s), the backward with dh 152 us (6.2 TB/s).
// Small calls are the host's: the kernel takes 2.7 us for one row of 7168, residual and bf16.
#include "common.hpp"
#include "plan.hpp"

namespace fp8q {

constexpr int NB = 128;  // elements of a block with one factor

struct NormArgs {
    const uint16_t* x;
    int64_t rows, cols, ld_x;
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

// Eight consecutive elements from 8 c on of a row of 8 or more, zeros past its end.  ACC & WIDE: rows are whole
// chunks that start on 16 bytes; else a wide access need not be aligned, and a chunk that the row's end cuts
// is read as the row's last eight, which stay inside it in one access, and moved down: reading it by elements
// costs the loop 7 registers for every such load.  20000 x 5457 in the backward: 322 us where it was moved at
// the load, 271 us where it is used.
constexpr int WIDE = 1, PAST = 2;  // PAST: past the caches
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// load_chunk only reads; settle moves a cut chunk down, where it is used: the loads ahead of it stay in flight.
template <int ACC>
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, int c, int cols) {
    if (ACC & WIDE) return ACC & PAST ? ld_nt16(row + 8 * c) : *reinterpret_cast<const uint4*>(row + 8 * c);
    const int over = 8 * c + 8 - cols;
    const u32x4_any* p = reinterpret_cast<const u32x4_any*>(row + 8 * c - (over > 0 ? over : 0));
    const u32x4_any v = ACC & PAST ? __builtin_nontemporal_load(p) : *p;
    return make_uint4(v.x, v.y, v.z, v.w);
}
template <int ACC>
__device__ __forceinline__ uint4 settle(uint4 v, int c, int cols) {
    const int over = 8 * c + 8 - cols;
    if ((ACC & WIDE) || over <= 0 || over >= 8) return v;
    uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
    const int k = 16 * over;  // bits, under 128
    lo = k >= 64 ? hi >> (k - 64) : lo >> k | hi << (64 - k);
    hi = k >= 64 ? 0 : hi >> k;
    return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
}
template <int ACC>
__device__ __forceinline__ void store_chunk(uint16_t* row, int c, int cols, uint4 v) {
    if ((ACC & WIDE) && (ACC & PAST)) {
        st_nt16(row + 8 * c, v);
    } else if (ACC & WIDE) {
        *reinterpret_cast<uint4*>(row + 8 * c) = v;
    } else if (8 * c + 8 <= cols) {
        u32x4_any* p = reinterpret_cast<u32x4_any*>(row + 8 * c);
        if (ACC & PAST) __builtin_nontemporal_store(u32x4_any{v.x, v.y, v.z, v.w}, p);
        else *p = u32x4_any{v.x, v.y, v.z, v.w};
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 7; i++)
            if (8 * c + i < cols) row[8 * c + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}
template <int ACC>
__device__ __forceinline__ void store_bytes(uint8_t* row, int c, int cols, uint32_t a, uint32_t b) {
    if ((ACC & WIDE) && (ACC & PAST)) {
        st_nt8(row + 8 * c, a, b);
    } else if (ACC & WIDE) {
        *reinterpret_cast<uint2*>(row + 8 * c) = make_uint2(a, b);
    } else if (8 * c + 8 <= cols) {
        u32x2_any* p = reinterpret_cast<u32x2_any*>(row + 8 * c);
        if (ACC & PAST) __builtin_nontemporal_store(u32x2_any{a, b}, p);
        else *p = u32x2_any{a, b};
    } else {
#pragma unroll
        for (int i = 0; i < 7; i++)
            if (8 * c + i < cols) row[8 * c + i] = (uint8_t)((i < 4 ? a : b) >> (8 * (i & 3)));
    }
}
__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {  // to the nearest, ties to even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
template <int ACC>
__device__ __forceinline__ void load_floats(const float* row, int c, int cols, float (&f)[8]) {
    const int over = ACC & WIDE ? 0 : 8 * c + 8 - cols;
    const f32x4_any* p = reinterpret_cast<const f32x4_any*>(row + 8 * c - (over > 0 ? over : 0));
    const f32x4_any a = ACC & PAST ? __builtin_nontemporal_load(p) : p[0], b = ACC & PAST ? __builtin_nontemporal_load(p + 1) : p[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <int ACC>
__device__ __forceinline__ void settle(float (&f)[8], int c, int cols) {
    const int over = 8 * c + 8 - cols;
    if ((ACC & WIDE) || over <= 0 || over >= 8) return;
#pragma unroll
    for (int k = 4; k > 0; k >>= 1)
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = over & k ? (i + k < 8 ? f[i + k] : 0.0f) : f[i];
}
template <int ACC>
__device__ __forceinline__ void store_floats(float* row, int c, int cols, const float (&f)[8]) {
    if ((ACC & WIDE) || 8 * c + 8 <= cols) {
        f32x4_any* p = reinterpret_cast<f32x4_any*>(row + 8 * c);
        const f32x4_any a = {f[0], f[1], f[2], f[3]}, b = {f[4], f[5], f[6], f[7]};
        if (ACC & PAST) {
            __builtin_nontemporal_store(a, p);
            __builtin_nontemporal_store(b, p + 1);
        } else {
            p[0] = a;
            p[1] = b;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 7; i++)
            if (8 * c + i < cols) row[8 * c + i] = f[i];
    }
}
template <int ACC>
__device__ __forceinline__ void load_weight(const void* w, bool w32, int c, int cols, float (&f)[8]) {
    if (w32) {
        load_floats<ACC & WIDE>(static_cast<const float*>(w), c, cols, f);
        settle<ACC>(f, c, cols);
    } else {
        unpack(settle<ACC>(load_chunk<ACC & WIDE>(static_cast<const uint16_t*>(w), c, cols), c, cols), f);
    }
}

// Sums (SUM) and maxima over a wave, the same in all lanes: by DPP 1 and 2 lanes away, then mirrored in 8 and
// in 16, then the four rows of 16.
template <bool SUM>
__device__ __forceinline__ float join(float a, float b) { return SUM ? a + b : fmaxf(a, b); }
template <bool SUM, int CTRL>
__device__ __forceinline__ float join_dpp(float v) {
    return join<SUM>(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false)));
}
template <bool SUM>
__device__ __forceinline__ float over16(float v) {
    return join_dpp<SUM, 0x140>(join_dpp<SUM, 0x141>(join_dpp<SUM, 0x4E>(join_dpp<SUM, 0xB1>(v))));
}
template <bool SUM>
__device__ __forceinline__ float over_wave(float v) {
    v = over16<SUM>(v);
    const auto lane = [&](int i) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), i)); };
    return join<SUM>(join<SUM>(lane(0), lane(16)), join<SUM>(lane(32), lane(48)));
}
// Over the WPR waves of a row; red: a float for each of the block's waves.
template <int WPR, bool SUM>
__device__ __forceinline__ float across(float v, float* red) {
    v = over_wave<SUM>(v);
    if (WPR == 1) return v;
    const int wave = threadIdx.x >> 6, w0 = wave / WPR * WPR;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = red[w0];
#pragma unroll
    for (int w = 1; w < WPR; w++) v = join<SUM>(v, red[w0 + w]);
    return v;
}

// Rows held in registers: WPR waves a row, NV chunks of 8 elements a lane.  Blocks take the rows in turn, so
// neighbouring rows are at work at once all over the chip.  (A run of rows for each XCD, whose factors then
// meet in one L2: 16384 x 7168 with residual, bf16 and block factors 198 us against 185, 32768 x 2048 124
// against 105; block rows alone 68 against 69.)
template <int SC, int FMT, int WPR, int NV, int ACC>
__global__ __launch_bounds__(64 * norm_waves(WPR)) void norm_kernel(const NormArgs p) {
    constexpr int WAVES = norm_waves(WPR), RPB = WAVES / WPR, TPR = 64 * WPR;
    __shared__ float red[3][WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), t = threadIdx.x % TPR;
    const int64_t r = (int64_t)blockIdx.x * RPB + wave / WPR;
    const bool row_ok = r < p.rows;
    const int64_t row = row_ok ? r : p.rows - 1;
    const int cols = row_ok ? (int)p.cols : 0;  // no columns of a row past the last
    const uint16_t* x = p.x + row * p.ld_x;
    uint4 h[NV], res[NV];
#pragma unroll
    for (int j = 0; j < NV; j++) {
        const int c = t + j * TPR;
        h[j] = res[j] = make_uint4(0, 0, 0, 0);
        if (8 * c < cols) h[j] = load_chunk<ACC>(x, c, cols);
    }
    if (p.residual) {
        const uint16_t* from = p.residual + row * p.ld_res;
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (8 * (t + j * TPR) < cols) res[j] = load_chunk<ACC>(from, t + j * TPR, cols);
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; j++) {
        const int c = t + j * TPR;
        float f[8];
        h[j] = settle<ACC>(h[j], c, cols);
        unpack(h[j], f);
        if (p.residual) {
            float g[8];
            unpack(settle<ACC>(res[j], c, cols), g);
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] += g[i];
            h[j] = pack(f);
            unpack(h[j], f);
            if (8 * c < cols) store_chunk<ACC>(p.h + row * p.ld_h, c, cols, h[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) sum += f[i] * f[i];
    }
    sum = across<WPR, true>(sum, red[0]);
    float rstd;
    if (sum == INFINITY) {  // (the same in the whole row)
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            float f[8];
            unpack(h[j], f);
#pragma unroll
            for (int i = 0; i < 8; i++) sum += (f[i] * kShrink) * (f[i] * kShrink);
        }
        rstd = rstd_of_shrunk(across<WPR, true>(sum, red[1]), (float)p.cols);
    } else {
        rstd = rstd_of(sum, (float)p.cols, p.eps);
        if (WPR > 1) __syncthreads();  // as many barriers as in the other case
    }
    if (t == 0 && row_ok && p.rstd) p.rstd[row] = rstd;
    float y[NV][8], amax = 0.0f, block_max[NV];
#pragma unroll
    for (int j = 0; j < NV; j++) {
        const int c = t + j * TPR;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = 0.0f;
        if (8 * c < cols) load_weight<ACC>(p.w, p.w32, c, cols, w);
        unpack(h[j], y[j]);
#pragma unroll
        for (int i = 0; i < 8; i++) y[j][i] = y[j][i] * rstd * w[i];
        if (p.y && 8 * c < cols) store_chunk<ACC>(p.y + row * p.ld_y, c, cols, pack(y[j]));
        if (SC == FP8Q_NORM_NONE) continue;
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(y[j][i]));
        if (SC == FP8Q_NORM_ROW) amax = fmaxf(amax, m);
        else block_max[j] = over16<false>(m);  // 16 lanes have a block
    }
    if (SC == FP8Q_NORM_BLOCK) {
        // the 16 lanes have NV blocks: 16 / NV lanes form each one's factors
        constexpr int EACH = 16 / NV;
        const int which = (t & 15) / EACH;
        float m = block_max[0];
#pragma unroll
        for (int j = 1; j < NV; j++) m = which == j ? block_max[j] : m;
        const float mine = scale_from_amax<FMT>(m);
        const int first = t / 16 + which * (TPR / 16);  // the block
        if (t % EACH == 0 && first * NB < cols) p.scales[first * p.ld_s + row] = 1.0f / mine;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int c = t + j * TPR;
            const float sm = (NV == 1 ? mine : __shfl(mine, (t & 48) + j * EACH, 64)) * Fmt<FMT>::mult;
            if (8 * c < cols)
                store_bytes<ACC>(p.q + row * p.ld_q, c, cols, enc4<FMT>(y[j][0] * sm, y[j][1] * sm, y[j][2] * sm, y[j][3] * sm),
                                 enc4<FMT>(y[j][4] * sm, y[j][5] * sm, y[j][6] * sm, y[j][7] * sm));
        }
    }
    if (SC != FP8Q_NORM_ROW) return;
    const float s = scale_from_amax<FMT>(across<WPR, false>(amax, red[2])), sm = s * Fmt<FMT>::mult;
    if (t == 0 && row_ok) p.scales[row] = s;
#pragma unroll
    for (int j = 0; j < NV; j++) {
        const int c = t + j * TPR;
        if (8 * c < cols)
            store_bytes<ACC>(p.q + row * p.ld_q, c, cols, enc4<FMT>(y[j][0] * sm, y[j][1] * sm, y[j][2] * sm, y[j][3] * sm),
                              enc4<FMT>(y[j][4] * sm, y[j][5] * sm, y[j][6] * sm, y[j][7] * sm));
    }
}

template <int SC, int FMT, int WPR, int NV>
static void launch_norm(const NormArgs& p, int acc, hipStream_t stream) {
    constexpr int WAVES = norm_waves(WPR), RPB = WAVES / WPR;
    const dim3 grid((unsigned)((p.rows + RPB - 1) / RPB)), block(64 * WAVES);
    if (acc == (WIDE | PAST)) norm_kernel<SC, FMT, WPR, NV, WIDE | PAST><<<grid, block, 0, stream>>>(p);
    else if (acc == WIDE) norm_kernel<SC, FMT, WPR, NV, WIDE><<<grid, block, 0, stream>>>(p);
    else if (acc == PAST) norm_kernel<SC, FMT, WPR, NV, PAST><<<grid, block, 0, stream>>>(p);
    else norm_kernel<SC, FMT, WPR, NV, 0><<<grid, block, 0, stream>>>(p);
}

// More than the last-level cache holds of what a call reads and writes: none of it will be found there.
// Backward 16384 x 7168 161 us past the caches, 182 through them; with fp32 gradients 288 and 314.
static inline bool past_caches(int64_t rows, int64_t cols, int bytes) { return (double)rows * cols * bytes > 2.0 * kStreamBytes; }

// Rows that start on whole vectors of 8 elements; none where there is no matrix.
static inline bool rows_wide(const void* p, int64_t ld, uintptr_t align) { return !p || (ld % 8 == 0 && fp8q_aligned(p, align)); }

template <int FMT>
__global__ void norm_generic_kernel(const NormArgs p);

template <int SC, int FMT>
static void start_norm(const NormArgs& p, hipStream_t stream) {
    const int each = (p.residual ? 6 : 2) + (p.y ? 2 : 0) + (p.q ? 1 : 0);  // bytes of an element
    const bool wide = p.cols % 8 == 0 && rows_wide(p.x, p.ld_x, 16) && rows_wide(p.residual, p.ld_res, 16) &&
                      rows_wide(p.h, p.ld_h, 16) && rows_wide(p.y, p.ld_y, 16) && rows_wide(p.q, p.ld_q, 8) &&
                      fp8q_aligned(p.w, 16);
    const int acc = (wide ? WIDE : 0) | (past_caches(p.rows, p.cols, each) ? PAST : 0);
    const NormShape n = pick_norm(p.rows, p.cols);
    switch (n.chunks ? 10 * n.waves + n.chunks : 0) {
        case 11: launch_norm<SC, FMT, 1, 1>(p, acc, stream); break;
        case 12: launch_norm<SC, FMT, 1, 2>(p, acc, stream); break;
        case 14: launch_norm<SC, FMT, 1, 4>(p, acc, stream); break;
        case 24: launch_norm<SC, FMT, 2, 4>(p, acc, stream); break;
        case 44: launch_norm<SC, FMT, 4, 4>(p, acc, stream); break;
        case 84: launch_norm<SC, FMT, 8, 4>(p, acc, stream); break;
        case 164: launch_norm<SC, FMT, 16, 4>(p, acc, stream); break;
        case 161: launch_norm<SC, FMT, 16, 1>(p, acc, stream); break;
        default: norm_generic_kernel<FMT><<<dim3((unsigned)p.rows), dim3(256), 0, stream>>>(p);
    }
}

// Rows longer than registers hold, or shorter than a vector: a block of 4 waves per row, a wave takes blocks
// of 128 columns in turn, a lane two of each; the row is read again (from cache) for the maximum and for the
// bytes.  A thread reads only what it wrote of h, so h may be x or the residual.  3000 x 40000 with residual,
// bf16 and blocks takes 644 us, 1.7 TB/s.
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
    int waves;     // of a row
    bool w32;
};

template <bool G32>
__device__ __forceinline__ float grad_at(const void* g, int64_t i) {
    return G32 ? static_cast<const float*>(g)[i] : bf16_f(static_cast<const uint16_t*>(g)[i]);
}

template <bool G32, int ACC>
struct Eight {  // eight gradients or weights
    uint4 v[G32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* g, int64_t at, int c, int cols) {
        if (G32) {
            float f[8];
            load_floats<ACC>(static_cast<const float*>(g) + at, c, cols, f);
            v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            v[G32 ? 1 : 0] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
        } else {
            v[0] = load_chunk<ACC>(static_cast<const uint16_t*>(g) + at, c, cols);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < (G32 ? 2 : 1); i++) v[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        if (G32) {
            const uint4 a = v[0], b = v[G32 ? 1 : 0];
            f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
            f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
        } else {
            unpack(v[0], f);
        }
    }
    __device__ __forceinline__ void settle_all(int c, int cols) {
        if (G32) {
            float f[8];
            get(f);
            settle<ACC>(f, c, cols);
            v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            v[G32 ? 1 : 0] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
        } else {
            v[0] = settle<ACC>(v[0], c, cols);
        }
    }
};

// What a lane has of a row.
template <bool G32, int NV, int ACC>
struct BackRow {
    uint4 h[NV];
    Eight<G32, ACC> dy[NV];
    float rstd;
    __device__ __forceinline__ void load(const NormBackArgs& p, int64_t row, int t, int tpr) {
        const bool ok = row < p.rows;
        const int cols = ok ? (int)p.cols : 0;
        rstd = ok ? p.rstd[row] : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int c = t + j * tpr;
            h[j] = make_uint4(0, 0, 0, 0);
            dy[j].clear();
            if (8 * c < cols) {
                h[j] = load_chunk<ACC>(p.h + row * p.ld_h, c, cols);
                dy[j].load(p.dy, row * p.ld_dy, c, cols);
            }
        }
    }
};

// Rows held in registers: p.waves waves a row, NV chunks of 8 columns a lane, the same ones of each of its
// rows, whose sums for dw it keeps; a row's loads go out while the one before it is worked on.  The rows of a
// block's waves are added at the end.  Two chunks do not fit the 128 registers of 16 waves: 4 to 8 of them spill
// with bf16 gradients (8192 x 16384 with dh 182 to 185 us, 5.8 TB/s, where one chunk at 8192 wide reaches 5.5 to
// 5.9), 19 to 32 with fp32 ones (412 to 424 us, 4.4 to 4.6 TB/s against 5.1 to 5.6).
template <bool G32, bool W32, int NV, int ACC>
__global__ __launch_bounds__(1024) void norm_back_kernel(const NormBackArgs p) {
    __shared__ float red[2][16];
    extern __shared__ float sums[];  // [rows of a block less one][8][threads of a row]
    const int waves = p.waves, tpr = 64 * waves, rpb = blockDim.x / tpr;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), mine = wave / waves, t = threadIdx.x - mine * tpr;
    float acc[NV][8];
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
        for (int i = 0; i < 8; i++) acc[j][i] = 0.0f;
    Eight<W32, ACC & WIDE> weight[NV];
#pragma unroll
    for (int j = 0; j < NV; j++) {
        const int c = t + j * tpr;
        weight[j].clear();
        if (8 * c < p.cols) weight[j].load(p.w, 0, c, (int)p.cols);
        weight[j].settle_all(c, (int)p.cols);
    }
    BackRow<G32, NV, ACC> cur, next;
    int64_t r0 = (int64_t)blockIdx.x * rpb;
    cur.load(p, r0 + mine, t, tpr);
    const float inv_cols = 1.0f / (float)p.cols;
    for (int turn = 0; r0 < p.rows; turn ^= 1) {  // the rows of a block stay together, for its barriers
        const int64_t row = r0 + mine;
        const int cols = row < p.rows ? (int)p.cols : 0;
        Eight<G32, ACC> dh[NV];  // used after the row's sum, so not a row ahead
#pragma unroll
        for (int j = 0; j < NV; j++) {
            dh[j].clear();
            if (p.dh && 8 * (t + j * tpr) < cols) dh[j].load(p.dh, row * p.ld_dh, t + j * tpr, cols);
        }
        r0 += (int64_t)gridDim.x * rpb;
        next.load(p, r0 + mine, t, tpr);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int c = t + j * tpr;
            float x[8], g[8], w[8];
            weight[j].get(w);
            cur.h[j] = settle<ACC>(cur.h[j], c, (int)p.cols);
            cur.dy[j].settle_all(c, (int)p.cols);
            unpack(cur.h[j], x);
            cur.dy[j].get(g);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float xh = x[i] * cur.rstd;
                sum += g[i] * w[i] * xh;
                acc[j][i] += g[i] * xh;
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
        if (waves > 1) {
            if ((threadIdx.x & 63) == 0) red[turn][wave] = sum;
            __syncthreads();
            sum = 0.0f;
            for (int i = 0; i < waves; i++) sum += red[turn][mine * waves + i];
        }
        const float mean = sum * inv_cols;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int c = t + j * tpr;
            if (8 * c >= cols) continue;
            float x[8], g[8], e[8], w[8];
            weight[j].get(w);
            unpack(cur.h[j], x);
            cur.dy[j].get(g);
            dh[j].settle_all(c, cols);
            dh[j].get(e);
#pragma unroll
            for (int i = 0; i < 8; i++) e[i] += cur.rstd * (g[i] * w[i] - (x[i] * cur.rstd) * mean);
            if (G32) store_floats<ACC>(static_cast<float*>(p.dx) + row * p.ld_dx, c, cols, e);
            else store_chunk<ACC>(static_cast<uint16_t*>(p.dx) + row * p.ld_dx, c, cols, pack(e));
        }
        cur = next;
    }
    float* part = p.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
    for (int j = 0; j < NV; j++) {
        const int c = t + j * tpr;
        if (rpb > 1) {
            __syncthreads();
            if (mine > 0)
#pragma unroll
                for (int i = 0; i < 8; i++) sums[((mine - 1) * 8 + i) * tpr + t] = acc[j][i];
            __syncthreads();
            if (mine == 0)
                for (int k = 0; k < rpb - 1; k++)
#pragma unroll
                    for (int i = 0; i < 8; i++) acc[j][i] += sums[(k * 8 + i) * tpr + t];
        }
        if (mine == 0 && 8 * c < p.cols) store_floats<ACC & WIDE>(part, c, (int)p.cols, acc[j]);
    }
}

// Rows longer than registers hold, or shorter than a vector: blocks take rows in turn, a thread the same
// columns of each; its columns' sums for dw are kept in the block's own piece of the workspace.  Element by
// element: 4096 x 20000 takes 1.9 to 2.3 ms, 0.3 to 0.6 TB/s.
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

// dw from the blocks' sums: a block takes 32 columns, 32 threads a column's parts in turn.
__global__ __launch_bounds__(1024) void norm_back_join_kernel(const float* part, int parts, int64_t cols, float* dw) {
    static_assert(NORM_JOIN == 32, "a column for each of 32 threads");
    __shared__ float red[32][33];
    const int i = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * NORM_JOIN + i;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int b = k; b < parts; b += 32) s += part[(int64_t)b * cols + c];
    }
    red[k][i] = s;
    __syncthreads();
    if (k == 0 && c < cols) {
#pragma unroll
        for (int j = 1; j < 32; j++) s += red[j][i];
        dw[c] = s;
    }
}

template <bool G32, bool W32, int NV>
static void launch_norm_back_rows(const NormBackArgs& p, int acc, dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
    if (acc == (WIDE | PAST)) norm_back_kernel<G32, W32, NV, WIDE | PAST><<<grid, block, lds, stream>>>(p);
    else if (acc == WIDE) norm_back_kernel<G32, W32, NV, WIDE><<<grid, block, lds, stream>>>(p);
    else if (acc == PAST) norm_back_kernel<G32, W32, NV, PAST><<<grid, block, lds, stream>>>(p);
    else norm_back_kernel<G32, W32, NV, 0><<<grid, block, lds, stream>>>(p);
}

template <bool G32, bool W32>
static void launch_norm_back(const NormBackArgs& p, const NormBackPlan& n, hipStream_t stream) {
    const bool wide = p.cols % 8 == 0 && rows_wide(p.h, p.ld_h, 16) && rows_wide(p.dy, p.ld_dy, 16) &&
                      rows_wide(p.dh, p.ld_dh, 16) && rows_wide(p.dx, p.ld_dx, 16) && fp8q_aligned(p.w, 16);
    const int acc = (wide ? WIDE : 0) | (past_caches(p.rows, p.cols, 2 + (G32 ? 4 : 2) * (p.dh ? 3 : 2)) ? PAST : 0);
    const dim3 grid((unsigned)n.blocks), block(64 * n.waves * n.rows);
    const size_t lds = (size_t)(n.rows - 1) * 8 * 64 * n.waves * 4;
    if (n.chunks == 0) norm_back_generic_kernel<G32><<<grid, dim3(256), 0, stream>>>(p);
    else if (n.chunks == 1) launch_norm_back_rows<G32, W32, 1>(p, acc, grid, block, lds, stream);
    else launch_norm_back_rows<G32, W32, 2>(p, acc, grid, block, lds, stream);
}

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
    if (rows > 0x7FFFFFFFLL || !norm_fits(rows, cols)) return FP8Q_ERR_UNSUPPORTED;
    NormArgs p{};
    p.x = x; p.rows = rows; p.cols = cols; p.ld_x = ld_x; p.residual = residual; p.ld_res = ld_res; p.w = weight; p.h = h; p.ld_h = ld_h;
    p.y = y; p.ld_y = ld_y; p.q = q; p.ld_q = ld_q; p.scales = scales; p.ld_s = ld_s; p.rstd = rstd; p.eps = eps;
    p.w32 = weight_dtype == FP8Q_OUT_FP32; p.scaling = scaling;
    if (scaling == FP8Q_NORM_NONE) start_norm<FP8Q_NORM_NONE, FP8Q_E4M3FN>(p, stream);
    else if (scaling == FP8Q_NORM_BLOCK) start_norm<FP8Q_NORM_BLOCK, FP8Q_E4M3FN>(p, stream);
    else if (fmt == FP8Q_E4M3FN) start_norm<FP8Q_NORM_ROW, FP8Q_E4M3FN>(p, stream);
    else start_norm<FP8Q_NORM_ROW, FP8Q_E4M3FNUZ>(p, stream);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

extern "C" size_t fp8_rms_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0) return 256;
    return (size_t)fp8q::norm_back_space(rows, cols);
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
    if (!norm_back_fits(rows, cols)) return FP8Q_ERR_UNSUPPORTED;
    if (rows > 0 && (!workspace || workspace_bytes < fp8_rms_norm_backward_workspace_size(rows, cols))) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 16)) return FP8Q_ERR_INVALID_ARG;
    NormBackArgs p{};
    p.dy = dy; p.ld_dy = ld_dy; p.dh = dh; p.ld_dh = ld_dh; p.h = h; p.rows = rows; p.cols = cols; p.ld_h = ld_h;
    p.rstd = rstd; p.w = weight; p.dx = dx; p.ld_dx = ld_dx; p.part = static_cast<float*>(workspace);
    p.w32 = weight_dtype == FP8Q_OUT_FP32;
    const NormBackPlan n = pick_norm_back(rows, cols);
    p.waves = n.waves;
    if (rows > 0) {
        const bool g32 = grad_dtype == FP8Q_OUT_FP32;
        if (g32 && p.w32) launch_norm_back<true, true>(p, n, stream);
        else if (g32) launch_norm_back<true, false>(p, n, stream);
        else if (p.w32) launch_norm_back<false, true>(p, n, stream);
        else launch_norm_back<false, false>(p, n, stream);
        FP8Q_CHECK_LAUNCH();
    }
    norm_back_join_kernel<<<dim3((unsigned)plan_up(cols, NORM_JOIN)), dim3(1024), 0, stream>>>(p.part, (int)n.blocks, cols, dweight);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}
