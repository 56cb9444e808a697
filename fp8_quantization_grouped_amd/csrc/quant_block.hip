// FP8 (OCP e4m3fn) quantization with one fp32 factor per block of 128: 1 x 128 blocks of an
// activation's rows, 128 x 1 blocks of its columns (written transposed), both from one read, and
// 128 x 128 blocks of expert weights in both layouts.
//
//   s = 448 / max(amax, 1e-12)        (IEEE quotient, fp32)
//   q = ENC(clamp(RN32(x * s), +-448)) (round to nearest even)
//   stored factor d = 1 / s           (IEEE quotient, fp32), so that x ~ q * d
//
// Bound: HBM.  Unlike a scale per whole column, every block's maximum is known inside one tile of
// 128 x 128, so each set of layouts needs exactly one read of x: 3 B per element for one layout, 4 B
// for two.  Measured: 16384 x 7168 in both layouts 81 us (5.8 TB/s), 64 experts of 1408 x 2048 142 us
// (5.2 TB/s), where a copy of large buffers reaches 4.9 TB/s and a fill 6.9; 49152 x 2048 in rows
// alone 49 us (6.1 TB/s); 1024 x 256 4.2 us, a launch's time.
//
// Tile: 256 threads; thread (rg, cg) holds the 8 x 8 elements at rows 8 rg.., columns 8 cg.. (eight
// 16-byte loads, 16 lanes per 256-byte row piece).  In that shape both layouts are encoded inside the
// lane: a row's 8 bytes and a column's 8 bytes are each two conversions of four.  Row maxima: 4 lane
// exchanges over the 16 lanes of a row; column maxima: 2 lane exchanges, then LDS across the 4 waves.
// The transposed bytes go through LDS (8-byte pieces, XOR-swizzled) so that each column leaves in runs
// of 128 bytes.  Tiles of 256 rows (runs of 256 bytes) are slower: 106 against 101 us at 16384 x 7168,
// 10.0 against 9.3 us at 1333 x 1104.
#include "common.hpp"

namespace fp8q {

constexpr int QB = 128;  // block edge

enum { LAY_ROW = 0, LAY_DUAL = 1, LAY_SQUARE = 2 };

struct BlockQuantArgs {
    const uint16_t* x;
    int64_t rows, cols, ld_x;  // LAY_SQUARE: rows of one matrix
    uint8_t* q;
    int64_t ld_q;
    float* s_rows;             // LAY_SQUARE: the factors [matrix][row block][column block]
    int64_t ld_sr;
    uint8_t* q_t;
    int64_t ld_qt;
    float* s_cols;
    int64_t ld_sc;
    int tiles_c;               // column tiles
    bool vec_x;                // 16-byte loads of x
    bool stream_q;             // q goes past the last-level cache
    int vec_q, vec_qt;         // bytes of one store: 8 or 1; 16, 8 or 1
};

// Maximum over the 16 lanes of a row, of packed or plain 16-bit magnitudes.
__device__ __forceinline__ uint32_t max16lanes(uint32_t v) {
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) v = pk_max_u16(v, (uint32_t)__shfl_xor((int)v, off, 64));
    return v;
}

__device__ __forceinline__ float elem(const uint4& v, int e) {  // e: compile-time after unrolling
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return (e & 1) ? bf16_hi(w) : bf16_lo(w);
}

// Slot of the 8-byte piece of column c for rows 8 rg..8 rg+7 in the transposed tile.
__device__ __forceinline__ int t_off(int c, int rg) {
    return c * QB + 8 * (rg ^ (2 * ((c >> 3) & 7)));
}

template <int LAY>
__global__ __launch_bounds__(256) void block_quant_kernel(const BlockQuantArgs p) {
    constexpr int NT = 256;
    __shared__ __align__(16) uint8_t tile[LAY == LAY_ROW ? 16 : QB * QB];
    __shared__ __align__(16) uint32_t cmax[LAY == LAY_ROW ? 4 : 4 * (QB / 2)];
    const int t = threadIdx.x, cg = t & 15, rg = t >> 4;
    const int64_t r0 = (int64_t)(blockIdx.x / p.tiles_c) * QB, c0 = (int64_t)(blockIdx.x % p.tiles_c) * QB;
    const int64_t mat = LAY == LAY_SQUARE ? (int64_t)blockIdx.y : 0;
    const uint16_t* x = p.x + mat * p.rows * p.ld_x;
    const int64_t c = c0 + 8 * cg;
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const int64_t r = r0 + 8 * rg + j;
        v[j] = make_uint4(0, 0, 0, 0);
        if (r < p.rows && c < p.cols) {
            const uint16_t* src = x + r * p.ld_x + c;
            if (p.vec_x) {
                v[j] = ld_nt16(src);
            } else {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; e++) w[e] = c + e < p.cols ? src[e] : 0;
                v[j] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
            }
        }
    }
    float sr[8];  // multipliers of the lane's rows (LAY_SQUARE: one for all)
    if (LAY != LAY_SQUARE) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const uint32_t m = pk_max_u16(pk_max_u16(mag2(v[j].x), mag2(v[j].y)), pk_max_u16(mag2(v[j].z), mag2(v[j].w)));
            sr[j] = scale_from_amax<FP8Q_E4M3FN>(__uint_as_float(hmax16(max16lanes(m)) << 16));
        }
    }
    uint32_t cm[4] = {0, 0, 0, 0};  // packed column maxima of the lane's 8 rows
    if (LAY != LAY_ROW) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            cm[0] = pk_max_u16(cm[0], mag2(v[j].x));
            cm[1] = pk_max_u16(cm[1], mag2(v[j].y));
            cm[2] = pk_max_u16(cm[2], mag2(v[j].z));
            cm[3] = pk_max_u16(cm[3], mag2(v[j].w));
        }
        // lanes 16 apart hold the same columns of other rows
#pragma unroll
        for (int i = 0; i < 4; i++) {
            cm[i] = pk_max_u16(cm[i], (uint32_t)__shfl_xor((int)cm[i], 16, 64));
            cm[i] = pk_max_u16(cm[i], (uint32_t)__shfl_xor((int)cm[i], 32, 64));
        }
        const int wave = t >> 6;
        if (LAY == LAY_SQUARE) {
            const uint32_t m = hmax16(max16lanes(pk_max_u16(pk_max_u16(cm[0], cm[1]), pk_max_u16(cm[2], cm[3]))));
            if ((t & 63) == 0) cmax[wave] = m;
        } else if ((t & 63) < 16) {
            *reinterpret_cast<uint4*>(&cmax[wave * (QB / 2) + 4 * cg]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
        }
        __syncthreads();
        if (LAY == LAY_SQUARE) {
            uint32_t m = cmax[0];
#pragma unroll
            for (int w = 1; w < 4; w++) m = m > cmax[w] ? m : cmax[w];
            const float s = scale_from_amax<FP8Q_E4M3FN>(__uint_as_float(m << 16));
#pragma unroll
            for (int j = 0; j < 8; j++) sr[j] = s;
            if (t == 0)
                p.s_rows[(mat * ((p.rows + QB - 1) / QB) + r0 / QB) * p.tiles_c + c0 / QB] = 1.0f / s;
        } else {
#pragma unroll
            for (int w = 0; w < 4; w++) {
                const uint4 o = *reinterpret_cast<const uint4*>(&cmax[w * (QB / 2) + 4 * cg]);
                cm[0] = pk_max_u16(cm[0], o.x);
                cm[1] = pk_max_u16(cm[1], o.y);
                cm[2] = pk_max_u16(cm[2], o.z);
                cm[3] = pk_max_u16(cm[3], o.w);
            }
        }
    }
    // rows: factors and bytes
    if (LAY != LAY_SQUARE) {
        // lane cg writes the factor of row 8 rg + cg (cg < 8), so a wave's 32 rows leave as one run
        float mine = sr[0];
#pragma unroll
        for (int j = 1; j < 8; j++) mine = cg == j ? sr[j] : mine;
        const int64_t r = r0 + 8 * rg + cg;
        if (cg < 8 && r < p.rows && p.s_rows) p.s_rows[(c0 / QB) * p.ld_sr + r] = 1.0f / mine;
    }
    if (p.q != nullptr && c < p.cols) {
        uint8_t* q = p.q + mat * p.rows * p.ld_q;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t r = r0 + 8 * rg + j;
            const float s = sr[j];
            const uint32_t a = enc4<FP8Q_E4M3FN>(elem(v[j], 0) * s, elem(v[j], 1) * s, elem(v[j], 2) * s, elem(v[j], 3) * s);
            const uint32_t b = enc4<FP8Q_E4M3FN>(elem(v[j], 4) * s, elem(v[j], 5) * s, elem(v[j], 6) * s, elem(v[j], 7) * s);
            if (r < p.rows) {
                uint8_t* dst = q + r * p.ld_q + c;
                if (p.vec_q == 8) {
                    if (p.stream_q) __builtin_nontemporal_store((uint64_t)b << 32 | a, reinterpret_cast<uint64_t*>(dst));
                    else *reinterpret_cast<uint2*>(dst) = make_uint2(a, b);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (c + e < p.cols) dst[e] = (uint8_t)((e < 4 ? a : b) >> (8 * (e & 3)));
                }
            }
        }
    }
    if (LAY == LAY_ROW || p.q_t == nullptr) return;
    // columns: bytes into the transposed tile, then out
#pragma unroll
    for (int e = 0; e < 8; e++) {
        float s = sr[0];
        if (LAY == LAY_DUAL) {
            const uint32_t m = (e & 1) ? cm[e >> 1] >> 16 : cm[e >> 1] & 0xFFFFu;
            s = scale_from_amax<FP8Q_E4M3FN>(__uint_as_float(m << 16));
            // one row group writes the block's 128 factors
            if (rg == 0 && c + e < p.cols) p.s_cols[(r0 / QB) * p.ld_sc + c + e] = 1.0f / s;
        }
        const uint32_t a = enc4<FP8Q_E4M3FN>(elem(v[0], e) * s, elem(v[1], e) * s, elem(v[2], e) * s, elem(v[3], e) * s);
        const uint32_t b = enc4<FP8Q_E4M3FN>(elem(v[4], e) * s, elem(v[5], e) * s, elem(v[6], e) * s, elem(v[7], e) * s);
        *reinterpret_cast<uint2*>(&tile[t_off(8 * cg + e, rg)]) = make_uint2(a, b);
    }
    __syncthreads();
    constexpr int CH = QB / 16;  // 16-byte pieces of a column
    uint8_t* q_t = p.q_t + mat * p.rows;
#pragma unroll
    for (int i = 0; i < QB * CH / NT; i++) {
        const int k = t + i * NT, col = k / CH, ch = k % CH;
        const uint4 w = *reinterpret_cast<const uint4*>(&tile[t_off(col, 2 * ch)]);
        const int64_t r = r0 + 16 * ch;
        if (c0 + col < p.cols && r < p.rows) {
            uint8_t* dst = q_t + (c0 + col) * p.ld_qt + r;
            const int n = p.rows - r < 16 ? (int)(p.rows - r) : 16;
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            if (n == 16 && p.vec_qt == 16) {
                *reinterpret_cast<uint4*>(dst) = w;
            } else if (n == 16 && p.vec_qt == 8) {
                reinterpret_cast<uint2*>(dst)[0] = make_uint2(w.x, w.y);
                reinterpret_cast<uint2*>(dst)[1] = make_uint2(w.z, w.w);
            } else {
#pragma unroll
                for (int e = 0; e < 16; e++)
                    if (e < n) dst[e] = (uint8_t)(u[e >> 2] >> (8 * (e & 3)));
            }
        }
    }
}

template <int LAY>
static fp8q_status_t launch_block_quant(BlockQuantArgs& p, int64_t mats, hipStream_t stream) {
    // a launch takes fewer than 2^32 threads along x
    constexpr int64_t most = (1LL << 32) / 256 - 1;
    if (p.rows > most * QB || p.cols > most * QB || mats > 65535) return FP8Q_ERR_UNSUPPORTED;
    const int64_t tr = (p.rows + QB - 1) / QB, tc = (p.cols + QB - 1) / QB;
    if (tr * tc > most) return FP8Q_ERR_UNSUPPORTED;
    p.tiles_c = (int)tc;
    p.vec_x = p.cols % 8 == 0 && p.ld_x % 8 == 0 && fp8q_aligned(p.x, 16);
    p.vec_q = p.cols % 8 == 0 && p.ld_q % 8 == 0 && fp8q_aligned(p.q, 8) ? 8 : 1;
    // With two layouts to write and more to read than stays in the last-level cache, q goes past it:
    // 16384 x 7168 101 -> 81 us, 64 experts of 1408 x 2048 149 -> 142 us (142 -> 139 and 81 -> 96 if q_t
    // does too).  q alone stays in reach of the product that reads it next: 49152 x 2048 and 64 experts'
    // product 247 us, past the cache 252.
    p.stream_q = LAY != LAY_ROW && (double)(mats * p.rows) * p.cols * 2.0 > kStreamBytes;
    // a matrix's columns start at byte mat * rows of q_t's rows
    const int64_t at = mats > 1 ? p.rows : 0;
    p.vec_qt = p.ld_qt % 16 == 0 && at % 16 == 0 && fp8q_aligned(p.q_t, 16) ? 16
             : p.ld_qt % 8 == 0 && at % 8 == 0 && fp8q_aligned(p.q_t, 8) ? 8 : 1;
    block_quant_kernel<LAY><<<dim3((unsigned)(tr * tc), (unsigned)mats), dim3(256), 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

}  // namespace fp8q

extern "C" fp8q_status_t fp8_block_quant_rowwise(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                                 uint8_t* q, int64_t ld_q, float* scales, int64_t ld_s,
                                                 hipStream_t stream) {
    using namespace fp8q;
    if (rows < 0 || cols < 0 || ld_x < cols || ld_q < cols || ld_s < rows) return FP8Q_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!x || !q || !scales) return FP8Q_ERR_INVALID_ARG;
    BlockQuantArgs p{};
    p.x = x; p.rows = rows; p.cols = cols; p.ld_x = ld_x; p.q = q; p.ld_q = ld_q; p.s_rows = scales; p.ld_sr = ld_s;
    return launch_block_quant<LAY_ROW>(p, 1, stream);
}

extern "C" fp8q_status_t fp8_block_quant_dual(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                                              uint8_t* q, int64_t ld_q, float* s_rows, int64_t ld_sr,
                                              uint8_t* q_t, int64_t ld_qt, float* s_cols, int64_t ld_sc,
                                              hipStream_t stream) {
    using namespace fp8q;
    const bool row_out = q || s_rows;  // both null: the transposed layout alone
    if (rows < 0 || cols < 0 || ld_x < cols || ld_qt < rows || ld_sc < cols) return FP8Q_ERR_INVALID_ARG;
    if (row_out && (ld_q < cols || ld_sr < rows)) return FP8Q_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!x || !q_t || !s_cols || (row_out && (!q || !s_rows))) return FP8Q_ERR_INVALID_ARG;
    BlockQuantArgs p{};
    p.x = x; p.rows = rows; p.cols = cols; p.ld_x = ld_x; p.q = q; p.ld_q = ld_q; p.s_rows = s_rows; p.ld_sr = ld_sr;
    p.q_t = q_t; p.ld_qt = ld_qt; p.s_cols = s_cols; p.ld_sc = ld_sc;
    return launch_block_quant<LAY_DUAL>(p, 1, stream);
}

extern "C" fp8q_status_t fp8_block_quant_weights(const uint16_t* w, int64_t experts, int64_t rows, int64_t cols,
                                                 int64_t ld_w, uint8_t* q, int64_t ld_q, uint8_t* q_t,
                                                 int64_t ld_qt, float* scales, hipStream_t stream) {
    using namespace fp8q;
    if (experts < 0 || rows < 0 || cols < 0 || ld_w < cols) return FP8Q_ERR_INVALID_ARG;
    if ((q && ld_q < cols) || (q_t && (experts > 0 && rows > ld_qt / experts))) return FP8Q_ERR_INVALID_ARG;
    if (experts == 0 || rows == 0 || cols == 0) return FP8Q_OK;
    if (!w || !scales || (!q && !q_t)) return FP8Q_ERR_INVALID_ARG;
    BlockQuantArgs p{};
    p.x = w; p.rows = rows; p.cols = cols; p.ld_x = ld_w; p.q = q; p.ld_q = ld_q; p.s_rows = scales;
    p.q_t = q_t; p.ld_qt = ld_qt;
    return launch_block_quant<LAY_SQUARE>(p, experts, stream);
}
