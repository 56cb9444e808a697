// What the grouped GEMMs share: the operand tiles' layout in LDS, byte masks, rounding to bf16.
#pragma once

#include "common.hpp"

namespace fp8q {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v4f_t __attribute__((ext_vector_type(4)));

constexpr int GK = 128;         // contraction bytes per step
constexpr int MODE_FWD = 0, MODE_WGRAD = 1;
constexpr int GMAX = 2048;  // groups whose schedule prefix fits in LDS

// 16-byte slot of chunk c in row r: c ^ (2*((r >> 2) & 3) + ((r >> 1) & 1)).  A fragment read
// is served as two 32-lane halves, each touching 16 consecutive rows at chunks kg ^ s and
// (kg+1) ^ s; the rows that share a 512-byte LDS window (same r & 3) get distinct
// 2*((r >> 2) & 3), so all 32 16-byte slots of a half are distinct (no bank conflicts).
__device__ __forceinline__ int swz(int r) { return (((r >> 2) & 3) << 1) | ((r >> 1) & 1); }
__device__ __forceinline__ int lds_off(int r, int ch) { return r * GK + ((ch ^ swz(r)) << 4); }
// N-side tile: its fragments take rows 32j' + 8q + 4h + e (q = lane%16 / 4, e = lane%4) so that
// each lane's results are 8 consecutive output columns; slot c ^ (2*((r>>3)&3) + ((r>>1)&1))
// puts those 16 rows in 16 distinct 16-byte bank slots.
__device__ __forceinline__ int swzB(int r) { return (((r >> 3) & 3) << 1) | ((r >> 1) & 1); }
__device__ __forceinline__ int lds_offB(int r, int ch) { return r * GK + ((ch ^ swzB(r)) << 4); }
// Row of the N-side tile that feeds MFMA row lr of column block j (see swzB).
__device__ __forceinline__ int brow(int j, int lr) {
    return 32 * (j >> 1) + 8 * (lr >> 2) + 4 * (j & 1) + (lr & 3);
}

// Bytes at positions base..base+3 of a chunk kept where lo <= pos < hi.
__device__ __forceinline__ uint32_t keep_mask4(int lo, int hi, int base) {
    int a = lo - base, b = hi - base;
    a = a < 0 ? 0 : (a > 4 ? 4 : a);
    b = b < 0 ? 0 : (b > 4 ? 4 : b);
    const uint32_t below_b = b >= 4 ? 0xFFFFFFFFu : ((1u << (8 * b)) - 1u);
    const uint32_t from_a = a >= 4 ? 0u : (0xFFFFFFFFu << (8 * a));
    return below_b & from_a;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
    a += 0x7FFFu + ((a >> 16) & 1u);
    b += 0x7FFFu + ((b >> 16) & 1u);
    return (a >> 16) | (b & 0xFFFF0000u);
}

static inline int num_cus() {
    static int cached[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (!cached[dev]) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            n <= 0)
            n = 256;
        cached[dev] = n;
    }
    return cached[dev];
}

}  // namespace fp8q
