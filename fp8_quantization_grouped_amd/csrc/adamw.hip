// One AdamW step over a list of tensors, with the states in 32 bits or in 8.
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,
//   p' = p - lr (m' / (1 - b1^t) / (sqrt(v' / (1 - b2^t)) + eps) + decay p)
//
// 8 bits: m and r = sqrt(v) are kept as e4m3fn values with one fp32 factor d per block of 128 elements
// (s = 448 / max(amax, 1e-12), d = 1 / s, as the block quantizers).  r instead of v, since a square has
// twice the range.  The new value goes to the grid's next value down or up, at random in proportion: with
// b2 = 0.999 one step changes r by 2^-11 of itself and the grid's steps are 2^-4 of it, so the nearest
// value would mostly be the old one for ever.  A nonzero r never becomes zero, which would divide a
// remaining m by eps.  What the step itself uses is m' and v' in 32 bits, before they are kept.  The kept r
// of a stationary gradient spreads about its true value by a sixth of it (b2 = 0.999) to a ninth (0.95),
// the mean being 1% above: a value on the grid that moves by a small e of itself is rounded with a variance
// of e times the step, so slow averages take little noise a step.  An element whose m' or v' is not finite in
// 32 bits (its gradient is not, or the square overflows) is kept as NaN and stays out of the factor: an infinite
// factor would cost the other 127 their states, and a finite byte would hide it.
//
// Random bits: word(tensor, element) = mix(mix(seed * 0x9E3779B1 + tensor) + element), mix two rounds of
// xor-shift and odd product as in the finalizers of published hash functions.  The constants are published ones
// too: a prime next to 2^32 over the golden ratio, the low half of splitmix64's increment (0x7F4A7C15) and the
// multiplier of the 32-bit PCG generators (0x2C9277B5).  m takes the word, r the word with its halves exchanged,
// the conversion the upper 20 bits of each.
//
// Bound: HBM.  Measured (MI355X, bytes of every tensor read and written once): 277M bf16 elements with 8-bit
// states 517 us (5.4 TB/s), 58M with masters, fp32 gradients and 32-bit states 321 us (5.4 TB/s), where a
// copy of large buffers reaches 5.2.  1.6M elements with 8-bit states take the kernel 9 us where their bytes take 3:
// 386 blocks, each one chain of loads, arithmetic and stores, on 256 CUs.
#include "common.hpp"

namespace fp8q {

constexpr int AB = 128;            // elements of a block with one factor
constexpr int ADAMW_TENSORS = 40;  // of one launch: its arguments fit the 4 KB that a launch takes
// Elements that a block of 256 threads takes: 8 of a thread, with 8-bit states twice 8, half a chunk apart,
// so that what a block's factors cost is shared by more of them.
constexpr int chunk_of(bool eight) { return eight ? 4096 : 2048; }

struct AdamTensor {
    void* param;
    float* master;
    const void* grad;
    void* m;
    float* m_scales;
    void* v;
    float* v_scales;
    int64_t n;
    uint32_t index;          // place in the caller's list
    uint8_t param32, grad32, wide, pad;
};

struct AdamArgs {
    AdamTensor t[ADAMW_TENSORS];
    int64_t chunk_end[ADAMW_TENSORS];  // chunks up to and with tensor i
    int count;
    float lr, b1, b2, one_b1, one_b2, eps, decay, inv_bc1, inv_bc2;
    float log_b1, log_b2;
    uint32_t seed;
    const float* lr_device;
    const int32_t* step_device;
    const float* grad_scale;
};

__device__ __forceinline__ float ad_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
typedef __bf16 ad_bf16x2 __attribute__((ext_vector_type(2)));
typedef float f2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t ad_pack(float a, float b) {  // to the nearest, ties to even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2_t{a, b}), ad_bf16x2));
}

// An access that is always one to global memory, also where the compiler would choose between this
// pointer and the address of an argument.
template <class T>
using Global = __attribute__((address_space(1))) T*;
template <class T>
__device__ __forceinline__ T global_at(const T* p, int64_t i) { return ((Global<const T>)p)[i]; }

__device__ __forceinline__ uint32_t mix(uint32_t z) {
    z = (z ^ z >> 16) * 0x7F4A7C15u;
    z = (z ^ z >> 15) * 0x2C9277B5u;
    return z ^ z >> 16;
}

// 16 bytes, with the non-temporal hint or without.
template <bool NT>
__device__ __forceinline__ uint4 get16(const void* p) { return NT ? ld_nt16(p) : *static_cast<const uint4*>(p); }
template <bool NT>
__device__ __forceinline__ void put16(void* p, uint4 v) {
    if (NT) st_nt16(p, v);
    else *static_cast<uint4*>(p) = v;
}
__device__ __forceinline__ uint32_t bits_of(float f) { return __float_as_uint(f); }

// Eight consecutive elements as 32-bit values; n of them exist.
template <bool F32, bool NT>
__device__ __forceinline__ void load8(const void* src, int64_t at, int n, bool wide, float (&out)[8]) {
    if (F32) {
        const float* p = static_cast<const float*>(src) + at;
        if (wide && n == 8) {
            const uint4 a = get16<NT>(p), b = get16<NT>(p + 4);
            out[0] = __uint_as_float(a.x); out[1] = __uint_as_float(a.y); out[2] = __uint_as_float(a.z); out[3] = __uint_as_float(a.w);
            out[4] = __uint_as_float(b.x); out[5] = __uint_as_float(b.y); out[6] = __uint_as_float(b.z); out[7] = __uint_as_float(b.w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) out[i] = i < n ? p[i] : 0.0f;
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(src) + at;
        if (wide && n == 8) {
            const uint4 a = get16<NT>(p);
            out[0] = bf16_lo(a.x); out[1] = bf16_hi(a.x); out[2] = bf16_lo(a.y); out[3] = bf16_hi(a.y);
            out[4] = bf16_lo(a.z); out[5] = bf16_hi(a.z); out[6] = bf16_lo(a.w); out[7] = bf16_hi(a.w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) out[i] = i < n ? ad_bf16(p[i]) : 0.0f;
        }
    }
}
template <bool F32, bool NT>
__device__ __forceinline__ void store8(void* dst, int64_t at, int n, bool wide, const float (&v)[8]) {
    if (F32) {
        float* p = static_cast<float*>(dst) + at;
        if (wide && n == 8) {
            put16<NT>(p, make_uint4(bits_of(v[0]), bits_of(v[1]), bits_of(v[2]), bits_of(v[3])));
            put16<NT>(p + 4, make_uint4(bits_of(v[4]), bits_of(v[5]), bits_of(v[6]), bits_of(v[7])));
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (i < n) p[i] = v[i];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(dst) + at;
        if (wide && n == 8) {
            put16<NT>(p, make_uint4(ad_pack(v[0], v[1]), ad_pack(v[2], v[3]), ad_pack(v[4], v[5]), ad_pack(v[6], v[7])));
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (i < n) p[i] = (uint16_t)ad_pack(v[i], 0.0f);
        }
    }
}

// Eight e4m3fn values.
__device__ __forceinline__ void load8_fp8(const void* src, int64_t at, int n, bool wide, float (&out)[8]) {
    const uint8_t* p = static_cast<const uint8_t*>(src) + at;
    uint32_t w[2] = {0, 0};
    if (wide && n == 8) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        w[0] = a.x; w[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const f2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
        out[4 * i] = lo.x; out[4 * i + 1] = lo.y; out[4 * i + 2] = hi.x; out[4 * i + 3] = hi.y;
    }
}

// Largest magnitude of eight values each of 16 lanes, in all of them, as its bits, whose order is the magnitudes'
// with the infinite behind the finite and NaN behind these: by DPP 1 and 2 lanes away, then mirrored in 8 and
// in 16.
constexpr uint32_t kInfBits = 0x7F800000u;
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}
__device__ __forceinline__ uint32_t block_amax(const float (&x)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = __builtin_elementwise_maximum(m, fabsf(x[i]));  // a NaN stays
    return dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(__float_as_uint(m)))));
}

// Eight values as bytes, by their block's multiplier and random bits.  ROOT: values of which none is negative
// and a nonzero one does not become zero: what lies under the grid's first value is taken for it.  lost: a bit
// for each of them that is zero here and kept as NaN.
template <bool ROOT, bool NT>
__device__ __forceinline__ void keep8(void* dst, int64_t at, int n, bool wide, float s, const float (&x)[8], const uint32_t (&bits)[8],
                                      uint32_t lost) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float y = __builtin_amdgcn_fmed3f(x[i] * s, ROOT ? (x[i] > 0.0f ? 0.001953125f : 0.0f) : -kFmaxFn, kFmaxFn);
        const uint32_t r = ROOT ? bits[i] << 16 | bits[i] >> 16 : bits[i];
        if ((i & 3) == 0) w[i >> 2] = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(y, r, 0, 0);
        if ((i & 3) == 1) w[i >> 2] = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(y, r, (int)w[i >> 2], 1);
        if ((i & 3) == 2) w[i >> 2] = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(y, r, (int)w[i >> 2], 2);
        if ((i & 3) == 3) w[i >> 2] = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(y, r, (int)w[i >> 2], 3);
    }
    if (lost) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (lost >> i & 1) w[i >> 2] |= 0x7Fu << (8 * (i & 3));
    }
    uint8_t* p = static_cast<uint8_t*>(dst) + at;
    if (wide && n == 8) {
        if (NT) st_nt8(p, w[0], w[1]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// The states' averages, each operation rounded by itself: what is kept of them can be told to the bit from
// elementary operations in 32 bits, and a value next to the grid's border falls where those say.
__device__ __forceinline__ void moments(const AdamArgs& a, float g, float& m, float& v) {
#pragma clang fp contract(off)
    m = a.b1 * m + a.one_b1 * g;
    v = a.b2 * v + a.one_b2 * g * g;
}

// NT: stores, and with 8-bit states loads too, go past the caches, where a launch moves more than stays in the
// last-level one.  277M bf16 elements, 8 bits: 545 us through the caches, 538 with the stores past them, 524
// with both; 58M with masters, 32 bits: 345, 321 and 333 us.
template <bool EIGHT, bool NT>
__global__ __launch_bounds__(256) void adamw_kernel(const AdamArgs a) {
    constexpr int H = EIGHT ? 2 : 1, CHUNK = chunk_of(EIGHT);
    constexpr bool NTL = NT && EIGHT;
    int lo = 0, hi = a.count - 1;  // the tensor of this chunk
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.chunk_end[mid] > (int64_t)blockIdx.x) hi = mid; else lo = mid + 1;
    }
    const AdamTensor& t = a.t[lo];
    const int64_t first = lo ? a.chunk_end[lo - 1] : 0;
    const int64_t at0 = ((int64_t)blockIdx.x - first) * CHUNK + 8 * threadIdx.x;
    const bool wide = t.wide;
    float p[H][8], g[H][8], m[H][8], v[H][8], dm[H], dv[H];
    int n[H];
#pragma unroll
    for (int h = 0; h < H; h++) {
        const int64_t at = at0 + h * 2048;
        n[h] = t.n - at >= 8 ? 8 : t.n > at ? (int)(t.n - at) : 0;
        if (t.master) load8<true, NTL>(t.master, at, n[h], wide, p[h]);
        else if (t.param32) load8<true, NTL>(t.param, at, n[h], wide, p[h]);
        else load8<false, NTL>(t.param, at, n[h], wide, p[h]);
        if (t.grad32) load8<true, NTL>(t.grad, at, n[h], wide, g[h]);
        else load8<false, NTL>(t.grad, at, n[h], wide, g[h]);
        if (EIGHT) {
            dm[h] = n[h] > 0 ? t.m_scales[at / AB] : 0.0f;
            dv[h] = n[h] > 0 ? t.v_scales[at / AB] : 0.0f;
            load8_fp8(t.m, at, n[h], wide, m[h]);
            load8_fp8(t.v, at, n[h], wide, v[h]);
        } else {
            load8<true, NTL>(t.m, at, n[h], wide, m[h]);
            load8<true, NTL>(t.v, at, n[h], wide, v[h]);
        }
    }
    const float lr = a.lr_device ? global_at(a.lr_device, 0) : a.lr;
    float inv_bc1 = a.inv_bc1, inv_bc2 = a.inv_bc2;
    uint32_t seed = a.seed;
    if (a.step_device) {
        const int32_t step = global_at(a.step_device, 0);
        inv_bc1 = -1.0f / expm1f((float)step * a.log_b1);
        inv_bc2 = -1.0f / expm1f((float)step * a.log_b2);
        seed += (uint32_t)step;
    }
    const float scale = a.grad_scale ? global_at(a.grad_scale, 0) : 1.0f, root_bc2 = sqrtf(inv_bc2);
    float r[H][8];
#pragma unroll
    for (int h = 0; h < H; h++) {
        if (EIGHT) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                m[h][i] *= dm[h];
                v[h][i] *= dv[h];
                v[h][i] *= v[h][i];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            moments(a, a.grad_scale ? g[h][i] * scale : g[h][i], m[h][i], v[h][i]);
            r[h][i] = sqrtf(v[h][i]);
            const float d = m[h][i] * inv_bc1 * __builtin_amdgcn_rcpf(r[h][i] * root_bc2 + a.eps);
            p[h][i] = p[h][i] - lr * (d + a.decay * p[h][i]);
        }
        const int64_t at = at0 + h * 2048;
        if (t.master) store8<true, NT>(t.master, at, n[h], wide, p[h]);
        if (t.param32) store8<true, NT>(t.param, at, n[h], wide, p[h]);
        else store8<false, NT>(t.param, at, n[h], wide, p[h]);
        if (!EIGHT) {
            store8<true, NT>(t.m, at, n[h], wide, m[h]);
            store8<true, NT>(t.v, at, n[h], wide, v[h]);
        }
    }
    if (!EIGHT) return;
    // 16 lanes share two blocks and so four factors: four lanes form each of them
    const int which = (threadIdx.x >> 2) & 3;
    uint32_t m0 = block_amax(m[0]), m1 = block_amax(m[H - 1]), r0 = block_amax(r[0]), r1 = block_amax(r[H - 1]);
    uint32_t amax = which & 2 ? (which & 1 ? r1 : m1) : which & 1 ? r0 : m0;
    uint32_t lost = 0;  // elements that 32 bits do not hold, which must not become their neighbours' factor
    if (__any(amax >= kInfBits)) {
#pragma unroll
        for (int i = 0; i < 8 * H; i++) {
            float &a = m[i / 8][i % 8], &b = r[i / 8][i % 8];
            if (!(fabsf(a) < INFINITY && b < INFINITY)) {
                lost |= 1u << i;
                a = b = 0.0f;
            }
        }
        m0 = block_amax(m[0]), m1 = block_amax(m[H - 1]), r0 = block_amax(r[0]), r1 = block_amax(r[H - 1]);
        amax = which & 2 ? (which & 1 ? r1 : m1) : which & 1 ? r0 : m0;
    }
    const float mine = scale_from_amax<FP8Q_E4M3FN>(__uint_as_float(amax));
    const int64_t at1 = at0 + (which & 2 ? 2048 : 0);
    if ((threadIdx.x & 3) == 0 && t.n > (at1 & ~(int64_t)(AB - 1))) (which & 1 ? t.v_scales : t.m_scales)[at1 / AB] = 1.0f / mine;
    const uint32_t key = mix(seed * 0x9E3779B1u + t.index);
#pragma unroll
    for (int h = 0; h < H; h++) {
        const int64_t at = at0 + h * 2048;
        const int from = (threadIdx.x & 48) + 8 * h;
        const float sm = __shfl(mine, from, 64), sr = __shfl(mine, from + 4, 64);
        const uint32_t base = key + (uint32_t)at + (uint32_t)(at >> 32) * 0x632BE5A7u;
        uint32_t bits[8];
#pragma unroll
        for (int i = 0; i < 8; i++) bits[i] = mix(base + i);
        keep8<false, NT>(t.m, at, n[h], wide, sm, m[h], bits, lost >> 8 * h & 0xFF);
        keep8<true, NT>(t.v, at, n[h], wide, sr, r[h], bits, lost >> 8 * h & 0xFF);
    }
}

static inline bool ad_real(const fp8q_adamw_tensor_t& t) { return t.n > 0 && t.grad; }

}  // namespace fp8q

extern "C" fp8q_status_t adamw_step(const fp8q_adamw_tensor_t* tensors, int32_t count, const fp8q_adamw_t* h, hipStream_t stream) {
    using namespace fp8q;
    if (count < 0 || !h || (count > 0 && !tensors) || (h->state_bits != 8 && h->state_bits != 32) || !(h->beta1 >= 0.0 && h->beta1 < 1.0) ||
        !(h->beta2 >= 0.0 && h->beta2 < 1.0) || !(h->eps > 0.0f) || (!h->step_device && h->step < 1))
        return FP8Q_ERR_INVALID_ARG;
    const bool eight = h->state_bits == 8;
    const int64_t chunk = chunk_of(eight);
    for (int32_t i = 0; i < count; i++) {  // all of them before the first launch
        const fp8q_adamw_tensor_t& t = tensors[i];
        if (t.n < 0 || (t.param_dtype != FP8Q_OUT_BF16 && t.param_dtype != FP8Q_OUT_FP32) ||
            (t.grad_dtype != FP8Q_OUT_BF16 && t.grad_dtype != FP8Q_OUT_FP32) || (t.master && t.param_dtype != FP8Q_OUT_BF16))
            return FP8Q_ERR_INVALID_ARG;
        if (!ad_real(t)) continue;
        if (!t.param || !t.exp_avg || !t.exp_avg_sq || (eight && (!t.exp_avg_scales || !t.exp_avg_sq_scales))) return FP8Q_ERR_INVALID_ARG;
        if (t.n > 1LL << 34) return FP8Q_ERR_UNSUPPORTED;  // a launch takes fewer than 2^32 threads
    }
    AdamArgs a{};
    a.b1 = (float)h->beta1; a.b2 = (float)h->beta2; a.one_b1 = (float)(1.0 - h->beta1); a.one_b2 = (float)(1.0 - h->beta2);
    a.eps = h->eps; a.decay = h->weight_decay; a.lr = h->lr; a.lr_device = h->lr_device; a.step_device = h->step_device;
    a.grad_scale = h->grad_scale; a.seed = (uint32_t)h->seed;
    if (h->step_device) {
        a.log_b1 = (float)log(h->beta1);
        a.log_b2 = (float)log(h->beta2);
    } else {
        a.inv_bc1 = (float)(1.0 / (1.0 - pow(h->beta1, (double)h->step)));
        a.inv_bc2 = (float)(1.0 / (1.0 - pow(h->beta2, (double)h->step)));
        a.seed += (uint32_t)h->step;
    }
    for (int32_t i = 0; i < count;) {
        int64_t chunks = 0;
        double bytes = 0.0;  // that the launch reads and writes
        a.count = 0;
        for (; i < count && a.count < ADAMW_TENSORS; i++) {
            const fp8q_adamw_tensor_t& t = tensors[i];
            if (!ad_real(t)) continue;
            const int64_t more = (t.n + chunk - 1) / chunk;
            if (chunks + more >= 1LL << 24) break;
            AdamTensor& to = a.t[a.count];
            to.param = t.param; to.master = t.master; to.grad = t.grad; to.m = t.exp_avg; to.m_scales = t.exp_avg_scales;
            to.v = t.exp_avg_sq; to.v_scales = t.exp_avg_sq_scales; to.n = t.n; to.index = (uint32_t)i;
            to.param32 = t.param_dtype == FP8Q_OUT_FP32; to.grad32 = t.grad_dtype == FP8Q_OUT_FP32;
            to.wide = fp8q_aligned(t.param, 16) && fp8q_aligned(t.master, 16) && fp8q_aligned(t.grad, 16) &&
                      fp8q_aligned(t.exp_avg, eight ? 8 : 16) && fp8q_aligned(t.exp_avg_sq, eight ? 8 : 16);
            chunks += more;
            bytes += (double)t.n * ((eight ? 4 : 16) + (to.param32 ? 8 : 4) + (to.grad32 ? 4 : 2) + (t.master ? 6 : 0));
            a.chunk_end[a.count++] = chunks;
        }
        if (a.count == 0) break;
        const dim3 grid((unsigned)chunks), block(256);
        if (eight && bytes > kStreamBytes) adamw_kernel<true, true><<<grid, block, 0, stream>>>(a);
        else if (eight) adamw_kernel<true, false><<<grid, block, 0, stream>>>(a);
        else if (bytes > kStreamBytes) adamw_kernel<false, true><<<grid, block, 0, stream>>>(a);
        else adamw_kernel<false, false><<<grid, block, 0, stream>>>(a);
        FP8Q_CHECK_LAUNCH();
    }
    return FP8Q_OK;
}
