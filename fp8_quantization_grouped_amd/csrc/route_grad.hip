// What a router's training needs beside the choice (moe_route): the balance loss with the experts' counts,
// and the gradient of the logits from that loss and from the chosen weights.
//
//   p[t,e]  = softmax(l)[e], or sigmoid(l[e]) / sum of the row's sigmoids
//   loss[s] = E / (k n^2) * sum_e count[s,e] * sum_{t in s} p[t,e]        (n tokens in sequence s)
//   dl      = p slope (dp - sum_e p dp),  dp[e] = dloss[s] E / (k n^2) count[s,e]
//           + the chosen weights' part;  slope = 1 (softmax) or 1 - sigmoid(l), of log(score) over l
//
// Bound: HBM for many tokens of few experts or of fp32 logits (65536 x 256: sums 23 us, gradient 29, 13 and 27
// at a copy's rate); with bf16 logits of 256 experts waits and exponentials (65536 x 256 sigmoid: sums 16 us and
// their join 7, gradient 30 or, on one input again and again, 25, of which a copy's rate would take 14); launches
// below (96 x 4: 3 us each).
#include "common.hpp"
#include "plan.hpp"

namespace fp8q {

constexpr int RG_MAX_E = 1024, RG_MAX_K = 32;

struct RouteGradArgs {
    const void* logits;
    int64_t T, ld_l;
    const int32_t* ids;          // [T][k]
    const int32_t* sequences;    // [S] ends, or null: one of all T
    const float* dweights;       // [T][k] or null
    const float* dloss;          // [S] or null
    float* loss;                 // [S]
    int32_t* counts;             // [S][E]
    void* dlogits;
    int64_t ld_d;
    float* mass;                 // [chunks + S][E] sums of p of a chunk's tokens of one sequence
    int32_t* part;               // [chunks + S][E] their counts
    float* group_sums;           // [S][groups] what groups of experts give a sequence's loss, or null
    int64_t rows;                // of a chunk
    int E, k, S;
    bool sigmoid, renorm, wide;  // wide: rows start on whole vectors of 4, and E is a multiple of 4
    float scale;
};

__device__ __forceinline__ float rg_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
typedef __bf16 rg_bf16x2 __attribute__((ext_vector_type(2)));
typedef float rg_f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t rg_pack(float a, float b) {  // to the nearest, ties to even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((rg_f32x2{a, b}), rg_bf16x2));
}

// The value of another lane of the 16 that a DPP operation reaches: 1 and 2 away, then mirrored in 8 and 16
// (whose lanes hold one value each by then).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
// Sum (SUM) or maximum over the L lanes that share a row, the same in all of them.
template <int L, bool SUM>
__device__ __forceinline__ float over_row(float v) {
    const auto join = [](float a, float b) { return SUM ? a + b : fmaxf(a, b); };
    if (L > 1) v = join(v, dpp<0xB1>(v));    // quad_perm 1 0 3 2
    if (L > 2) v = join(v, dpp<0x4E>(v));    // quad_perm 2 3 0 1
    if (L > 4) v = join(v, dpp<0x141>(v));   // row_half_mirror
    if (L > 8) v = join(v, dpp<0x140>(v));   // row_mirror
    if (L > 16) v = join(v, __shfl_xor(v, 16, 64));
    if (L > 32) v = join(v, __shfl_xor(v, 32, 64));
    return v;
}
template <int L>
__device__ __forceinline__ float row_sum(float v) { return over_row<L, true>(v); }
template <int L>
__device__ __forceinline__ float row_max(float v) { return over_row<L, false>(v); }

// Sum over the 64 / L rows of a wave, in each of its lanes: by rotations of 16 lanes, then across these.
template <int L>
__device__ __forceinline__ float over_rows(float v) {
    if (L <= 8) v += dpp<0x128>(v);  // row_ror 8
    if (L <= 4) v += dpp<0x124>(v);
    if (L <= 2) v += dpp<0x122>(v);
    if (L <= 1) v += dpp<0x121>(v);
    if (L <= 16) v += __shfl_xor(v, 16, 64);
    if (L <= 32) v += __shfl_xor(v, 32, 64);
    return v;
}

// exp(x) for x <= 0 within two units and |x| / 4 of the last place: 2^(x log2(e)), the product's rounding made
// good to first order.  Results under 2^-126 are zero.
__device__ __forceinline__ float exp_neg(float x) {
    x = x < -200.0f ? -200.0f : x;  // a NaN stays
    const float t = x * 1.44269504f, r = fmaf(x, 1.44269504f, -t);
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r * 0.693147181f, e);
}

// The sequences' ends, inside [0, T] whatever is stored.  Lane l of a wave reads the l-th at the kernel's start, so
// that up to 64 of them are at hand without another load.  All lanes of a wave call these together.
struct Ends {
    const int32_t* all;
    int64_t T;
    int S, mine;
    __device__ __forceinline__ explicit Ends(const RouteGradArgs& p) : all(p.sequences), T(p.T), S(p.S), mine(0) {
        const int lane = threadIdx.x & 63;
        if (all && lane < S) mine = all[lane];
    }
    // Of sequence s, which may differ from lane to lane; 0 for s < 0.
    __device__ __forceinline__ int64_t end(int s) const {
        int64_t e = T;
        if (all) e = S <= 64 ? __shfl(mine, s < 0 ? 0 : s, 64) : all[s < 0 ? 0 : s];
        return s < 0 || e < 0 ? 0 : e > T ? T : e;
    }
    // The first sequence behind s whose end lies behind row r, S for none; each lane by itself.
    __device__ __forceinline__ int after(int s, int64_t r) const {
        int lo = s + 1, hi = S;
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if ((int64_t)all[mid] > r) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }
    // The sequence of row r, the same in the whole wave: the first whose end lies behind it, S for rows behind
    // the last; of more than 64, by looking at 64 places at a time.
    __device__ __forceinline__ int of(int64_t r) const {
        if (!all) return r < T ? 0 : 1;
        const int lane = threadIdx.x & 63;
        if (S <= 64) return __popcll(__ballot(lane < S && (int64_t)mine <= r));
        int lo = 0, n = S;  // the answer lies in lo .. lo + n
        while (n > 0) {
            const int step = (n + 63) / 64, at = lane * step;
            const int before = __popcll(__ballot(at < n && (int64_t)all[lo + (at < n ? at : 0)] <= r));
            if (before == 0) return lo;
            const int skip = (before - 1) * step + 1;
            lo += skip;
            n = n - skip < step - 1 ? n - skip : step - 1;
        }
        return lo;
    }
};

// A row's logits: L lanes with 4 * NV experts each, lane j's at 4 (j + L v) .. + 3; minus infinity past E.
// They are held as they are read until get.
template <int L, int NV, bool F32, bool WIDE>
struct Logits {
    uint32_t w[NV][F32 ? 4 : 2];
    __device__ __forceinline__ void load(const RouteGradArgs& p, int64_t r, int j) {
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int e = 4 * (j + L * v);
            if (F32) {
#pragma unroll
                for (int i = 0; i < 4; i++) w[v][F32 ? i : 0] = 0xFF800000u;
                if (e >= p.E) continue;
                const uint32_t* src = static_cast<const uint32_t*>(p.logits) + r * p.ld_l + e;
                if (WIDE) {
                    const uint4 a = *reinterpret_cast<const uint4*>(src);
                    w[v][0] = a.x; w[v][1] = a.y; w[v][F32 ? 2 : 0] = a.z; w[v][F32 ? 3 : 0] = a.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (e + i < p.E) w[v][F32 ? i : 0] = src[i];
                }
            } else {
                w[v][0] = w[v][1] = 0xFF80FF80u;
                if (e >= p.E) continue;
                const uint16_t* src = static_cast<const uint16_t*>(p.logits) + r * p.ld_l + e;
                if (WIDE) {
                    const uint2 a = *reinterpret_cast<const uint2*>(src);
                    w[v][0] = a.x; w[v][1] = a.y;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (e + i < p.E) w[v][i >> 1] = i & 1 ? (w[v][i >> 1] & 0xFFFFu) | (uint32_t)src[i] << 16 : (w[v][i >> 1] & 0xFFFF0000u) | src[i];
                }
            }
        }
    }
    __device__ __forceinline__ void get(float (&l)[4 * NV]) const {
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                l[4 * v + i] = F32 ? __uint_as_float(w[v][F32 ? i : 0]) : i & 1 ? bf16_hi(w[v][i >> 1]) : bf16_lo(w[v][i >> 1]);
    }
};

// Scores under this sum are formed from the logits less their maximum: sigmoids of logits so far below
// zero are their exponentials, and a softmax's scores have the exponentials' ratios.
constexpr float kTinyScores = 5.421010862427522e-20f;  // 2^-64

// exp(l - m) and its row's 1 / sum.
template <int L, int N>
__device__ __forceinline__ void exponentials(const float (&l)[N], float (&t)[N], float& m, float& inv) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; i++) m = fmaxf(m, l[i]);
    m = row_max<L>(m);
    m = m == -INFINITY ? 0.0f : m;  // every logit at minus infinity: no probabilities
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        t[i] = exp_neg(l[i] - m);
        sum += t[i];
    }
    sum = row_sum<L>(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
}

// A row's scores: probabilities are t a, the scores that weights are made of t b, and slope (sigmoids alone;
// 1 else) is the derivative of a score's logarithm by its logit.
template <int L, bool SIG, int N>
__device__ __forceinline__ void scores_of(const float (&l)[N], float (&t)[N], float (&slope)[N], float& a, float& b) {
    if (!SIG) {
        float m;
        exponentials<L>(l, t, m, a);
        b = a;
        return;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float u = exp_neg(-fabsf(l[i])), one = __builtin_amdgcn_rcpf(1.0f + u), rest = u * one;  // neither end overflows or cancels
        t[i] = l[i] > 0.0f ? one : rest;
        slope[i] = l[i] > 0.0f ? rest : one;
        sum += t[i];
    }
    sum = row_sum<L>(sum);
    a = 1.0f / sum;
    b = 1.0f;
    if (sum < kTinyScores) {
        float m;
        exponentials<L>(l, t, m, a);
        b = expf(m);  // sigmoids so small are exponentials
    }
}

// E / (k n^2), what a sequence of n tokens' sum of counts times probabilities is multiplied by.
__device__ __forceinline__ float balance_over(const RouteGradArgs& p, int64_t n) {
    return (float)p.E / ((float)p.k * (float)n * (float)n);
}
// Sum over a block of up to 16 waves, in thread 0.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int i = 1; i < (int)blockDim.x / 64; i++) v += red[i];
    return v;
}

// One chunk of rows: for each sequence in it, the probabilities' sums and the counts go to slot chunk +
// sequence of the workspace: both only grow along the rows, so no two pairs share one.  A thread keeps
// the sums of its experts; rows of the block's waves are added in a fixed order.  Where one block takes all
// rows (p.mass is null) it leaves the losses and counts, those of empty sequences among them.
template <int L, int NV, bool F32, bool SIG, bool WIDE>
__global__ __launch_bounds__(64 * BAL_WAVES) void balance_kernel(const RouteGradArgs p) {
    constexpr int R = 64 / L, ROWS = BAL_WAVES * R, N = 4 * NV;  // rows of a wave and of the block at a time
    __shared__ float sums[BAL_WAVES][4 * L * NV];
    __shared__ int32_t count[4 * L * NV];
    __shared__ float red[BAL_WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane % L, mine = wave * R + lane / L;
    const int64_t begin = (int64_t)blockIdx.x * p.rows;
    const int64_t end = begin + p.rows < p.T ? begin + p.rows : p.T;
    int64_t r0 = begin;
    Logits<L, NV, F32, WIDE> cur, next;  // a row's loads go out while the one before it is worked on
    if (r0 + mine < end) cur.load(p, r0 + mine, j);
    const int64_t id_at = begin * p.k + threadIdx.x;
    const int first_id = id_at < end * p.k ? p.ids[id_at] : -1;
    const Ends ends(p);
    const bool small = p.mass == nullptr;
    for (int s = small ? 0 : ends.of(begin); s < p.S && (small || r0 < end); s++) {
        const int64_t e1 = ends.end(s), r1 = e1 < end ? e1 : end;
        if (r1 <= r0) {
            if (small) {
                for (int e = threadIdx.x; e < p.E; e += 64 * BAL_WAVES) p.counts[(int64_t)s * p.E + e] = 0;
                if (threadIdx.x == 0) p.loss[s] = 0.0f;
            } else {  // on past all that are empty, and never back, whatever the ends say
                const int at = ends.of(r0) - 1;
                s = at > s ? at : s;
            }
            continue;
        }
        for (int i = threadIdx.x; i < p.E; i += 64 * BAL_WAVES) count[i] = 0;
        __syncthreads();
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; i++) acc[i] = 0.0f;
        if (r0 != begin && r0 + mine < r1) cur.load(p, r0 + mine, j);
        for (int64_t r = r0 + mine; r < r1; r += ROWS) {
            next.load(p, r + ROWS < r1 ? r + ROWS : r, j);
            float l[N], t[N], slope[N], a, b;
            cur.get(l);
            scores_of<L, SIG>(l, t, slope, a, b);
#pragma unroll
            for (int i = 0; i < N; i++) acc[i] += t[i] * a;
            cur = next;
        }
        for (int64_t i = id_at; i < r1 * p.k; i += 64 * BAL_WAVES) {
            if (i < r0 * p.k) continue;
            const int e = i == id_at ? first_id : p.ids[i];
            if (e >= 0 && e < p.E) atomicAdd(&count[e], 1);  // whole numbers: any order
        }
#pragma unroll
        for (int i = 0; i < N; i++) acc[i] = over_rows<L>(acc[i]);
        if (lane < L)
#pragma unroll
            for (int i = 0; i < N; i++) sums[wave][4 * (j + L * (i / 4)) + i % 4] = acc[i];
        __syncthreads();
        const int64_t slot = (int64_t)blockIdx.x + s;
        float loss = 0.0f;
        for (int e = threadIdx.x; e < p.E; e += 64 * BAL_WAVES) {
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < BAL_WAVES; i++) a += sums[i][e];
            if (small) {
                p.counts[(int64_t)s * p.E + e] = count[e];
                loss += (float)count[e] * a;
            } else {
                p.mass[slot * p.E + e] = a;
                p.part[slot * p.E + e] = count[e];
            }
        }
        if (small) {
            loss = block_sum(loss, red);
            if (threadIdx.x == 0) p.loss[s] = loss * balance_over(p, r1 - r0);
        }
        __syncthreads();
        r0 = r1;
    }
}

// A sequence's loss and counts from its chunks: a block per sequence; C threads take an expert each, up to
// 16 rows of them the chunks in turn.  With p.group_sums a block per sequence and C experts, whose parts of the
// loss are added by a third launch: one block alone reads 130 GB/s.
__global__ __launch_bounds__(1024) void balance_join_kernel(const RouteGradArgs p, int C) {
    __shared__ float mass[1024], red[16];
    __shared__ int32_t count[1024];
    const int s = blockIdx.x, e = blockIdx.y * C + (threadIdx.x & (C - 1)), row = threadIdx.x / C, rows = blockDim.x / C;
    const Ends ends(p);
    const int64_t a = ends.end(s - 1), b = ends.end(s), n = b - a;
    float m = 0.0f;
    int32_t k = 0;
    if (n > 0 && e < p.E) {
        const int64_t last = (b - 1) / p.rows;
#pragma unroll 8
        for (int64_t c = a / p.rows + row; c <= last; c += rows) {
            m += p.mass[(c + s) * p.E + e];
            k += p.part[(c + s) * p.E + e];
        }
    }
    mass[threadIdx.x] = m;
    count[threadIdx.x] = k;
    __syncthreads();
    float sum = 0.0f;
    if (row == 0 && e < p.E) {
        for (int i = 1; i < rows; i++) {
            m += mass[i * C + threadIdx.x];
            k += count[i * C + threadIdx.x];
        }
        p.counts[(int64_t)s * p.E + e] = k;
        sum = (float)k * m;
    }
    sum = block_sum(sum, red);
    if (threadIdx.x != 0) return;
    if (p.group_sums) p.group_sums[(int64_t)s * gridDim.y + blockIdx.y] = sum;
    else p.loss[s] = n > 0 ? sum * balance_over(p, n) : 0.0f;
}

// The losses from the groups' parts: a wave a sequence.
__global__ __launch_bounds__(64) void balance_loss_kernel(const RouteGradArgs p, int groups) {
    const int s = blockIdx.x;
    const Ends ends(p);
    const int64_t n = ends.end(s) - ends.end(s - 1);
    float sum = (int)threadIdx.x < groups ? p.group_sums[(int64_t)s * groups + threadIdx.x] : 0.0f;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (threadIdx.x == 0) p.loss[s] = n > 0 ? sum * balance_over(p, n) : 0.0f;
}

// Lanes of a wave see what others of it have written to LDS.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// p.rows rows of a block.  What the chosen experts' weights add goes through LDS: a row's scores are read
// there by its choices, and each choice leaves its part at its expert's place.  (Comparing each choice with
// each expert in registers: 52 us where this takes 30, 65536 x 256, 8 of them.)  Where an expert is named
// twice for a token, which a choice learns by not finding its own number at the place, the lane that holds
// the expert adds its parts in the order of the choices.
template <int L, int NV, bool F32, bool SIG, bool WIDE>
__global__ __launch_bounds__(256) void route_back_kernel(const RouteGradArgs p) {
    constexpr int R = 64 / L, ROWS = 4 * R, N = 4 * NV;
    __shared__ float4 lds[2][4][R][NV][L];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane % L;
    float4(*scores)[L] = lds[0][wave][lane / L];
    float4(*parts)[L] = lds[1][wave][lane / L];
    float* score = reinterpret_cast<float*>(scores);  // expert e's at score[e]
    float* part = reinterpret_cast<float*>(parts);
    int32_t* tag = reinterpret_cast<int32_t*>(parts);
    const int64_t begin = (int64_t)blockIdx.x * p.rows;
    const int64_t end = begin + p.rows < p.T ? begin + p.rows : p.T;
    const Ends ends(p);
    int s = p.dloss ? ends.of(begin + wave * R) - 1 : p.S;
    int64_t seq_last = -1;  // end of sequence s
    float dp[N];
#pragma unroll
    for (int i = 0; i < N; i++) dp[i] = 0.0f;
    for (int64_t r0 = begin; r0 < end; r0 += ROWS) {
        const int64_t r = r0 + wave * R + lane / L;
        const int64_t row = r < p.T ? r : p.T - 1;  // the lanes of a wave stay together
        Logits<L, NV, F32, WIDE> raw;
        raw.load(p, row, j);
        const int32_t* ids = p.ids + row * p.k;
        const float* dw = p.dweights + row * p.k;
        const auto expert = [&](int c) {  // of choice c, E for none
            const int id = ids[c];
            return id >= 0 && id < p.E ? id : p.E;
        };
        int first = p.E;  // the lane's first choice and its weight's gradient
        float first_dw = 0.0f;
        if (p.dweights && j < p.k) {
            first = expert(j);
            first_dw = dw[j];
        }
        const auto choices = [&](auto&& f) {  // the lane's: number, expert, gradient
            if (first < p.E) f(j, first, first_dw);
            for (int c = j + L; c < p.k; c += L) {
                const int e = expert(c);
                if (e < p.E) f(c, e, dw[c]);
            }
        };
        // the row's sequence, and what its loss gives each expert
        bool ahead = s < p.S && row >= seq_last, other = ahead;
        int64_t seq_first = 0;
        for (int turn = 0; __any(ahead); turn++) {  // a few steps, then by halves
            if (ahead) s = turn < 4 || p.S <= 64 ? s + 1 : ends.after(s, row);
            const int at = s < p.S ? s : p.S - 1;
            const int64_t from = ends.end(at - 1), to = ends.end(at);
            if (ahead) {
                seq_first = from;
                seq_last = to;
            }
            ahead = ahead && s < p.S && row >= seq_last;
        }
        if (other) {
            const float over = s < p.S ? p.dloss[s] * balance_over(p, seq_last - seq_first) : 0.0f;
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int e = 4 * (j + L * v) + i;
                    dp[4 * v + i] = s < p.S && e < p.E ? over * (float)p.counts[(int64_t)s * p.E + e] : 0.0f;
                }
        }
        float t[N], slope[N], a, b;
        {
            float l[N];
            raw.get(l);
            scores_of<L, SIG>(l, t, slope, a, b);
        }
        float mean = 0.0f;  // of dp over p
        if (p.dloss) {
#pragma unroll
            for (int i = 0; i < N; i++) mean += t[i] * dp[i];
            mean = row_sum<L>(mean) * a;
        }
        float x[N], all = 0.0f;  // what the weights add: slope (x - t all)
        if (p.dweights) {
            wave_sync();
#pragma unroll
            for (int v = 0; v < NV; v++) {
                scores[v][j] = make_float4(t[4 * v], t[4 * v + 1], t[4 * v + 2], t[4 * v + 3]);
                parts[v][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            wave_sync();
            float total = 0.0f, dot = 0.0f;
            choices([&](int c, int e, float g) {
                const float v = score[e];
                total += v;
                dot += v * g;
                tag[e] = c;
            });
            total = row_sum<L>(total);
            dot = row_sum<L>(dot);
            float by = p.scale * b;
            if (!p.renorm) {
                if (!SIG) all = by * b * dot;  // a softmax's scores hang together
                dot = 0.0f;
            } else if (total >= kTinyScores || total != total) {
                by = p.scale / total;
                dot /= total;
            } else {  // the weights are a softmax of the chosen logits alone
                const auto logit = [&](int e) {
                    const int64_t at = row * p.ld_l + e;
                    return F32 ? static_cast<const float*>(p.logits)[at] : rg_bf16(static_cast<const uint16_t*>(p.logits)[at]);
                };
                float m = -INFINITY;
                choices([&](int, int e, float) { m = fmaxf(m, logit(e)); });
                m = row_max<L>(m);
                m = m == -INFINITY ? 0.0f : m;
                total = dot = 0.0f;
                choices([&](int, int e, float g) {
                    const float v = exp_neg(logit(e) - m);
                    score[e] = v;
                    total += v;
                    dot += v * g;
                });
                total = row_sum<L>(total);
                dot = row_sum<L>(dot);
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                by = p.scale * inv;
                dot *= inv;
            }
            wave_sync();
            bool twice = false;
            choices([&](int c, int e, float) { twice = twice || tag[e] != c; });
            twice = __any(twice);
            wave_sync();
            if (!twice) {
                choices([&](int, int e, float g) { part[e] = score[e] * by * (g - dot); });
            } else {
#pragma unroll
                for (int v = 0; v < NV; v++) parts[v][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                wave_sync();
                for (int c = 0; c < p.k; c++) {
                    const int e = expert(c);
                    if (e < p.E && (e >> 2) % L == j) part[e] += score[e] * by * (dw[c] - dot);
                }
            }
            wave_sync();
        }
#pragma unroll
        for (int v = 0; v < NV; v++) {
            float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (p.dweights) w = parts[v][j];
            x[4 * v] = w.x; x[4 * v + 1] = w.y; x[4 * v + 2] = w.z; x[4 * v + 3] = w.w;
        }
        if (r >= end) continue;
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int e = 4 * (j + L * v);
            if (e >= p.E) continue;
            float d[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int k = 4 * v + i;
                d[i] = t[k] * (a * (dp[k] - mean) - all) + x[k];
                if (SIG) d[i] *= slope[k];
            }
            if (F32) {
                float* dst = static_cast<float*>(p.dlogits) + r * p.ld_d + e;
                if (WIDE) {
                    *reinterpret_cast<float4*>(dst) = make_float4(d[0], d[1], d[2], d[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (e + i < p.E) dst[i] = d[i];
                }
            } else {
                uint16_t* dst = static_cast<uint16_t*>(p.dlogits) + r * p.ld_d + e;
                if (WIDE) {
                    *reinterpret_cast<uint2*>(dst) = make_uint2(rg_pack(d[0], d[1]), rg_pack(d[2], d[3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (e + i < p.E) dst[i] = (uint16_t)rg_pack(d[i], 0.0f);
                }
            }
        }
    }
}

template <int L, int NV, bool F32, bool SIG>
static void launch_route_grad(RouteGradArgs& p, bool back, hipStream_t stream) {
    constexpr int ROWS = 4 * (64 / L);
    // four blocks of the gradient for each of 256 CUs: as many as these hold at once of sigmoids with 16 experts a
    // lane (115 to 126 registers; 65536 x 256 bf16 sigmoid, on one input: 25.2 us; 512 blocks 28.4, 768 29.2, 2048
    // 28.3).  A softmax's (81 to 95) would fit five, few experts' (54 to 77) six to eight: not measured apart.
    constexpr int64_t AT_ONCE = 1024 * ROWS;
    if (back) p.rows = p.T <= AT_ONCE ? ROWS : (p.T + AT_ONCE - 1) / AT_ONCE * ROWS;
    const unsigned blocks = (unsigned)((p.T + p.rows - 1) / p.rows);
    if (back && p.wide) route_back_kernel<L, NV, F32, SIG, true><<<dim3(blocks), dim3(256), 0, stream>>>(p);
    else if (back) route_back_kernel<L, NV, F32, SIG, false><<<dim3(blocks), dim3(256), 0, stream>>>(p);
    else if (p.wide) balance_kernel<L, NV, F32, SIG, true><<<dim3(blocks), dim3(64 * BAL_WAVES), 0, stream>>>(p);
    else balance_kernel<L, NV, F32, SIG, false><<<dim3(blocks), dim3(64 * BAL_WAVES), 0, stream>>>(p);
}

template <bool F32, bool SIG>
static void pick_route_grad(RouteGradArgs& p, bool back, hipStream_t stream) {
    switch (route_lanes(p.E)) {
        case 1:
            if (p.E <= 4) launch_route_grad<1, 1, F32, SIG>(p, back, stream);
            else if (p.E <= 8) launch_route_grad<1, 2, F32, SIG>(p, back, stream);
            else launch_route_grad<1, 4, F32, SIG>(p, back, stream);
            break;
        case 2: launch_route_grad<2, 4, F32, SIG>(p, back, stream); break;
        case 4: launch_route_grad<4, 4, F32, SIG>(p, back, stream); break;
        case 8: launch_route_grad<8, 4, F32, SIG>(p, back, stream); break;
        case 16: launch_route_grad<16, 4, F32, SIG>(p, back, stream); break;
        case 32: launch_route_grad<32, 4, F32, SIG>(p, back, stream); break;
        default: launch_route_grad<64, 4, F32, SIG>(p, back, stream); break;
    }
}

static void start_route_grad(RouteGradArgs& p, bool f32, bool back, hipStream_t stream) {
    if (f32 && p.sigmoid) pick_route_grad<true, true>(p, back, stream);
    else if (f32) pick_route_grad<true, false>(p, back, stream);
    else if (p.sigmoid) pick_route_grad<false, true>(p, back, stream);
    else pick_route_grad<false, false>(p, back, stream);
}

static inline bool rg_wide(const void* p, int64_t ld, int64_t E, bool f32) {
    return E % 4 == 0 && ld % 4 == 0 && fp8q_aligned(p, f32 ? 16 : 8);
}

}  // namespace fp8q

extern "C" size_t moe_balance_workspace_size(int64_t T, int64_t E, int32_t sequences) {
    if (T <= 0 || E <= 0 || sequences <= 0 || fp8q::balance_is_small(T, E, sequences)) return 0;
    return (size_t)fp8q::balance_space(T, E, sequences);
}

extern "C" fp8q_status_t moe_balance(const void* logits, fp8q_out_t logits_dtype, int64_t T, int64_t E, int64_t ld_l,
                                     fp8q_scoring_t scoring, const int32_t* ids, int32_t top_k, const int32_t* sequences,
                                     int32_t S, float* loss, int32_t* counts, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream) {
    using namespace fp8q;
    const bool f32 = logits_dtype == FP8Q_OUT_FP32;
    if (T < 0 || E < 1 || ld_l < E || top_k < 1 || S < 1 || (!sequences && S != 1) || (!f32 && logits_dtype != FP8Q_OUT_BF16) ||
        (scoring != FP8Q_SCORE_SOFTMAX && scoring != FP8Q_SCORE_SIGMOID) || !loss || !counts || (T > 0 && (!logits || !ids)))
        return FP8Q_ERR_INVALID_ARG;
    if (E > RG_MAX_E || top_k > RG_MAX_K || T > 0x7FFFFFFFLL || S >= 1 << 22) return FP8Q_ERR_UNSUPPORTED;
    const bool small = T == 0 || balance_is_small(T, E, S);  // neither takes a workspace
    if (!small && (!workspace || workspace_bytes < moe_balance_workspace_size(T, E, S))) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 16)) return FP8Q_ERR_INVALID_ARG;
    RouteGradArgs p{};
    p.logits = logits; p.T = T; p.ld_l = ld_l; p.ids = ids; p.sequences = sequences; p.loss = loss; p.counts = counts;
    p.rows = balance_rows(T, E);
    if (!small) {
        p.mass = static_cast<float*>(workspace);
        p.part = reinterpret_cast<int32_t*>(p.mass + balance_slots(T, E, S) * E);
    }
    p.E = (int)E; p.k = top_k; p.S = S; p.sigmoid = scoring == FP8Q_SCORE_SIGMOID; p.wide = rg_wide(logits, ld_l, E, f32);
    if (T > 0) {
        start_route_grad(p, f32, false, stream);
        FP8Q_CHECK_LAUNCH();
        if (small) return FP8Q_OK;
    }
    const int groups = balance_groups(T, E, S);
    if (!small && groups > 1) {
        p.group_sums = reinterpret_cast<float*>(p.part + balance_slots(T, E, S) * E);
        balance_join_kernel<<<dim3((unsigned)S, (unsigned)groups), dim3(1024), 0, stream>>>(p, BAL_GROUP);
        FP8Q_CHECK_LAUNCH();
        balance_loss_kernel<<<dim3((unsigned)S), dim3(64), 0, stream>>>(p, groups);
    } else {
        int C = 4;
        while (C < E) C *= 2;
        balance_join_kernel<<<dim3((unsigned)S), dim3(C < 64 ? 16 * C : 1024), 0, stream>>>(p, C);
    }
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

extern "C" fp8q_status_t moe_route_backward(const void* logits, fp8q_out_t logits_dtype, int64_t T, int64_t E, int64_t ld_l,
                                            fp8q_scoring_t scoring, const int32_t* ids, int32_t top_k, const float* dweights,
                                            int renormalize, float scale, const float* dloss, const int32_t* counts,
                                            const int32_t* sequences, int32_t S, void* dlogits, int64_t ld_d,
                                            hipStream_t stream) {
    using namespace fp8q;
    const bool f32 = logits_dtype == FP8Q_OUT_FP32;
    if (T < 0 || E < 1 || ld_l < E || ld_d < E || top_k < 1 || (!f32 && logits_dtype != FP8Q_OUT_BF16) ||
        (scoring != FP8Q_SCORE_SOFTMAX && scoring != FP8Q_SCORE_SIGMOID))
        return FP8Q_ERR_INVALID_ARG;
    if (dloss && (!counts || S < 1 || (!sequences && S != 1))) return FP8Q_ERR_INVALID_ARG;
    if (T == 0) return FP8Q_OK;
    if (!logits || !ids || !dlogits || (dlogits == logits && ld_d != ld_l)) return FP8Q_ERR_INVALID_ARG;
    if (E > RG_MAX_E || top_k > RG_MAX_K || T > 0x7FFFFFFFLL || (dloss && S >= 1 << 22)) return FP8Q_ERR_UNSUPPORTED;
    RouteGradArgs p{};
    p.logits = logits; p.T = T; p.ld_l = ld_l; p.ids = ids; p.dweights = dweights; p.renorm = renormalize != 0; p.scale = scale;
    p.dlogits = dlogits; p.ld_d = ld_d;
    if (dloss) {  // else none of them is looked at
        p.dloss = dloss; p.counts = const_cast<int32_t*>(counts); p.sequences = sequences; p.S = S;
    }
    p.E = (int)E; p.k = top_k; p.sigmoid = scoring == FP8Q_SCORE_SIGMOID;
    p.wide = rg_wide(logits, ld_l, E, f32) && rg_wide(dlogits, ld_d, E, f32);
    start_route_grad(p, f32, true, stream);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}
