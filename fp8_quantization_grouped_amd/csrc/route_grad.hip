// What a router's training needs beside the choice (moe_route): the balance loss with the experts' counts,
// and the gradient of the logits from that loss and from the chosen weights.
//
//   p[t,e]  = softmax(l)[e], or sigmoid(l[e]) / sum of the row's sigmoids
//   loss[s] = E / (k n^2) * sum_e count[s,e] * sum_{t in s} p[t,e]        (n tokens in sequence s)
//   dl      = p slope (dp - sum_e p dp),  dp[e] = dloss[s] E / (k n^2) count[s,e]
//           + the chosen weights' part;  slope = 1 (softmax) or 1 - sigmoid(l), of log(score) over l
//
// Bound: HBM for large T * E, launches below.
#include "common.hpp"

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
    int64_t rows;                // of a chunk
    int E, k, S;
    bool sigmoid, renorm, wide;  // wide: rows start on whole vectors of 4, and E is a multiple of 4
    float scale;
};

__device__ __forceinline__ float rg_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t rg_to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);  // NaN stays NaN
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// Sums and maxima over the L lanes that share a row.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
template <int L>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

// End of sequence s, inside [0, T] whatever is stored.
__device__ __forceinline__ int64_t seq_end(const RouteGradArgs& p, int s) {
    if (!p.sequences) return p.T;
    const int64_t e = p.sequences[s];
    return e < 0 ? 0 : e > p.T ? p.T : e;
}
// Sequence of row r: the first whose end lies behind it, S for rows behind the last.
__device__ __forceinline__ int seq_of(const RouteGradArgs& p, int64_t r) {
    if (!p.sequences) return 0;
    int lo = 0, hi = p.S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)p.sequences[mid] > r) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// A row's logits: L lanes with 4 * NV experts each, lane j's at 4 (j + L v) .. + 3; minus infinity past E.
template <int L, int NV, bool WIDE32>
__device__ __forceinline__ void load_logits(const RouteGradArgs& p, int64_t r, int j, float (&l)[4 * NV]) {
#pragma unroll
    for (int v = 0; v < NV; v++) {
        const int e = 4 * (j + L * v);
#pragma unroll
        for (int i = 0; i < 4; i++) l[4 * v + i] = -INFINITY;
        if (e >= p.E) continue;
        if (WIDE32) {
            const float* src = static_cast<const float*>(p.logits) + r * p.ld_l + e;
            if (p.wide) {
                const float4 w = *reinterpret_cast<const float4*>(src);
                l[4 * v] = w.x; l[4 * v + 1] = w.y; l[4 * v + 2] = w.z; l[4 * v + 3] = w.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (e + i < p.E) l[4 * v + i] = src[i];
            }
        } else {
            const uint16_t* src = static_cast<const uint16_t*>(p.logits) + r * p.ld_l + e;
            if (p.wide) {
                const uint2 w = *reinterpret_cast<const uint2*>(src);
                l[4 * v] = bf16_lo(w.x); l[4 * v + 1] = bf16_hi(w.x); l[4 * v + 2] = bf16_lo(w.y); l[4 * v + 3] = bf16_hi(w.y);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (e + i < p.E) l[4 * v + i] = rg_bf16(src[i]);
            }
        }
    }
}

// Scores under this sum are formed from the logits less their maximum: sigmoids of logits so far below
// zero are their exponentials, and a softmax's scores have the exponentials' ratios.
constexpr float kTinyScores = 5.421010862427522e-20f;  // 2^-64

template <int L, int N>
__device__ __forceinline__ void softmax_of(const float (&l)[N], float (&out)[N]) {
    float m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) m = fmaxf(m, l[i]);
    m = row_max<L>(m);
    m = m == -INFINITY ? 0.0f : m;  // every logit at minus infinity: no probabilities
#pragma unroll
    for (int i = 0; i < N; i++) {
        out[i] = expf(l[i] - m);
        sum += out[i];
    }
    sum = row_sum<L>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < N; i++) out[i] *= inv;
}

// Probabilities p, and the scores s and slopes of log(s) that the chosen weights are made of.
template <int L, int N>
__device__ __forceinline__ void scores_of(bool sigmoid, const float (&l)[N], float (&p)[N], float (&s)[N], float (&slope)[N]) {
    if (!sigmoid) {
        softmax_of<L>(l, p);
#pragma unroll
        for (int i = 0; i < N; i++) {
            s[i] = p[i];
            slope[i] = 1.0f;
        }
        return;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float u = expf(-fabsf(l[i])), one = 1.0f / (1.0f + u), rest = u * one;  // neither end overflows or cancels
        s[i] = l[i] > 0.0f ? one : rest;
        slope[i] = l[i] > 0.0f ? rest : one;
        sum += s[i];
    }
    sum = row_sum<L>(sum);
    if (sum < kTinyScores) {
        softmax_of<L>(l, p);
    } else {
        const float inv = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < N; i++) p[i] = s[i] * inv;
    }
}

// One chunk of rows: for each sequence in it, the probabilities' sums and the counts go to slot chunk +
// sequence of the workspace: both only grow along the rows, so no two pairs share one.  A thread keeps
// the sums of its experts; rows of the block's waves are added in a fixed order.
template <int L, int NV, bool WIDE32>
__global__ __launch_bounds__(256) void balance_kernel(const RouteGradArgs p) {
    constexpr int R = 64 / L, ROWS = 4 * R, N = 4 * NV;  // rows of a wave and of the block at a time
    extern __shared__ float lds[];
    float* sums = lds;                                           // [ROWS][E]
    int32_t* count = reinterpret_cast<int32_t*>(lds + ROWS * p.E);  // [E]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane % L, mine = wave * R + lane / L;
    const int64_t begin = (int64_t)blockIdx.x * p.rows;
    const int64_t end = begin + p.rows < p.T ? begin + p.rows : p.T;
    int64_t r0 = begin;
    for (int s = seq_of(p, begin); s < p.S && r0 < end; s++) {
        const int64_t e1 = seq_end(p, s), r1 = e1 < end ? e1 : end;
        if (r1 <= r0) continue;
        for (int i = threadIdx.x; i < p.E; i += 256) count[i] = 0;
        __syncthreads();
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; i++) acc[i] = 0.0f;
        for (int64_t r = r0 + mine; r < r1; r += ROWS) {
            float l[N], q[N], sc[N], sl[N];
            load_logits<L, NV, WIDE32>(p, r, j, l);
            scores_of<L>(p.sigmoid, l, q, sc, sl);
#pragma unroll
            for (int i = 0; i < N; i++) acc[i] += q[i];
        }
        for (int64_t i = r0 * p.k + threadIdx.x; i < r1 * p.k; i += 256) {
            const int e = p.ids[i];
            if (e >= 0 && e < p.E) atomicAdd(&count[e], 1);  // whole numbers: any order
        }
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int e = 4 * (j + L * v) + i;
                if (e < p.E) sums[mine * p.E + e] = acc[4 * v + i];
            }
        __syncthreads();
        const int64_t slot = (int64_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < p.E; e += 256) {
            float a = 0.0f;
            for (int i = 0; i < ROWS; i++) a += sums[i * p.E + e];
            p.mass[slot * p.E + e] = a;
            p.part[slot * p.E + e] = count[e];
        }
        __syncthreads();
        r0 = r1;
    }
}

// A sequence's loss and counts from its chunks: a block per sequence, a thread an expert at a time.
__global__ __launch_bounds__(256) void balance_join_kernel(const RouteGradArgs p) {
    __shared__ float red[4];
    const int s = blockIdx.x;
    const int64_t a = s == 0 ? 0 : seq_end(p, s - 1), b = seq_end(p, s), n = b - a;
    float sum = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += 256) {
        float mass = 0.0f;
        int32_t count = 0;
        if (n > 0)
            for (int64_t c = a / p.rows; c <= (b - 1) / p.rows; c++) {
                mass += p.mass[(c + s) * p.E + e];
                count += p.part[(c + s) * p.E + e];
            }
        p.counts[(int64_t)s * p.E + e] = count;
        sum += (float)count * mass;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = (red[0] + red[1]) + (red[2] + red[3]);
        p.loss[s] = n > 0 ? sum * ((float)p.E / ((float)p.k * (float)n * (float)n)) : 0.0f;
    }
}

template <int L, int NV, bool WIDE32>
__global__ __launch_bounds__(256) void route_back_kernel(const RouteGradArgs p) {
    constexpr int R = 64 / L, ROWS = 4 * R, N = 4 * NV;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane % L;
    const int64_t r = (int64_t)blockIdx.x * ROWS + wave * R + lane / L;
    const int64_t row = r < p.T ? r : p.T - 1;  // the lanes of a wave stay together
    float l[N], q[N], sc[N], sl[N], dl[N];
    load_logits<L, NV, WIDE32>(p, row, j, l);
    scores_of<L>(p.sigmoid, l, q, sc, sl);
#pragma unroll
    for (int i = 0; i < N; i++) dl[i] = 0.0f;
    const int s = seq_of(p, row);
    if (p.dloss && s < p.S) {
        const float n = (float)(seq_end(p, s) - (s == 0 ? 0 : seq_end(p, s - 1)));
        const float over = p.dloss[s] * ((float)p.E / ((float)p.k * n * n));
        float dp[N], dot = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int e = 4 * (j + L * v) + i;
                dp[4 * v + i] = e < p.E ? over * (float)p.counts[(int64_t)s * p.E + e] : 0.0f;
                dot += q[4 * v + i] * dp[4 * v + i];
            }
        dot = row_sum<L>(dot);
#pragma unroll
        for (int i = 0; i < N; i++) dl[i] = q[i] * sl[i] * (dp[i] - dot);
    }
    if (p.dweights) {
        float times[N], dw[N];  // how often an expert is chosen, and its weights' gradients
#pragma unroll
        for (int i = 0; i < N; i++) times[i] = dw[i] = 0.0f;
        for (int c = 0; c < p.k; c++) {
            const int id = p.ids[row * p.k + c];
            const float g = p.dweights[row * p.k + c];
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const bool hit = id == 4 * (j + L * v) + i;
                    times[4 * v + i] += hit ? 1.0f : 0.0f;
                    dw[4 * v + i] += hit ? g : 0.0f;
                }
        }
        if (p.renorm) {
            float total = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < N; i++) total += times[i] * sc[i];
            total = row_sum<L>(total);
            if (total < kTinyScores) {  // the weights are a softmax of the chosen logits alone
                float m = -INFINITY;
#pragma unroll
                for (int i = 0; i < N; i++) m = times[i] > 0.0f ? fmaxf(m, l[i]) : m;
                m = row_max<L>(m);
                total = 0.0f;
#pragma unroll
                for (int i = 0; i < N; i++) {
                    sc[i] = times[i] > 0.0f && m > -INFINITY ? expf(l[i] - m) : 0.0f;
                    total += times[i] * sc[i];
                }
                total = row_sum<L>(total);
            }
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
            for (int i = 0; i < N; i++) dot += dw[i] * (sc[i] * inv);
            dot = row_sum<L>(dot);
#pragma unroll
            for (int i = 0; i < N; i++)
                if (times[i] > 0.0f) dl[i] += p.scale * (sc[i] * inv) * sl[i] * (dw[i] - times[i] * dot);
        } else if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < N; i++) dl[i] += p.scale * sc[i] * sl[i] * dw[i];
        } else {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < N; i++) dot += q[i] * dw[i];
            dot = row_sum<L>(dot);
#pragma unroll
            for (int i = 0; i < N; i++) dl[i] += p.scale * q[i] * (dw[i] - dot);
        }
    }
    if (r >= p.T) return;
#pragma unroll
    for (int v = 0; v < NV; v++) {
        const int e = 4 * (j + L * v);
        if (e >= p.E) continue;
        const float* d = &dl[4 * v];
        if (WIDE32) {
            float* dst = static_cast<float*>(p.dlogits) + r * p.ld_d + e;
            if (p.wide) {
                *reinterpret_cast<float4*>(dst) = make_float4(d[0], d[1], d[2], d[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (e + i < p.E) dst[i] = d[i];
            }
        } else {
            uint16_t* dst = static_cast<uint16_t*>(p.dlogits) + r * p.ld_d + e;
            if (p.wide) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(rg_to_bf16(d[0]) | (uint32_t)rg_to_bf16(d[1]) << 16,
                                                            rg_to_bf16(d[2]) | (uint32_t)rg_to_bf16(d[3]) << 16);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (e + i < p.E) dst[i] = rg_to_bf16(d[i]);
            }
        }
    }
}

// Rows of a chunk: enough for a block's waves several times over, at most 512 chunks.
static inline int64_t balance_rows(int64_t T) {
    const int64_t r = (T + 511) / 512;
    return r < 16 ? 16 : r;
}
static inline int64_t balance_slots(int64_t T, int64_t S) { return (T + balance_rows(T) - 1) / balance_rows(T) + S; }

template <int L, int NV, bool WIDE32>
static void launch_route_grad(const RouteGradArgs& p, bool back, hipStream_t stream) {
    constexpr int ROWS = 4 * (64 / L);
    if (back) {
        route_back_kernel<L, NV, WIDE32><<<dim3((unsigned)((p.T + ROWS - 1) / ROWS)), dim3(256), 0, stream>>>(p);
    } else {
        const unsigned blocks = (unsigned)((p.T + p.rows - 1) / p.rows);
        balance_kernel<L, NV, WIDE32><<<dim3(blocks), dim3(256), (size_t)(ROWS + 1) * p.E * 4, stream>>>(p);
    }
}

// Lanes of a row by the number of experts, 4 to a lane.
template <bool WIDE32>
static void pick_route_grad(const RouteGradArgs& p, bool back, hipStream_t stream) {
    if (p.E <= 4) launch_route_grad<1, 1, WIDE32>(p, back, stream);
    else if (p.E <= 8) launch_route_grad<2, 1, WIDE32>(p, back, stream);
    else if (p.E <= 16) launch_route_grad<4, 1, WIDE32>(p, back, stream);
    else if (p.E <= 32) launch_route_grad<8, 1, WIDE32>(p, back, stream);
    else if (p.E <= 64) launch_route_grad<16, 1, WIDE32>(p, back, stream);
    else if (p.E <= 128) launch_route_grad<32, 1, WIDE32>(p, back, stream);
    else if (p.E <= 256) launch_route_grad<64, 1, WIDE32>(p, back, stream);
    else if (p.E <= 512) launch_route_grad<64, 2, WIDE32>(p, back, stream);
    else launch_route_grad<64, 4, WIDE32>(p, back, stream);
}

static inline bool rg_wide(const void* p, int64_t ld, int64_t E, bool f32) {
    return E % 4 == 0 && ld % 4 == 0 && fp8q_aligned(p, f32 ? 16 : 8);
}

}  // namespace fp8q

extern "C" size_t moe_balance_workspace_size(int64_t T, int64_t E, int32_t sequences) {
    if (T <= 0 || E <= 0 || sequences <= 0) return 256;
    return (size_t)fp8q::balance_slots(T, sequences) * (size_t)E * 8;
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
    if (E > RG_MAX_E || top_k > RG_MAX_K || T > 0x7FFFFFFFLL) return FP8Q_ERR_UNSUPPORTED;
    if (T > 0 && (!workspace || workspace_bytes < moe_balance_workspace_size(T, E, S))) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 16)) return FP8Q_ERR_INVALID_ARG;
    RouteGradArgs p{};
    p.logits = logits; p.T = T; p.ld_l = ld_l; p.ids = ids; p.sequences = sequences; p.loss = loss; p.counts = counts;
    p.rows = balance_rows(T);
    p.mass = static_cast<float*>(workspace);
    p.part = reinterpret_cast<int32_t*>(p.mass + balance_slots(T, S) * E);
    p.E = (int)E; p.k = top_k; p.S = S; p.sigmoid = scoring == FP8Q_SCORE_SIGMOID; p.wide = rg_wide(logits, ld_l, E, f32);
    if (T > 0) {
        if (f32) pick_route_grad<true>(p, false, stream);
        else pick_route_grad<false>(p, false, stream);
        FP8Q_CHECK_LAUNCH();
    }
    balance_join_kernel<<<dim3((unsigned)S), dim3(256), 0, stream>>>(p);
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
    if (E > RG_MAX_E || top_k > RG_MAX_K || T > 0x7FFFFFFFLL) return FP8Q_ERR_UNSUPPORTED;
    RouteGradArgs p{};
    p.logits = logits; p.T = T; p.ld_l = ld_l; p.ids = ids; p.dweights = dweights; p.renorm = renormalize != 0; p.scale = scale;
    p.dloss = dloss; p.counts = const_cast<int32_t*>(counts); p.sequences = sequences; p.S = S; p.dlogits = dlogits; p.ld_d = ld_d;
    p.E = (int)E; p.k = top_k; p.sigmoid = scoring == FP8Q_SCORE_SIGMOID;
    p.wide = rg_wide(logits, ld_l, E, f32) && rg_wide(dlogits, ld_d, E, f32);
    if (f32) pick_route_grad<true>(p, true, stream);
    else pick_route_grad<false>(p, true, stream);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}
