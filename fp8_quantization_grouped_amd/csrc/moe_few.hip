// A mixture-of-experts layer for a few tokens: routing, and the experts' SwiGLU feed-forward on
// block-scaled FP8 weights.
//
//   route    logits = x Wr^T, scores = softmax or sigmoid, the top_k of scores (+ bias), weights
//   experts  y[t] = sum_j w[t,j] W2_e ( silu(G_e x_t) * (U_e x_t) ),  e = ids[t,j]
//            ([G_e; U_e] = w13[e], 2 I x H; W2_e = w2[e], H x I; one fp32 factor per 128 x 128)
//
// Bound: HBM.  With few tokens every chosen expert's 3 H I weight bytes are read for a handful of
// multiplications each, so the kernels are built around streaming them once: no operand goes
// through LDS, a lane's 16-byte weight loads feed the matrix cores directly, and the activations
// (small, shared by all blocks) come from the caches.  The weights are widened to bf16 (exact) and
// multiply the bf16 activations as they are: nothing is quantized on the way, and the matrix
// cores, which would be idle otherwise, take up to 16 tokens for the price of one.
//
// Matrix instruction: 16 x 16 x 32 bf16.  Its A rows are tokens, its B rows are weight rows: lane l
// holds token or weight row l % 16, and its 8 k values may be any 8 as long as both operands agree.  Here
// lane group l / 16 of a 64-byte piece of a weight row takes bytes 16 (l / 16) .. + 15, one 16-byte
// load for two instructions.  Result register i of lane l is token 4 (l / 16) + i, weight row l % 16.
//
// Every sum has a fixed order: a block's waves split the contraction (gate and up) or the experts
// (down) the same way for the same sizes and ids, and are added in wave order.
#include "common.hpp"

namespace fp8q {

typedef float f4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

constexpr int MB = 128;           // weight factor block
constexpr int MOE_MAX_T = 128;    // tokens of one call
constexpr int MOE_MAX_E = 1024;   // experts
constexpr int MOE_MAX_K = 32;     // experts of one token

// 8 e4m3fn bytes as bf16 (exact: 4 significant bits, exponents -9 .. 8).
__device__ __forceinline__ bf8_t widen8(uint32_t a, uint32_t b) {
    const bf2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf2_t v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf2_t v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf2_t v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return bf8_t{v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}
__device__ __forceinline__ bf8_t as_bf8(uint4 v) { return __builtin_bit_cast(bf8_t, v); }
__device__ __forceinline__ f4_t mma(bf8_t a, bf8_t b, f4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ uint16_t to_bf16(float f) {
    uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);  // NaN stays NaN
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// ------------------------------------------------------------------------------------- routing

struct RouteArgs {
    const uint16_t* x;
    int64_t ld_x;
    const uint16_t* router;
    int64_t ld_r;
    const float* bias;
    float* part;       // [splits][T][E] partial logits
    int32_t* ids;
    float* weights;
    int T, E, H, top_k, splits, sigmoid, renorm;
    float scale;
};

// Partial logits of 16 tokens x 16 experts over one split of H; the block's 4 waves share the split.
__global__ __launch_bounds__(256) void route_logits_kernel(const RouteArgs p) {
    __shared__ f4_t red[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int e = blockIdx.x * 16 + r, t = blockIdx.z * 16 + r;
    const int chunks = (p.H + 31) / 32;                          // 32 k values of one instruction
    const int parts = p.splits * 4, me = blockIdx.y * 4 + wave;  // waves over H
    const int k0 = (int)((int64_t)chunks * me / parts), k1 = (int)((int64_t)chunks * (me + 1) / parts);
    f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kc = k0; kc < k1; kc++) {
        const int k = kc * 32 + 8 * g;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (k < p.H) {  // H is a multiple of 8
            if (t < p.T) a = *reinterpret_cast<const uint4*>(p.x + t * p.ld_x + k);
            if (e < p.E) b = *reinterpret_cast<const uint4*>(p.router + e * p.ld_r + k);
        }
        acc = mma(as_bf8(a), as_bf8(b), acc);
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && e < p.E) {
        const f4_t s = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int tt = blockIdx.z * 16 + 4 * g + i;
            if (tt < p.T) p.part[((int64_t)blockIdx.y * p.T + tt) * p.E + e] = s[i];
        }
    }
}

// Order of choice: NaN last, then by value; the lower index wins a tie.
__device__ __forceinline__ bool goes_before(float a, int ia, float b, int ib) {
    return a > b || (a == b && ia < ib);
}

// One wave per token: scores, top_k rounds of a wave-wide maximum, weights.
template <int NV>  // experts per lane
__global__ __launch_bounds__(64) void route_select_kernel(const RouteArgs p) {
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    float score[NV], by[NV];
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; v++) {
        const int e = v * 64 + lane;
        float l = 0.0f;
        if (e < p.E)
            for (int s = 0; s < p.splits; s++) l += p.part[((int64_t)s * p.T + t) * p.E + e];
        score[v] = l;
        if (e < p.E) top = fmaxf(top, l);
    }
    if (!p.sigmoid) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    }
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; v++) {
        const int e = v * 64 + lane;
        const float l = score[v];
        score[v] = p.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top);
        if (e < p.E) sum += score[v];
        // without a bias the logits give the same order, and no ties that the scores' rounding makes
        by[v] = e < p.E ? l : -INFINITY;
    }
    if (!p.sigmoid) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
#pragma unroll
        for (int v = 0; v < NV; v++) score[v] /= sum;
    }
    if (p.bias) {
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int e = v * 64 + lane;
            if (e < p.E) by[v] = score[v] + p.bias[e];
        }
    }
    uint32_t used = 0;  // the lane's experts that are chosen, or do not exist
#pragma unroll
    for (int v = 0; v < NV; v++) {
        if (v * 64 + lane >= p.E) used |= 1u << v;
        if (!(by[v] == by[v])) by[v] = -INFINITY;
    }
    float mine = 0.0f, total = 0.0f;  // lane j: weight of choice j
    int my_id = 0;
    for (int j = 0; j < p.top_k; j++) {
        float best = -INFINITY, best_score = 0.0f;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int v = 0; v < NV; v++)
            if (!(used >> v & 1) && (at == 0x7FFFFFFF || by[v] > best)) {
                best = by[v];
                best_score = score[v];
                at = v * 64 + lane;
            }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const float ob = __shfl_xor(best, off, 64), os = __shfl_xor(best_score, off, 64);
            const int oa = __shfl_xor(at, off, 64);
            if (goes_before(ob, oa, best, at)) {
                best = ob;
                best_score = os;
                at = oa;
            }
        }
        if ((at & 63) == lane) used |= 1u << (at >> 6);
        if (lane == j) {
            mine = best_score;
            my_id = at;
        }
        total += best_score;
    }
    if (lane < p.top_k) {
        // a sum that vanished (every chosen score underflowed) gives zeros, not 0 / 0
        const float w = p.renorm ? mine / fmaxf(total, 1e-30f) : mine;
        p.ids[t * p.top_k + lane] = my_id;
        // fmaxf drops a NaN: keep it visible
        p.weights[t * p.top_k + lane] = (total == total ? w : total) * p.scale;
    }
}

// ------------------------------------------------------------------------------------- experts

struct MoeArgs {
    const uint16_t* x;
    int64_t ld_x;
    const int32_t* ids;
    const float* weights;
    const uint8_t *w13, *w2;
    int64_t ld13, gs13, ld2, gs2;          // strides of rows and experts, bytes
    const float *s13, *s2;
    int64_t s13_n, s13_k, s13_g, s2_n, s2_k, s2_g;
    uint16_t* h;                           // [T * top_k][I] bf16
    uint16_t* y;
    int64_t ld_y;
    int T, H, I, E, top_k;
    bool by_choice;                        // gate/up blocks go by choice, not by expert
};

// Writes the first `cap` choices of expert e from rank `first` on to list, and returns their total
// number; one wave's work, in choice order.
__device__ __forceinline__ int choices_of(const int32_t* __restrict__ ids, int n, int e, int first, int cap,
                                          uint16_t* list, int lane) {
    int count = 0;
    for (int a0 = 0; a0 < n; a0 += 64) {
        const int a = a0 + lane;
        const bool hit = a < n && ids[a] == e;
        const uint64_t m = __ballot(hit);
        const int rank = count + __popcll(m & ((1ull << lane) - 1)) - first;
        if (hit && rank >= 0 && rank < cap) list[rank] = (uint16_t)a;
        count += __popcll(m);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's lanes read each other's entries
    return count;
}

// acc[ct][m] += rows of `wrow[ct]` times token rows `xrow[m]` over the 128-blocks kb0..kb1 of a
// contraction of K values.  Token tiles at or past mt are left out (their rows are not read).
template <int CT, int MT>
__device__ __forceinline__ void stream_blocks(f4_t (&acc)[CT][MT], const uint8_t* const (&wrow)[CT], const float* const (&srow)[CT],
                                              int64_t s_k, const uint16_t* const (&xrow)[MT], int mt, int K, int kb0, int kb1, int g) {
    constexpr int U = MT == 1 ? 2 : 1;  // blocks whose loads are in flight together
    for (int kb = kb0; kb < kb1; kb += U) {
        uint4 w[U][CT][2];
        float s[U][CT];
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int c = 0; c < CT; c++) {
                s[u][c] = 0.0f;
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    const int k = (kb + u) * MB + 64 * hf + 16 * g;
                    w[u][c][hf] = make_uint4(0, 0, 0, 0);
                    if (kb + u < kb1 && k < K && wrow[c]) w[u][c][hf] = ld_nt16(wrow[c] + k);
                }
                if (kb + u < kb1 && wrow[c]) s[u][c] = srow[c][(kb + u) * s_k];
            }
#pragma unroll
        for (int u = 0; u < U; u++) {
            bf8_t b[CT][4];
#pragma unroll
            for (int c = 0; c < CT; c++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    b[c][2 * hf] = widen8(w[u][c][hf].x, w[u][c][hf].y);
                    b[c][2 * hf + 1] = widen8(w[u][c][hf].z, w[u][c][hf].w);
                }
#pragma unroll
            for (int m = 0; m < MT; m++) {
                if (m < mt) {
                    uint4 a[4];
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const int k = (kb + u) * MB + 64 * (q >> 1) + 16 * g + 8 * (q & 1);
                        a[q] = make_uint4(0, 0, 0, 0);
                        if (kb + u < kb1 && k < K && xrow[m]) a[q] = *reinterpret_cast<const uint4*>(xrow[m] + k);
                    }
#pragma unroll
                    for (int c = 0; c < CT; c++) {
                        f4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int q = 0; q < 4; q++) d = mma(as_bf8(a[q]), b[c][q], d);
#pragma unroll
                        for (int i = 0; i < 4; i++) acc[c][m][i] = fmaf(d[i], s[u][c], acc[c][m][i]);
                    }
                }
            }
        }
    }
}

// h[a] = silu(G x) * (U x) for 16 columns of one expert and all its choices a.  The block's NW
// waves split H; their sums meet in LDS.
template <int MT, int NW>
__global__ __launch_bounds__(64 * NW) void moe_gate_up_kernel(const MoeArgs p) {
    __shared__ f4_t red[NW][2][64];
    __shared__ uint16_t list[16 * MT];
    __shared__ int s_n;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int n = p.T * p.top_k;
    int e = blockIdx.y;
    if (p.by_choice) {  // the first choice of an expert has its block, the others end here
        e = p.ids[blockIdx.y];
        if (e < 0 || e >= p.E) return;
        bool earlier = false;
        for (int a = threadIdx.x; a < (int)blockIdx.y; a += 64 * NW) earlier |= p.ids[a] == e;
        if (__syncthreads_or(earlier)) return;
    }
    const int col = blockIdx.x * 16 + r;  // I is a multiple of 16
    const uint8_t* wrow[2];
    const float* srow[2];
#pragma unroll
    for (int c = 0; c < 2; c++) {
        const int row = c * p.I + col;
        wrow[c] = p.w13 + e * p.gs13 + row * p.ld13;
        srow[c] = p.s13 + e * p.s13_g + (row / MB) * p.s13_n;
    }
    const int kbs = (p.H + MB - 1) / MB, kb0 = kbs * wave / NW, kb1 = kbs * (wave + 1) / NW;
    for (int first = 0;; first += 16 * MT) {
        if (wave == 0) {
            const int c = choices_of(p.ids, n, e, first, 16 * MT, list, lane);
            if (lane == 0) s_n = c;
        }
        __syncthreads();
        const int left = s_n - first;
        if (left <= 0) return;
        const int mt = left >= 16 * MT ? MT : (left + 15) / 16;
        const uint16_t* xrow[MT];
#pragma unroll
        for (int m = 0; m < MT; m++)
            xrow[m] = 16 * m + r < left ? p.x + (list[16 * m + r] / p.top_k) * p.ld_x : nullptr;
        f4_t acc[2][MT];
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
            for (int m = 0; m < MT; m++) acc[c][m] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
        stream_blocks<2, MT>(acc, wrow, srow, p.s13_k, xrow, mt, p.H, kb0, kb1, g);
#pragma unroll
        for (int m = 0; m < MT; m++) {
            if (m < mt) {
                red[wave][0][lane] = acc[0][m];
                red[wave][1][lane] = acc[1][m];
                __syncthreads();
                // thread t < 256 adds element (lane t % 64, register t / 64) of all waves
                for (int t = threadIdx.x; t < 256; t += 64 * NW) {
                    const int l = t & 63, i = t >> 6, row = 16 * m + 4 * (l >> 4) + i;
                    float a = 0.0f, b = 0.0f;
#pragma unroll
                    for (int w = 0; w < NW; w++) {
                        a += red[w][0][l][i];
                        b += red[w][1][l][i];
                    }
                    // h is rounded to bf16, as activations between two layers are: the down
                    // product's operand has to be bf16 for the matrix cores
                    if (row < left)
                        p.h[(int64_t)list[row] * p.I + blockIdx.x * 16 + (l & 15)] = to_bf16(a / (1.0f + expf(-a)) * b);
                }
                __syncthreads();
            }
        }
        if (left <= 16 * MT) return;
    }
}

// y[:, 16 columns] over all chosen experts.  Units of work (chosen expert, part of I) go to the
// block's waves in turn; each wave has its own sums of all tokens in LDS, added at the end.
template <int MT, int TMAX, int NW>
__global__ __launch_bounds__(64 * NW) void moe_down_kernel(const MoeArgs p) {
    __shared__ float ysum[NW][TMAX][16];
    __shared__ uint16_t lists[NW][16 * MT];
    __shared__ uint16_t s_active[MOE_MAX_E];
    __shared__ uint8_t s_flag[MOE_MAX_E];
    __shared__ int s_n;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, r = lane & 15, g = lane >> 4;
    const int n = p.T * p.top_k;
    for (int i = t; i < p.E; i += 64 * NW) s_flag[i] = 0;
    for (int i = lane; i < p.T * 16; i += 64) (&ysum[wave][0][0])[i] = 0.0f;
    __syncthreads();
    for (int a = t; a < n; a += 64 * NW) {
        const int e = p.ids[a];
        if (e >= 0 && e < p.E) s_flag[e] = 1;
    }
    __syncthreads();
    if (wave == 0) {
        int c = 0;
        for (int e0 = 0; e0 < p.E; e0 += 64) {
            const bool on = e0 + lane < p.E && s_flag[e0 + lane];
            const uint64_t m = __ballot(on);
            if (on) s_active[c + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(e0 + lane);
            c += __popcll(m);
        }
        if (lane == 0) s_n = c;
    }
    __syncthreads();
    const int active = s_n, kbs = (p.I + MB - 1) / MB;
    // parts of I so that every wave has a unit
    int parts = 1;
    while (parts < NW && active * parts < NW && 2 * parts <= kbs) parts *= 2;
    const int row = blockIdx.x * 16 + r;
    uint16_t* list = lists[wave];
    for (int u = wave; u < active * parts; u += NW) {
        const int e = s_active[u / parts], part = u % parts;
        const uint8_t* wrow[1] = {row < p.H ? p.w2 + e * p.gs2 + row * p.ld2 : nullptr};
        const float* srow[1] = {p.s2 + e * p.s2_g + (row / MB) * p.s2_n};
        const int kb0 = kbs * part / parts, kb1 = kbs * (part + 1) / parts;
        for (int first = 0;; first += 16 * MT) {
            const int left = choices_of(p.ids, n, e, first, 16 * MT, list, lane) - first;
            if (left <= 0) break;
            const int mt = left >= 16 * MT ? MT : (left + 15) / 16;
            const uint16_t* xrow[MT];
#pragma unroll
            for (int m = 0; m < MT; m++) xrow[m] = 16 * m + r < left ? p.h + (int64_t)list[16 * m + r] * p.I : nullptr;
            f4_t acc[1][MT];
#pragma unroll
            for (int m = 0; m < MT; m++) acc[0][m] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
            stream_blocks<1, MT>(acc, wrow, srow, p.s2_k, xrow, mt, p.I, kb0, kb1, g);
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = 16 * m + 4 * g + i;
                    if (at < left) {
                        const int a = list[at];
                        // one wave owns these sums; an LDS addition, because a token may be listed
                        // twice for one expert and then two lanes meet here
                        atomicAdd(&ysum[wave][a / p.top_k][r], p.weights[a] * acc[0][m][i]);
                    }
                }
            if (left <= 16 * MT) break;
        }
    }
    __syncthreads();
    for (int i = t; i < p.T * 16; i += 64 * NW) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; w++) s += (&ysum[w][0][0])[i];
        const int c = blockIdx.x * 16 + (i & 15);
        if (c < p.H) p.y[(i >> 4) * p.ld_y + c] = to_bf16(s);
    }
}

template <int MT, int TMAX>
static fp8q_status_t launch_moe(const MoeArgs& p, hipStream_t stream) {
    const int n = p.T * p.top_k;
    moe_gate_up_kernel<MT, 8><<<dim3((unsigned)(p.I / 16), (unsigned)(p.by_choice ? n : p.E)), dim3(512), 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    moe_down_kernel<MT, TMAX, 8><<<dim3((unsigned)((p.H + 15) / 16)), dim3(512), 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

static int route_splits(int64_t T, int64_t H, int64_t E) {
    // enough blocks for the chip's CUs, at least 8 instructions' worth of H for each of a block's waves
    const int64_t blocks = ((T + 15) / 16) * ((E + 15) / 16);
    int64_t s = 128 / blocks;
    const int64_t most = H / (4 * 8 * 32);
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

}  // namespace fp8q

extern "C" size_t moe_route_workspace_size(int64_t T, int64_t H, int64_t E) {
    if (T <= 0 || H <= 0 || E <= 0) return 256;
    return (size_t)fp8q::route_splits(T, H, E) * (size_t)T * (size_t)E * 4;
}

extern "C" fp8q_status_t moe_route(const uint16_t* x, int64_t T, int64_t H, int64_t ld_x, const uint16_t* router,
                                   int64_t E, int64_t ld_r, const float* bias, fp8q_scoring_t scoring, int32_t top_k,
                                   int renormalize, float scale, int32_t* ids, float* weights, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
    using namespace fp8q;
    if (T < 0 || H < 1 || E < 1 || ld_x < H || ld_r < H || top_k < 1 || top_k > E ||
        (scoring != FP8Q_SCORE_SOFTMAX && scoring != FP8Q_SCORE_SIGMOID))
        return FP8Q_ERR_INVALID_ARG;
    if (T == 0) return FP8Q_OK;
    if (!x || !router || !ids || !weights) return FP8Q_ERR_INVALID_ARG;
    if (E > MOE_MAX_E || top_k > MOE_MAX_K || H % 8 || ld_x % 8 || ld_r % 8 || !fp8q_aligned(x, 16) ||
        !fp8q_aligned(router, 16) || H > 0x3FFFFFFF || T > 16LL * 65535)
        return FP8Q_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < moe_route_workspace_size(T, H, E)) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 4)) return FP8Q_ERR_INVALID_ARG;
    RouteArgs p{};
    p.x = x; p.ld_x = ld_x; p.router = router; p.ld_r = ld_r; p.bias = bias; p.part = reinterpret_cast<float*>(workspace);
    p.ids = ids; p.weights = weights; p.T = (int)T; p.E = (int)E; p.H = (int)H; p.top_k = top_k;
    p.splits = route_splits(T, H, E); p.sigmoid = scoring == FP8Q_SCORE_SIGMOID; p.renorm = renormalize != 0; p.scale = scale;
    route_logits_kernel<<<dim3((unsigned)((E + 15) / 16), (unsigned)p.splits, (unsigned)((T + 15) / 16)), dim3(256), 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    const dim3 grid((unsigned)T), block(64);
    if (E <= 64) route_select_kernel<1><<<grid, block, 0, stream>>>(p);
    else if (E <= 256) route_select_kernel<4><<<grid, block, 0, stream>>>(p);
    else route_select_kernel<16><<<grid, block, 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

extern "C" size_t fp8_moe_few_tokens_workspace_size(int64_t T, int64_t I, int32_t top_k) {
    if (T <= 0 || I <= 0 || top_k <= 0) return 256;
    return (size_t)T * (size_t)top_k * (size_t)I * 2;
}

extern "C" fp8q_status_t fp8_moe_few_tokens(const uint16_t* x, int64_t T, int64_t H, int64_t ld_x, const int32_t* ids,
                                            const float* weights, int32_t top_k, const uint8_t* w13, int64_t ld13,
                                            int64_t w13_group_stride, const float* s13, int64_t s13_n, int64_t s13_k,
                                            int64_t s13_group_stride, const uint8_t* w2, int64_t ld2,
                                            int64_t w2_group_stride, const float* s2, int64_t s2_n, int64_t s2_k,
                                            int64_t s2_group_stride, int64_t E, int64_t I, uint16_t* y, int64_t ld_y,
                                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace fp8q;
    if (T < 0 || H < 1 || I < 1 || E < 1 || top_k < 1 || ld_x < H || ld13 < H || ld2 < I || ld_y < H ||
        w13_group_stride < 0 || w2_group_stride < 0 || s13_n < 0 || s13_k < 0 || s13_group_stride < 0 || s2_n < 0 ||
        s2_k < 0 || s2_group_stride < 0)
        return FP8Q_ERR_INVALID_ARG;
    if (T == 0) return FP8Q_OK;
    if (!x || !ids || !weights || !w13 || !s13 || !w2 || !s2 || !y) return FP8Q_ERR_INVALID_ARG;
    if (T > MOE_MAX_T || E > MOE_MAX_E || top_k > MOE_MAX_K || H % 16 || I % 16 || H > 0x3FFFFFFF || I > 0x3FFFFFFF ||
        ld_x % 8 || ld13 % 16 || ld2 % 16 || w13_group_stride % 16 || w2_group_stride % 16 || !fp8q_aligned(x, 16) ||
        !fp8q_aligned(w13, 16) || !fp8q_aligned(w2, 16))
        return FP8Q_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < fp8_moe_few_tokens_workspace_size(T, I, top_k)) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 16)) return FP8Q_ERR_INVALID_ARG;
    MoeArgs p{};
    p.x = x; p.ld_x = ld_x; p.ids = ids; p.weights = weights; p.w13 = w13; p.w2 = w2; p.ld13 = ld13; p.gs13 = w13_group_stride;
    p.ld2 = ld2; p.gs2 = w2_group_stride; p.s13 = s13; p.s2 = s2; p.s13_n = s13_n; p.s13_k = s13_k; p.s13_g = s13_group_stride;
    p.s2_n = s2_n; p.s2_k = s2_k; p.s2_g = s2_group_stride; p.h = reinterpret_cast<uint16_t*>(workspace); p.y = y; p.ld_y = ld_y;
    p.T = (int)T; p.H = (int)H; p.I = (int)I; p.E = (int)E; p.top_k = top_k;
    p.by_choice = T * top_k < E;
    if (T <= 16) return launch_moe<1, 16>(p, stream);
    if (T <= 64) return launch_moe<2, 64>(p, stream);
    return launch_moe<2, MOE_MAX_T>(p, stream);
}
