// A mixture-of-experts layer for a few tokens: routing, and the experts' SwiGLU feed-forward on
// block-scaled FP8 weights.
//
//   route    logits = x Wr^T, scores = softmax or sigmoid, the top_k of scores (+ bias), weights
//   experts  y[t] = sum_j w[t,j] W2_e ( silu(G_e x_t) * (U_e x_t) ),  e = ids[t,j]
//            ([G_e; U_e] = w13[e], 2 I x H; W2_e = w2[e], H x I; one fp32 factor per 128 x 128)
//
// Bound: HBM.  With few tokens every chosen expert's 3 H I weight bytes are read for a handful of
// multiplications each, so the kernels are built around streaming them once: a lane's 16-byte
// weight loads feed the matrix cores directly.  The weights are widened to bf16 (exact) and
// multiply the bf16 activations as they are: nothing is quantized on the way, and the matrix
// cores, which would be idle otherwise, take up to 16 tokens for the price of one.
//
// Matrix instruction: 16 x 16 x 32 bf16.  Its A rows are tokens, its B rows are weight rows: lane l
// holds token or weight row l % 16, and its 8 k values may be any 8 as long as both operands agree.  Here
// lane group l / 16 of a 64-byte piece of a weight row takes bytes 16 (l / 16) .. + 15, one 16-byte
// load for two instructions.  Result register i of lane l is token 4 (l / 16) + i, weight row l % 16.
//
// Every sum has a fixed order: a contraction's parts are added in wave order, a token's experts in
// the order of its choices.
//
// Measured (32 experts of 2048 x 7168, 8 of them a token): 1 token's gate and up products 47 us (4.9
// TB/s of weights) and down product 27 us (4.4 TB/s), 64 tokens' 198 and 117 us (4.8 and 4.0 TB/s),
// where a copy of large buffers reaches 4.9 TB/s and a kernel that only reads as these do 5.4 at 240
// MB and 6.2 at 960 MB.  64 experts of 1408 x 2048, 6 of them, 5 tokens: 37 and 20 us (3.8 TB/s: each
// wave has 16 and 11 blocks to stream, so starting and ending count).  Routing and the join take 2
// to 6 us each, a launch's time.
//
// Measured and not kept: 4 blocks ahead instead of 2 (spills: 340 against 242 us for 64 tokens), 8
// waves a CU with twice the registers (242 to 265 us), non-temporal weight loads, a second pass over
// the weights for more than 32 tokens (65 us), h in one bf16 (its rounding shows in the result).
#include "common.hpp"
#include "gemm_tile.hpp"
#include "lds_dma.hpp"
#include "plan.hpp"

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

// The same, but a finite value past bf16's largest gives that one, so that the rest is finite too.
__device__ __forceinline__ uint16_t to_bf16_finite(float f) {
    const uint32_t u = __float_as_uint(f);
    const uint16_t r = to_bf16(f);
    return (r & 0x7FFFu) == 0x7F80u && (u & 0x7FFFFFFFu) < 0x7F800000u ? (uint16_t)(r - 1) : r;
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
    constexpr int U = 4;  // chunks whose loads are in flight together
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int e = blockIdx.x * 16 + r, t = blockIdx.z * 16 + r;
    const int chunks = (p.H + 31) / 32;                          // 32 k values of one instruction
    const int parts = p.splits * 4, me = blockIdx.y * 4 + wave;  // waves over H
    const int k0 = (int)((int64_t)chunks * me / parts), k1 = (int)((int64_t)chunks * (me + 1) / parts);
    const uint16_t* xr = p.x + (t < p.T ? t : 0) * p.ld_x;
    const uint16_t* wr = p.router + (e < p.E ? e : 0) * p.ld_r;  // rows past the last: results not used
    f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kc = k0; kc < k1; kc += U) {
        uint4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int k = (kc + u) * 32 + 8 * g;
            a[u] = b[u] = make_uint4(0, 0, 0, 0);
            if (kc + u < k1 && k < p.H) {  // H is a multiple of 8
                a[u] = *reinterpret_cast<const uint4*>(xr + k);
                b[u] = *reinterpret_cast<const uint4*>(wr + k);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) acc = mma(as_bf8(a[u]), as_bf8(b[u]), acc);
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

// Renormalized weights come from the scores where their sum is at least this: a score that underflows
// then weighs less than 2^-62.  Below it they come from the chosen logits l_j and their maximum m, as
// exp(l_j - m) / sum exp(l_i - m): a softmax's chosen scores have these ratios, and so have sigmoids
// of logits below -44, whose 1 + exp(l) is 1 in 32 bits.
constexpr float kTinySum = 5.421010862427522e-20f;  // 2^-64

// What a block needs beside the logits to choose a token's experts.
struct Choice {
    float logit[256], by[256], chosen[MOE_MAX_K], chosen_logit[MOE_MAX_K];
};

// Scores, choice and weights of one token from its logits in LDS, by a whole block of at least E
// threads: an expert's place is the number of experts that go before it.
__device__ __forceinline__ void choose(const RouteArgs& p, int64_t t, Choice& s) {
    const float* logit = s.logit;
    float* by = s.by;
    const int e = threadIdx.x;
    const float l = e < p.E ? logit[e] : 0.0f;
    float score = 1.0f / (1.0f + expf(-l));
    if (!p.sigmoid) {
        float top = -INFINITY;
        for (int j = 0; j < p.E; j++) top = fmaxf(top, logit[j]);
        score = expf(l - top);
        if (e < p.E) by[e] = score;
        __syncthreads();
        float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // four sums in turn
        for (int j = 0; j < p.E; j++) s4[j & 3] += by[j];
        score /= (s4[0] + s4[1]) + (s4[2] + s4[3]);
        __syncthreads();
    }
    if (e < p.E) {
        // without a bias the logits give the same order, and no ties that the scores' rounding makes
        const float v = p.bias ? score + p.bias[e] : l;
        by[e] = v == v ? v : -INFINITY;  // NaN goes last
    }
    __syncthreads();
    int place = p.top_k;
    if (e < p.E) {
        const float v = by[e];
        place = 0;
        for (int j = 0; j < p.E; j++) place += by[j] > v || (by[j] == v && j < e);
        if (place < p.top_k) {
            s.chosen[place] = score;
            s.chosen_logit[place] = l;
        }
    }
    __syncthreads();
    if (place < p.top_k) {
        float total = 0.0f;
        for (int j = 0; j < p.top_k; j++) total += s.chosen[j];
        float w = score;
        if (p.renorm && total < kTinySum) {
            float m = -INFINITY, sum = 0.0f;
            for (int j = 0; j < p.top_k; j++) m = fmaxf(m, s.chosen_logit[j]);
            for (int j = 0; j < p.top_k; j++) sum += expf(s.chosen_logit[j] - m);
            w = m > -INFINITY ? expf(l - m) / sum : 0.0f;  // all of them at minus infinity: no weight
        } else if (p.renorm) {
            w = score / total;
        }
        p.ids[t * p.top_k + place] = e;
        p.weights[t * p.top_k + place] = (total == total ? w : total) * p.scale;  // a NaN stays visible
    }
}

__global__ __launch_bounds__(256) void route_choose_kernel(const RouteArgs p) {
    __shared__ Choice s;
    const int64_t t = blockIdx.x;
    const int e = threadIdx.x;
    if (e < p.E) {
        float part[16], l = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) part[i] = i < p.splits ? p.part[((int64_t)i * p.T + t) * p.E + e] : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) l += part[i];
        s.logit[e] = l;
    }
    __syncthreads();
    choose(p, t, s);
}

// Small routers in one kernel: a block of 16 waves per token, each wave an expert at a time.
__global__ __launch_bounds__(1024) void route_small_kernel(const RouteArgs p) {
    __shared__ Choice s;
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint16_t* xr = p.x + t * p.ld_x;
    for (int e = wave; e < p.E; e += 16) {
        const uint16_t* wr = p.router + e * p.ld_r;
        float acc = 0.0f;
        for (int k = lane * 8; k < p.H; k += 512) {
            const uint4 a = *reinterpret_cast<const uint4*>(xr + k), b = *reinterpret_cast<const uint4*>(wr + k);
            const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                acc = fmaf(bf16_lo(u[q]), bf16_lo(v[q]), acc);
                acc = fmaf(bf16_hi(u[q]), bf16_hi(v[q]), acc);
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) acc += __shfl_xor(acc, off, 64);
        if (lane == 0) s.logit[e] = acc;
    }
    __syncthreads();
    choose(p, t, s);
}

// Order of choice: NaN last, then by value; the lower index wins a tie.
__device__ __forceinline__ bool goes_before(float a, int ia, float b, int ib) {
    return a > b || (a == b && ia < ib);
}

// More experts: one wave per token, top_k rounds of a wave-wide maximum (the places above cost E^2
// comparisons).
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
    float w = mine;
    if (p.renorm && total < kTinySum) {  // (the same in every lane)
        float l = -INFINITY;
        if (lane < p.top_k) {
            l = 0.0f;
            for (int s = 0; s < p.splits; s++) l += p.part[((int64_t)s * p.T + t) * p.E + my_id];
        }
        float m = l;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
        float all = m > -INFINITY ? expf(l - m) : 0.0f;  // all of them at minus infinity: no weight
        w = all;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) all += __shfl_xor(all, off, 64);
        w = m > -INFINITY ? w / all : 0.0f;
    } else if (p.renorm) {
        w = mine / total;
    }
    if (lane < p.top_k) {
        p.ids[t * p.top_k + lane] = my_id;
        p.weights[t * p.top_k + lane] = (total == total ? w : total) * p.scale;  // a NaN stays visible
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
    uint16_t* h;                           // two planes of [T * top_k][I]: bf16 and what it leaves
    float* o;                              // [T * top_k][H] the experts' outputs
    uint16_t* y;
    int64_t ld_y;
    int T, H, I, E, top_k;
    int pass;                              // tokens of an expert that one pass takes: a power of two
    bool by_choice;                        // gate/up blocks go by choice, not by expert
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_buffer(const uint8_t* base, int64_t bytes) {
    const uint64_t a = (uint64_t)base;  // wave-uniform: keep the descriptor in scalar registers
    const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) << 32;
    return __builtin_amdgcn_make_buffer_rsrc((void*)u, (short)0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// put(i, a) for the choices a of expert e with ranks first + i, i < cap, in choice order; returns how
// many there are in all.  One wave's work.
template <class F>
__device__ __forceinline__ int choices_of(const int32_t* __restrict__ ids, int n, int e, int first, int cap, int lane, F put) {
    int count = 0;
    for (int a0 = 0; a0 < n; a0 += 64) {
        const int a = a0 + lane;
        const bool hit = a < n && ids[a] == e;
        const uint64_t m = __ballot(hit);
        const int rank = count + __popcll(m & ((1ull << lane) - 1)) - first;
        if (hit && rank >= 0 && rank < cap) put(rank, a);
        count += __popcll(m);
    }
    return count;
}

// One expert's product with its chosen tokens.  DOWN = false: h[a] = silu(G x) * (U x), a wave's two
// weight tiles being 16 gate rows and the same 16 up rows; DOWN = true: o[a] = W2 h[a], two
// neighbouring tiles of 16 rows.  A block's NW waves are NW / S such pairs times S parts of the
// contraction, whose sums meet in LDS.
//
// A wave streams its 32 weight rows through registers, D contraction blocks (4 KB each) ahead of the
// matrix instructions.  The block's waves share the tokens' activations, brought into LDS a chunk of
// contraction blocks ahead, a few instructions a step, so that the weights' loads (which complete in
// order with them) never wait for a burst.  h keeps 16 significant bits: two bf16 planes, each
// multiplied, since the matrix cores wait for memory anyway.
template <int MT, int S, bool DOWN, int NW>
__global__ __launch_bounds__(64 * NW, 4) void moe_stream_kernel(const MoeArgs p) {
    constexpr int D = 2, PAIRS = NW / S, PL = DOWN ? 2 : 1, NT = 64 * NW, LDS = moe_lds(NW);
    __shared__ __align__(16) uint8_t stage[LDS];
    __shared__ uint16_t list[16 * MT];     // choices of this pass
    __shared__ uint32_t at_byte[16 * MT];  // and where their activations start
    __shared__ int s_n;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = wave % S;
    const int n = p.T * p.top_k;
    const int K = DOWN ? p.I : p.H, rows = DOWN ? p.H : p.I;  // multiples of 16
    int e = blockIdx.y;
    if (p.by_choice) {  // the first choice of an expert has its block, the others end below
        e = p.ids[blockIdx.y];
        if (e < 0 || e >= p.E) return;
    }
    // first row of each tile; a tile never straddles a factor block, so its factors are uniform
    const int pair = blockIdx.x * PAIRS + wave / S;
    const int row0 = DOWN ? 32 * pair : 16 * pair, row1 = DOWN ? row0 + 16 : p.I + row0;
    const bool on0 = row0 < rows, on1 = DOWN ? row1 < rows : on0;
    const uint8_t* w = DOWN ? p.w2 + e * p.gs2 : p.w13 + e * p.gs13;
    const int64_t ld = DOWN ? p.ld2 : p.ld13;
    // a tile's 16 rows as a buffer: a lane past K, or a tile past the last row, reads zeros
    const __amdgpu_buffer_rsrc_t wbuf[2] = {tile_buffer(w + row0 * ld, on0 ? 15 * ld + K : 0),
                                            tile_buffer(w + row1 * ld, on1 ? 15 * ld + K : 0)};
    // activations: x, or the two planes of h
    const uint32_t plane = (uint32_t)n * (uint32_t)p.I * 2;
    const i32x4_t abuf = make_rsrc4(DOWN ? p.h : p.x, DOWN ? 2 * plane : (uint32_t)((p.T - 1) * p.ld_x + K) * 2);
    const uint32_t stage_at = lds_addr(stage);
    const uint32_t lane_off = (uint32_t)(r * ld) + 16 * g;
    const bool on[2] = {on0, on1};
    const float* s = DOWN ? p.s2 + e * p.s2_g : p.s13 + e * p.s13_g;
    const int64_t s_n_ = DOWN ? p.s2_n : p.s13_n, s_k = DOWN ? p.s2_k : p.s13_k;
    const float* srow[2] = {s + (row0 / MB) * s_n_, s + (row1 / MB) * s_n_};
    const int kbs = (K + MB - 1) / MB, kb0 = kbs * part / S, len = kbs * (part + 1) / S - kb0;
    const int most = (kbs + S - 1) / S;  // the longest part's blocks
    // A block begins at its own place of the contraction and goes round: rows often lie a power of two
    // apart, and waves at one place of all of them ask few of the memory's channels at a time (16 tokens
    // of 8 experts of 14336 x 4096 312 -> 284 us, 128 tokens 528 -> 492; 32 of 2048 x 7168 288 -> 290 and
    // 357 -> 352).
    const int turn = (int)(blockIdx.x * 5u % (unsigned)most);
    auto place = [&](int i) { return i + turn < most ? i + turn : i + turn - most; };

    for (int first = 0;; first += p.pass) {
        uint4 wv[D][2][2];
        auto load = [&](int d, int hf, int i) {  // half of block i of the part into register set d
            const int j = place(i), k = (kb0 + j) * MB + 64 * hf;
            const uint32_t off = k + 16 * g < K && i < most && j < len ? lane_off + k : OOB;
#pragma unroll
            for (int c = 0; c < 2; c++)
                wv[d][c][hf] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(wbuf[c], off, 0, 0));
        };
#pragma unroll
        for (int d = 0; d < D; d++) {
            load(d, 0, d);
            load(d, 1, d);
        }
        // the weights are on their way while the tokens are looked up
        if (wave == 0) {
            const int c = choices_of(p.ids, n, e, first, p.pass, lane, [&](int i, int a) {
                list[i] = (uint16_t)a;
                at_byte[i] = (uint32_t)(DOWN ? a * p.I : a / p.top_k * (int)p.ld_x) * 2;
            });
            if (lane == 0) s_n = c;
        }
        __syncthreads();
        const int left = __builtin_amdgcn_readfirstlane(s_n) - first;
        if (left <= 0 || (p.by_choice && first == 0 && list[0] != blockIdx.y)) return;
        const int toks = left < p.pass ? left : p.pass, mt = (toks + 15) / 16;
        // rows of the staged chunk: lanes past the last take any row, their results are not used
        int lr = 0;
        while ((1 << lr) < toks) lr++;
        // contraction blocks of each part in a chunk, of which two are held: a power of two, and
        // pick_stream sees to it that one fits
        int lc = 0;
        while ((LDS / 2 >> (lc + 1 + lr + 8)) >= PL * S && (1 << lc) < most) lc++;

        // One instruction of staging: 4 rows of 256 bytes, rows of a (part, block) and plane following
        // each other, of the chunk that starts at block i0 of every part; q counts them.
        auto bring = [&](int i0, int q, uint32_t to) {
            const int unit = 4 * q + g, row = unit & ((1 << lr) - 1), rest = unit >> lr, bl = rest / PL;
            const int kb = kbs * (bl >> lc) / S + place(i0 + (bl & ((1 << lc) - 1)));
            const int k = kb * MB + 8 * (r ^ (row & 15));
            uint32_t off = OOB;
            if (row < toks && k < K) off = at_byte[row] + 2 * k + (PL == 2 && (rest & 1) ? plane : 0);
            dma16(abuf, off, to + q * 1024);
        };
        const int bring_all = (((S * PL) << (lc + lr)) + 3) >> 2;     // instructions of a chunk
        const int bring_step = ((bring_all + NW - 1) / NW + (1 << lc) - 1) >> lc;  // one wave's in a step
        uint32_t buf = 0;  // the buffer being read

        f4_t acc[2][MT];
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
            for (int m = 0; m < MT; m++) acc[c][m] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
        float sv[2] = {0.0f, 0.0f};  // lane l: factors of blocks 64 j + l of the part
#pragma unroll 1
        for (int q = wave; q < bring_all; q += NW) bring(0, q, stage_at);
        wait_vm0();
        for (int i0 = 0; i0 < most; i0 += D) {
            if ((i0 & 63) == 0) {
#pragma unroll
                for (int c = 0; c < 2; c++)
                    sv[c] = on[c] && i0 + lane < most && place(i0 + lane) < len ? srow[c][(kb0 + place(i0 + lane)) * s_k] : 0.0f;
            }
#pragma unroll
            for (int d = 0; d < D; d++) {
                const int i = i0 + d;
                if (i >= most) break;
                const int i1 = i & ((1 << lc) - 1), next = i - i1 + (1 << lc);
                if (i1 == 0) {
                    // this chunk has landed, in every wave: only the last step's 4 weight loads are
                    // younger than its instructions; and the buffer read until now is free
                    if (i > 0) {
                        asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
                        buf ^= LDS / 2;
                    }
                    __syncthreads();
                }
                if (next < most) {
#pragma unroll 1
                    for (int q = 0; q < bring_step; q++) {
                        const int at = wave + NW * (i1 * bring_step + q);
                        if (at < bring_all) bring(next, at, stage_at + (buf ^ (LDS / 2)));
                    }
                }
                const int bl = (part << lc) + i1;
                const float f0 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sv[0]), i & 63));
                const float f1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sv[1]), i & 63));
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    bf8_t b[2][2];
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        b[c][0] = widen8(wv[d][c][hf].x, wv[d][c][hf].y);
                        b[c][1] = widen8(wv[d][c][hf].z, wv[d][c][hf].w);
                    }
                    load(d, hf, i + D);
#pragma unroll
                    for (int m = 0; m < MT; m++) {
                        if (m < mt && place(i) < len) {
                            const int row = (16 * m + r) & ((1 << lr) - 1);
                            f4_t sum0 = {0.0f, 0.0f, 0.0f, 0.0f}, sum1 = sum0;
#pragma unroll
                            for (int pl = 0; pl < PL; pl++) {
                                const uint8_t* src = stage + buf + ((((bl * PL + pl) << lr) + row) << 8);
#pragma unroll
                                for (int q = 0; q < 2; q++) {
                                    const int ch = 8 * hf + 2 * g + q;
                                    const bf8_t a = as_bf8(*reinterpret_cast<const uint4*>(src + ((ch ^ (row & 15)) << 4)));
                                    sum0 = mma(a, b[0][q], sum0);
                                    sum1 = mma(a, b[1][q], sum1);
                                }
                            }
#pragma unroll
                            for (int q = 0; q < 4; q++) {
                                acc[0][m][q] = fmaf(sum0[q], f0, acc[0][m][q]);
                                acc[1][m][q] = fmaf(sum1[q], f1, acc[1][m][q]);
                            }
                        }
                    }
                }
            }
        }
        if (S > 1) {
            f4_t* red = reinterpret_cast<f4_t*>(stage);  // [wave][tile][m][lane]
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 2; c++)
#pragma unroll
                for (int m = 0; m < MT; m++) red[((wave * 2 + c) * MT + m) * 64 + lane] = acc[c][m];
            __syncthreads();
            if (part == 0) {
#pragma unroll
                for (int c = 0; c < 2; c++)
#pragma unroll
                    for (int m = 0; m < MT; m++)
#pragma unroll
                        for (int q = 1; q < S; q++) acc[c][m] += red[(((wave + q) * 2 + c) * MT + m) * 64 + lane];
            }
        }
        if (part == 0) {
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = 16 * m + 4 * g + i;
                    if (at < toks) {
                        const int64_t a = list[at];
                        const float u = acc[0][m][i], v = acc[1][m][i];
                        if (!DOWN) {
                            const float h = u / (1.0f + expf(-u)) * v;
                            const uint16_t hi = to_bf16_finite(h);
                            const float rest = h - __uint_as_float((uint32_t)hi << 16);
                            if (on0) {
                                p.h[a * p.I + row0 + r] = hi;
                                p.h[(int64_t)n * p.I + a * p.I + row0 + r] = to_bf16(rest == rest ? rest : 0.0f);  // inf - inf
                            }
                        } else {
                            if (on0) p.o[a * p.H + row0 + r] = u;
                            if (on1) p.o[a * p.H + row1 + r] = v;
                        }
                    }
                }
        }
        if (left <= p.pass) return;
        __syncthreads();  // the list is written again
    }
}

// y[t] = sum_j weights[t,j] o[t,j], in order of j; 4 columns a thread.
__global__ __launch_bounds__(256) void moe_join_kernel(const MoeArgs p) {
    const int64_t n4 = (int64_t)p.T * p.H / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    const int64_t t = i * 4 / p.H, c = i * 4 - t * p.H;
    f4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < p.top_k; j0 += 8) {  // 8 loads in flight
        f4_t o[8];
        float w[8];
        bool on[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t a = t * p.top_k + (j0 + j < p.top_k ? j0 + j : p.top_k - 1);
            const int e = p.ids[a];
            on[j] = j0 + j < p.top_k && e >= 0 && e < p.E;
            w[j] = p.weights[a];
            o[j] = *reinterpret_cast<const f4_t*>(p.o + a * p.H + c);  // unwritten where !on[j]
        }
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
            for (int q = 0; q < 4; q++) s[q] = on[j] ? fmaf(w[j], o[j][q], s[q]) : s[q];
    }
    uint16_t* y = p.y + t * p.ld_y + c;
#pragma unroll
    for (int q = 0; q < 4; q++) y[q] = to_bf16(s[q]);
}

template <int MT, bool DOWN>
static void launch_stream(MoeArgs p, const StreamPlan& plan, hipStream_t stream) {
    constexpr int NW = moe_waves(MT), SMAX = moe_parts(MT, DOWN);
    static_assert(moe_lds(NW) / 2 >= SMAX * (DOWN ? 2 : 1) * (MT == 1 ? 1 : 16 * MT) * 256, "a block of every part fits");
    p.pass = plan.pass;
    const int pairs = DOWN ? (p.H + 31) / 32 : p.I / 16;
    const dim3 grid((unsigned)((pairs * plan.parts + NW - 1) / NW), (unsigned)(p.by_choice ? p.T * p.top_k : p.E)), block(64 * NW);
    if (plan.parts == 1) moe_stream_kernel<MT, 1, DOWN, NW><<<grid, block, 0, stream>>>(p);
    else if (plan.parts == 2) moe_stream_kernel<MT, SMAX < 2 ? 1 : 2, DOWN, NW><<<grid, block, 0, stream>>>(p);
    else moe_stream_kernel<MT, SMAX, DOWN, NW><<<grid, block, 0, stream>>>(p);
}

template <bool DOWN>
static void launch_product(const MoeArgs& p, hipStream_t stream) {
    const StreamPlan plan = pick_stream(DOWN, p.T, p.top_k, p.E, p.H, p.I, num_cus());
    if (plan.mt == 1) launch_stream<1, DOWN>(p, plan, stream);
    else if (plan.mt == 2) launch_stream<2, DOWN>(p, plan, stream);
    else launch_stream<4, DOWN>(p, plan, stream);
}

static fp8q_status_t launch_moe(const MoeArgs& p, hipStream_t stream) {
    launch_product<false>(p, stream);
    FP8Q_CHECK_LAUNCH();
    launch_product<true>(p, stream);
    FP8Q_CHECK_LAUNCH();
    moe_join_kernel<<<dim3((unsigned)(((int64_t)p.T * p.H / 4 + 255) / 256)), dim3(256), 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

}  // namespace fp8q

extern "C" size_t moe_route_workspace_size(int64_t T, int64_t H, int64_t E) {
    if (T <= 0 || H <= 0 || E <= 0) return 256;
    if (fp8q::route_is_small(H, E)) return 0;
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
    if ((!workspace || workspace_bytes < moe_route_workspace_size(T, H, E)) && !route_is_small(H, E)) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 4)) return FP8Q_ERR_INVALID_ARG;
    RouteArgs p{};
    p.x = x; p.ld_x = ld_x; p.router = router; p.ld_r = ld_r; p.bias = bias; p.part = reinterpret_cast<float*>(workspace);
    p.ids = ids; p.weights = weights; p.T = (int)T; p.E = (int)E; p.H = (int)H; p.top_k = top_k;
    p.splits = route_splits(T, H, E); p.sigmoid = scoring == FP8Q_SCORE_SIGMOID; p.renorm = renormalize != 0; p.scale = scale;
    if (route_is_small(H, E)) {
        route_small_kernel<<<dim3((unsigned)T), dim3(1024), 0, stream>>>(p);
        FP8Q_CHECK_LAUNCH();
        return FP8Q_OK;
    }
    route_logits_kernel<<<dim3((unsigned)((E + 15) / 16), (unsigned)p.splits, (unsigned)((T + 15) / 16)), dim3(256), 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    const dim3 grid((unsigned)T), block(64);
    if (E <= 256) route_choose_kernel<<<grid, dim3(256), 0, stream>>>(p);
    else route_select_kernel<16><<<grid, block, 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

// Workspace: h, then the experts' outputs, both 32-bit.
extern "C" size_t fp8_moe_few_tokens_workspace_size(int64_t T, int64_t H, int64_t I, int32_t top_k) {
    if (T <= 0 || H <= 0 || I <= 0 || top_k <= 0) return 256;
    return (size_t)T * (size_t)top_k * (size_t)(I + H) * 4;
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
    if (T > MOE_MAX_T || E > MOE_MAX_E || top_k > MOE_MAX_K || H % 16 || I % 16 || H > 0x3FFFFFFF || I > 0x3FFFFFFF || ld13 >= (1 << 26) ||
        ld2 >= (1 << 26) || ld_x > ((1 << 30) - 1) / T ||
        T * top_k * I >= (1 << 29) || ld_x % 8 || ld13 % 16 || ld2 % 16 || w13_group_stride % 16 || w2_group_stride % 16 || !fp8q_aligned(x, 16) ||
        !fp8q_aligned(w13, 16) || !fp8q_aligned(w2, 16))
        return FP8Q_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < fp8_moe_few_tokens_workspace_size(T, H, I, top_k)) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 16)) return FP8Q_ERR_INVALID_ARG;
    MoeArgs p{};
    p.x = x; p.ld_x = ld_x; p.ids = ids; p.weights = weights; p.w13 = w13; p.w2 = w2; p.ld13 = ld13; p.gs13 = w13_group_stride;
    p.ld2 = ld2; p.gs2 = w2_group_stride; p.s13 = s13; p.s2 = s2; p.s13_n = s13_n; p.s13_k = s13_k; p.s13_g = s13_group_stride;
    p.s2_n = s2_n; p.s2_k = s2_k; p.s2_g = s2_group_stride; p.h = reinterpret_cast<uint16_t*>(workspace);
    p.o = reinterpret_cast<float*>(workspace) + T * top_k * I; p.y = y; p.ld_y = ld_y;
    p.T = (int)T; p.H = (int)H; p.I = (int)I; p.E = (int)E; p.top_k = top_k;
    p.by_choice = T * top_k < E;
    return launch_moe(p, stream);
}
