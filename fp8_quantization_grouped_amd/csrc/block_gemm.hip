// Block-scaled FP8 grouped GEMM on gfx950 matrix cores: e4m3fn operands with one fp32 factor per
// 128 elements of the contraction (1 x 128 blocks of activations and gradients, 128 x 128 blocks of
// weights).
//
//   forward, M-grouped:  c[m,n]   = sum_kb sa[kb,m] sb[g,n/128,kb] sum_{k in kb} A[m,k] B_g[n,k]
//   wgrad, K-grouped:    c[g,k,n] = sum_tb sa[tb,k] sb[tb,n] sum_{m in tb, g} A[k,m] B[n,m]
//
// One contraction step is one block, so v_mfma_f32_16x16x128_f8f6f4 makes a block's whole sum from
// zero, and each of its results is added to an accumulator times its factors by one fused
// multiply-add (the weight gradient: a product more).  Those run on the vector units while the
// matrix cores work on the next row of results: the sums of row i are added while row i + 1 is
// multiplied, four multiply-adds per 32-cycle matrix instruction.
//
// Tiles: TM x TN outputs by 8 waves, 128-byte steps, operands straight from memory into NS LDS
// stages (layout and swizzles: gemm_tile.hpp), one barrier per step, before its last row of results:
// by then every fragment of the step is in registers, so its stage takes the loads of the step NS
// later, and the next step's first fragments come during that row.  A step's load offsets are the
// tile's plus the step's position: they are held in registers (formed anew at each step, they delay
// the last row: 7% slower), and only steps that end or begin inside a block form masked ones.
//   256 x 256, 2 stages, one block per CU: a wave's 128 x 64 results fill its registers, and with
//     them the waves read 192 KB of LDS a step, the least that eight of them can.
//   128 x 128, 2 stages, two blocks per CU; 128 x 64, 3 stages, and 64 x 64, 4 stages, one block per
//     CU: for problems whose larger tiles would leave CUs without work (see pick_block_tile).
//
// Bound: delivery of the operands to the matrix cores, which are busy half of the time (49% by
// counters); at 256 x 256 a step's matrix instructions take 2048 cycles of a SIMD, and the step 3700.
// Measured: 8192 x 14336 x 4096 in one group 423 us, 2.3 PFLOP/s (20 us less with the loads taken away
// after the first step, half without the reads of A's fragments, 6% less without the factors); 49152
// rows in 64 groups, 1408 x 2048, 209 us (1.4 PFLOP/s of the products asked for: groups and columns
// that end inside a tile add a third); data gradient of 16384 rows in 32 groups, 2048 x 7168, 326 us,
// their weight gradient 498 us, of which 40 are stores, 56 the columns' factors and a quarter of the
// rest the groups' ends inside blocks.  Small: 512 x 2048 x 7168 26 us, a chain of 56 steps of 0.4 us.
//
// Measured and not kept: 16 waves per block, fragments of A read two rows ahead, wave priorities, the
// loads issued later in a step and B two steps ahead of the arithmetic (all within 1%); leaving out
// the multiplications of waves without rows or columns of the tile (64 experts 1% faster, dense 1%
// slower: the loads take as long), and the loads with them (2 to 4% slower); long and short tiles of
// the weight gradient in turn (same).
//
// Schedule (persistent blocks, no cross-block waits): as the other grouped GEMM.  Forward tiles go
// by group, in bands of 8 row tiles, an XCD's share in one piece; weight-gradient tiles by group
// size, largest first, in rounds.  Offsets are clamped into [0, M] before use, so any offsets
// content keeps every access in range.
#include <type_traits>

#include "common.hpp"
#include "gemm_tile.hpp"
#include "lds_dma.hpp"
#include "plan.hpp"

namespace fp8q {

struct BlockGemmArgs {
    const uint8_t* a;
    int64_t lda;
    const float* sa;
    int64_t ld_sa;
    const uint8_t* b;
    int64_t ldb, bgs;
    const float* sb;
    int64_t sb_n, sb_k, sb_g;  // strides by column block (forward), contraction block and group
    const int32_t* offsets;    // null: one group
    int G;
    int M, N, K;
    uint8_t* c;
    int64_t ldc;
    int32_t* status;           // null: not reported
    int nt_n, nt_k;            // column tiles; weight gradient: row tiles
    bool out_f32, vec_store, stream_out;
};

__device__ __forceinline__ v8i_t two_chunks(const uint8_t* lo, const uint8_t* hi) {
    const uint4 a = *reinterpret_cast<const uint4*>(lo), b = *reinterpret_cast<const uint4*>(hi);
    return v8i_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Group g's end, as the caller gave it.  Read as constant memory: a uniform group's comes by a scalar
// load, which the waits on the operands' loads do not count.
__device__ __forceinline__ int group_end(const BlockGemmArgs& p, int g) {
    typedef const __attribute__((address_space(4))) int32_t* const_i32;
    return p.offsets ? ((const_i32)(uintptr_t)p.offsets)[g] : p.M;
}

// The offsets check's two words, by one wave.
__device__ __forceinline__ void report_offsets(const BlockGemmArgs& p, int lane) {
    int bad = 0x7FFFFFFF;
    for (int i = lane; i < p.G; i += 64) {
        const int64_t lo = i == 0 ? 0 : group_end(p, i - 1), hi = group_end(p, i);
        if ((hi < lo || hi > p.M || (i == p.G - 1 && hi != p.M)) && i < bad) bad = i;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const int o = __shfl_xor(bad, off, 64);
        bad = o < bad ? o : bad;
    }
    if (lane == 0) {
        p.status[0] = bad == 0x7FFFFFFF ? (int32_t)FP8Q_OK : (int32_t)FP8Q_ERR_INVALID_ARG;
        p.status[1] = bad == 0x7FFFFFFF ? -1 : bad;
    }
}

template <int MODE, int TM, int TN, int NS>
__global__ __launch_bounds__(512, TM == 256 ? 2 : 4) void block_gemm_kernel(const BlockGemmArgs p) {
    constexpr bool FWD = MODE == MODE_FWD;
    constexpr int STAGE_A = TM * GK, STAGE_B = TN * GK, STAGE = STAGE_A + STAGE_B;  // bytes of a step's operands
    constexpr int NA = TM / 64, NB = TN / 64;      // each wave's loads of either
    constexpr int WC = TN > 64 ? 4 : 2;            // waves side by side
    constexpr int WM = TM * WC / 8, WN = TN / WC;  // a wave's rows and columns
    constexpr int MI = WM / 16, NJ = WN / 16;
    constexpr int NT = 512;
    __shared__ __align__(16) uint8_t smem[NS][STAGE];
    __shared__ __align__(16) float sscale[NS][TM + TN];  // by stage: factors of the tile's rows, columns
    __shared__ int s_pref[FWD ? GMAX + 1 : 1];           // forward: row tiles before each group
    __shared__ unsigned short s_perm[FWD ? 1 : GMAX];    // weight gradient: groups, most steps first
    __shared__ int s_busy;                               // and how many have any
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave / WC, wn = wave % WC;
    const int lr = lane & 15, lq = lane >> 4;

    auto end_of = [&](int g) -> int { return group_end(p, g); };
    // group g's rows, clamped so that any offsets content stays in range
    auto rows_of = [&](int lo, int hi, int& l, int& h) {
        l = lo < 0 ? 0 : lo > p.M ? p.M : lo;
        h = hi < l ? l : hi > p.M ? p.M : hi;
    };
    auto group_rows = [&](int g, int& l, int& h) { rows_of(g == 0 ? 0 : end_of(g - 1), end_of(g), l, h); };

    // --- the offsets check (block 0's last wave) and the schedule's table
    if (p.status != nullptr && blockIdx.x == 0 && wave == 7) report_offsets(p, lane);
    if (FWD) {
        if (wave == 0) {
            int base = 0;
            for (int g0 = 0; g0 < p.G; g0 += 64) {
                int l = 0, h = 0;
                if (g0 + lane < p.G) group_rows(g0 + lane, l, h);
                int n = (h - l + TM - 1) / TM;
#pragma unroll
                for (int off = 1; off < 64; off <<= 1) {
                    const int o = __shfl_up(n, off, 64);
                    if (lane >= off) n += o;
                }
                if (g0 + lane < p.G) s_pref[g0 + lane + 1] = base + n;
                base += __shfl(n, 63, 64);
            }
            if (lane == 0) s_pref[0] = 0;
        }
    } else {
        // a group's place is the number of groups with more steps, or as many and a lower index
        int* steps = reinterpret_cast<int*>(&smem[0][0]);
        if (t == 0) s_busy = 0;
        for (int g = t; g < p.G; g += NT) {
            int l, h;
            group_rows(g, l, h);
            l &= ~(GK - 1);
            steps[g] = h > l ? (h - l + GK - 1) / GK : 0;
        }
        __syncthreads();
        for (int g = t; g < p.G; g += NT) {
            const int mine = steps[g];
            int place = 0;
            for (int o = 0; o < p.G; o++) place += steps[o] > mine || (steps[o] == mine && o < g);
            s_perm[place] = (unsigned short)g;
            if (mine > 0) atomicMax(&s_busy, place + 1);
        }
    }
    __syncthreads();

    const int nb = gridDim.x, nx = nb % 8 == 0 ? 8 : 1;  // blocks are dealt to the 8 XCDs round-robin
    const int xcd = (int)blockIdx.x % nx, lb = (int)blockIdx.x / nx, bpx = nb / nx;
    // forward: the next tile and the last of the XCD's share; weight gradient: the next round
    struct Walk {
        int next, end;
    };
    Walk lead{0, 0};
    if (FWD) {
        const long long total = (long long)s_pref[p.G] * p.nt_n;  // < 2^31 (host check)
        lead.next = __builtin_amdgcn_readfirstlane((int)(total * xcd / nx) + lb);
        lead.end = __builtin_amdgcn_readfirstlane((int)(total * (xcd + 1) / nx));
    }
    // weight gradient: the groups with rows come first in the order
    const int tpg = p.nt_k * p.nt_n, w_tiles = FWD ? 0 : __builtin_amdgcn_readfirstlane(s_busy) * tpg;

    struct Tile {
        int g;
        int row, n0, rows, cols;       // first output row and column, rows and columns inside
        int k_lo, k_hi, k0, steps;     // contraction range, its first step's position, steps
    };
    auto next_tile = [&](Walk& w, Tile& x) -> bool {
        if (FWD) {
            const int ti = w.next;
            if (ti >= w.end) return false;
            int lo = 0, hi = p.G - 1;  // last group whose tiles start at or before ti
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_pref[mid] * p.nt_n <= ti) lo = mid; else hi = mid - 1;
            }
            x.g = lo;
            const int rt = s_pref[lo + 1] - s_pref[lo], l = ti - s_pref[lo] * p.nt_n;
            constexpr int BAND = 8;
            const int bt = BAND * p.nt_n, b = l / bt, r = l - b * bt;
            const int in_band = rt - b * BAND < BAND ? rt - b * BAND : BAND;
            x.n0 = (r / in_band) * TN;
            x.row = (b * BAND + r % in_band) * TM;  // relative to the group's start
            w.next += bpx;
        } else {
            const int round = w.next;
            int idx;
            if (nx == 8) {
                const int chunk = (round & 1) ? 7 - xcd : xcd;
                idx = round * nb + chunk * bpx + ((round & 1) ? bpx - 1 - lb : lb);
            } else {
                idx = round * nb + ((round & 1) ? nb - 1 - (int)blockIdx.x : (int)blockIdx.x);
            }
            if (idx >= w_tiles) return false;
            w.next++;
            x.g = s_perm[idx / tpg];
            const int l = idx % tpg;
            x.row = (l / p.nt_n) * TM;
            x.n0 = (l % p.nt_n) * TN;
        }
        // uniform, though read from LDS: keep the tile in scalar registers
        x.g = __builtin_amdgcn_readfirstlane(x.g);
        x.row = __builtin_amdgcn_readfirstlane(x.row);
        x.n0 = __builtin_amdgcn_readfirstlane(x.n0);
        int l, h;
        rows_of(x.g == 0 ? 0 : end_of(x.g - 1), end_of(x.g), l, h);
        if (FWD) {
            x.row += l;
            x.rows = h - x.row < TM ? h - x.row : TM;
            x.k_lo = 0;
            x.k_hi = p.K;
        } else {
            x.rows = p.K - x.row < TM ? p.K - x.row : TM;
            x.k_lo = l;
            x.k_hi = h;
        }
        x.k0 = x.k_lo & ~(GK - 1);
        x.steps = x.k_hi > x.k0 ? (x.k_hi - x.k0 + GK - 1) / GK : 0;
        x.cols = p.N - x.n0 < TN ? p.N - x.n0 : TN;
        return true;
    };

    // The loads run NS - 1 steps ahead of the arithmetic, across tiles.  What they are at: a tile, the
    // step's position, descriptors at the tile's first rows, and this lane's offset in each of the
    // wave's parts (8 rows x 128 bytes) of either operand.
    Tile src;
    int src_k = 0;
    bool src_ok;
    i32x4_t ra, rb;
    uint32_t oa[NA], ob[NB];
    const uint32_t smem_at = lds_addr(&smem[0][0]), scale_at = lds_addr(&sscale[0][0]);
    auto aim = [&]() {  // at the next tile
        src_ok = next_tile(lead, src);
        if (!src_ok) return;
        src_k = src.k0;
        ra = make_rsrc4(p.a + (int64_t)src.row * p.lda, (uint32_t)(src.rows * p.lda));
        rb = make_rsrc4(p.b + (FWD ? (int64_t)src.g * p.bgs : 0) + (int64_t)src.n0 * p.ldb, (uint32_t)(src.cols * p.ldb));
        int l = lane;
        asm volatile("" : "+v"(l));  // formed here, not held through the steps
        const int ch = l & 7;
#pragma unroll
        for (int i = 0; i < NA; i++) {
            const int row = wave * (8 * NA) + 8 * i + (l >> 3);
            oa[i] = row < src.rows ? (uint32_t)row * (uint32_t)p.lda + 16 * (ch ^ swz(row)) : OOB;
        }
#pragma unroll
        for (int i = 0; i < NB; i++) {
            const int row = wave * (8 * NB) + 8 * i + (l >> 3);
            ob[i] = row < src.cols ? (uint32_t)row * (uint32_t)p.ldb + 16 * (ch ^ swzB(row)) : OOB;
        }
    };
    // The loads of one step into a stage; each of the first waves also brings 64 factors.
    constexpr int FW = (TM + TN) / 64;
    int ahead = 0;                        // steps whose loads are on their way
    int cut_lo[NS - 1], cut_hi[NS - 1];  // weight gradient: the tokens of each that count
    auto issue = [&](int stage) {
        const uint32_t at_a = smem_at + stage * STAGE + wave * (NA * 1024), at_b = smem_at + stage * STAGE + STAGE_A + wave * (NB * 1024);
        const int kpos = __builtin_amdgcn_readfirstlane(src_k);
        if (kpos >= src.k_lo && kpos + GK <= src.k_hi) {
#pragma unroll
            for (int i = 0; i < (NA > NB ? NA : NB); i++) {
                if (i < NA) dma16_at(ra, oa[i < NA ? i : 0], kpos, at_a + i * 1024);
                if (i < NB) dma16_at(rb, ob[i < NB ? i : 0], kpos, at_b + i * 1024);
            }
        } else {  // chunks outside the range read as zeros
            int l = lane;
            asm volatile("" : "+v"(l));
            const int ch = l & 7;
#pragma unroll
            for (int i = 0; i < NA; i++) {
                const int pa = kpos + 16 * (ch ^ swz(wave * (8 * NA) + 8 * i + (l >> 3)));
                dma16(ra, pa < src.k_hi && pa + 16 > src.k_lo ? oa[i] + kpos : OOB, at_a + i * 1024);
            }
#pragma unroll
            for (int i = 0; i < NB; i++) {
                const int pb = kpos + 16 * (ch ^ swzB(wave * (8 * NB) + 8 * i + (l >> 3)));
                dma16(rb, pb < src.k_hi && pb + 16 > src.k_lo ? ob[i] + kpos : OOB, at_b + i * 1024);
            }
        }
        if (wave < FW) {
            const int row = (wave < NA ? wave : wave - NA) * 64 + lane;
            const int64_t kb = kpos / GK;
            const float* f;
            uint32_t o = (uint32_t)row * 4u;
            if (wave < NA) {
                f = p.sa + kb * p.ld_sa + src.row;
            } else if (FWD) {
                f = p.sb + (int64_t)src.g * p.sb_g + kb * p.sb_k;
                o = (uint32_t)((src.n0 + row) / GK) * (uint32_t)p.sb_n * 4u;
            } else {
                f = p.sb + kb * p.sb_k + src.n0;
            }
            dma4(make_rsrc4(f, 0x7FFFFFFFu), row < (wave < NA ? src.rows : src.cols) ? o : OOB, scale_at + stage * (4 * (TM + TN)) + wave * 256);
        }
        if (!FWD) {
#pragma unroll
            for (int d = 0; d < NS - 1; d++) {
                if (d == ahead) {
                    cut_lo[d] = src.k_lo - kpos;
                    cut_hi[d] = src.k_hi - kpos;
                }
            }
        }
        ahead++;
        src_k += GK;
        if (src_k >= src.k_hi) aim();
    };

    Walk follow = lead;
    aim();
    Tile cur;
    bool have = next_tile(follow, cur);
    int st = 0;  // stage of the current step
#pragma unroll
    for (int d = 0; d < NS - 1; d++)
        if (src_ok) issue(d);
    // The oldest step's loads, to a stage, have landed in every wave (NS - 2 steps' are younger), and
    // every wave has read what it takes from the stage before.
    auto arrive = [&](int stage) {
        if (NS > 2 && ahead == NS - 1) {
            if (wave < FW) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * (NA + NB + 1)) : "memory");
            else asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * (NA + NB)) : "memory");
        } else {
            wait_vm0();
        }
        if (!FWD) {
            const int lo = cut_lo[0], hi = cut_hi[0];
#pragma unroll
            for (int d = 0; d + 1 < NS - 1; d++) {
                cut_lo[d] = cut_lo[d + 1];
                cut_hi[d] = cut_hi[d + 1];
            }
            if (lo > 0 || hi < GK) {
                // zero the bytes of other groups' tokens (or of the padding past M) in the chunks that
                // the range cuts, in both operands: such a byte may be a NaN code.  Each wave does the
                // rows that it loaded, so its own wait suffices.
                int l = lane;
                asm volatile("" : "+v"(l));
                static_assert(FWD || TM == TN, "one count of rows");
                constexpr int OWN = 8 * NA;
                if (l < 2 * OWN) {
                    const int row = wave * OWN + (l & (OWN - 1));
                    const bool in_a = l < OWN;
                    uint8_t* side = smem[stage] + (in_a ? 0 : STAGE_A);
#pragma unroll
                    for (int ch = 0; ch < 8; ch++) {
                        const int b0 = 16 * ch;
                        if ((lo > b0 && lo < b0 + 16) || (hi > b0 && hi < b0 + 16)) {
                            uint4* q = reinterpret_cast<uint4*>(side + (in_a ? lds_off(row, ch) : lds_offB(row, ch)));
                            uint4 w = *q;
                            w.x &= keep_mask4(lo, hi, b0);
                            w.y &= keep_mask4(lo, hi, b0 + 4);
                            w.z &= keep_mask4(lo, hi, b0 + 8);
                            w.w &= keep_mask4(lo, hi, b0 + 12);
                            *q = w;
                        }
                    }
                }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // LDS reads and writes done
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        ahead--;
    };
    // this lane's fragments: A row wm * WM + lr (+ 16 i), B row brow(j, lr) of its columns
    const int fa0 = lds_off(wm * WM + lr, lq), fa1 = lds_off(wm * WM + lr, 4 + lq);
    const int fb0 = STAGE_A + lds_offB(wn * WN + brow(0, lr), lq), fb1 = STAGE_A + lds_offB(wn * WN + brow(0, lr), 4 + lq);
    v8i_t bf[NJ], af[2];  // rows of A in turn
    auto load_b = [&](const uint8_t* at, int j) {
        const int o = 32 * GK * (j >> 1) + 4 * GK * (j & 1);
        bf[j] = two_chunks(at + fb0 + o, at + fb1 + o);
    };
    auto load_a = [&](const uint8_t* at, int i) { af[i & 1] = two_chunks(at + fa0 + 16 * GK * i, at + fa1 + 16 * GK * i); };
    if (have) {
        arrive(0);
        if (src_ok) issue(NS - 1);
        load_a(smem[0], 0);
#pragma unroll
        for (int j = 0; j < NJ; j++) load_b(smem[0], j);
    }

    while (have) {
        v4f_t acc[MI][NJ];
#pragma unroll
        for (int i = 0; i < MI; i++)
#pragma unroll
            for (int j = 0; j < NJ; j++) acc[i][j] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
        // sums of the row multiplied last, waiting to be added times f (forward: across steps too)
        v4f_t sum[NJ];
        float f = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; j++) sum[j] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
        auto add_sums = [&](int i, int j, const v4f_t* sbv) {
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][j][e] = fmaf(FWD ? sum[j][e] : sum[j][e] * sbv[FWD ? 0 : j][e], f, acc[i][j][e]);
        };
        float fa[MI], sbu = 1.0f;
        v4f_t sbv[FWD ? 1 : NJ];
        // The order below is the order of issue (no scheduling across the barriers): while a matrix
        // instruction runs, the vector unit adds the sums that the same column block gave for the row
        // before, and the next row's fragment is read; in the last row the next step's first ones.
        auto row = [&](int i, const uint8_t* now, const uint8_t* next) {
            if (i + 1 < MI) load_a(now, i + 1);
            else if (MI > 1) load_a(next, 0);  // (MI even)
            const float f_new = FWD ? fa[i] * sbu : fa[i];
#pragma unroll
            for (int j = 0; j < NJ; j++) {
                if (FWD || i > 0) add_sums(i > 0 ? i - 1 : MI - 1, j, sbv);
                sum[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    bf[j], af[i & 1], v4f_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
                if (i == MI - 1) load_b(next, j);
                __builtin_amdgcn_sched_barrier(0);
            }
            f = f_new;
            if (i == MI - 1) {
                if (MI == 1) load_a(next, 0);
                if (!FWD) {
#pragma unroll
                    for (int j = 0; j < NJ; j++) add_sums(MI - 1, j, sbv);
                }
            }
        };
        auto first_rows = [&]() {  // factors, and all rows but the last
            const float* sa = &sscale[st][wm * WM + lr];
            const float* sb = &sscale[st][TM + wn * WN];
#pragma unroll
            for (int i = 0; i < MI; i++) fa[i] = sa[16 * i];
            if (FWD) sbu = sb[0];  // a wave's columns lie in one weight block
            else
#pragma unroll
                for (int j = 0; j < NJ; j++) sbv[FWD ? 0 : j] = *reinterpret_cast<const v4f_t*>(sb + 32 * (j >> 1) + 8 * lq + 4 * (j & 1));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i + 1 < MI; i++) row(i, smem[st], smem[st]);
        };
        first_rows();
        for (int s = 1; s < cur.steps; s++) {
            const int st_next = st + 1 < NS ? st + 1 : 0;
            arrive(st_next);
            if (src_ok) issue(st);
            __builtin_amdgcn_sched_barrier(0);
            row(MI - 1, smem[st], smem[st_next]);
            st = st_next;
            first_rows();
        }
        {
            const int st_next = st + 1 < NS ? st + 1 : 0;
            if (ahead > 0) {
                arrive(st_next);
                if (src_ok) issue(st);
            }
            row(MI - 1, smem[st], smem[st_next]);
            st = st_next;
        }
        if (FWD) {
#pragma unroll
            for (int j = 0; j < NJ; j++) {
#pragma unroll
                for (int e = 0; e < 4; e++) acc[MI - 1][j][e] = fmaf(sum[j][e], f, acc[MI - 1][j][e]);
            }
        }

        // Epilogue: lane rows wm * WM + 16 i + lr, and per pair of column blocks 8 consecutive
        // columns.  A row or column past the tile's last gets an offset past the buffer.
        const int64_t row0 = FWD ? (int64_t)cur.row : (int64_t)cur.g * p.K + cur.row;
        auto epilogue = [&](auto f32, auto stream) {
            constexpr bool F32 = decltype(f32)::value;
            constexpr int AUX = decltype(stream)::value ? 2 : 0;  // streaming stores
            constexpr uint32_t ESZ = F32 ? 4 : 2;
            const uint32_t ldc = (uint32_t)p.ldc * ESZ;
            const __amdgpu_buffer_rsrc_t rc =
                make_rsrc(p.c + (row0 * p.ldc + cur.n0) * ESZ, (uint32_t)(cur.rows - 1) * ldc + (uint32_t)cur.cols * ESZ);
            int el = lane;
            asm volatile("" : "+v"(el));  // the addresses are formed here, not held through the steps
            const int elr = el & 15, elq = el >> 4;
            if (p.vec_store && !F32 && NJ == 4) {
                // A wave's row is one 128-byte line.  Lanes 8 apart exchange half of what they hold, so
                // that an instruction writes 8 whole lines instead of 16 halves.
                const bool hi = elr >= 8;
                const int col = wn * WN + 8 * elq + (hi ? 32 : 0), row = wm * WM + (elr & 7);
                const uint32_t at = row * ldc + col * ESZ;
                const bool col_ok = col < cur.cols;
#pragma unroll
                for (int i = 0; i < MI; i++) {
                    i32x4_t keep, give;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const v4f_t v = acc[i][e >> 1], w = acc[i][(NJ > 2 ? 2 : 0) + (e >> 1)];
                        const int a = (int)pack_bf16x2(v[2 * (e & 1)], v[2 * (e & 1) + 1]);
                        const int b = (int)pack_bf16x2(w[2 * (e & 1)], w[2 * (e & 1) + 1]);
                        keep[e] = hi ? b : a;
                        give[e] = __builtin_amdgcn_mov_dpp(hi ? a : b, 0x128, 0xF, 0xF, true);  // row_ror:8
                    }
                    const i32x4_t first = hi ? give : keep, second = hi ? keep : give;
                    const uint32_t off = at + 16 * i * ldc;
                    __builtin_amdgcn_raw_buffer_store_b128(first, rc, col_ok && row + 16 * i < cur.rows ? off : OOB, 0, AUX);
                    __builtin_amdgcn_raw_buffer_store_b128(second, rc, col_ok && row + 16 * i + 8 < cur.rows ? off + 8 * ldc : OOB, 0, AUX);
                }
            } else if (p.vec_store) {
                const uint32_t at = (wm * WM + elr) * ldc + (wn * WN + 8 * elq) * ESZ;
#pragma unroll
                for (int jp = 0; jp < NJ / 2; jp++) {
                    const bool col_ok = wn * WN + 32 * jp + 8 * elq < cur.cols;
#pragma unroll
                    for (int i = 0; i < MI; i++) {
                        const uint32_t off = col_ok && wm * WM + 16 * i + elr < cur.rows ? at + 16 * i * ldc + 32 * jp * ESZ : OOB;
                        const v4f_t v = acc[i][2 * jp], w = acc[i][2 * jp + 1];
                        if (F32) {
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4_t, v), rc, off, 0, 0);
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4_t, w), rc, off + 16u, 0, 0);
                        } else {
                            __builtin_amdgcn_raw_buffer_store_b128(
                                i32x4_t{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3]), (int)pack_bf16x2(w[0], w[1]), (int)pack_bf16x2(w[2], w[3])},
                                rc, off, 0, 0);
                        }
                    }
                }
            } else {
                // any N, ldc and alignment: the same 8 columns of a lane in stores that need no alignment
                // but the element's, one by one where the tile's last columns cut them
                typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(2)));
                typedef __attribute__((address_space(1))) uint8_t* gptr;
                const gptr base = (gptr)(uintptr_t)(p.c + (row0 * p.ldc + cur.n0) * ESZ);
#pragma unroll
                for (int i = 0; i < MI; i++) {
                    const int row = wm * WM + 16 * i + elr;
                    if (row >= cur.rows) continue;
#pragma unroll
                    for (int jp = 0; jp < NJ / 2; jp++) {
                        const int col = wn * WN + 32 * jp + 8 * elq;
                        const gptr at = base + (uint32_t)row * ldc + (uint32_t)col * ESZ;
                        const v4f_t v = acc[i][2 * jp], w = acc[i][2 * jp + 1];
                        if (col + 8 <= cur.cols) {
                            if (F32) {
                                *(__attribute__((address_space(1))) i32x4_any*)at = __builtin_bit_cast(i32x4_t, v);
                                *(__attribute__((address_space(1))) i32x4_any*)(at + 16) = __builtin_bit_cast(i32x4_t, w);
                            } else {
                                *(__attribute__((address_space(1))) i32x4_any*)at =
                                    i32x4_t{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3]), (int)pack_bf16x2(w[0], w[1]), (int)pack_bf16x2(w[2], w[3])};
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; e++) {
                                const float x = e < 4 ? v[e & 3] : w[e & 3];
                                if (col + e >= cur.cols) continue;
                                if (F32) ((__attribute__((address_space(1))) float*)at)[e] = x;
                                else ((__attribute__((address_space(1))) uint16_t*)at)[e] = (uint16_t)pack_bf16x2(x, 0.0f);
                            }
                        }
                    }
                }
            }
        };
        if (p.out_f32) epilogue(std::true_type{}, std::false_type{});
        else if (NJ == 4 && p.stream_out) epilogue(std::false_type{}, std::true_type{});
        else epilogue(std::false_type{}, std::false_type{});
        have = next_tile(follow, cur);
    }
    // weight gradient: the groups without rows
    if (!FWD) {
        const int esz = p.out_f32 ? 4 : 2;
        for (int idx = w_tiles + (int)blockIdx.x; idx < p.G * tpg; idx += nb) {
            const int g = s_perm[idx / tpg], l = idx % tpg, r0 = l / p.nt_n * TM, c0 = l % p.nt_n * TN;
            const int width = p.vec_store ? 8 : 1;  // columns of a thread
            for (int i = t; i < TM * TN / width; i += NT) {
                const int row = r0 + i * width / TN, col = c0 + i * width % TN;
                if (row < p.K && col < p.N) {
                    uint8_t* dst = p.c + (((int64_t)g * p.K + row) * p.ldc + col) * esz;
                    if (p.vec_store) {
                        reinterpret_cast<uint4*>(dst)[0] = make_uint4(0, 0, 0, 0);
                        if (p.out_f32) reinterpret_cast<uint4*>(dst)[1] = make_uint4(0, 0, 0, 0);
                    } else if (p.out_f32) {
                        *reinterpret_cast<float*>(dst) = 0.0f;
                    } else {
                        *reinterpret_cast<uint16_t*>(dst) = 0;
                    }
                }
            }
        }
    }
}

// The forward's output where there is nothing to sum (K == 0), and its offsets check.
__global__ __launch_bounds__(256) void block_zero_kernel(const BlockGemmArgs p) {
    if (p.status != nullptr && blockIdx.x == 0 && threadIdx.x < 64) report_offsets(p, threadIdx.x);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)p.M * p.N; i += (int64_t)gridDim.x * 256) {
        const int64_t at = i / p.N * p.ldc + i % p.N;
        if (p.out_f32) reinterpret_cast<float*>(p.c)[at] = 0.0f;
        else reinterpret_cast<uint16_t*>(p.c)[at] = 0;
    }
}

template <int MODE, int TM, int TN, int NS>
static fp8q_status_t launch_block_gemm(BlockGemmArgs p, hipStream_t stream) {
    p.nt_n = (p.N + TN - 1) / TN;
    p.nt_k = MODE == MODE_FWD ? 1 : (p.K + TM - 1) / TM;
    if (MODE == MODE_FWD && p.K == 0) {
        block_zero_kernel<<<dim3(1024), dim3(256), 0, stream>>>(p);
        FP8Q_CHECK_LAUNCH();
        return FP8Q_OK;
    }
    const int64_t tiles = MODE == MODE_FWD ? ((int64_t)(p.M + TM - 1) / TM + p.G) * p.nt_n : (int64_t)p.G * p.nt_k * p.nt_n;
    // offsets that go up and down can make every group as long as M
    const int64_t most = MODE == MODE_FWD ? (int64_t)p.G * ((p.M + TM - 1) / TM) * p.nt_n : tiles;
    if (tiles >= 0x7FFF0000LL || most >= 0x7FFF0000LL) return FP8Q_ERR_UNSUPPORTED;
    int64_t grid = (int64_t)num_cus() * (TM == 256 || NS > 2 ? 1 : 2);
    if (tiles < grid) grid = (tiles + 7) / 8 * 8;  // whole rounds of the XCDs
    block_gemm_kernel<MODE, TM, TN, NS><<<dim3((unsigned)grid), dim3(512), 0, stream>>>(p);
    FP8Q_CHECK_LAUNCH();
    return FP8Q_OK;
}

template <int MODE>
static fp8q_status_t launch_picked(const BlockGemmArgs& p, hipStream_t stream) {
    constexpr bool FWD = MODE == MODE_FWD;
    switch (pick_block_tile(FWD, p.M, p.N, p.K, p.G, num_cus())) {
        case TILE_64: return launch_block_gemm<MODE, 64, 64, 4>(p, stream);
        case TILE_128X64: return launch_block_gemm<MODE_FWD, 128, 64, 3>(p, stream);
        case TILE_128: return launch_block_gemm<MODE, 128, 128, 2>(p, stream);
        case TILE_256: break;
    }
    return launch_block_gemm<MODE, 256, 256, 2>(p, stream);
}

}  // namespace fp8q

extern "C" fp8q_status_t fp8_block_grouped_gemm(fp8q_gemm_mode_t mode, const uint8_t* a, int64_t lda,
                                                const float* a_scales, int64_t ld_sa, const uint8_t* b,
                                                int64_t ldb, int64_t b_group_stride, const float* b_scales,
                                                int64_t sb_n, int64_t sb_k, int64_t sb_group_stride,
                                                const int32_t* offsets, int32_t groups, int64_t M, int64_t N,
                                                int64_t K, void* c, int64_t ldc, fp8q_out_t out_dtype,
                                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace fp8q;
    const bool fwd = mode == FP8Q_GEMM_FWD_MGROUPED;
    if (!fwd && mode != FP8Q_GEMM_WGRAD_KGROUPED) return FP8Q_ERR_INVALID_ARG;
    if (groups < 1 || M < 0 || N < 0 || K < 0 || ldc < N || (!offsets && groups != 1) || sb_n < 0 || sb_k < 0 ||
        sb_group_stride < 0 || b_group_stride < 0)
        return FP8Q_ERR_INVALID_ARG;
    if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_FP32) return FP8Q_ERR_INVALID_ARG;
    const int64_t esz = out_dtype == FP8Q_OUT_FP32 ? 4 : 2;
    if (workspace && workspace_bytes < 256) return FP8Q_ERR_WORKSPACE;
    if (!fp8q_aligned(workspace, 4) || !fp8q_aligned(a_scales, 4) || !fp8q_aligned(b_scales, 4) || !fp8q_aligned(c, (uintptr_t)esz))
        return FP8Q_ERR_INVALID_ARG;
    const int64_t inner = fwd ? K : M, rows = fwd ? M : K;
    if (lda < inner || ldb < inner || ld_sa < rows) return FP8Q_ERR_INVALID_ARG;
    if (!fwd && (b_group_stride != 0 || sb_group_stride != 0 || sb_n != 1 || sb_k < N)) return FP8Q_ERR_INVALID_ARG;
    if (N == 0 || rows == 0) return FP8Q_OK;
    if (!c || (inner > 0 && (!a || !b || !a_scales || !b_scales))) return FP8Q_ERR_INVALID_ARG;
    if (lda % 16 || ldb % 16 || !fp8q_aligned(a, 16) || !fp8q_aligned(b, 16)) return FP8Q_ERR_UNSUPPORTED;
    if (fwd && (K % 16 || b_group_stride % 16)) return FP8Q_ERR_UNSUPPORTED;
    // 32-bit tile indices, contraction positions and offsets within 256 rows; a column block's
    // factor is reached with a 32-bit byte offset
    constexpr int64_t most = 0x7FFFFF00LL;
    if (groups > GMAX || M > most || N > most || K > most || lda > most / 256 || ldb > most / 256 || ldc > most / (256 * esz) ||
        (fwd && sb_n > (1LL << 29) / (N / GK + 1)))
        return FP8Q_ERR_UNSUPPORTED;
    BlockGemmArgs p{};
    p.a = a; p.lda = lda; p.sa = a_scales; p.ld_sa = ld_sa; p.b = b; p.ldb = ldb; p.bgs = b_group_stride;
    p.sb = b_scales; p.sb_n = sb_n; p.sb_k = sb_k; p.sb_g = sb_group_stride; p.offsets = offsets; p.G = groups;
    p.M = (int)M; p.N = (int)N; p.K = (int)K; p.c = reinterpret_cast<uint8_t*>(c); p.ldc = ldc;
    p.status = reinterpret_cast<int32_t*>(workspace); p.out_f32 = out_dtype == FP8Q_OUT_FP32;
    // an output that cannot stay in the last-level cache goes past it (dense 466 -> 454 us, gradients of
    // 32 experts 862 -> 839 us)
    p.stream_out = (double)(fwd ? M : groups * K) * N * esz > kStreamBytes;
    p.vec_store = N % 8 == 0 && ldc % 8 == 0 && fp8q_aligned(c, 16);
    return fwd ? launch_picked<MODE_FWD>(p, stream) : launch_picked<MODE_WGRAD>(p, stream);
}
