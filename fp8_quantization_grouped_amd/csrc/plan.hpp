// Which variant of the block-scaled kernels a call takes: rules on sizes and the chip's CUs alone, in
// plain C++ so that they can be checked without a GPU.  Times are of an MI355X (256 CUs), those of one
// comparison taken together.
#pragma once

#include <stdint.h>

namespace fp8q {

static inline int64_t plan_up(int64_t n, int64_t by) { return (n + by - 1) / by; }

// ------------------------------------------------------------------ block-scaled grouped product

enum BlockTile { TILE_64 = 0, TILE_128X64 = 1, TILE_128 = 2, TILE_256 = 3 };

// Output tile of a product.  fwd: M x N outputs in G groups of rows; else G outputs of K x N.
static inline BlockTile pick_block_tile(bool fwd, int64_t M, int64_t N, int64_t K, int64_t G, int64_t cus) {
    // Where CUs would be left over, smaller tiles and loads further ahead, one block per CU (1 group, 7168
    // long): 512 x 2048 in 64-tiles 24 us, in 128 x 64-tiles 27, in 128-tiles 42; 1024 x 2048 in 128 x
    // 64-tiles 28 us, in 128-tiles 42, in 64-tiles, two for every CU, 34.  Every group but one ends inside
    // a tile, on average half way.
    const int64_t ends = (G - 1) / 2;
    if (fwd) {
        if ((plan_up(M, 64) + ends) * plan_up(N, 64) <= cus) return TILE_64;
        if ((plan_up(M, 128) + ends) * plan_up(N, 64) <= cus) return TILE_128X64;
    } else if (G * plan_up(K, 64) * plan_up(N, 64) <= cus) {
        return TILE_64;
    }
    // 128-tiles where 256-tiles would not give every CU one: 2048 x 2048 x 2048 in one group 26 against
    // 40 us, 4096 x 2048 x 2048 34 against 43 us; with a tile for each, 256 is faster: 4096 x 4096 x
    // 2048 47 against 53 us, weight gradient of 8 groups of 1024 x 2048 28 against 31 us
    if (plan_up(fwd ? M : G * K, 256) * plan_up(N, 256) < cus) return TILE_128;
    // Forward tiles are of one length, so a launch takes whole rounds of them: a round of two 128-tiles a
    // CU takes 0.65 as long as one of a 256-tile each, and few rounds of cut tiles can come out shorter
    // (16384 rows in 64 groups, 1408 x 2048: 76 against 92 us; 4096 rows in 8 groups, 4096 x 4096: 91
    // against 110).  The rule knows the groups' ends by their number alone and loses where they fall well:
    // 6000 x 4096 x 4096 takes 115 us, in 256-tiles 110.  Past three rounds the larger tile's fewer loads
    // count (49152 rows in 64 groups: 235 against 207 us, though the rounds are even).
    if (fwd) {
        const int64_t r256 = plan_up((plan_up(M, 256) + ends) * plan_up(N, 256), cus);
        const int64_t r128 = plan_up((plan_up(M, 128) + ends) * plan_up(N, 128), 2 * cus);
        if (r256 <= 3 && 65 * r128 < 100 * r256) return TILE_128;
    }
    return TILE_256;
}

// ----------------------------------------------------------------------- layer for a few tokens

constexpr int moe_lds(int nw) { return 8192 * nw; }  // staged activations of a block: 16 waves share a CU
// Waves of a block, and the most parts of the contraction, by token tiles of 16 in a pass; the down
// product stages two planes.
constexpr int moe_waves(int mt) { return mt == 1 ? 4 : 8; }
constexpr int moe_parts(int mt, bool down) { return mt == 1 ? 4 : mt == 2 ? (down ? 2 : 4) : 1; }

struct StreamPlan {
    int mt;     // token tiles of 16 in a pass
    int pass;   // tokens of an expert that one pass takes: a power of two
    int parts;  // of the contraction: 1, 2 or 4
};

// One of the layer's two products: gate and up (rows = I pairs of 16, contraction H) or down (rows = H,
// contraction I).
static inline StreamPlan pick_stream(bool down, int64_t T, int64_t top_k, int64_t E, int64_t H, int64_t I, int64_t cus) {
    const int64_t experts = T * top_k < E ? T * top_k : E;
    const int64_t waves = experts * (down ? plan_up(H, 32) : I / 16);  // of one part
    const int64_t blocks = plan_up(down ? I : H, 128), chip = 16 * cus;  // waves that run at a time
    StreamPlan p;
    // The tokens of an expert that one pass takes: as many as may come, since a second pass reads the
    // weights again (65 us for 64 tokens of 32 experts of 2048 x 7168 in passes of 32).  Where the waves
    // leave half of the chip idle, the chain of one wave's blocks counts instead, and passes of 32 leave
    // room for two parts of it: 34 tokens of 4 experts of 4096 x 1024, 2 a token, 78 -> 52 us, 128 tokens
    // 165 -> 125; 64 tokens of 4 experts of 816 x 1920, all four of them, 63 -> 52 us.  Passes of 16 were
    // slower than those of 32 from 17 tokens on (1024 x 4096, 28 tokens: 52 against 45 us).
    const bool idle = waves < chip / 2 && blocks >= 3;
    p.mt = T <= 16 ? 1 : T <= 32 || idle ? 2 : 4;
    p.pass = 1;
    while (p.pass < T && p.pass < 16 * p.mt) p.pass *= 2;
    // Parts of the contraction: two unless there are waves for the chip twice over, four below half of
    // that, each with 4 blocks or more, or 3 for two parts where most of the chip is idle (layers of 32
    // experts of 2048 x 7168, 8 of them a token: 1 token 78 us in four parts, 79 in two, 88 in one; 5
    // tokens 231, 230 and 252; 24 tokens of 64 experts of 1408 x 2048 120 us in two, 129 in one).  In
    // passes of 64 tokens one part stages them best (64 tokens 315 us, in two parts 326).  One block of
    // every part has to fit half the staging buffer (2^8 bytes a row and plane).
    const int planes = down ? 2 : 1;
    p.parts = 1;
    while (2 * p.parts <= moe_parts(p.mt, down) && 2 * p.parts * planes * p.pass * 256 <= moe_lds(moe_waves(p.mt)) / 2 &&
           waves * p.parts < (p.parts == 1 ? 2 * chip : chip) && blocks >= (waves * p.parts < chip / 2 ? 3 : 8) * p.parts)
        p.parts *= 2;
    return p;
}

// One block takes a token's whole router: 4 x 256 in 3.4 us against 5.5 us in two launches, but 64 x
// 2048 in 15 us against 10 us.
static inline bool route_is_small(int64_t H, int64_t E) { return E <= 256 && E * H <= (1 << 14); }

// Parts of the contraction: blocks for half of the CUs, at least 8 instructions' worth of H for each of a
// block's waves.  The workspace's size goes by them, so they do not depend on the device.
static inline int route_splits(int64_t T, int64_t H, int64_t E) {
    const int64_t blocks = plan_up(T, 16) * plan_up(E, 16);
    int64_t s = 128 / blocks;
    const int64_t most = H / (4 * 8 * 32);
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

}  // namespace fp8q
