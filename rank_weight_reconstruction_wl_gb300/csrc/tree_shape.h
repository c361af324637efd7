// tree_shape.h -- tile shapes of the tree attention kernel and the order of its
// ring.  Plain C++: the host compiles it as well, to check the ring's waits.
#pragma once

namespace wl {

constexpr int kTaTile = 128;     // positions per tile
constexpr int kTaFlush = 64;     // tiles summed in tensor memory before the sums move to fp32 partials

template <bool kE4M3, int DP, int RT>
struct TaShape {
    static constexpr int ES = kE4M3 ? 1 : 2;
    static constexpr int PARTS = kE4M3 ? 2 : 1;
    static constexpr int N = PARTS * RT;             // columns of both products
    static constexpr int ROWB = DP * ES;             // bytes of a cache row
    static constexpr int SLOTROW = ROWB < 256 ? ROWB : 256;
    static constexpr int NS = ROWB / SLOTROW;        // ring slots per K or V tile
    static constexpr int SLOT = kTaTile * SLOTROW;
    static constexpr int QB = N * ROWB;
    static constexpr int PW = 2 * RT;                // bytes of a position's weights
    static constexpr int PB1 = kTaTile * PW, PB = kE4M3 ? PB1 : 2 * PB1;  // bf16: the weights, then their remainders
    static constexpr int ROOM = (232448 - 3072 - QB - 2 * PB) / SLOT;
    static constexpr int SLOTS = ROOM < 10 ? ROOM : 10;
    // e4m3: an exponent for each row, behind the barriers where a small ring
    // leaves room there (and none elsewhere)
    static constexpr int QEXP = SLOTS < 10 ? 1728 : 3072;
    static constexpr int MISC = SLOTS < 10 ? 3072 : 3136;
    static constexpr int SMEM = MISC + QB + 2 * PB + SLOTS * SLOT;
    static constexpr int MT = DP / 128;              // M tiles of the second product
    static constexpr bool PP = RT <= 32;             // each softmax warpgroup has tiles and sums of its own
    static constexpr int USED = (2 + (PP ? 2 : 1) * MT) * N;  // two score buffers, the sums
    static constexpr int COLS = USED <= 64 ? 64 : USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
    static constexpr int KSTEP = 32 / ES;            // contraction elements per MMA: 32 bytes of a K-major row
    static constexpr int CW = PP ? RT : RT / 2;      // columns per softmax thread
    // Exponents of weights: the limit, and how far below it a moved reference
    // puts the largest weight.  e4m3 ends at 448, so the limit is 2^8, and the
    // gap is precision lost for fewer moves (8 trees of 20 to 32 tokens on 18000
    // to 32000 positions, and 8 of 39 to 61 on 3375 to 6000: 55 and 79 us with a
    // gap of 3, 51 and 73 with 5, which leaves two bits less).  bf16 has range to
    // spare.  kNear: a column that another column's move finds so near the limit
    // moves along.
    static constexpr float kTop = kE4M3 ? 8.0f : 64.0f, kGap = kE4M3 ? 3.0f : 64.0f, kNear = kE4M3 ? 2.0f : 0.0f;
    static constexpr int SWP = PW == 128 ? 2 : PW == 64 ? 4 : 6;  // swizzle code of the weights' rows
    // K and V boxes come from a warp each.  A warp waits for a free slot by
    // parity, which cannot tell "item X - SLOTS consumed" from "item X - 2 SLOTS
    // not yet": it needs to know the latter from its item before X (or, where
    // the two warps keep in step, from the other's).  The widest step from one
    // of a warp's items to its next is 2 NS + 1, at a change of segment, so a
    // ring of fewer slots has its warps keep in step there.
    static constexpr bool PACED = SLOTS < 2 * NS + 1;
    static_assert((2 * SLOTS + 11) * 8 <= (SLOTS < 10 ? QEXP : 1792) - 1536, "barriers");
    static_assert(SLOTS >= 2 * NS && SLOTS >= 4 && SMEM <= 232448 && USED <= 512 && RT % 16 == 0, "tile shape");
};

// Place of K or V of a segment's tile r (of n) among its ring items, which go
// K0, K1, V0, K2, V1, ..., K(n-1), V(n-2), V(n-1).
constexpr int ta_item(int r, int n, bool isv)
{
    return isv ? (r + 1 < n ? 2 * r + 2 : 2 * n - 1) : (r > 0 ? 2 * r - 1 : 0);
}

}  // namespace wl
