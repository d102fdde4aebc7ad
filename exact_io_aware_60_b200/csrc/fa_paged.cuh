// fa_paged.cuh -- attention of a step's new tokens over a paged key/value cache.
//
// Sequence b holds cache_len[b] tokens and new_len[b] new ones (one token, a chain or a tree
// of drafted tokens), all in the cache's pages.  New token t of b sees every held key and the
// new keys its mask row names (chain: keys up to itself).  The G query heads of a key/value
// head are packed with the tokens into tiles of ROWS rows (row r = token r / G, head r % G),
// so that the cache is read once for all of them:
//   S = Q K^T on tcgen05 (M = 128 rows, 128 keys), online softmax with a running maximum m
//   and sum l per row, O += P V.
//
// Bound by memory for up to about 256 rows per key/value head (4 R flop per 2 bytes against
// 260 flop per byte of the card): a 128-key tile of one SM's share of HBM takes 1.5 us at
// d = 128, 0.75 us at d = 64.  Measured on B200 (kernels in a graph, three sets of inputs in
// turn): one token for each of 8 sequences of 32768 keys, 16 heads over 4, d = 128, 86 us, 6.3
// TB/s = 0.96 of the measured copy rate; at d = 64 50 us, 0.82; a chunk of 512 tokens against
// 15872 keys, 16 heads, d = 128, 83 us, 810 TFLOP/s; 16 sequences of up to 8000 keys, trees of
// 16 tokens, 32 heads over 8, pages of 16, 58 us.
//
// Precision: scores, maxima, sums, O and the pieces are fp32.  The weights are rounded to the
// element type, as the tensor cores take one 16-bit type for P and V and a second product for
// the rest of P would double the time of P V; O is divided by the sum of the rounded weights,
// so that their rounding has no bias.  Against 64 bits O is then off by 1.3 to 1.4 times what
// fp32 weights give with the same last rounding (bf16 2.2e-3 against 1.7e-3 of the norm, fp16
// 2.8e-4 against 2.1e-4); the log-sum-exp is of the unrounded weights.
//
// Work: the 128-key tiles of all (sequence, key/value head, row tile) items form one flat
// list that is cut into equal shares, one per CTA, wherever the cuts fall (lengths are only
// known on the device).  An item inside one share is written to O directly; the pieces of a
// cut item go to the workspace as fp32 (normalised O, log-sum-exp) and a second kernel,
// launched early by PDL, merges them in a fixed order.
//
// CTA: softmax warps (one row per thread, 4 per row tile), then one or two loaders (page table
// and TMA of K and V), one issuer of S, one of P V, and one that works out the CTA's pieces of
// work two ahead of the others (its lookups of lengths, about 1 us an item, are off everybody's
// path), loads Q and repairs V tiles (see repair).  Two issuers, because a commit leaves the
// tensor core idle for about 150 cycles in the stream of one: S and P V of 128 keys x 128 rows
// at d = 128, committed each, took 1330 cycles from one thread and 1075 from two.
//
// Few rows (REP = 4: a tile of 32 rows, REP = 2: 64): the rows are repeated in the tile's
// REP lane quarters / halves, and each copy takes 1 / REP of the keys of every tile as a
// softmax of its own (P is zero elsewhere); the copies are merged in the epilogue.  The
// exponentials of a tile then take 1 / REP of the time.
// At d = 64, where a tile's bytes take less than its 128 exponentials a row, one row tile can
// have two groups of softmax warps (KS = 2) that take the key tiles in turn, each with an O of
// its own, merged in the epilogue (16 sequences of 4000 keys, 32 new tokens, 32 heads over 8:
// 52 us with one group, 44 with two; of 600 keys 18.2 and 18.8, so that fa_fwd_paged chooses).
// Many rows (RT = 2): two tiles of 128 rows share every K and V tile, each with softmax warps
// of its own, so that one tile's products run beside the other's exponentials.
#pragma once

#include <cuda.h>

#include "fa_rope.cuh"
#include "sm100.cuh"

namespace fa {

struct PagedParams {
    Rows o;              // [B, H, T, d]
    Rows vc;             // the value cache (also behind the tensor map)
    float *lse;          // [B, H, T]
    PageTable pt;
    const uint8_t *tree; // [B or 1, T, T], nullptr: chain
    long long tree_sb;   // bytes between sequences (0: shared)
    float *part_o;       // [2 * gridDim.x][rows of an item][D]
    float *part_lse;     // [2 * gridDim.x][rows of an item], base 2
    int B, Hk, G, T;
    unsigned gp_magic;   // r / GP = r * gp_magic >> 16 for r < 128
    int GP, GT;          // heads of a row tile; row tiles that a token's G heads take (1 up to
                         // 128 heads to a key/value head)
    int TPT;             // tokens of a row tile: (rows of a tile) / GP
    int uncut;           // items are not cut: a share is a number of whole items
    int row_tiles;       // items of a (sequence, key/value head): ceil(T / (TPT * RT)) * GT
    int ctas;            // shares
    float scale_log2;
};

template <int D, int REP, int RT, int KS_ = 1>
struct PagedCfg {
    static_assert(REP == 1 || RT == 1, "copies of one row tile, or two row tiles");
    static constexpr int BN = 128;              // keys per tile
    static constexpr int ROWS = 128 / REP;      // rows of a row tile
    static_assert(KS_ == 1 || (KS_ == 2 && D == 64 && REP == 1 && RT == 1), "two groups: one row tile at d = 64");
    static constexpr int KS = KS_;              // softmax groups of a row tile
    static constexpr int HALVES = D / 64;
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int TILE = BN * D * 2;     // K or V tile
    static constexpr int HALF = BN * 128;       // one 64-element column block of a tile
    // rings of K and V tiles (V, used later, has the odd slot: 62 -> 56 us for decoding 32K
    // keys at d = 64 from pages of 16)
    static constexpr int NK = (D == 64) ? 5 : 2;
    static constexpr int NV = (D == 64) ? (RT == 1 && KS == 1 ? 6 : 5) : (RT == 1 ? 3 : 2);
    // epilogue: REP > 1, a 32-column block of every row and copy, rows padded to 36 columns;
    // else 32 rows x 32 columns of 16 bits for each softmax warp (with two groups too: the one
    // that writes changes from piece to piece, and no barrier stands between a piece of one tile,
    // which its group writes, and a piece of none, which the first does)
    static constexpr int SOFT = 4 * RT * KS;    // softmax warps
    static constexpr int STAGE = SOFT * 2048;
    static constexpr int MERGE = (REP > 1) ? 128 * 36 * 4 : STAGE + (KS > 1 ? 128 * 36 * 4 + 3 * 256 * 4 : 0);
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = OFF_Q + RT * QTILE;
    static constexpr int OFF_MERGE = OFF_RING + (NK + NV) * TILE;
    static constexpr int OFF_BAR = OFF_MERGE + MERGE;
    static constexpr int USED = OFF_BAR + 3200 + 8192;
    static constexpr int SMEM = USED + 1024;
    // K and V come from a warp each where the registers allow one more: a box takes about
    // 45 ns to issue, and pages of 16 tokens are 32 boxes a tile at d = 128.
    static constexpr int LOADERS = (SOFT == 4) ? 2 : 1;
    static constexpr int THREADS = 32 * (SOFT + 3 + LOADERS);
    // The softmax goes in steps: whole tiles (RT = 1) or 64 keys (RT = 2), whose scores a
    // thread holds in registers, so that the one score buffer that TMEM has room for at
    // d = 128 is free for the next step's S at once.  (A chunk of 512 tokens against 16K keys,
    // d = 128: 103 us in steps of 128 with P over S, 93 us in steps of 64 with two buffers and
    // P over S, 87 us in this form.)
    static constexpr int SPT = RT;              // steps of a tile
    static constexpr int STEP = BN / SPT;       // keys of a step
    static constexpr int NSB = (RT == 1 || D == 64) ? 2 : 1;  // score buffers of a row tile
    // TMEM columns of a row tile: scores, two buffers of P; then O of both
    static constexpr uint32_t S_BUF = STEP;
    static constexpr uint32_t COL_P = NSB * STEP;
    static constexpr uint32_t S_TILE = NSB * STEP + STEP;
    static constexpr uint32_t P_BUF = STEP / 2;
    static constexpr uint32_t COL_O = RT * S_TILE;
    static_assert(COL_O + RT * KS * D <= 512, "TMEM budget");
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct PagedBars {
    uint64_t q_full, q_empty, o_empty;
    // The MMA issuer asks for the repair of a tile's V once the tile's S is issued: from then
    // on the tile's vfull phase is the current or the last one, so that the parity that the repairing
    // warp waits for is unambiguous.  (Four in turn: S runs at most four tiles ahead of a
    // repair, as P V of the first waits for it.)
    uint64_t need[4];
    uint64_t s_full[4], s_empty[4];   // index: NSB * row tile + score buffer
    uint64_t p_full[4], pv_done[4];   // index: 2 * row tile + buffer of P
    // Fills are announced per tile (mod 8; a ring holds at most 6), slots released per slot.
    // fixed: V repaired.
    uint64_t kfull[8], vfull[8], fixed[8];
    uint64_t kempty[6], vempty[6];
    uint64_t seg_full[4], seg_empty[4];
    uint64_t mask_full[2], mask_empty[2];
    uint32_t tmem_base;
    int4 seg[4][3];         // ring of pieces (PagedSeg)
    uint32_t bad[16];       // per tile: sub-pages whose page number is outside the cache
    // Item t & 3 hides keys whose V is not finite.  (Four: the repairing warp reaches item
    // t + 4 only after the softmax of item t + 1 began.)
    int poison[4];
    float stat[3][128];     // merge of copies: m, l, l of the rounded weights
    uint32_t mask[2][1024]; // per token of the piece, up to 128 bits: the new keys it sees
};

// Work units of a sequence: for each of its items with a new token the key tiles and kItemCost
// for what an item costs by itself (its first scores, its epilogue: about 4 us against 1 to
// 1.5 us a tile; 16 ragged sequences with trees of 16 tokens: 69, 64, 60 us at 1, 2, 3), one for an item without (its rows are written as empty).
constexpr int kItemCost = 3;
struct PagedSeq {
    int past, fresh, tiles, valid;  // valid: items that hold a new token
    int per_head;
};
template <int RT>
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams &p, int b) {
    PagedSeq s;
    page_lengths(p.pt, p.T, b, s.past, s.fresh);
    s.tiles = (s.past + s.fresh + 127) >> 7;
    s.valid = (s.fresh + p.TPT * RT - 1) / (p.TPT * RT) * p.GT;
    s.per_head = s.valid * (s.tiles + kItemCost) + (p.row_tiles - s.valid);
    return s;
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive prefix sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// The shares: W units over G CTAs, the first W % G of them with one unit more.
struct PagedShares {
    int q, extra;  // units of a share; shares with one more
    __device__ __forceinline__ void init(int W, int ctas) {
        const int G = max(min(ctas, W), 1);
        q = W / G;
        extra = W - q * G;
    }
    __device__ __forceinline__ int begin(int c) const { return c * q + min(c, extra); }
    __device__ __forceinline__ int of(int u) const {  // the share of unit u
        const int lead = extra * (q + 1);
        return u < lead ? u / (q + 1) : extra + (u - lead) / q;
    }
};

// One piece of work: key tiles [j0, j1) of one item.
struct PagedSeg {
    int b, hk;          // sequence, key/value head
    int tok0, g0;       // first token of the rows, first of its heads
    int past, total;    // keys held, keys with the new ones
    int fresh;
    int j0, j1;
    int slot;           // of the workspace, if the item was cut
    int whole;
    // Keys that every new token from `tok` on sees: the held ones, and in a chain the new
    // ones up to `tok`.
    __device__ __forceinline__ int open(const PagedParams &p, int tok) const {
        return p.tree ? past : min(past + tok + 1, total);
    }
    // Whether V tile j is gone over: slots behind the last key, whose contents are
    // unspecified, are cleared (0 * NaN would reach O), and so are values that are not
    // finite in keys that some row does not see.
    __device__ __forceinline__ bool repair(const PagedParams &p, int j) const {
        return (j + 1) * 128 > open(p, tok0);
    }
};

// All ones in the halves of a 16-bit pair that are infinite or NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
    constexpr uint32_t e = BF16 ? 0x7F807F80u : 0x7C007C00u;
    return __vcmpeq2(w & e, e);
}

// Works out this CTA's pieces, in order (one whole warp; the lanes share the lookups: a group
// of 32 sequences, one per lane), and hands them over.
template <int RT>
struct PagedWalk {
    int u, u1;          // the share's next unit, its end
    int k0, base;       // the group with unit u, the units before it
    int mine, upto;     // units of the lane's sequence, sums up to it
    PagedSeq sq;
    int n;              // pieces handed over
    bool first, done;

    __device__ __forceinline__ void load(const PagedParams &p, int k, int lane) {
        k0 = k;
        mine = 0;
        if (k + lane < p.B) {
            sq = paged_seq<RT>(p, k + lane);
            mine = sq.per_head * p.Hk;
        }
    }
    // Share c of all units; returns the shares.
    __device__ __forceinline__ PagedShares init(const PagedParams &p, int c, int lane) {
        int W = p.B * p.Hk * p.row_tiles;  // uncut: a unit is an item, no length is needed
        if (!p.uncut) {
            W = 0;
            for (int k = 0; k < p.B; k += 32) {
                load(p, k, lane);
                W += warp_sum(mine);
            }
            if (p.B > 32) load(p, 0, lane);
            base = 0;
            upto = warp_scan(mine, lane);
        }
        PagedShares sh;
        sh.init(W, p.ctas);
        u = min(sh.begin(c), W);
        u1 = min(sh.begin(c + 1), W);
        n = 0;
        first = true;
        done = false;
        return sh;
    }
    // The sequence with unit u, and u's place in its head `hk` (u must not go back).
    struct Place {
        int b, hk, r, past, fresh, tiles, valid;
    };
    __device__ __forceinline__ Place place(const PagedParams &p, int lane) {
        if (p.uncut) {
            const int per = p.Hk * p.row_tiles, b = (unsigned)u / (unsigned)per, r0 = u - b * per;
            const int hk = (unsigned)r0 / (unsigned)p.row_tiles;
            const PagedSeq s = paged_seq<RT>(p, b);
            return Place{b, hk, r0 - hk * p.row_tiles, s.past, s.fresh, s.tiles, s.valid};
        }
        for (int all; base + (all = __shfl_sync(0xffffffffu, upto, 31)) <= u;) {
            base += all;
            load(p, k0 + 32, lane);
            upto = warp_scan(mine, lane);
        }
        Place x;
        const int f = __ffs(__ballot_sync(0xffffffffu, base + upto > u)) - 1;
        const int r0 = u - base - __shfl_sync(0xffffffffu, upto - mine, f);
        const int per_head = __shfl_sync(0xffffffffu, sq.per_head, f);
        x.b = k0 + f;
        x.past = __shfl_sync(0xffffffffu, sq.past, f);
        x.fresh = __shfl_sync(0xffffffffu, sq.fresh, f);
        x.tiles = __shfl_sync(0xffffffffu, sq.tiles, f);
        x.valid = __shfl_sync(0xffffffffu, sq.valid, f);
        x.hk = (unsigned)r0 / (unsigned)per_head;
        x.r = r0 - x.hk * per_head;
        return x;
    }
    // The next piece goes to the ring (b = -1 after the last); false if a wait gave up.
    __device__ __forceinline__ bool step(const PagedParams &p, PagedBars *bars, int lane) {
        if (done) return true;
        PagedSeg g;
        g.b = -1;
        while (u < u1) {
            const Place x = place(p, lane);
            const int r = x.r, tiles = x.tiles, valid = x.valid;
            g.past = x.past;
            g.fresh = x.fresh;
            g.total = g.past + g.fresh;
            g.hk = x.hk;
            const int cost = tiles + kItemCost;
            g.slot = 2 * blockIdx.x + (first ? 0 : 1);
            first = false;
            int rt;
            if (p.uncut) {
                rt = r;
                g.j0 = 0;
                g.j1 = rt < valid ? tiles : 0;
                g.whole = 1;
                u += 1;
            } else if (r < valid * cost) {
                rt = (unsigned)r / (unsigned)cost;
                g.j0 = min(r - rt * cost, tiles);
                const int end = min(cost, r - rt * cost + (u1 - u));
                g.j1 = min(end, tiles);
                u += end - (r - rt * cost);
                if (g.j0 == g.j1) continue;  // nothing but the item's own cost
                g.whole = g.j0 == 0 && g.j1 == tiles;
            } else {
                rt = valid + (r - valid * cost);
                g.j0 = g.j1 = 0;
                g.whole = 1;
                u += 1;
            }
            g.b = x.b;
            const int tt = p.GT == 1 ? rt : rt / p.GT;
            g.tok0 = tt * RT * p.TPT;
            g.g0 = p.GT == 1 ? 0 : (rt - tt * p.GT) * p.GP;
            if (p.tree == nullptr)  // a chain's rows see no key behind their last token
                g.j1 = min(g.j1, (g.past + min(g.fresh, g.tok0 + RT * p.TPT) + 127) >> 7);
            break;
        }
        done = g.b < 0;
        if (n >= 4 && !__all_sync(0xffffffffu, mbar_wait(&bars->seg_empty[n & 3], ((n >> 2) - 1) & 1)))
            return false;
        if (lane == 0) {
            int4 *d = bars->seg[n & 3];
            d[0] = make_int4(g.b, g.hk, g.tok0, g.g0);
            d[1] = make_int4(g.past, g.total, g.fresh, g.j0);
            d[2] = make_int4(g.j1, g.slot, g.whole, 0);
            mbar_arrive(&bars->seg_full[n & 3]);
        }
        __syncwarp();
        ++n;
        return true;
    }
};

// Takes piece n (all lanes that use it; lane 0 among them); false after the last one, or when
// the wait gave up.
__device__ __forceinline__ bool paged_take(PagedBars *bars, int n, int lane, bool warp_wide,
                                           PagedSeg &g) {
    bool ok = mbar_wait(&bars->seg_full[n & 3], (n >> 2) & 1);
    if (warp_wide) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    const int4 *d = bars->seg[n & 3];
    const int4 x = d[0], y = d[1], z = d[2];
    g.b = x.x, g.hk = x.y, g.tok0 = x.z, g.g0 = x.w;
    g.past = y.x, g.total = y.y, g.fresh = y.z, g.j0 = y.w;
    g.j1 = z.x, g.slot = z.y, g.whole = z.z;
    if (warp_wide) __syncwarp();
    if (lane == 0) mbar_arrive(&bars->seg_empty[n & 3]);
    return g.b >= 0;
}

__device__ __forceinline__ void tma_load_4d(void *smem_dst, const void *tmap, uint64_t *bar, int x,
                                            int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// C columns of 32 TMEM lanes.
template <int C>
__device__ __forceinline__ void tmem_ldn(uint32_t a, uint32_t (&r)[C]) {
    if constexpr (C == 128) tmem_ld128(a, r);
    else if constexpr (C == 64) tmem_ld64(a, r);
    else tmem_ld32(a, r);
}

// Registers -> TMEM, 32 lanes x 16 columns, complete after tmem_wait_st().
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two fp32 operations at once (packed registers).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The row of key j in the value cache (nullptr: its page lies outside).
__device__ __forceinline__ const uint16_t *paged_value(const PagedParams &p, const PagedSeg &it, int j) {
    const int id = p.pt.table[(long long)it.b * p.pt.max_blocks + (j >> p.pt.page_shift)];
    if (id < 0 || id >= p.pt.num_pages) return nullptr;
    return p.vc.p + id * p.vc.sb + it.hk * p.vc.sh + (j & ((1 << p.pt.page_shift) - 1)) * p.vc.st;
}

// Puts the values that are not finite of the keys that a row sees into its output or piece: their
// sum, as every visible key's weight is above 0, where P V has 0 * inf = NaN for weights that
// round to 0 and for the keys of other copies, and nothing for values that the repair cleared.
// A whole warp calls this for what its threads stored: rows r0, r0 + step, .. < used of row tile
// ti and n columns from c4 on (in every block of 32, or `once`: in c4's).  held: some output of
// the warp is not finite, so the keys that all rows see are gone over (32 at a time, one per
// lane); cleared: so are the others.  ok: a row's weights are numbers (copies: its sums, `sums`).
// (Out of line, as are the next: rare, and the code that every piece runs through comes in from
// memory at each launch.)
template <int D, bool BF16, int REP, int RT>
__device__ __noinline__ void paged_put_not_finite(const PagedParams &p, const PagedSeg &it, int ti, int r0, int step,
                                                  int used, int c4, int n, bool once, bool held, bool cleared,
                                                  bool ok, const float *sums) {
    constexpr int ROWS = 128 / REP;
    const int k0 = it.j0 * 128, k1 = min(it.total, it.j1 * 128);
    const int mid = max(k0, min(k1, it.open(p, it.tok0)));
#pragma unroll 1
    for (int cb = 0; cb < D; cb += 32) {
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = 0.f;
        if (held) {
#pragma unroll 1
            for (int j = k0 + (int)(threadIdx.x & 31); j < mid; j += 32) {
                const uint16_t *src = paged_value(p, it, j);
                if (src == nullptr) continue;
                uint4 x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = reinterpret_cast<const uint4 *>(src + cb)[e];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack2<BF16>(w[i]);
                        const uint32_t bad = not_finite2<BF16>(w[i]);
                        if (bad & 0xffffu) y[8 * e + 2 * i] += f.x;
                        if (bad >> 16) y[8 * e + 2 * i + 1] += f.y;
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 32; ++e)
                for (int o = 16; o > 0; o >>= 1) y[e] += __shfl_xor_sync(0xffffffffu, y[e], o);
        }
        if (once && c4 >> 5 != cb >> 5) continue;
#pragma unroll 1
        for (int r = r0; r < used; r += step) {
            const int tl = r * p.gp_magic >> 16, tok = it.tok0 + ti * p.TPT + tl, h = it.g0 + (r - tl * p.GP);
            if (tl >= p.TPT || tok >= it.fresh || h >= p.G) continue;
            if (REP > 1) {
                float l = 0.f;
                for (int k = 0; k < REP; ++k) l += sums[k * ROWS + r];
                ok = l > 0.f;
            }
            if (!ok) continue;
            float s[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = y[e];
            const int e0 = c4 & 31;
#pragma unroll 1
            for (int j = mid; cleared && j < k1; ++j) {
                const int x = j - it.past;
                if (!(p.tree ? p.tree[it.b * p.tree_sb + (long long)tok * p.T + x] != 0 : x <= tok)) continue;
                const uint16_t *src = paged_value(p, it, j);
                if (src == nullptr) continue;
#pragma unroll 4
                for (int e = e0; e < e0 + n; ++e) {
                    const uint32_t w = src[cb + e];
                    if (not_finite2<BF16>(w) & 0xffffu) s[e] += unpack2<BF16>(w).x;
                }
            }
            const long long at = (long long)it.slot * (RT * ROWS) + ti * ROWS;
#pragma unroll 1
            for (int e = e0; e < e0 + n; ++e) {
                const int c = cb + e;
                if (s[e] == 0.f) continue;
                if (it.whole)
                    const_cast<uint16_t *>(p.o.p)[it.b * p.o.sb + (it.hk * p.G + h) * p.o.sh + tok * p.o.st + c] =
                        (uint16_t)pack2<BF16>(s[e], s[e]);
                else if (REP > 1)
                    p.part_o[(at + r) * D + c] = s[e];
                else
                    p.part_o[at * D + ((c >> 2) * ROWS + r) * 4 + (c & 3)] = s[e];
            }
        }
    }
}

// NaN if one of N values is not finite, else 0.
template <int N>
__device__ __forceinline__ float paged_finite(const float (&v)[N]) {
    float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < N; ++e) z[e & 3] = fmaf(v[e], 0.f, z[e & 3]);
    return (z[0] + z[1]) + (z[2] + z[3]);
}

// New keys x0 .. x0 + 31 (x0 > -32) that token tok sees, from a mask of more than 128 columns.
__device__ __noinline__ uint32_t paged_tree_bits(const PagedParams &p, int b, int fresh, int tok, int x0) {
    uint32_t bits = x0 >= 0 ? 0u : (1u << -x0) - 1u;
    const uint8_t *mr = p.tree + b * p.tree_sb + (long long)tok * p.T + x0;
    const int lo = max(0, -x0), hi = min(32, fresh - x0);
    for (int c = lo; c < hi; ++c) bits |= (__ldg(mr + c) != 0 ? 1u : 0u) << c;
    return bits;
}

// Keys of 32 from place kt of a tile on whose pages lie outside the cache.
__device__ __noinline__ uint32_t paged_bad_bits(uint32_t bad, int page_shift, int kt) {
    const int sh = min(page_shift, 7), sub = min(1 << sh, 32);
    uint32_t bits = 0u;
    for (int c = 0; c < 32; c += sub)
        if ((bad >> ((kt + c) >> sh)) & 1u) bits |= (sub == 32 ? 0xffffffffu : (1u << sub) - 1u) << c;
    return bits;
}

template <int D, bool BF16, int REP, int RT, int KS_>
__global__ void __launch_bounds__(PagedCfg<D, REP, RT, KS_>::THREADS, 1)
fa_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
    using C = PagedCfg<D, REP, RT, KS_>;
    constexpr int ROWS = C::ROWS;
    constexpr int CW = C::STEP / REP; // keys of a step that one thread handles
    constexpr int SPT = C::SPT, KS = C::KS;
    constexpr int W_S = C::SOFT, W_PV = C::SOFT + 1, W_FIX = C::SOFT + 2, W_TMA = C::SOFT + 3;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem + C::OFF_Q;
    uint8_t *ring = smem + C::OFF_RING;
    PagedBars *bars = reinterpret_cast<PagedBars *>(smem + C::OFF_BAR);
    static_assert(sizeof(PagedBars) <= 3200 + 8192, "barrier area");
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // Step n, row tile i: score buffer's barrier and phase, P buffer's barrier and phase.
    constexpr int NSB = C::NSB;
    auto sb_of = [](int n, int i) { return NSB == 2 ? 2 * i + (n & 1) : i; };
    auto sb_at = [](int n, int i) { return i * C::S_TILE + (NSB == 2 ? (n & 1) * C::S_BUF : 0u); };
    auto sb_ph = [](int n) { return NSB == 2 ? (n >> 1) & 1 : n & 1; };
    auto pb_of = [](int n, int i) { return 2 * i + (n & 1); };
    auto pb_ph = [](int n) { return (n >> 1) & 1; };

    if (threadIdx.x == W_S * 32) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        mbar_init(&bars->o_empty, 32 * C::SOFT);
        for (int i = 0; i < 4; ++i) mbar_init(&bars->need[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->mask_full[i], 1);
            mbar_init(&bars->mask_empty[i], C::SOFT);
        }
        for (int i = 0; i < NSB * RT; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->s_empty[i], 128);
        }
        for (int i = 0; i < 2 * RT; ++i) {
            mbar_init(&bars->p_full[i], 128);
            mbar_init(&bars->pv_done[i], 1);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&bars->kfull[i], 1);
            mbar_init(&bars->vfull[i], 1);
            mbar_init(&bars->fixed[i], 1);
        }
        for (int i = 0; i < 6; ++i) {
            mbar_init(&bars->kempty[i], 1);
            mbar_init(&bars->vempty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars->seg_full[i], 1);
            mbar_init(&bars->seg_empty[i], C::SOFT + 3 + C::LOADERS);
        }
        fence_mbar_init();
    }
    if (warp == W_FIX) tmem_alloc(&bars->tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_FIX) {  // (hints only: nothing is read before the wait)
        for (int b = lane * 32; b < p.B; b += 1024) {
            prefetch_l2(p.pt.cache_len + b);
            if (p.pt.new_len) prefetch_l2(p.pt.new_len + b);
        }
    }
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t tmem = bars->tmem_base;
    PagedSeg it;
    int np = 0;  // pieces taken

    if (warp >= W_TMA) {
        // ------------------------------ K and V: a whole warp each ----------------------
        // A tile's pages: npt boxes (a page, or 128 rows of a larger one) per 64-element
        // column block; lane l loads box l % npt of block l / npt.  Page numbers are read one
        // tile ahead.
        const int kv0 = C::LOADERS == 2 ? warp - W_TMA : 0, kv1 = C::LOADERS == 2 ? kv0 + 1 : 2;
        const int page = 1 << p.pt.page_shift;
        const int box_rows = min(page, 128);
        const int npt = 128 / box_rows;
        const int mine = lane % npt, half = lane / npt;
        int gj = 0;  // tiles so far
        bool ok = true;
        while (ok && paged_take(bars, np++, lane, true, it)) {
            const int *row = p.pt.table + (long long)it.b * p.pt.max_blocks;
            auto page_at = [&](int j) -> int {  // (a place behind the last key: -1)
                const int key = j * 128 + mine * box_rows;
                return key < it.total ? __ldg(row + (key >> p.pt.page_shift)) : -1;
            };
            int next = page_at(it.j0);
            for (int j = it.j0; ok && j < it.j1; ++j, ++gj) {
                const int key = j * 128 + mine * box_rows, id = next;
                if (j + 1 < it.j1) next = page_at(j + 1);
                const bool bad = key < it.total && (id < 0 || id >= p.pt.num_pages);
                // outside the cache: the box is filled with zeros
                const int z = key < it.total && !bad ? id : p.pt.num_pages;
                if (kv0 == 0) {
                    const unsigned bads = __ballot_sync(0xffffffffu, bad && half == 0);
                    if (lane == 0) {
                        bars->bad[gj & 15] = bads;
                        if (bads) report_bad_page();
                    }
                }
                const int y = key & (page - 1);
                for (int kv = kv0; kv < kv1; ++kv) {
                    const int N = kv ? C::NV : C::NK, s = gj % N;
                    if (gj >= N)
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait(kv ? &bars->vempty[s] : &bars->kempty[s], (gj / N - 1) & 1));
                    if (!ok) break;
                    uint64_t *full = kv ? &bars->vfull[gj & 7] : &bars->kfull[gj & 7];
                    if (lane == 0) mbar_arrive_expect_tx(full, C::TILE);
                    __syncwarp();
                    if (half < C::HALVES)
                        tma_load_4d(ring + (kv ? C::NK + s : s) * C::TILE + half * C::HALF + mine * box_rows * 128,
                                    kv ? &tmV : &tmK, full, half * 64, y, it.hk, z);
                }
            }
        }
        if (!ok)  // a wait gave up: the copies in flight land before the CTA's memory goes
            for (int kv = kv0; kv < kv1; ++kv)
                for (int g = max(0, gj - 6); g < gj; ++g)
                    (void)mbar_wait(kv ? &bars->vfull[g & 7] : &bars->kfull[g & 7], (g >> 3) & 1);
    } else if (warp == W_S) {
        // ------------------------------ issuer of S -------------------------------------
        if (lane == 0) {
            constexpr uint32_t kIdesc = idesc_f16(BF16, false, false, 128, C::STEP);
            const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t k_desc = smem_desc_sw128(smem_u32(ring), 16, 1024);
            bool ok = true;
            int n0 = 0, t = 0;  // steps and pieces so far
            int asked = 0;
            while (ok && paged_take(bars, np++, lane, false, it)) {
                const int steps = (it.j1 - it.j0) * SPT;
                if (steps <= 0) continue;
                if (!mbar_wait(&bars->q_full, t & 1)) break;
                for (int x = 0; ok && x < steps; ++x) {
                    const int n = n0 + x, h = x % SPT;
                    const int g = n / SPT, s = g % C::NK;  // tile, K's slot
                    if (h == 0 && !mbar_wait(&bars->kfull[g & 7], (g >> 3) & 1)) { ok = false; break; }
                    const uint64_t kd = k_desc + (uint64_t)((s * C::TILE + h * C::STEP * 128) >> 4);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const int b = sb_of(n, i);
                        if (n >= NSB && !mbar_wait(&bars->s_empty[b], sb_ph(n - NSB))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t qd = q_desc + (uint64_t)((i * C::QTILE) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t qo = (uint64_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4);
                            const uint64_t ko = (uint64_t)(((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4);
                            mma_ss(tmem + sb_at(n, i), qd + qo, kd + ko, kIdesc, kk > 0);
                        }
                        // (the barriers that nobody waits for at the end come first, so that no
                        // arrival is outstanding when the CTA ends)
                        if (i == RT - 1 && h == SPT - 1) mma_commit(&bars->kempty[s]);
                        if (i == RT - 1 && x == steps - 1) mma_commit(&bars->q_empty);
                        mma_commit(&bars->s_full[b]);
                    }
                    if (!ok) break;
                    if (h == 0 && it.repair(p, it.j0 + x / SPT)) mbar_arrive(&bars->need[asked++ & 3]);
                }
                n0 += steps;
                ++t;
            }
        }
    } else if (warp == W_PV) {
        // ------------------------------ issuer of P V -----------------------------------
        if (lane == 0) {
            constexpr uint32_t kIdesc = idesc_f16(BF16, false, true, 128, D);
            const uint64_t v_desc = smem_desc_sw128(smem_u32(ring), C::HALF, 1024);
            bool ok = true;
            int n0 = 0, t = 0;
            uint32_t fixes = 0;  // parity of the next repair of each of the eight
            while (ok && paged_take(bars, np++, lane, false, it)) {
                const int steps = (it.j1 - it.j0) * SPT;
                if (steps <= 0) continue;
                for (int x = 0; ok && x < steps; ++x) {
                    const int n = n0 + x, h = x % SPT;
                    const int g = n / SPT, s = C::NK + g % C::NV;  // tile, V's slot
                    if (h == 0) {
                        if (!mbar_wait(&bars->vfull[g & 7], (g >> 3) & 1)) { ok = false; break; }
                        if (it.repair(p, it.j0 + x / SPT)) {
                            if (!mbar_wait(&bars->fixed[g & 7], (fixes >> (g & 7)) & 1)) { ok = false; break; }
                            fixes ^= 1u << (g & 7);
                        }
                        if (x == 0 && t > 0 && !mbar_wait(&bars->o_empty, (t - 1) & 1)) { ok = false; break; }
                    }
                    const uint64_t vd = v_desc + (uint64_t)((s * C::TILE + h * C::STEP * 128) >> 4);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const int b = pb_of(n, i);
                        if (!mbar_wait(&bars->p_full[b], pb_ph(n))) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t pa = tmem + C::COL_P + i * C::S_TILE + (n & 1) * C::P_BUF;
#pragma unroll
                        for (int kk = 0; kk < C::STEP / 16; ++kk)
                            mma_ts(tmem + C::COL_O + (KS == 2 ? n & 1 : i) * D, pa + kk * 8,
                                   vd + (uint64_t)((kk * 16 * 128) >> 4), kIdesc, x >= KS || kk > 0);
                        if (i == RT - 1 && h == SPT - 1) mma_commit(&bars->vempty[g % C::NV]);
                        mma_commit(&bars->pv_done[b]);
                    }
                }
                n0 += steps;
                ++t;
            }
        }
    } else if (warp == W_FIX) {
        // ------------------------------ pieces, Q loads, V repairs ----------------------
        PagedWalk<RT> walk;
        walk.init(p, blockIdx.x, lane);
        bool ok = walk.step(p, bars, lane);
        int loads = 0;
        int gj = 0, t = 0, served = 0, masks = 0;
        while (ok && paged_take(bars, np++, lane, true, it)) {
            const int nt = it.j1 - it.j0;
            if (nt <= 0) {
                if (!(ok = walk.step(p, bars, lane))) break;
                continue;
            }
            if (t > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->q_empty, (t - 1) & 1))) break;
            if (lane == 0) {
                // a box of TPT tokens x GP heads is a row tile (zeros behind the last token)
                mbar_arrive_expect_tx(&bars->q_full, p.TPT * p.GP * 128 * C::HALVES * REP * RT);
#pragma unroll
                for (int i = 0; i < RT * REP; ++i)
#pragma unroll
                    for (int hf = 0; hf < C::HALVES; ++hf)
                        tma_load_4d(sQ + (RT > 1 ? i * C::QTILE : i * ROWS * 128) + hf * (128 * 128), &tmQ,
                                    &bars->q_full, hf * 64, it.hk * p.G + it.g0,
                                    it.tok0 + (RT > 1 ? i * p.TPT : 0), it.b);
            }
            __syncwarp();
            ++loads;
            // The next piece (after the first Q, which is waited for, the next two) is worked out
            // behind the load: 512 items of 2 tiles, 128 rows, d = 64: 28.1 -> 26.1 us.
            if (t == 0) ok = walk.step(p, bars, lane);
            if (!(ok = ok && walk.step(p, bars, lane))) break;
            // The rows' masks as bits, one (token, 32 new keys) per lane at a time.
            if (p.tree != nullptr && p.T <= 128 && it.j1 * 128 > it.past) {
                uint32_t *mask = bars->mask[masks & 1];
                if (masks >= 2 &&
                    !(ok = __all_sync(0xffffffffu, mbar_wait(&bars->mask_empty[masks & 1], ((masks >> 1) - 1) & 1))))
                    break;
                const int nw = (it.fresh + 31) >> 5, toks = min(RT * p.TPT, it.fresh - it.tok0);
                for (int k = lane; k < toks * nw; k += 32) {
                    const int tk = k / nw, w = k - tk * nw;
                    const uint8_t *mr = p.tree + it.b * p.tree_sb + (long long)(it.tok0 + tk) * p.T + w * 32;
                    const int n = it.fresh - w * 32;
                    uint32_t bits = 0u;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c < n) bits |= (__ldg(mr + c) != 0 ? 1u : 0u) << c;
                    mask[tk * 4 + w] = bits;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->mask_full[masks & 1]);
                ++masks;
            }
            // V tiles with new keys that some row does not see, or slots behind the last
            bool found = false;
            for (int i = 0; ok && i < nt; ++i) {
                const int j = it.j0 + i;
                if (!it.repair(p, j)) continue;
                const int g = gj + i, s = C::NK + g % C::NV;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->need[served & 3], (served >> 2) & 1) &&
                                                 mbar_wait(&bars->vfull[g & 7], (g >> 3) & 1));
                if (!ok) break;
                ++served;
                // (the swizzle permutes 16-byte chunks within a row only)
                uint8_t *tile = ring + s * C::TILE;
                const int tail = min(128, it.total - j * 128);
                for (int x = tail * 8 + lane; x < 128 * 8; x += 32)
#pragma unroll
                    for (int hf = 0; hf < C::HALVES; ++hf)
                        *reinterpret_cast<uint4 *>(tile + hf * C::HALF + x * 16) = make_uint4(0, 0, 0, 0);
                // (the exponent's all ones carry into the sign's place)
                constexpr uint32_t kCarry = BF16 ? 0x00800080u : 0x04000400u;
                const int x1 = tail * 8;
                for (int x = max(0, it.open(p, it.tok0) - j * 128) * 8 + lane; x < x1; x += 128) {
                    uint32_t hit = 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int hf = 0; hf < C::HALVES; ++hf)
                            if (x + e * 32 < x1) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(tile + hf * C::HALF + (x + e * 32) * 16);
                                hit |= ((v.x & 0x7FFF7FFFu) + kCarry) | ((v.y & 0x7FFF7FFFu) + kCarry) |
                                       ((v.z & 0x7FFF7FFFu) + kCarry) | ((v.w & 0x7FFF7FFFu) + kCarry);
                            }
                    if (hit & 0x80008000u) {
                        found = true;
#pragma unroll 1
                        for (int e = 0; e < 4 * C::HALVES; ++e) {
                            const int xx = C::HALVES == 2 ? x + (e >> 1) * 32 : x + e * 32;
                            if (xx >= x1) break;
                            uint32_t *w = reinterpret_cast<uint32_t *>(tile + (C::HALVES == 2 ? (e & 1) * C::HALF : 0) + xx * 16);
#pragma unroll
                            for (int c = 0; c < 4; ++c) w[c] &= ~not_finite2<BF16>(w[c]);
                        }
                    }
                }
                found = __any_sync(0xffffffffu, found);
                if (lane == 0) bars->poison[t & 3] = found ? 1 : 0;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->fixed[g & 7]);
            }
            ++t;
            gj += nt;
        }
        if (blockIdx.x == 0)
            for (int b = lane; b < p.B; b += 32) page_lengths_check(p.pt, p.T, b);
        // the last Q load has landed before the CTA's memory goes (at once unless a wait gave up)
        if (loads > 0) (void)mbar_wait(&bars->q_full, (loads - 1) & 1);
    } else {
        // ------------------------------ softmax warps -----------------------------------
        constexpr int WPC = 4 / REP;                       // warps of one copy of the rows
        const int ti = RT == 1 ? 0 : warp >> 2;            // row tile
        const int ks = KS == 1 ? 0 : warp >> 2;            // group: tiles n with n % KS == ks
        const int wq = warp & 3;                           // lane quarter of TMEM
        const int row = (wq % WPC) * 32 + lane;            // row of the tile
        const int kw = wq / WPC;                           // the copy: keys [kw * CW, + CW)
        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        const uint32_t ob = tmem + lane_base + C::COL_O + (ti + ks) * D;
        const float sl2 = p.scale_log2;
        const int tl = row * p.gp_magic >> 16, gl = row - tl * p.GP;  // the row's token and head
        if constexpr (REP > 1) {  // P is zero outside the copy's own keys
            uint32_t zero[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) zero[i] = 0u;
#pragma unroll
            for (int i = 0; i < 2 * (int)C::P_BUF / 32; ++i) tmem_st32(tmem + lane_base + C::COL_P + i * 32, zero);
        }
        bool ok = true;
        int n0 = 0, t = 0, masks = 0;  // steps, pieces and masks so far
        while (paged_take(bars, np++, lane, true, it)) {
            const int tok = it.tok0 + ti * p.TPT + tl;
            const int head = it.g0 + gl;                   // among the key/value head's
            const bool mine = tl < p.TPT && tok < p.T && head < p.G;  // a row of the call
            const bool live = mine && tok < it.fresh;      // a new token's row
            const int nt = max(it.j1 - it.j0, 0);
            // (keys in front of it need no mask)
            const int open = it.open(p, it.tok0 + ti * p.TPT);
            // the piece's masks are in place (see the repairing warp)
            const bool bits_used = p.tree != nullptr && p.T <= 128 && nt > 0 && it.j1 * 128 > it.past;
            if (bits_used) ok = __all_sync(0xffffffffu, mbar_wait(&bars->mask_full[masks & 1], (masks >> 1) & 1));
            float m = -INFINITY;   // running maximum, base 2
            float l = 0.f;         // running sum
            float lr = 0.f;        // the same sum of the rounded weights
            const int i0 = KS == 1 ? 0 : ((n0 ^ ks) & 1);  // the group's first tile of the piece
            const bool has = KS == 1 ? nt > 0 : i0 < nt;
            for (int i = i0; ok && i < nt * SPT; i += KS) {
                const int n = n0 + i, b = sb_of(n, ti);
                const int kt = i % SPT * C::STEP + kw * CW;        // this thread's keys of the tile
                const int k0 = (it.j0 + i / SPT) * 128 + kt;
                const uint32_t sb = tmem + lane_base + sb_at(n, ti) + kw * CW;
                const bool masked = k0 + CW > open;
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[b], sb_ph(n)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t bad = bars->bad[(n / SPT) & 15];
                // The row's visible ones of 32 keys (held keys all are).
                auto visible = [&](int w) -> uint32_t {
                    const int x0 = k0 + w * 32 - it.past;  // new key of bit 0
                    uint32_t bits = 0u;
                    if (!masked) {
                        bits = 0xffffffffu;
                    } else if (!live) {
                    } else if (p.tree == nullptr) {
                        const int c = tok + 1 - x0;        // keys up to the row's token
                        bits = c >= 32 ? 0xffffffffu : (c <= 0 ? 0u : (1u << c) - 1u);
                    } else if (p.T <= 128) {
                        const uint32_t *mr = bars->mask[masks & 1] + (tok - it.tok0) * 4;
                        const int q = x0 >> 5, nw = (it.fresh + 31) >> 5;  // (floor)
                        const uint32_t lo = q < 0 ? 0xffffffffu : (q < nw ? mr[q] : 0u);
                        const uint32_t hi = q + 1 < 0 ? 0xffffffffu : (q + 1 < nw ? mr[q + 1] : 0u);
                        bits = __funnelshift_r(lo, hi, x0 & 31);
                    } else {
                        bits = x0 <= -32 ? 0xffffffffu : paged_tree_bits(p, it.b, it.fresh, tok, x0);
                    }
                    // keys of pages outside the cache are not visible
                    if (bad) bits &= ~paged_bad_bits(bad, p.pt.page_shift, kt + w * 32);
                    return bits;
                };
                // The maximum.  Up to 64 scores stay in registers; 128 are read from TMEM in two
                // passes, 64 and 32 at a time in loops: unrolled, the code took 4 us to come in
                // from memory at a kernel's first tile, against 1.1 us a tile once there.
                // Hidden scores become -inf (in TMEM where they are read again).
                constexpr bool HELD = CW <= 64;
                constexpr int N = HELD ? CW : 64;
                uint32_t sc[N];
                float mxv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mxv[e] = -INFINITY;
#pragma unroll 1
                for (int w = 0; w < CW / N; ++w) {
                    tmem_ldn<N>(sb + w * N, sc);
                    if (HELD) {
                        tc_fence_before();
                        mbar_arrive(&bars->s_empty[b]);
                    }
                    if (masked || bad != 0) {
#pragma unroll
                        for (int v = 0; v < N / 32; ++v) {
                            const uint32_t bits = visible(w * (N / 32) + v);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!((bits >> c) & 1u)) sc[v * 32 + c] = 0xff800000u;
                        }
                        if constexpr (!HELD) {
                            uint32_t lo[32], hi[32];
#pragma unroll
                            for (int c = 0; c < 32; ++c) lo[c] = sc[c], hi[c] = sc[32 + c];
                            tmem_st32(sb + w * N, lo);
                            tmem_st32(sb + w * N + 32, hi);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < N; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mxv[e] = fmax3(mxv[e], __uint_as_float(sc[c + e]), __uint_as_float(sc[c + 4 + e]));
                }
                const float mx = fmaxf(fmax3(mxv[0], mxv[1], mxv[2]), mxv[3]) * sl2;
                // Lazy rescale: m moves when the maximum grew by more than 2^8.
                const bool any_grow = __any_sync(0xffffffffu, mx > m + 8.0f);
                float alpha = 1.f;
                if (any_grow && mx > m) {
                    alpha = ex2(m - mx);
                    m = mx;
                }
                const float m_use = (m == -INFINITY) ? 0.f : m;
                // P's buffer is free once P V of step n - 2 is done; O may be rescaled once that
                // of step n - 1 is (two groups: n - 2, the group's last).
                if (n >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bars->pv_done[pb_of(n, ti)], pb_ph(n - 2)))) {
                    ok = false;
                    break;
                }
                if (i >= KS && any_grow) {
                    if (KS == 1 && !__all_sync(0xffffffffu, mbar_wait(&bars->pv_done[pb_of(n - 1, ti)], pb_ph(n - 1)))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t rr[32];
                        tmem_ld32(ob + c * 32, rr);
#pragma unroll
                        for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
                        tmem_st32(ob + c * 32, rr);
                    }
                }
                tc_fence_after();
                // The weights, their sums, P.
                float2 ls = make_float2(0.f, 0.f), rs = make_float2(0.f, 0.f);
                const float2 sc2 = make_float2(sl2, sl2), nm = make_float2(-m_use, -m_use);
                const uint32_t pb = tmem + lane_base + C::COL_P + ti * C::S_TILE + (n & 1) * C::P_BUF + kw * (CW / 2);
                auto weights = [&](const uint32_t *rr, uint32_t dst) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float2 x = fma2(make_float2(__uint_as_float(rr[c]), __uint_as_float(rr[c + 1])), sc2, nm);
                        const float2 w = make_float2(ex2(x.x), ex2(x.y));
                        ls = add2(ls, w);
                        pk[c >> 1] = pack2<BF16>(w.x, w.y);
                        rs = add2(rs, unpack2<BF16>(pk[c >> 1]));
                    }
                    tmem_st16_async(dst, pk);
                };
                if constexpr (HELD) {
#pragma unroll
                    for (int w = 0; w < CW / 32; ++w) weights(sc + w * 32, pb + w * 16);
                } else {
                    uint32_t ra[32], rb[32];
                    tmem_ld32(sb, ra);
#pragma unroll 1
                    for (int w = 0; w < CW / 32; w += 2) {  // the next 32 are on their way
                        tmem_ld32_async(sb + (w + 1) * 32, rb);
                        weights(ra, pb + w * 16);
                        tmem_wait_ld(rb);
                        // (behind the last: a load that nobody uses, so that the loop's
                        // registers are not merged before the wait)
                        tmem_ld32_async(sb + min(w + 2, CW / 32 - 1) * 32, ra);
                        weights(rb, pb + (w + 1) * 16);
                        tmem_wait_ld(ra);
                    }
                }
                tmem_wait_st();
                l = l * alpha + (ls.x + ls.y);
                lr = lr * alpha + (rs.x + rs.y);
                tc_fence_before();
                if (!HELD) mbar_arrive(&bars->s_empty[b]);
                mbar_arrive(&bars->p_full[pb_of(n, ti)]);
            }

            if (bits_used) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->mask_empty[masks & 1]);
                ++masks;
            }
            // ------------------------------ epilogue of the piece ------------------------
            if (ok && has) {
                int n = n0 + nt * SPT - 1;
                if (KS == 2 && (n & 1) != ks) --n;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[pb_of(n, ti)], pb_ph(n)));
                tc_fence_after();
            }
            // (the merge of the copies has barriers of all four warps: they leave together)
            if constexpr (REP > 1 || KS > 1)
                if (nt > 0) ok = named_bar_and(1, 128 * KS, ok);
            if (!ok) break;
            if (!live) m = -INFINITY, l = lr = 0.f;  // rows behind the last new token are empty
            bool none = l == 0.f;                    // (a NaN sum is carried to O and LSE)
            float inv = none ? 0.f : 1.f / lr;
            const bool writer = KS == 1 || (nt == 1 ? has : ks == 0);  // (one tile: its group alone)
            float lse2 = none ? -INFINITY : m + lg2(l);
            // Values that the repair cleared reach the rows that do see them (see paged_put_not_finite).
            const bool poison = nt > 0 && it.repair(p, it.j1 - 1) && bars->poison[t & 3] != 0;
            auto out_row = [&](int h, int tk) {
                return const_cast<uint16_t *>(p.o.p) + it.b * p.o.sb + (it.hk * p.G + h) * p.o.sh + tk * p.o.st;
            };
            const long long prow0 = (long long)it.slot * (RT * ROWS) + ti * ROWS;  // first row of the partial
            if constexpr (REP == 1) {
                float *other = reinterpret_cast<float *>(smem + C::OFF_MERGE + C::STAGE) + row * 36;
                if constexpr (KS == 2) {
                    if (nt > 1) {  // the groups' statistics; inv becomes 2^(m - M) / R, as with copies
                        float *stat = reinterpret_cast<float *>(smem + C::OFF_MERGE + C::STAGE + 128 * 36 * 4);
                        stat[threadIdx.x] = m;
                        stat[256 + threadIdx.x] = l;
                        stat[512 + threadIdx.x] = lr;
                        named_bar_sync(1, 256);
                        const int x = threadIdx.x ^ 128;
                        const float m2 = stat[x], M = fmaxf(m, m2);
                        const float f = (m == -INFINITY) ? 0.f : ex2(m - M);
                        const float f2 = (m2 == -INFINITY) ? 0.f : ex2(m2 - M);
                        l = f * l + f2 * stat[256 + x];
                        none = l == 0.f;
                        inv = f / (f * lr + f2 * stat[512 + x]);
                        lse2 = none ? -INFINITY : M + lg2(l);
                    }
                }
                float z = 0.f;  // NaN where an output is not finite
#pragma unroll 1
                for (int c32 = 0; c32 < D / 32; ++c32) {
                    float v[32];
                    if (has) {
                        uint32_t rr[32];
                        tmem_ld32(ob + c32 * 32, rr);
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = none ? 0.f : __uint_as_float(rr[e]) * inv;
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0.f;
                    }
                    if constexpr (KS == 2) {  // the second group's O through shared memory
                        if (nt > 1) {
                            if (c32 > 0) named_bar_sync(1, 256);
                            if (ks == 1)
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    *reinterpret_cast<float4 *>(other + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                            named_bar_sync(1, 256);
                            if (ks == 0)
#pragma unroll
                                for (int e = 0; e < 32; e += 4) {
                                    const float4 y = *reinterpret_cast<const float4 *>(other + e);
                                    v[e] += y.x, v[e + 1] += y.y, v[e + 2] += y.z, v[e + 3] += y.w;
                                }
                        }
                    }
                    if (c32 == D / 32 - 1 && nt > 0) {
                        tc_fence_before();
                        mbar_arrive(&bars->o_empty);
                    }
                    if (KS == 2 && !writer) continue;
                    z += paged_finite(v);
                    if (it.whole) {
                        // through shared memory, so that a store covers 64 bytes of 8 rows
                        // instead of 16 bytes of 32 (16-byte chunks permuted by row pairs)
                        uint4 *st = reinterpret_cast<uint4 *>(smem + C::OFF_MERGE + warp * 2048);
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            st[lane * 4 + (e ^ ((lane >> 1) & 3))] =
                                make_uint4(pack2<BF16>(v[8 * e], v[8 * e + 1]),
                                           pack2<BF16>(v[8 * e + 2], v[8 * e + 3]),
                                           pack2<BF16>(v[8 * e + 4], v[8 * e + 5]),
                                           pack2<BF16>(v[8 * e + 6], v[8 * e + 7]));
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int rl = e * 8 + (lane >> 2), r = (wq << 5) + rl, q = lane & 3;
                            const int tr = r * p.gp_magic >> 16, hr = r - tr * p.GP + it.g0;
                            const int tk = it.tok0 + ti * p.TPT + tr;
                            if (tr < p.TPT && tk < p.T && hr < p.G)
                                reinterpret_cast<uint4 *>(out_row(hr, tk))[c32 * 4 + q] =
                                    st[rl * 4 + (q ^ ((rl >> 1) & 3))];
                        }
                    } else {
                        // a piece: [column / 4][row] of four columns, whole lines at a time
                        float4 *dst = reinterpret_cast<float4 *>(p.part_o + prow0 * D) + c32 * 8 * ROWS + row;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e * ROWS] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                }
                const bool held = __any_sync(0xffffffffu, live && z != 0.f);
                if (writer && (poison || held)) {
                    const PagedSeg piece = it;  // (copies: the piece stays in registers)
                    __syncwarp();
                    paged_put_not_finite<D, BF16, REP, RT>(p, piece, ti, row, 128, 128, 0, 32, false, held, poison,
                                                           l > 0.f, nullptr);
                }
            } else {
                // The copies meet in shared memory (the vote above is also the barrier behind
                // the last piece's reads): first their maxima and sums, then O scaled by
                // f_k / R, f_k = 2^(m_k - M), R = sum_k f_k lr_k, all columns at once where the
                // used rows are few, else 32 at a time.  O = sum_k (f_k / R) O_k.
                float *buf = reinterpret_cast<float *>(smem + C::OFF_MERGE);
                const int used = min(p.TPT, p.T) * p.GP;
                constexpr int MAXR = 4;                        // rows of a thread at most
                const bool once = REP * used * (D + 4) * 4 <= C::MERGE && used <= MAXR * (512 / D);
                const int pitch = (once ? D : 32) + 4;
                const int qs = once ? (D == 64 ? 4 : 5) : 3;   // log2 of 4-column groups
                const int x = wq * 32 + lane;
                const int c4 = (x & ((1 << qs) - 1)) * 4;      // this thread's columns
                void *dst[MAXR];                               // of its rows, at column c4
                int dtok[MAXR];
#pragma unroll
                for (int e = 0; e < MAXR; ++e) {
                    const int r = (x >> qs) + e * (128 >> qs);
                    const int rl = r * p.gp_magic >> 16, h = it.g0 + (r - rl * p.GP);
                    dtok[e] = it.tok0 + rl;
                    dst[e] = nullptr;
                    if (r < used && dtok[e] < p.T && h < p.G)
                        dst[e] = it.whole ? (void *)(out_row(h, dtok[e]) + c4)
                                          : (void *)(p.part_o + (prow0 + r) * D + c4);
                }
                float scale = 0.f, z = 0.f;  // z: NaN where an output is not finite
                if (nt > 0) {
                    bars->stat[0][x] = m;
                    bars->stat[1][x] = l;
                    bars->stat[2][x] = lr;
                    named_bar_sync(1, 128);
                    float M = -INFINITY, L = 0.f, R = 0.f;
#pragma unroll
                    for (int k = 0; k < REP; ++k) M = fmaxf(M, bars->stat[0][k * ROWS + row]);
#pragma unroll
                    for (int k = 0; k < REP; ++k) {
                        const float mk = bars->stat[0][k * ROWS + row];
                        const float fk = (mk == -INFINITY) ? 0.f : ex2(mk - M);
                        L = fmaf(fk, bars->stat[1][k * ROWS + row], L);
                        R = fmaf(fk, bars->stat[2][k * ROWS + row], R);
                    }
                    none = L == 0.f;
                    scale = ((m == -INFINITY) ? 0.f : ex2(m - M)) / R;
                    lse2 = none ? -INFINITY : M + lg2(L);
                }
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += pitch - 4) {
                    if (nt > 0) {
                        if (c0 > 0) named_bar_sync(1, 128);
#pragma unroll 1
                        for (int c = 0; c < pitch - 4; c += 32) {
                            uint32_t rr[32];
                            tmem_ld32(ob + c0 + c, rr);
                            if (c0 + c == D - 32) {
                                tc_fence_before();
                                mbar_arrive(&bars->o_empty);
                            }
                            if (row < used) {
                                float4 *dst = reinterpret_cast<float4 *>(buf + (kw * used + row) * pitch + c);
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    dst[e] = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                  : make_float4(__uint_as_float(rr[4 * e]) * scale,
                                                                __uint_as_float(rr[4 * e + 1]) * scale,
                                                                __uint_as_float(rr[4 * e + 2]) * scale,
                                                                __uint_as_float(rr[4 * e + 3]) * scale);
                            }
                        }
                        named_bar_sync(1, 128);
                    }
#pragma unroll
                    for (int e = 0; e < MAXR; ++e) {
                        if (dst[e] == nullptr) continue;
                        const float *src = buf + ((x >> qs) + e * (128 >> qs)) * pitch + c4;
                        float v[4] = {0.f, 0.f, 0.f, 0.f};
                        if (nt > 0) {
#pragma unroll
                            for (int k = 0; k < REP; ++k) {
                                const float4 y = *reinterpret_cast<const float4 *>(src + k * used * pitch);
                                v[0] += y.x;
                                v[1] += y.y;
                                v[2] += y.z;
                                v[3] += y.w;
                            }
                        }
                        z += paged_finite(v);
                        if (it.whole)
                            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(dst[e]) + c0) =
                                make_uint2(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]));
                        else
                            *reinterpret_cast<float4 *>(static_cast<float *>(dst[e]) + c0) =
                                make_float4(v[0], v[1], v[2], v[3]);
                    }
                }
                const bool held = __any_sync(0xffffffffu, z != 0.f);
                if (poison || held) {
                    const PagedSeg piece = it;  // (copies: the piece stays in registers)
                    paged_put_not_finite<D, BF16, REP, RT>(p, piece, 0, x >> qs, 128 >> qs, used, c4, 4, once, held,
                                                           poison, false, bars->stat[1]);
                }
            }
            if (mine && kw == 0 && writer) {
                if (it.whole)
                    p.lse[((long long)it.b * p.Hk * p.G + it.hk * p.G + head) * p.T + tok] =
                        lse2 * 0.69314718055994531f;
                else
                    p.part_lse[prow0 + row] = lse2;
            }
            n0 += nt * SPT;
            if (nt > 0) ++t;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_FIX) tmem_dealloc(tmem, 512);
}

// Merges the pieces of the items that were cut: with the pieces' log-sum-exps L_s (base 2),
//   LSE = M + log2 sum_s 2^(L_s - M), O = sum_s 2^(L_s - LSE) O_s.
// An O_s may be infinite (a visible key's value is), and 0 * inf would be NaN, so no weight is 0:
// 2^x, which is from x = -127 on and for the repeats of the last piece that fill up a round, gets
// the smallest fp32 number added (2^-149 of the largest 16-bit value is below 5e-7).
// A share leaves at most one item unfinished that it began: grid.x = shares.  The item, its
// pieces and their places are worked out before the wait for the attention kernel (which
// triggers this launch behind its own wait, so that the lengths are final by then).
// Without copies (TRANS, rows of a piece as [column / 4][row]): grid.y = groups of 32 rows, a
// lane is a row, a warp 1 / 8 of the columns.  With copies a block takes all rows, so that the
// whole grid is in place beside the attention kernel's when that ends: a warp is a row at a
// time, a lane 1 / 32 of the columns.
// (64 registers: what the attention kernel leaves of an SM's is 17000)
template <int D, bool BF16, int REP, int RT>
__global__ void __launch_bounds__(256, 4) fa_paged_merge_kernel(const __grid_constant__ PagedParams p) {
    constexpr bool TRANS = REP == 1;
    constexpr int ROWS = 128 / REP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = blockIdx.x;
    pdl_launch_dependents();  // (whoever comes next waits for this grid's end in its turn)
    PagedWalk<RT> walk;
    const PagedShares sh = walk.init(p, c0, lane);
    bool cut = false;
    int b = 0, hk = 0, rt = 0, c1 = 0, first = 0;
    if (walk.u < walk.u1) {
        const int begin = walk.u, end = walk.u1;
        walk.u = end - 1;
        const auto x = walk.place(p, lane);
        const int cost = x.tiles + kItemCost;
        if (x.r < x.valid * cost) {
            rt = (unsigned)x.r / (unsigned)cost;
            const int u0 = end - 1 - (x.r - rt * cost);  // the item's first unit
            cut = u0 >= begin && u0 + x.tiles > end;
            b = x.b;
            hk = x.hk;
            c1 = sh.of(u0 + x.tiles - 1);
            first = begin < u0 ? 1 : 0;  // (its first piece is not the share's first)
        }
    }
    pdl_wait();
    if (!cut) return;
    // Each round takes U pieces of R rows, log-sum-exps and outputs together, into a running
    // maximum and sum: one wait on L2 (about 0.7 us) a round.  Few rows come in many pieces
    // (decoding), many rows in few.  (Three pieces at d = 128: four do not fit 64 registers.  128
    // rows, 16 sequences of 4000 keys: 61.7 us with three, 63.0 with four, 60.7 with two; one item
    // in 148 pieces: 48.1 with three, 50.2 with four, 57.1 with two.)
    constexpr int E = TRANS ? D / 8 : D / 32;             // columns of a thread
    constexpr int R = TRANS ? 1 : (REP == 4 ? 1 : 2), U = TRANS ? (D == 128 ? 3 : 4) : (REP == 4 ? 8 : 3);
    constexpr int NR = TRANS ? 1 : (REP == 4 ? 4 : 8);    // rows of a thread
    constexpr float kTiny = 1.401298464324817e-45f;       // 2^-149
#pragma unroll 1
    for (int k = 0; k < NR; k += R) {
        int row[R], tok[R], head[R];
        bool in[R], any = false;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            row[j] = TRANS ? blockIdx.y * 32 + lane : (k + j) * 8 + warp;  // of the item
            const int tile = row[j] / ROWS, r = row[j] - tile * ROWS;
            const int tl = r * p.gp_magic >> 16, tt = rt / p.GT;
            tok[j] = (tt * RT + tile) * p.TPT + tl;
            head[j] = (rt - tt * p.GT) * p.GP + (r - tl * p.GP);
            in[j] = tile < RT && tl < p.TPT && tok[j] < p.T && head[j] < p.G;
            any = any || in[j];
            if (!in[j]) row[j] = 0;
        }
        if (!any) continue;
        float acc[R][E], sum[R], M[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            sum[j] = 0.f;
            M[j] = -3.402823466e38f;  // (finite, so that the differences below are numbers)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[j][e] = 0.f;
        }
        for (int s0 = c0; s0 <= c1; s0 += U) {
            float ls[U][R], v[U][R][E];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = min(s0 + u, c1);
                const long long at = (2LL * c + (c == c0 ? first : 0)) * (RT * ROWS);
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    ls[u][j] = s0 + u <= c1 ? p.part_lse[at + row[j]] : -INFINITY;
                    if constexpr (TRANS) {
                        const int tile = row[j] / ROWS, r = row[j] - tile * ROWS;
                        const float4 *src = reinterpret_cast<const float4 *>(p.part_o + (at + tile * ROWS) * D) +
                                            warp * (E / 4) * ROWS + r;
#pragma unroll
                        for (int e = 0; e < E / 4; ++e) {
                            const float4 x = src[e * ROWS];
                            v[u][j][4 * e] = x.x, v[u][j][4 * e + 1] = x.y;
                            v[u][j][4 * e + 2] = x.z, v[u][j][4 * e + 3] = x.w;
                        }
                    } else if constexpr (E == 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(p.part_o + (at + row[j]) * D + lane * E);
                        v[u][j][0] = x.x, v[u][j][1] = x.y, v[u][j][2] = x.z, v[u][j][3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2 *>(p.part_o + (at + row[j]) * D + lane * E);
                        v[u][j][0] = x.x, v[u][j][1] = x.y;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float M1 = M[j];
#pragma unroll
                for (int u = 0; u < U; ++u) M1 = fmaxf(M1, ls[u][j]);
                const float alpha = ex2(M[j] - M1) + kTiny;
                M[j] = M1;
                sum[j] *= alpha;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[j][e] *= alpha;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float w = ex2(ls[u][j] - M1) + kTiny;  // (NaN is carried on)
                    sum[j] += w;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[j][e] = fmaf(w, v[u][j][e], acc[j][e]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (!in[j]) continue;
            const bool none = sum[j] < 0.5f;  // no piece with a key: else the largest weight is 1
            const float inv = none ? 0.f : 1.f / sum[j];
            const int h = hk * p.G + head[j];
            uint32_t *o = reinterpret_cast<uint32_t *>(const_cast<uint16_t *>(p.o.p) + b * p.o.sb + h * p.o.sh +
                                                       tok[j] * p.o.st + (TRANS ? warp : lane) * E);
            uint32_t w[E / 2];
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
                w[e] = none ? 0u : pack2<BF16>(acc[j][2 * e] * inv, acc[j][2 * e + 1] * inv);
            if constexpr (E / 2 >= 4) {
#pragma unroll
                for (int e = 0; e < E / 8; ++e)
                    reinterpret_cast<uint4 *>(o)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            } else if constexpr (E / 2 == 2) {
                *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
            } else {
                *o = w[0];
            }
            if (TRANS ? warp == 0 : lane == 0)
                p.lse[((long long)b * p.Hk * p.G + h) * p.T + tok[j]] =
                    none ? -INFINITY : (M[j] + lg2(sum[j])) * 0.69314718055994531f;
        }
    }
}

}  // namespace fa
