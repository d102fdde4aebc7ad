// fa_paged.cuh -- attention of a step's new tokens over a paged key/value cache.
//
// Sequence b holds cache_len[b] tokens and new_len[b] new ones (one token, a chain or a tree
// of drafted tokens), all in the cache's pages.  New token t of b sees every held key and the
// new keys its mask row names (chain: keys up to itself).  With G query heads to a key/value
// head, the R = T * G rows that share a key/value head are packed into tiles of 128 rows
// (row r = token r / G, head r % G), so that the cache is read once for all of them:
//   S = Q K^T on tcgen05 (M = 128 rows, 128 keys), online softmax with a running maximum m
//   and sum l per row, O += P V.
//
// Bound by memory for up to about 256 rows per key/value head (4 R flop per 2 bytes against
// 260 flop per byte of the card): a 128-key tile of one SM's share of HBM takes 1.5 us at
// d = 128, 0.75 us at d = 64.
//
// Work: the 128-key tiles of all (sequence, key/value head, row tile) items form one flat
// list that is cut into equal shares, one per CTA, wherever the cuts fall (lengths are only
// known on the device).  An item inside one share is written to O directly; the pieces of a
// cut item go to the workspace as fp32 (normalised O, log-sum-exp) and a second kernel,
// launched early by PDL, merges them in a fixed order.
//
// CTA: warps 0..3 softmax (one row per thread), warp 4 producer (page table and TMA), warp 5
// MMA issuer, warp 6 loads Q and repairs V tiles with slots behind the sequence's end (their
// contents are unspecified, and 0 * NaN would reach O).
//
// Few rows (REP = 4: a tile of 32 rows, REP = 2: 64): the rows are repeated in the tile's
// REP lane quarters / halves, and each copy takes 1 / REP of the keys of every tile as a
// softmax of its own (P is zero elsewhere); the copies are merged in the epilogue.  The
// exponentials of a tile then take 1 / REP of the time.
#pragma once

#include <cuda.h>

#include "fa_rope.cuh"
#include "sm100.cuh"

namespace fa {

struct PagedParams {
    Rows q, o;           // [B, H, T, d]
    Rows vc;             // the value cache (also behind the tensor map)
    float *lse;          // [B, H, T]
    PageTable pt;
    const uint8_t *tree; // [B or 1, T, T], nullptr: chain
    long long tree_sb;   // bytes between sequences (0: shared)
    float *part_o;       // [2 * gridDim.x][rows of a tile][D]
    float *part_lse;     // [2 * gridDim.x][rows of a tile], base 2
    int B, Hk, G, T;
    int row_tiles;       // tiles of an item's R rows
    int ctas;            // shares
    float scale_log2;
};

template <int D>
struct PagedCfg {
    static constexpr int BN = 128;              // keys per tile
    static constexpr int HALVES = D / 64;
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int TILE = BN * D * 2;     // K or V tile
    static constexpr int HALF = BN * 128;       // one 64-element column block of a tile
    static constexpr int NS = (D == 64) ? 11 : 5;  // ring of K and V tiles, alternating
    static constexpr int MERGE = 4 * 32 * 33 * 4;  // REP merge: a padded 32 x 32 block per warp
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = OFF_Q + QTILE;
    static constexpr int OFF_MERGE = OFF_RING + NS * TILE;
    static constexpr int OFF_BAR = OFF_MERGE + MERGE;
    static constexpr int USED = OFF_BAR + 2560;
    static constexpr int SMEM = USED + 1024;
    static constexpr int THREADS = 224;
    static constexpr uint32_t COL_S = 0;        // two score buffers
    static constexpr uint32_t COL_P = 256;      // two P buffers of 64 columns
    static constexpr uint32_t COL_O = 384;
    static_assert(COL_O + D <= 512, "TMEM budget");
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct PagedBars {
    uint64_t q_full, q_empty, o_empty;
    uint64_t s_full[2], s_empty[2], p_full[2], pv_done[2];
    uint64_t full[12], empty[12], fixed[12];  // per ring slot; fixed: V repaired by warp 6
    uint32_t tmem_base;
    int b0;                 // this CTA's share: first sequence, its first unit, the share
    long long base0, u0, u1;
    uint32_t bad[16];       // per tile: sub-pages whose page number is outside the cache
    // Item t & 3 hides keys whose V is not finite.  (Four: warp 6 reaches item t + 4 only
    // after the softmax of item t + 1 began.)
    int poison[4];
    float stat[3][128];     // REP merge: m, l, l of the rounded weights
};

// Work units of a sequence: `tiles` per (head, row tile with new tokens), one for a row tile
// without (its rows are written as empty).
struct PagedSeq {
    int past, fresh, tiles, valid;  // valid: row tiles that hold a new token
    int per_head;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams &p, int rows, int b) {
    PagedSeq s;
    page_lengths(p.pt, p.T, b, s.past, s.fresh);
    s.tiles = (s.past + s.fresh + 127) >> 7;
    s.valid = (int)(((long long)s.fresh * p.G + rows - 1) / rows);
    s.per_head = s.valid * s.tiles + (p.row_tiles - s.valid);
    return s;
}

// All units, and the sequence in which unit u lies with its first unit (one whole warp).
__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ long long paged_units(const PagedParams &p, int rows, int lane, int upto) {
    long long n = 0;
    for (int b = lane; b < upto; b += 32) n += (long long)paged_seq(p, rows, b).per_head * p.Hk;
    return warp_sum(n);
}

// One piece of work: key tiles [j0, j1) of one item.
struct PagedSeg {
    int b, hk, rt;      // sequence, key/value head, row tile
    int past, total;    // keys held, keys with the new ones
    int fresh;
    int j0, j1;
    int index;          // 0: the share's first piece
    bool whole;
    // Whether some row may see fewer new keys than another.
    __device__ __forceinline__ bool hides(const PagedParams &p) const {
        return fresh > 1 || p.tree != nullptr;
    }
    // Whether warp 6 goes over V tile j: slots behind the last key, whose contents are
    // unspecified, are cleared (0 * NaN would reach O), and so are values that are not
    // finite in keys that some row may not see.
    __device__ __forceinline__ bool repair(const PagedParams &p, int j) const {
        return (j + 1) * 128 > (hides(p) ? past : total);
    }
};

// All ones in the halves of a 16-bit pair that are infinite or NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
    constexpr uint32_t e = BF16 ? 0x7F807F80u : 0x7C007C00u;
    return __vcmpeq2(w & e, e);
}

struct PagedWalk {
    long long u, u1, base;
    int b, index;
    PagedSeq s;
    __device__ __forceinline__ void init(const PagedParams &p, int rows, const PagedBars *bars) {
        u = bars->u0;
        u1 = bars->u1;
        b = bars->b0;
        base = bars->base0;
        index = 0;
        if (u < u1) s = paged_seq(p, rows, b);
    }
    __device__ __forceinline__ bool next(const PagedParams &p, int rows, PagedSeg &g) {
        if (u >= u1) return false;
        while (u >= base + (long long)s.per_head * p.Hk) {
            base += (long long)s.per_head * p.Hk;
            s = paged_seq(p, rows, ++b);
        }
        const unsigned r0 = (unsigned)(u - base);
        g.hk = (int)(r0 / (unsigned)s.per_head);
        const int r = (int)(r0 - (unsigned)g.hk * (unsigned)s.per_head);
        g.b = b;
        g.past = s.past;
        g.fresh = s.fresh;
        g.total = s.past + s.fresh;
        g.index = index++;
        if (r < s.valid * s.tiles) {
            g.rt = r / s.tiles;
            g.j0 = r - g.rt * s.tiles;
            const long long left = u1 - u;
            g.j1 = (int)min((long long)s.tiles, g.j0 + left);
            u += g.j1 - g.j0;
            g.whole = g.j0 == 0 && g.j1 == s.tiles;
            if (p.tree == nullptr) {  // a chain's rows see no key behind their last token
                const int t1 = min(s.fresh, (g.rt * rows + rows - 1) / p.G + 1);
                g.j1 = min(g.j1, (s.past + t1 + 127) >> 7);
            }
        } else {
            g.rt = s.valid + (r - s.valid * s.tiles);
            g.j0 = g.j1 = 0;
            g.whole = true;
            u += 1;
        }
        return true;
    }
};

__device__ __forceinline__ void tma_load_4d(void *smem_dst, const void *tmap, uint64_t *bar, int x,
                                            int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// 16 bytes global -> shared, asynchronous; zeros where !valid.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// C columns of 32 TMEM lanes.
template <int C>
__device__ __forceinline__ void tmem_ldn(uint32_t a, uint32_t (&r)[C]) {
    if constexpr (C == 128) tmem_ld128(a, r);
    else if constexpr (C == 64) tmem_ld64(a, r);
    else tmem_ld32(a, r);
}

template <int D, bool BF16, int REP>
__global__ void __launch_bounds__(224, 1)
fa_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ PagedParams p) {
    using C = PagedCfg<D>;
    constexpr int ROWS = 128 / REP;   // rows of a tile
    constexpr int CW = 128 / REP;     // keys of a tile that one thread handles
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem + C::OFF_Q;
    uint8_t *ring = smem + C::OFF_RING;
    PagedBars *bars = reinterpret_cast<PagedBars *>(smem + C::OFF_BAR);
    static_assert(sizeof(PagedBars) <= 2560, "barrier area");
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 160) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        mbar_init(&bars->o_empty, 128);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->s_empty[i], 128);
            mbar_init(&bars->p_full[i], 128);
            mbar_init(&bars->pv_done[i], 1);
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
            mbar_init(&bars->fixed[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 6) tmem_alloc(&bars->tmem_base, 512);
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 4) {
        if (blockIdx.x == 0)
            for (int b = lane; b < p.B; b += 32) page_lengths_check(p.pt, p.T, b);
        // this CTA's share of the units
        const long long W = paged_units(p, ROWS, lane, p.B);
        const long long G = min((long long)p.ctas, W);
        const long long c = blockIdx.x;
        const long long u0 = c < G ? c * W / G : 0, u1 = c < G ? (c + 1) * W / G : 0;
        // the sequence of u0: 32 sequences at a time
        long long base = 0;
        int b0 = 0;
        if (u0 < u1) {
            for (int k = 0; k < p.B; k += 32) {
                const long long mine =
                    k + lane < p.B ? (long long)paged_seq(p, ROWS, k + lane).per_head * p.Hk : 0;
                long long upto = mine;  // inclusive prefix sum
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                const unsigned past = __ballot_sync(0xffffffffu, base + upto > u0);
                if (past) {
                    const int f = __ffs(past) - 1;
                    b0 = k + f;
                    base += __shfl_sync(0xffffffffu, upto - mine, f);
                    break;
                }
                base += __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        if (lane == 0) {
            bars->b0 = b0;
            bars->base0 = base;
            bars->u0 = u0;
            bars->u1 = u1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    PagedWalk walk;
    walk.init(p, ROWS, bars);
    PagedSeg it;

    if (warp == 4) {
        // ------------------------------ producer: whole warp ---------------------------
        // A tile's pages: npt boxes (a page, or 128 rows of a larger one) per 64-element
        // column block; lane l loads box l % npt of block l / npt.
        const int page = 1 << p.pt.page_shift;
        const int box_rows = min(page, 128);
        const int npt = 128 / box_rows;
        const int mine = lane % npt, half = lane / npt;
        int gj = 0;  // tiles so far
        bool ok = true;
        while (ok && walk.next(p, ROWS, it)) {
            const int *row = p.pt.table + (long long)it.b * p.pt.max_blocks;
            for (int j = it.j0; j < it.j1; ++j, ++gj) {
                const int key = j * 128 + mine * box_rows;
                int z = p.pt.num_pages;  // outside the cache: the box is filled with zeros
                bool bad = false;
                if (key < it.total) {
                    const int id = __ldg(row + (key >> p.pt.page_shift));
                    bad = id < 0 || id >= p.pt.num_pages;
                    if (!bad) z = id;
                }
                const unsigned bads = __ballot_sync(0xffffffffu, bad && half == 0);
                if (lane == 0) {
                    bars->bad[gj & 15] = bads;
                    if (bads) atomicExch(&g_status, 6);
                }
                const int y = key & (page - 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int n = 2 * gj + kv, s = n % C::NS;
                    if (n >= C::NS)
                        ok = __all_sync(0xffffffffu, mbar_wait(&bars->empty[s], (n / C::NS - 1) & 1));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bars->full[s], C::TILE);
                    __syncwarp();
                    if (half < C::HALVES)
                        tma_load_4d(ring + s * C::TILE + half * C::HALF + mine * box_rows * 128,
                                    kv ? &tmV : &tmK, &bars->full[s], half * 64, y, it.hk, z);
                }
                if (!ok) break;
            }
        }
        if (!ok)  // a wait gave up: the copies in flight land before the CTA's memory goes
            for (int n = max(0, 2 * gj + 1 - C::NS); n < 2 * gj + 2; ++n)
                (void)mbar_wait(&bars->full[n % C::NS], (n / C::NS) & 1);
    } else if (warp == 5) {
        // ------------------------------ MMA issuer --------------------------------------
        if (lane == 0) {
            constexpr uint32_t kIdescS = idesc_f16(BF16, false, false, 128, 128);
            constexpr uint32_t kIdescO = idesc_f16(BF16, false, true, 128, D);
            const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t k_desc = smem_desc_sw128(smem_u32(ring), 16, 1024);
            const uint64_t v_desc = smem_desc_sw128(smem_u32(ring), C::HALF, 1024);
            auto issue_s = [&](int g) -> bool {
                const int n = 2 * g, s = n % C::NS;
                if (!mbar_wait(&bars->full[s], (n / C::NS) & 1)) return false;
                if (g >= 2 && !mbar_wait(&bars->s_empty[g & 1], (g / 2 - 1) & 1)) return false;
                tc_fence_after();
                const uint64_t kd = k_desc + (uint64_t)((s * C::TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t qo = (uint64_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4);
                    const uint64_t ko = (uint64_t)(((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4);
                    mma_ss(tmem + C::COL_S + (g & 1) * 128, q_desc + qo, kd + ko, kIdescS, kk > 0);
                }
                mma_commit(&bars->empty[s]);
                mma_commit(&bars->s_full[g & 1]);
                return true;
            };
            bool ok = true;
            int gj = 0, t = 0;
            uint32_t fixes = 0;  // parity of each slot's next repair
            while (ok && walk.next(p, ROWS, it)) {
                const int nt = it.j1 - it.j0;
                if (nt <= 0) continue;
                if (!mbar_wait(&bars->q_full, t & 1)) break;
                tc_fence_after();
                if (!issue_s(gj)) break;
                for (int i = 0; i < nt; ++i) {
                    const int g = gj + i;
                    if (i + 1 < nt) {
                        if (!issue_s(g + 1)) { ok = false; break; }
                    } else {
                        mma_commit(&bars->q_empty);
                    }
                    const int n = 2 * g + 1, s = n % C::NS;
                    if (!mbar_wait(&bars->p_full[g & 1], (g / 2) & 1) ||
                        !mbar_wait(&bars->full[s], (n / C::NS) & 1)) { ok = false; break; }
                    if (it.repair(p, it.j0 + i)) {
                        if (!mbar_wait(&bars->fixed[s], (fixes >> s) & 1)) { ok = false; break; }
                        fixes ^= 1u << s;
                    }
                    if (i == 0 && t > 0 && !mbar_wait(&bars->o_empty, (t - 1) & 1)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t vd = v_desc + (uint64_t)((s * C::TILE) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + C::COL_O, tmem + C::COL_P + (g & 1) * 64 + kk * 8,
                               vd + (uint64_t)((kk * 16 * 128) >> 4), kIdescO, i > 0 || kk > 0);
                    mma_commit(&bars->empty[s]);
                    mma_commit(&bars->pv_done[g & 1]);
                }
                gj += nt;
                ++t;
            }
        }
    } else if (warp == 6) {
        // ------------------------------ Q loads, V tails --------------------------------
        bool ok = true;
        int gj = 0, t = 0;
        while (ok && walk.next(p, ROWS, it)) {
            const int nt = it.j1 - it.j0;
            if (nt <= 0) continue;
            if (t > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->q_empty, (t - 1) & 1))) break;
            constexpr int CH = D / 8;        // 16-byte chunks of a row
            constexpr int RPI = 32 / CH;     // rows per step
            const int ch = lane % CH;
            const long long qb = it.b * p.q.sb;
            for (int i = lane / CH; i < 128; i += RPI) {
                const int r = it.rt * ROWS + (i % ROWS);
                const int tok = r / p.G, h = it.hk * p.G + (r - tok * p.G);
                const bool valid = tok < it.fresh;
                const uint16_t *src = p.q.p + (valid ? qb + h * p.q.sh + tok * p.q.st : 0) + ch * 8;
                const uint32_t dst = smem_u32(sQ) + (ch >> 3) * (128 * 128) + i * 128 +
                                     (((ch & 7) ^ (i & 7)) << 4);
                cp_async16(dst, src, valid);
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_full);
            // V tiles with new keys or slots behind them
            bool found = false;
            for (int i = 0; ok && i < nt; ++i) {
                const int j = it.j0 + i;
                if (!it.repair(p, j)) continue;
                const int n = 2 * (gj + i) + 1, s = n % C::NS;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[s], (n / C::NS) & 1));
                if (!ok) break;
                // (the swizzle permutes 16-byte chunks within a row only)
                uint8_t *tile = ring + s * C::TILE;
                const int tail = min(128, it.total - j * 128);
                for (int x = tail * 8 + lane; x < 128 * 8; x += 32)
#pragma unroll
                    for (int hf = 0; hf < C::HALVES; ++hf)
                        *reinterpret_cast<uint4 *>(tile + hf * C::HALF + x * 16) = make_uint4(0, 0, 0, 0);
                if (it.hides(p)) {
                    for (int x = max(0, it.past - j * 128) * 8 + lane; x < tail * 8; x += 32)
#pragma unroll
                        for (int hf = 0; hf < C::HALVES; ++hf) {
                            uint32_t *w = reinterpret_cast<uint32_t *>(tile + hf * C::HALF + x * 16);
                            uint4 v = *reinterpret_cast<uint4 *>(w);
                            const uint32_t hit = not_finite2<BF16>(v.x) | not_finite2<BF16>(v.y) |
                                                 not_finite2<BF16>(v.z) | not_finite2<BF16>(v.w);
                            if (hit) {
                                found = true;
                                v.x &= ~not_finite2<BF16>(v.x);
                                v.y &= ~not_finite2<BF16>(v.y);
                                v.z &= ~not_finite2<BF16>(v.z);
                                v.w &= ~not_finite2<BF16>(v.w);
                                *reinterpret_cast<uint4 *>(w) = v;
                            }
                        }
                    found = __any_sync(0xffffffffu, found);
                }
                if (lane == 0) bars->poison[t & 3] = found ? 1 : 0;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->fixed[s]);
            }
            ++t;
            gj += nt;
        }
    } else {
        // ------------------------------ softmax warps -----------------------------------
        constexpr int WPC = 4 / REP;                       // warps of one copy of the rows
        const int row = (warp % WPC) * 32 + lane;          // row of the tile
        const int kw = warp / WPC;                         // the copy: keys [kw * CW, + CW)
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const uint32_t ob = tmem + lane_base + C::COL_O;
        const float sl2 = p.scale_log2;
        if constexpr (REP > 1) {  // P is zero outside the copy's own keys
            uint32_t zero[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) zero[i] = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_st32(tmem + lane_base + C::COL_P + i * 32, zero);
        }
        bool ok = true;
        int gj = 0, t = 0;
        while (walk.next(p, ROWS, it)) {
            const int r = it.rt * ROWS + row;
            const int tok = r / p.G;
            const bool live = tok < it.fresh;              // a new token's row
            const int nt = max(it.j1 - it.j0, 0);
            float m = -INFINITY;   // running maximum, base 2
            float l = 0.f;         // running sum
            float lr = 0.f;        // the same sum of the rounded weights
            for (int i = 0; ok && i < nt; ++i) {
                const int g = gj + i;
                const int k0 = (it.j0 + i) * 128 + kw * CW;  // first key of this thread
                // visibility of keys from the first new one on (held keys are all visible)
                const bool need_mask = k0 + CW > it.past;
                uint32_t vis[CW / 32];
                if (need_mask) {
#pragma unroll
                    for (int w = 0; w < CW / 32; ++w) {
                        const int x0 = k0 + w * 32 - it.past;  // new key of bit 0
                        uint32_t bits = 0u;
                        if (live) {
                            if (p.tree == nullptr) {
                                const int n = tok + 1 - x0;    // keys up to the row's token
                                bits = n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
                            } else {
                                bits = x0 >= 0 ? 0u : (x0 <= -32 ? 0xffffffffu : (1u << -x0) - 1u);
                                const uint8_t *mr = p.tree + it.b * p.tree_sb + (long long)tok * p.T;
                                const int lo = max(0, -x0), hi = min(32, it.fresh - x0);
                                for (int c = lo; c < hi; ++c)
                                    bits |= (__ldg(mr + x0 + c) != 0 ? 1u : 0u) << c;
                            }
                        }
                        vis[w] = bits;
                    }
                }
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[g & 1], (g / 2) & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float s[CW];
                {
                    uint32_t rr[CW];
                    tmem_ldn<CW>(tmem + lane_base + C::COL_S + (g & 1) * 128 + kw * CW, rr);
#pragma unroll
                    for (int c = 0; c < CW; ++c) s[c] = __uint_as_float(rr[c]);
                }
                const uint32_t bad = bars->bad[g & 15];
                tc_fence_before();
                mbar_arrive(&bars->s_empty[g & 1]);
                if (need_mask) {
#pragma unroll
                    for (int c = 0; c < CW; ++c)
                        if (!((vis[c >> 5] >> (c & 31)) & 1u)) s[c] = -INFINITY;
                }
                if (bad) {  // keys of pages outside the cache are not visible
                    const int sh = min(p.pt.page_shift, 7);
#pragma unroll
                    for (int c = 0; c < CW; ++c)
                        if ((bad >> ((kw * CW + c) >> sh)) & 1u) s[c] = -INFINITY;
                }
                float mxv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mxv[e] = fmaxf(s[e], s[8 + e]);
#pragma unroll
                    for (int c = 16; c < CW; c += 16) mxv[e] = fmax3(mxv[e], s[c + e], s[c + 8 + e]);
                }
                const float mx = fmax3(fmax3(mxv[0], mxv[1], mxv[2]), fmax3(mxv[3], mxv[4], mxv[5]),
                                       fmaxf(mxv[6], mxv[7])) * sl2;
                // Lazy rescale: m moves when the maximum grew by more than 2^8.
                const bool any_grow = __any_sync(0xffffffffu, mx > m + 8.0f);
                float alpha = 1.f;
                if (any_grow && mx > m) {
                    alpha = ex2(m - mx);
                    m = mx;
                }
                const float m_use = (m == -INFINITY) ? 0.f : m;
                float s0 = 0.f, s1 = 0.f, r0 = 0.f, r1 = 0.f;
                uint32_t pk[CW / 2];
#pragma unroll
                for (int c = 0; c < CW; c += 2) {
                    const float p0 = ex2(fmaf(s[c], sl2, -m_use));
                    const float p1 = ex2(fmaf(s[c + 1], sl2, -m_use));
                    s0 += p0;
                    s1 += p1;
                    pk[c >> 1] = pack2<BF16>(p0, p1);
                    const float2 q = unpack2<BF16>(pk[c >> 1]);
                    r0 += q.x;
                    r1 += q.y;
                }
                l = l * alpha + (s0 + s1);
                lr = lr * alpha + (r0 + r1);
                // P's buffer is free once P_{g-2} V_{g-2} is done; O may be rescaled once
                // P_{g-1} V_{g-1} is.
                if (g >= 2 &&
                    !__all_sync(0xffffffffu, mbar_wait(&bars->pv_done[g & 1], (g / 2 - 1) & 1))) {
                    ok = false;
                    break;
                }
                if (i > 0 && any_grow) {
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait(&bars->pv_done[(g - 1) & 1], ((g - 1) / 2) & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t rr[32];
                        tmem_ld32(ob + c * 32, rr);
#pragma unroll
                        for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
                        tmem_st32(ob + c * 32, rr);
                    }
                }
                tc_fence_after();
                {
                    const uint32_t pb = tmem + lane_base + C::COL_P + (g & 1) * 64 + kw * (CW / 2);
                    if constexpr (CW == 32) {
                        uint32_t rr[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) rr[e] = pk[e];
                        tmem_st16(pb, rr);
                    } else {
#pragma unroll
                        for (int h = 0; h < CW / 64; ++h) {
                            uint32_t rr[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) rr[e] = pk[h * 32 + e];
                            tmem_st32(pb + h * 32, rr);
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(&bars->p_full[g & 1]);
            }

            // ------------------------------ epilogue of the piece ------------------------
            if (ok && nt > 0) {
                const int g = gj + nt - 1;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[g & 1], (g / 2) & 1));
                tc_fence_after();
            }
            // (the merge of the copies has barriers of all four warps: they leave together)
            if constexpr (REP > 1)
                if (nt > 0) ok = named_bar_and(1, 128, ok);
            if (!ok) break;
            if (!live) m = -INFINITY, l = lr = 0.f;  // rows behind the last new token are empty
            // weights of the copies: O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) lr_k
            float f = 1.f;
            if constexpr (REP > 1) {
                if (nt > 0) {
                    bars->stat[0][threadIdx.x] = m;
                    bars->stat[1][threadIdx.x] = l;
                    bars->stat[2][threadIdx.x] = lr;
                    named_bar_sync(1, 128);
                    float M = -INFINITY;
#pragma unroll
                    for (int k = 0; k < REP; ++k) M = fmaxf(M, bars->stat[0][k * ROWS + row]);
                    f = (m == -INFINITY) ? 0.f : ex2(m - M);
                    l = lr = 0.f;
#pragma unroll
                    for (int k = 0; k < REP; ++k) {
                        const float mk = bars->stat[0][k * ROWS + row];
                        const float fk = (mk == -INFINITY) ? 0.f : ex2(mk - M);
                        l = fmaf(fk, bars->stat[1][k * ROWS + row], l);
                        lr = fmaf(fk, bars->stat[2][k * ROWS + row], lr);
                    }
                    m = M;
                }
            }
            const bool none = l == 0.f;                    // (a NaN sum is carried to O and LSE)
            const float inv = none ? 0.f : f / lr;
            const float lse2 = none ? -INFINITY : m + lg2(l);
            const bool mine = r < p.G * p.T;               // a row of the call
            const int h = it.hk * p.G + (r - tok * p.G);
            const long long slot = 2 * (long long)blockIdx.x + (it.index != 0 ? 1 : 0);
            uint16_t *orow = const_cast<uint16_t *>(p.o.p) + it.b * p.o.sb + h * p.o.sh + tok * p.o.st;
            float *prow = p.part_o + (slot * ROWS + row) * D;
            float *merge = reinterpret_cast<float *>(smem + C::OFF_MERGE);
            // Values that warp 6 cleared reach the rows that do see them (rare: only where a
            // new key's V is not finite, and slow).
            const bool poison = nt > 0 && it.hides(p) && it.j1 * 128 > it.past && bars->poison[t & 3] != 0;
            auto add_not_finite = [&](float *v, int n, int col) {
                if (!live) return;
                for (int j = max(it.past, it.j0 * 128); j < min(it.total, it.j1 * 128); ++j) {
                    const int x = j - it.past;
                    const bool seen = p.tree ? p.tree[it.b * p.tree_sb + (long long)tok * p.T + x] != 0
                                             : x <= tok;
                    const int id = p.pt.table[(long long)it.b * p.pt.max_blocks + (j >> p.pt.page_shift)];
                    if (!seen || id < 0 || id >= p.pt.num_pages) continue;
                    const uint16_t *src = p.vc.p + id * p.vc.sb + it.hk * p.vc.sh +
                                          (j & ((1 << p.pt.page_shift) - 1)) * p.vc.st + col;
                    for (int e = 0; e < n; ++e) {
                        const uint32_t w = src[e];
                        if (not_finite2<BF16>(w) & 0xffffu) v[e] += unpack2<BF16>(w).x;
                    }
                }
            };
#pragma unroll
            for (int c32 = 0; c32 < D / 32; ++c32) {
                uint32_t rr[32];
                if (nt > 0) {
                    tmem_ld32(ob + c32 * 32, rr);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        rr[e] = none ? 0u : __float_as_uint(__uint_as_float(rr[e]) * inv);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) rr[e] = 0u;
                }
                if (c32 == D / 32 - 1 && nt > 0) {
                    tc_fence_before();
                    mbar_arrive(&bars->o_empty);
                }
                if constexpr (REP == 1) {
                    if (!mine) continue;
                    if (poison) {
                        float v[32];
                        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(rr[e]);
                        add_not_finite(v, 32, c32 * 32);
                        for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(v[e]);
                    }
                    if (it.whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(orow) + c32 * 4;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e] = make_uint4(
                                pack2<BF16>(__uint_as_float(rr[8 * e]), __uint_as_float(rr[8 * e + 1])),
                                pack2<BF16>(__uint_as_float(rr[8 * e + 2]), __uint_as_float(rr[8 * e + 3])),
                                pack2<BF16>(__uint_as_float(rr[8 * e + 4]), __uint_as_float(rr[8 * e + 5])),
                                pack2<BF16>(__uint_as_float(rr[8 * e + 6]), __uint_as_float(rr[8 * e + 7])));
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(prow) + c32 * 8;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_float4(__uint_as_float(rr[4 * e]), __uint_as_float(rr[4 * e + 1]),
                                                 __uint_as_float(rr[4 * e + 2]), __uint_as_float(rr[4 * e + 3]));
                    }
                } else {
                    // sum of the copies: each warp lays its 32 x 32 block out (padded rows),
                    // copy kw then sums columns [kw * 32 / REP, + 32 / REP) of its row
                    float *buf = merge;
                    if (c32 > 0) named_bar_sync(1, 128);
#pragma unroll
                    for (int e = 0; e < 32; ++e) buf[(warp * 32 + lane) * 33 + e] = __uint_as_float(rr[e]);
                    named_bar_sync(1, 128);
                    constexpr int N = 32 / REP;
                    float v[N];
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        v[e] = 0.f;
#pragma unroll
                        for (int k = 0; k < REP; ++k) v[e] += buf[(k * ROWS + row) * 33 + kw * N + e];
                    }
                    if (poison) add_not_finite(v, N, c32 * 32 + kw * N);
                    if (mine) {
                        if (it.whole) {
                            uint4 *dst = reinterpret_cast<uint4 *>(orow + c32 * 32 + kw * N);
#pragma unroll
                            for (int e = 0; e < N / 8; ++e)
                                dst[e] = make_uint4(pack2<BF16>(v[8 * e], v[8 * e + 1]),
                                                    pack2<BF16>(v[8 * e + 2], v[8 * e + 3]),
                                                    pack2<BF16>(v[8 * e + 4], v[8 * e + 5]),
                                                    pack2<BF16>(v[8 * e + 6], v[8 * e + 7]));
                        } else {
                            float4 *dst = reinterpret_cast<float4 *>(prow + c32 * 32 + kw * N);
#pragma unroll
                            for (int e = 0; e < N / 4; ++e)
                                dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                        }
                    }
                }
            }
            if (mine && kw == 0) {
                if (it.whole)
                    p.lse[((long long)it.b * p.Hk * p.G + h) * p.T + tok] =
                        lse2 * 0.69314718055994531f;
                else
                    p.part_lse[slot * ROWS + row] = lse2;
            }
            if constexpr (REP > 1) named_bar_sync(1, 128);  // stat and the buffers are free again
            gj += nt;
            if (nt > 0) ++t;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 6) tmem_dealloc(tmem, 512);
}

// Merges the pieces of the items that were cut: with the pieces' log-sum-exps L_s (base 2),
//   LSE = M + log2 sum_s 2^(L_s - M), O = sum_s 2^(L_s - LSE) O_s.
// One warp per row; grid = (items, groups of 4 rows).
template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_paged_merge_kernel(const __grid_constant__ PagedParams p,
                                                             const int rows) {
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int item = blockIdx.x;
    const int rt = item % p.row_tiles, hk = (item / p.row_tiles) % p.Hk, b = item / p.row_tiles / p.Hk;
    const int row = blockIdx.y * 4 + warp;
    const int r = rt * rows + row;
    if (row >= rows || r >= p.T * p.G) return;
    const PagedSeq s = paged_seq(p, rows, b);
    if (rt >= s.valid) return;
    const long long W = paged_units(p, rows, lane, p.B), base = paged_units(p, rows, lane, b);
    const long long G = min((long long)p.ctas, W);
    const long long u0 = base + (long long)hk * s.per_head + (long long)rt * s.tiles, u1 = u0 + s.tiles;
    const int c0 = (int)(((u0 + 1) * G - 1) / W), c1 = (int)((u1 * G - 1) / W);
    if (c0 == c1) return;
    // the first piece lies in CTA c0's second slot if that share began before the item
    const int first = (c0 * W / G < u0) ? 1 : 0;
    auto slot = [&](int c) -> long long { return 2LL * c + (c == c0 ? first : 0); };
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.part_lse[slot(c) * rows + row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    constexpr int E = D / 32;  // columns of a lane
    float acc[E], sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
        const float ls = p.part_lse[slot(c) * rows + row];
        const float w = ls == -INFINITY ? 0.f : ex2(ls - M);
        const float *src = p.part_o + (slot(c) * rows + row) * D + lane * E;
        float v[E];
        if constexpr (E == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(src);
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2 *>(src);
            v[0] = x.x; v[1] = x.y;
        }
        sum += w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[e], acc[e]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int tok = r / p.G, h = hk * p.G + (r - tok * p.G);
    uint16_t *o = const_cast<uint16_t *>(p.o.p) + b * p.o.sb + h * p.o.sh + tok * p.o.st + lane * E;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(o) = make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv),
                                                   pack2<BF16>(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(o) = pack2<BF16>(acc[0] * inv, acc[1] * inv);
    if (lane == 0)
        p.lse[((long long)b * p.Hk * p.G + h) * p.T + tok] =
            sum == 0.f ? -INFINITY : (M + lg2(sum)) * 0.69314718055994531f;
}

}  // namespace fa
