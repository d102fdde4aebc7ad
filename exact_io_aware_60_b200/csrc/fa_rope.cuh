// fa_rope.cuh -- rotary positions, and the paged cache's append with the rotation on the way.
//
// Pair i of a head's first `rot` elements, at position p, turns by the angle a = p f_i:
//   (y1, y2) = g (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
// (x1, x2) = (x_i, x_{i + rot/2}) in the half layout, (x_{2i}, x_{2i+1}) in the interleaved
// one; the other elements are copied.  The gradient's map is the transpose: the same with
// sin a negated.
//
// The angle: p f_i / 2 pi reaches 10^5 turns and more at far positions, where a 32-bit
// product keeps no digits of the fraction that matters.  The plan holds each frequency as
// the 64-bit fixed-point fraction of a turn, turns_i = f_i / 2 pi * 2^64 mod 2^64, so that
// the low 64 bits of p * turns_i ARE the fraction of a turn (whole turns drop out exactly,
// for negative p too).  Its top 32 bits, as a signed number, go to sincospif in fp32: an
// error below 2^-25 turns.  No table of angles is read.
//
// Bound by memory: every element is read and written once.  A thread owns 8 pairs (two
// 16-byte vectors) of a token, computes their sines and cosines once and applies them to
// several heads of that token, four heads' loads in flight at a time.  Measured on B200: queries
// and keys of B1 H16 N65536 d128 (1.07 GB read and written) 160 us, 6.7 TB/s, the rate of a plain
// copy; B8 H12 N1024 d64 (50 MB) 10.7 us of which 7.7 are the bytes; appending 2 x 4096 tokens of
// 32 query and 8 key/value heads, d = 128 (201 MB) 34.8 us, 0.88 of the copy rate.
#pragma once

#include "sm100.cuh"

namespace fa {

// A [B, heads, tokens, d] tensor of 16-bit elements, d contiguous: strides in elements.
struct Rows {
    const uint16_t *p;
    long long sb, sh, st;
};

struct RopeParams {
    Rows q, k;        // k.p == nullptr: no keys
    Rows qo, ko;      // outputs (written)
    int H, HT;        // query heads, all heads (queries first)
    int N;            // tokens of a sequence
    int tokens;       // B * N
    int heads_per_thread;
    const int *positions;      // nullptr: 0 .. N-1
    int positions_sb;          // elements between sequences (0: shared)
    const unsigned long long *turns;
    int rot;
    float mag;
    float sign;       // +1 forward, -1 backward
};

// cos and sin (times the magnitude) of 8 consecutive pairs at one position.
__device__ __forceinline__ void rope_angles(const unsigned long long *turns, int pair0, int pos,
                                            float mag, float sign, float (&c)[8], float (&s)[8]) {
    const unsigned long long p = (unsigned long long)(long long)pos;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int frac = (int)(unsigned)((p * __ldg(turns + pair0 + i)) >> 32);
        float si, co;
        sincospif((float)frac * 4.656612873077393e-10f, &si, &co);  // 2^-31: half turns
        c[i] = co * mag;
        s[i] = si * (mag * sign);
    }
}

// Rotates 8 pairs held in two 16-byte vectors: (a_i, b_i) in the half layout, adjacent
// elements of a then b in the interleaved one.  One rounding, to the element type.
template <bool BF16, bool INTER>
__device__ __forceinline__ void rope_turn(uint4 &a, uint4 &b, const float (&c)[8],
                                          const float (&s)[8]) {
    uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2<BF16>(aw[i]), y = unpack2<BF16>(bw[i]);
            aw[i] = pack2<BF16>(x.x * c[i] - x.y * s[i], x.y * c[i] + x.x * s[i]);
            bw[i] = pack2<BF16>(y.x * c[4 + i] - y.y * s[4 + i], y.y * c[4 + i] + y.x * s[4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2<BF16>(aw[i]), y = unpack2<BF16>(bw[i]);
            const int e = 2 * i, o = 2 * i + 1;
            aw[i] = pack2<BF16>(x.x * c[e] - y.x * s[e], x.y * c[o] - y.y * s[o]);
            bw[i] = pack2<BF16>(y.x * c[e] + x.x * s[e], y.y * c[o] + x.y * s[o]);
        }
    }
    a = make_uint4(aw[0], aw[1], aw[2], aw[3]);
    b = make_uint4(bw[0], bw[1], bw[2], bw[3]);
}

// Element offsets of chunk c's two vectors (c < rot / 16 rotates, the rest is copied).
template <bool INTER>
__device__ __forceinline__ void rope_chunk(int c, int rot, int &e1, int &e2) {
    const bool half = !INTER && c * 16 < rot;
    e1 = half ? c * 8 : c * 16;
    e2 = half ? rot / 2 + c * 8 : c * 16 + 8;
}

// Threads: x = (token, chunk of 16 elements), y = group of heads.
template <bool BF16, bool INTER, int D>
__global__ void __launch_bounds__(256) fa_rope_kernel(const RopeParams p) {
    constexpr int CPT = D / 16;
    pdl_wait();
    pdl_launch_dependents();
    const int c = threadIdx.x % CPT;
    const long long token = (long long)blockIdx.x * (blockDim.x / CPT) + threadIdx.x / CPT;
    const int h0 = (blockIdx.y * blockDim.y + threadIdx.y) * p.heads_per_thread;
    if (token >= p.tokens || h0 >= p.HT) return;
    const int h1 = min(h0 + p.heads_per_thread, p.HT);
    const int b = (int)token / p.N, n = (int)token - b * p.N;
    const bool turn = c * 16 < p.rot;
    int e1, e2;
    rope_chunk<INTER>(c, p.rot, e1, e2);
    float co[8], si[8];
    if (turn) {
        const int pos = p.positions ? __ldg(p.positions + (long long)b * p.positions_sb + n) : n;
        rope_angles(p.turns, c * 8, pos, p.mag, p.sign, co, si);
    }
    for (int h = h0; h < h1; h += 4) {
        uint4 a[4], v[4];
        uint16_t *dst[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int hh = h + i;
            if (hh >= h1) break;
            const bool is_q = hh < p.H;
            const Rows &in = is_q ? p.q : p.k, &out = is_q ? p.qo : p.ko;
            const int x = is_q ? hh : hh - p.H;
            const uint16_t *src = in.p + b * in.sb + x * in.sh + n * in.st;
            dst[i] = const_cast<uint16_t *>(out.p) + b * out.sb + x * out.sh + n * out.st;
            a[i] = *reinterpret_cast<const uint4 *>(src + e1);
            v[i] = *reinterpret_cast<const uint4 *>(src + e2);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (h + i >= h1) break;
            if (turn) rope_turn<BF16, INTER>(a[i], v[i], co, si);
            *reinterpret_cast<uint4 *>(dst[i] + e1) = a[i];
            *reinterpret_cast<uint4 *>(dst[i] + e2) = v[i];
        }
    }
}

// A paged cache's table and lengths.
struct PageTable {
    const int *table;  // [B, max_blocks] page numbers
    int max_blocks;
    int num_pages;
    int page_shift;    // page size = 1 << page_shift
    const int *cache_len;  // [B] tokens held before the call
    const int *new_len;    // [B] new tokens (nullptr: T)
};

// FA_ERR_BAD_PAGE in the status word, unless it already holds something (a wait that gave up is
// the graver: it takes the word whatever it holds).
__device__ __forceinline__ void report_bad_page() { atomicCAS(&g_status, 0, 6); }

// Tokens held before the call and new tokens of sequence b, made safe: 0 <= past,
// past + fresh <= the table's capacity, fresh <= T.
__device__ __forceinline__ void page_lengths(const PageTable &t, int T, int b, int &past,
                                             int &fresh) {
    const long long cap = (long long)t.max_blocks << t.page_shift;
    const int pl = __ldg(t.cache_len + b);
    past = pl < 0 ? 0 : ((long long)pl > cap ? (int)cap : pl);
    fresh = t.new_len ? __ldg(t.new_len + b) : T;
    fresh = fresh < 0 ? 0 : (fresh > T ? T : fresh);
    if (past + (long long)fresh > cap) fresh = (int)(cap - past);
}

// Sets the status word if sequence b's lengths are not what page_lengths() makes of them.
__device__ __forceinline__ void page_lengths_check(const PageTable &t, int T, int b) {
    const int pl = __ldg(t.cache_len + b), nl = t.new_len ? __ldg(t.new_len + b) : T;
    if (pl < 0 || nl < 0 || nl > T || pl + (long long)nl > ((long long)t.max_blocks << t.page_shift))
        report_bad_page();
}

struct AppendParams {
    Rows q, k, v, qo;     // q.p == nullptr: no queries
    Rows kc, vc;          // caches: sb = between pages, sh = heads, st = rows of a page
    int H, Hk, HT;        // query heads (0 without q), key/value heads, H + 2 Hk
    int T;
    int tokens;           // B * T
    int heads_per_thread;
    const int *positions; // [B, T] (nullptr: cache_len + t)
    const unsigned long long *turns;  // nullptr: no rotation
    int rot;
    float mag;
    PageTable pt;
};

// Heads in the order q, k, v.  Rows t >= new_len and everything outside the new tokens'
// slots are left as they are.  A new token whose slot lies behind the table's capacity, or
// whose page number is outside the cache, is not written and sets the status word.
template <bool BF16, bool INTER, int D>
__global__ void __launch_bounds__(256) fa_kv_append_kernel(const AppendParams p) {
    constexpr int CPT = D / 16;
    pdl_wait();
    pdl_launch_dependents();
    const int c = threadIdx.x % CPT;
    const long long token = (long long)blockIdx.x * (blockDim.x / CPT) + threadIdx.x / CPT;
    const int h0 = (blockIdx.y * blockDim.y + threadIdx.y) * p.heads_per_thread;
    if (token >= p.tokens || h0 >= p.HT) return;
    const int h1 = min(h0 + p.heads_per_thread, p.HT);
    const int b = (int)token / p.T, t = (int)token - b * p.T;
    if (t == 0 && c == 0 && h0 == 0) page_lengths_check(p.pt, p.T, b);
    const int want = p.pt.new_len ? __ldg(p.pt.new_len + b) : p.T;
    if (t >= want) return;
    const int len = __ldg(p.pt.cache_len + b);
    const long long slot = (long long)(len < 0 ? 0 : len) + t;
    int page = -1;
    const int row = (int)(slot & ((1 << p.pt.page_shift) - 1));
    if (h1 > p.H) {
        const long long block = slot >> p.pt.page_shift;
        if (block < p.pt.max_blocks) page = __ldg(p.pt.table + (long long)b * p.pt.max_blocks + block);
        if (page < 0 || page >= p.pt.num_pages) {
            page = -1;
            report_bad_page();
        }
    }
    const bool turn = p.turns != nullptr && c * 16 < p.rot && h0 < p.H + p.Hk;
    int e1, e2;
    rope_chunk<INTER>(c, p.rot, e1, e2);
    float co[8], si[8];
    if (turn) {
        const int pos = p.positions ? __ldg(p.positions + token) : (int)slot;
        rope_angles(p.turns, c * 8, pos, p.mag, 1.f, co, si);
    }
    for (int h = h0; h < h1; h += 4) {
        uint4 a[4], v[4];
        uint16_t *dst[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int hh = h + i;
            dst[i] = nullptr;
            if (hh >= h1) continue;
            const Rows *in, *out;
            int x;
            if (hh < p.H) {
                in = &p.q, out = &p.qo, x = hh;
            } else if (hh < p.H + p.Hk) {
                in = &p.k, out = &p.kc, x = hh - p.H;
            } else {
                in = &p.v, out = &p.vc, x = hh - p.H - p.Hk;
            }
            if (hh < p.H) {
                dst[i] = const_cast<uint16_t *>(out->p) + b * out->sb + x * out->sh + t * out->st;
            } else {
                if (page < 0) continue;
                dst[i] = const_cast<uint16_t *>(out->p) + page * out->sb + x * out->sh + row * out->st;
            }
            const uint16_t *src = in->p + b * in->sb + x * in->sh + t * in->st;
            a[i] = *reinterpret_cast<const uint4 *>(src + e1);
            v[i] = *reinterpret_cast<const uint4 *>(src + e2);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (dst[i] == nullptr) continue;
            if (turn && h + i < p.H + p.Hk) rope_turn<BF16, INTER>(a[i], v[i], co, si);
            *reinterpret_cast<uint4 *>(dst[i] + e1) = a[i];
            *reinterpret_cast<uint4 *>(dst[i] + e2) = v[i];
        }
    }
}

}  // namespace fa
