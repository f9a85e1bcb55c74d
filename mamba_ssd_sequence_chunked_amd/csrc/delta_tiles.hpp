// delta_tiles.hpp - what the gated delta rule's chunk kernels share: sequences cut into blocks of 32 tokens,
// the per-(block, head) record of matrices and decay tables, LDS tiles and operand fragments.
//
// Within a block of C = 32 tokens (cs = inclusive prefix sum of g, G_ij = exp(cs_i - cs_j)):
//
//   X_ij = G_ij (k_i . k_j), j < i         A = (I + X diag(beta))^-1        M_ij = G_ij (q_i . k_j), j <= i
//   E = V - diag(gam) K S^T    e = A E    U = diag(beta) e                  gam_i = exp(cs_i)
//   Y = diag(gam) Q S^T + M U             S+ = gam_last S + U^T diag(del) K  del_j = exp(cs_last - cs_j)
//
// A and M do not need the state: delta_prep makes them for all blocks at once, and the walk over the blocks is
// left with products against the state.
//
// Contraction slots (see common.hpp). In the walks over the blocks lane group g's 8 slots stand for indices 8g .. 8g + 7
// of a block of 32, and an accumulator's rows go with that: row 4g + m of tile x (0, 1) of a pair stands for index
// 8g + 4x + m, so that two accumulator tiles are an operand fragment as they are and a fragment along a row of LDS is
// one 16-byte read (perm32). In the dq, dk step, slots stand for {4g .. 4g + 3, 16 + 4g .. 16 + 4g + 3} and rows
// for themselves.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace ssd {

constexpr int kDC = 32;      // tokens of a block

// what row (or column) i of 16 of tile x of a pair stands for within its 32
__device__ __forceinline__ int perm32(int x, int i) { return 8 * (i >> 2) + 4 * x + (i & 3); }

// ---- sequences ------------------------------------------------------------------------------------------

struct DeltaSeq {
    int64_t start;           // first token on the token axis
    int64_t slot;            // number of its first block among all blocks
    int len;                 // tokens
};

// With offsets, sequence s's blocks get the numbers start / 32 + s on: ceil(len / 32) of them end before
// (start + len) / 32 + s + 1, so no two sequences share one and all are below tokens / 32 + seqs.
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaDims& d, int64_t s)
{
    DeltaSeq q;
    if (d.cu) {
        q.start = min(max((int64_t)d.cu[s], (int64_t)0), d.tokens);
        q.len = (int)(min(max((int64_t)d.cu[s + 1], q.start), d.tokens) - q.start);
        q.slot = q.start / kDC + s;
    } else {
        q.start = s * d.seqlen;
        q.len = (int)d.seqlen;
        q.slot = s * ((d.seqlen + kDC - 1) / kDC);
    }
    return q;
}

inline int64_t delta_slots(const DeltaDims& d)
{
    return d.cu ? d.tokens / kDC + d.seqs : d.seqs * ((d.seqlen + kDC - 1) / kDC);
}

// The sequence that block number `slot` belongs to and its block within it; false if it is no block of any.
__device__ __forceinline__ bool delta_slot(const DeltaDims& d, int64_t slot, DeltaSeq& q, int& c)
{
    int64_t s;
    if (d.cu) {
        int64_t lo = 0, hi = d.seqs - 1;          // the last s with start / 32 + s <= slot
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            const int64_t at = min(max((int64_t)d.cu[mid], (int64_t)0), d.tokens) / kDC + mid;
            if (at <= slot) lo = mid; else hi = mid - 1;
        }
        s = lo;
    } else {
        s = slot / ((d.seqlen + kDC - 1) / kDC);
    }
    q = delta_seq(d, s);
    const int64_t cc = slot - q.slot;
    c = (int)cc;
    return cc >= 0 && cc * kDC < q.len;
}

// ---- records --------------------------------------------------------------------------------------------

// What delta_prep leaves for a block and head: 32 x 32 matrices in T as LDS tiles (WTile), bf16 ones as a hi and a lo
// plane, and tables of 32 floats.  A and B are kept without their unit diagonals: what they multiply is added in
// fp32, so that a rounding of the pairs counts for the rest only.
//   forward:  A - I (hi, lo), M diag(beta) (hi only), tables gam, del beta
//   backward: A - I, M below its diagonal (both as pairs), tables gam, del, beta and M's diagonal q_i . k_i, B - I with
//             B = (I + diag(beta) X)^-1 (pair); the walk forward reads A to the tables, the walk back M to B
template <typename T, bool kBwd> struct DeltaRec {
    static constexpr int kPair = sizeof(T) == 2 ? 2 : 1;
    static constexpr int kMat = 32 * 32 * (int)sizeof(T);
    static constexpr int kA = 0, kM = kPair * kMat;
    static constexpr int kTab = kM + (kBwd ? kPair : 1) * kMat;
    static constexpr int kB = kTab + 512;
    static constexpr int kBytes = kB + (kBwd ? kPair * kMat : 0);
    static constexpr int kFwdBytes = kB;               // what the walk forward reads, from the record's start
    static constexpr int kRevBytes = kBytes - kM;      // what the walk back reads, from kM on
};

// ---- LDS tiles ------------------------------------------------------------------------------------------

// A tile of 32 rows of CH 16-byte chunks; chunk c of row r lies at slot c ^ key(r).  A pass of LDS reads covers 256
// bytes: 16 lanes of a 16-byte read, 32 of an 8-byte one, which need different slots of 16 (rows of fewer than 16
// chunks take the upper part of the slot from the row).  Three ways of reading, three keys:
//   DTile  8-byte reads of 16 rows and transpose reads of 8 rows x 2 adjacent chunks (the dq, dk step)
//   WTile  16-byte reads of the 16 rows perm32(x, .) at one chunk: 16 slots; transpose reads of 8 rows x the same
//          half of 4 chunks: two lanes to a slot (no key does better: all want the same half)
//   VTile  transpose reads of 8 rows (4 of each of two lane groups) x 2 adjacent chunks
template <int CH>
struct DTile {
    static constexpr int kShift = CH >= 16 ? 0 : CH == 8 ? 1 : CH == 4 ? 2 : 3;
    __device__ __forceinline__ static int key(int r)
    {
        return ((((r >> kShift) & (7 >> kShift)) << 1) | ((r >> 3) & 1)) & (CH - 1);
    }
    __device__ __forceinline__ static int offset(int r, int c) { return r * (CH * 16) + ((c ^ key(r)) << 4); }
    static constexpr int kBytes = 32 * CH * 16;
    static constexpr int kInst = CH / 2;          // copies of 64 chunks
};

template <int CH>
struct WTile {
    // the row's bits 0, 1, 3, 4 (bit 2 is x), the lowest first where they do not already choose the slot
    __device__ __forceinline__ static int key(int r)
    {
        const int low = ((r >> 3) & 1) << 1 | ((r >> 4) & 1);
        return CH >= 16 ? (r & 1) << 3 | (r & 2) << 1 | low : CH == 8 ? (r & 2) << 1 | low : low;
    }
    __device__ __forceinline__ static int offset(int r, int c) { return r * (CH * 16) + ((c ^ key(r)) << 4); }
};
template <int CH>
struct VTile {
    // the row's bits 0, 1, 3 above the lowest slot bit
    __device__ __forceinline__ static int key(int r)
    {
        const int k = ((r >> 3) & 1) | (r & 2) | (r & 1) << 2;
        return CH >= 16 ? k << 1 : CH == 8 ? (k & 3) << 1 : CH == 4 ? (k & 1) << 1 : 0;
    }
    __device__ __forceinline__ static int offset(int r, int c) { return r * (CH * 16) + ((c ^ key(r)) << 4); }
};

// One wavefront's share of a tile's copies: row r from base + r * row_bytes, its first `valid` chunks only; rows from
// `rows` on are written as zeros.
// The source offsets of a whole tile are worked out once (plan), so that a copy in the loop costs its issue and a
// scalar add; lds is the tile's LDS address.
template <int CH, int NW, class TL = DTile<CH>>
struct DTileCopy {
    static constexpr int kI = DTile<CH>::kInst, kK = (kI + NW - 1) / NW;
    static constexpr bool kPlan = kK <= 16;       // more offsets would crowd the registers: worked out each time
    unsigned off[kPlan ? kK : 1];
    __device__ __forceinline__ static void place(int q, int lane, int& r, int& c)
    {
        const int pos = q * 64 + lane;
        r = pos / CH;
        c = (pos % CH) ^ TL::key(r);
    }
    __device__ __forceinline__ void plan(unsigned row_bytes, int wave, int lane)
    {
        if constexpr (kPlan) {
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                int r, c;
                place(wave + NW * k, lane, r, c);
                off[k] = (unsigned)r * row_bytes + 16u * c;
            }
        }
    }
    __device__ __forceinline__ void issue(const void* base, unsigned row_bytes, int rows, int valid, unsigned lds,
                                          int wave, int lane) const
    {
        if (kPlan && valid == CH && rows >= 32) {
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                const int q = wave + NW * k;
                if (kI % NW != 0 && q >= kI) break;
                dma16_off(base, off[kPlan ? k : 0], lds + q * 1024u);
            }
        } else {
            for (int q = wave; q < kI; q += NW) {
                int r, c;
                place(q, lane, r, c);
                if (c < valid) {
                    if (r < rows)
                        dma16_off(base, (unsigned)r * row_bytes + 16u * c, lds + q * 1024u);
                    else
                        *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(lds + q * 1024u + lane * 16u) = u32x4{0, 0, 0, 0};
                }
            }
        }
    }
};

// Reads of a tile's operand fragments. The per-lane parts of the addresses are worked out once (the constructors); what
// changes with the tile, the stage and the row or column block is an instruction's constant offset. All addresses
// are LDS addresses as integers.
template <typename V>
__device__ __forceinline__ V lds_at(unsigned a)
{
    return *(const __attribute__((address_space(3))) V*)(uintptr_t)a;
}

// Slots along a row: row 16 t + r, elements {32 kb + 4g .. + 3, 32 kb + 16 + 4g .. + 3}.
template <typename T, int CH> struct DRows;
template <int CH> struct DRows<bf16, CH> {
    static constexpr int kPer = CH / 4 < 4 ? CH / 4 : 4;      // row blocks whose chunk bits the key reaches
    unsigned a[kPer][2];
    __device__ __forceinline__ DRows(int r, int g)
    {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            a[k][0] = DTile<CH>::offset(r, 4 * k + (g >> 1)) + (g & 1) * 8;
            a[k][1] = DTile<CH>::offset(r, 4 * k + 2 + (g >> 1)) + (g & 1) * 8;
        }
    }
    __device__ __forceinline__ void load(Vec8<bf16>& f, unsigned tile, int t, int kb) const
    {
        const unsigned o = tile + t * (16 * CH * 16) + (kb / kPer) * 256;
        const bf16x4 x = lds_at<bf16x4>(a[kb % kPer][0] + o), y = lds_at<bf16x4>(a[kb % kPer][1] + o);
        f.v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};
template <int CH> struct DRows<float, CH> {
    int r, g;
    __device__ __forceinline__ DRows(int r_, int g_) : r(r_), g(g_) {}
    __device__ __forceinline__ void load(Vec8<float>& f, unsigned tile, int t, int kb) const
    {
        const f32x4 x = lds_at<f32x4>(tile + DTile<CH>::offset(16 * t + r, 8 * kb + g));
        const f32x4 y = lds_at<f32x4>(tile + DTile<CH>::offset(16 * t + r, 8 * kb + 4 + g));
#pragma unroll
        for (int m = 0; m < 4; ++m) { f.v[m] = x[m]; f.v[4 + m] = y[m]; }
    }
};

// Slots down the rows: column 16 t + r of rows {4g .. 4g + 3, 16 + 4g .. 16 + 4g + 3}.
template <typename T, int CH> struct DCols;
template <int CH> struct DCols<bf16, CH> {
    static constexpr int kPer = CH / 2 < 8 ? CH / 2 : 8;      // column tiles whose chunk bits the key reaches
    unsigned a[kPer];
    __device__ __forceinline__ DCols(int r, int g)
    {
#pragma unroll
        for (int t = 0; t < kPer; ++t)
            a[t] = DTile<CH>::offset(4 * g + (r >> 2), 2 * t + ((r & 3) >> 1)) + (r & 1) * 8;
    }
    __device__ __forceinline__ void load(Vec8<bf16>& f, unsigned tile, int t) const
    {
        typedef short v4i16 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4i16* P;
        const unsigned o = a[t % kPer] + tile + (t / kPer) * 256;
        const v4i16 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)o);
        const v4i16 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)(o + 16 * CH * 16));
        f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // the same for a tile number that is not a constant
    __device__ __forceinline__ static void load_any(Vec8<bf16>& f, unsigned tile, int t, int r, int g)
    {
        typedef short v4i16 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4i16* P;
        const unsigned o = tile + DTile<CH>::offset(4 * g + (r >> 2), 2 * t + ((r & 3) >> 1)) + (r & 1) * 8;
        const v4i16 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)o);
        const v4i16 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)(o + 16 * CH * 16));
        f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};
template <int CH> struct DCols<float, CH> {
    int r, g;
    __device__ __forceinline__ DCols(int r_, int g_) : r(r_), g(g_) {}
    __device__ __forceinline__ void load(Vec8<float>& f, unsigned tile, int t) const { load_any(f, tile, t, r, g); }
    __device__ __forceinline__ static void load_any(Vec8<float>& f, unsigned tile, int t, int r, int g)
    {
        const int c = 4 * t + (r >> 2), h = 4 * (r & 3);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            f.v[m] = lds_at<float>(tile + DTile<CH>::offset(4 * g + m, c) + h);
            f.v[4 + m] = lds_at<float>(tile + DTile<CH>::offset(16 + 4 * g + m, c) + h);
        }
    }
};

// Fragments of WTiles. Along a row: row perm32(x, r), elements 32 kb + 8g .. + 7. Down the rows: column perm32(x, r) of
// the 32 from 32 kb on, rows 8g .. 8g + 7.
template <typename T, int CH> struct WRows;
template <int CH> struct WRows<bf16, CH> {
    static constexpr int kPer = CH / 4 < 4 ? CH / 4 : 4;      // blocks of 32 whose chunk bits the key reaches
    unsigned a[kPer];
    __device__ __forceinline__ WRows(int r, int g)
    {
#pragma unroll
        for (int k = 0; k < kPer; ++k) a[k] = WTile<CH>::offset(perm32(0, r), 4 * k + g);
    }
    __device__ __forceinline__ void load(Vec8<bf16>& f, unsigned tile, int x, int kb) const
    {
        // (the key leaves out bit 2 of the row, which is x)
        f.v = lds_at<bf16x8>(a[kb % kPer] + tile + x * (4 * CH * 16) + (kb / kPer) * (64 * kPer));
    }
};
template <int CH> struct WRows<float, CH> {
    int r, g;
    __device__ __forceinline__ WRows(int r_, int g_) : r(r_), g(g_) {}
    __device__ __forceinline__ void load(Vec8<float>& f, unsigned tile, int x, int kb) const
    {
        const f32x4 p = lds_at<f32x4>(tile + WTile<CH>::offset(perm32(x, r), 8 * kb + 2 * g));
        const f32x4 q = lds_at<f32x4>(tile + WTile<CH>::offset(perm32(x, r), 8 * kb + 2 * g + 1));
#pragma unroll
        for (int m = 0; m < 4; ++m) { f.v[m] = p[m]; f.v[4 + m] = q[m]; }
    }
};
template <typename T, int CH> struct WCols;
template <int CH> struct WCols<bf16, CH> {
    static constexpr int kPer = CH / 4 < 4 ? CH / 4 : 4;
    unsigned a[kPer];
    __device__ __forceinline__ WCols(int r, int g)
    {
#pragma unroll
        for (int k = 0; k < kPer; ++k) a[k] = WTile<CH>::offset(8 * g + (r >> 2), 4 * k + (r & 3));
    }
    __device__ __forceinline__ void load(Vec8<bf16>& f, unsigned tile, int x, int kb) const
    {
        typedef short v4i16 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4i16* P;
        const unsigned o = a[kb % kPer] + tile + 8 * x + (kb / kPer) * (64 * kPer);
        const v4i16 p = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)o);
        const v4i16 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)(o + 4 * CH * 16));
        f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(p, q, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};
template <int CH> struct WCols<float, CH> {
    int r, g;
    __device__ __forceinline__ WCols(int r_, int g_) : r(r_), g(g_) {}
    __device__ __forceinline__ void load(Vec8<float>& f, unsigned tile, int x, int kb) const
    {
        const int n = 32 * kb + perm32(x, r);
#pragma unroll
        for (int m = 0; m < 8; ++m) f.v[m] = lds_at<float>(tile + WTile<CH>::offset(8 * g + m, n >> 2) + 4 * (n & 3));
    }
};
// Column 16 w + r of a VTile, rows 8g .. 8g + 7.
template <int CH>
__device__ __forceinline__ void vtile_cols(Vec8<bf16>& f, unsigned tile, int w, int r, int g)
{
    typedef short v4i16 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4i16* P;
    const unsigned o = tile + VTile<CH>::offset(8 * g + (r >> 2), 2 * w + ((r & 3) >> 1)) + (r & 1) * 8;
    const v4i16 p = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)o);
    const v4i16 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)(o + 4 * CH * 16));
    f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(p, q, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int CH>
__device__ __forceinline__ void vtile_cols(Vec8<float>& f, unsigned tile, int w, int r, int g)
{
    const int c = 16 * w + r;
#pragma unroll
    for (int m = 0; m < 8; ++m) f.v[m] = lds_at<float>(tile + VTile<CH>::offset(8 * g + m, c >> 2) + 4 * (c & 3));
}

// ---- operands -------------------------------------------------------------------------------------------

// An fp32 operand of a product: for bf16 inputs a pair hi + lo (the value to 2^-18), so that products keep fp32's
// accuracy to about 2^-17 on the bf16 matrix cores; for fp32 inputs the value.
template <typename T> struct Pair;
template <> struct Pair<bf16> {
    Vec8<bf16> hi, lo;
    __device__ __forceinline__ void set(const float (&v)[8]) { pack8_split(hi, lo, v); }
};
template <> struct Pair<float> {
    Vec8<float> hi;
    __device__ __forceinline__ void set(const float (&v)[8]) { pack8(hi, v); }
};

// a exact, b a pair and the other way round; both pairs: without the product of the two low parts (2^-18), or with it
__device__ __forceinline__ void mma_px(f32x4& acc, const Pair<bf16>& a, const Vec8<bf16>& b) { mma(acc, a.lo, b); mma(acc, a.hi, b); }
__device__ __forceinline__ void mma_px(f32x4& acc, const Pair<float>& a, const Vec8<float>& b) { mma(acc, a.hi, b); }
__device__ __forceinline__ void mma_xp(f32x4& acc, const Vec8<bf16>& a, const Pair<bf16>& b) { mma(acc, a, b.lo); mma(acc, a, b.hi); }
__device__ __forceinline__ void mma_xp(f32x4& acc, const Vec8<float>& a, const Pair<float>& b) { mma(acc, a, b.hi); }
template <bool kLow = false>
__device__ __forceinline__ void mma_pp(f32x4& acc, const Pair<bf16>& a, const Pair<bf16>& b)
{
    if constexpr (kLow) mma(acc, a.lo, b.lo);
    mma(acc, a.lo, b.hi);
    mma(acc, a.hi, b.lo);
    mma(acc, a.hi, b.hi);
}
template <bool kLow = false>
__device__ __forceinline__ void mma_pp(f32x4& acc, const Pair<float>& a, const Pair<float>& b) { mma(acc, a.hi, b.hi); }
// The product of b with what the pair a of v leaves of it.
__device__ __forceinline__ void mma_rest(f32x4& acc, const Pair<bf16>& a, const float (&v)[8], const Vec8<bf16>& b)
{
    float left[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) left[i] = v[i] - a.hi.get(i) - a.lo.get(i);
    Vec8<bf16> f;
    pack8(f, left);
    mma(acc, f, b);
}
__device__ __forceinline__ void mma_rest(f32x4&, const Pair<float>&, const float (&)[8], const Vec8<float>&) {}

// The matrices of a record (tiles of kRecCH chunks a row): pairs by rows and by columns (tile x).
template <typename T> constexpr int kRecCH = 32 * (int)sizeof(T) / 16;
template <class A>
__device__ __forceinline__ void load_pair(Pair<bf16>& f, const A& a, unsigned m, int x)
{
    a.load(f.hi, m, x, 0);
    a.load(f.lo, m + 2048, x, 0);
}
template <class A>
__device__ __forceinline__ void load_pair(Pair<float>& f, const A& a, unsigned m, int x) { a.load(f.hi, m, x, 0); }

// The unit matrix's fragment with rows (or columns) of tile x: slot s of lane group g is index 8g + s.
template <typename T>
__device__ __forceinline__ void unit_frag(Vec8<T>& f, int x, int r, int g)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) f.set(i, 8 * g + i == perm32(x, r) ? 1.f : 0.f);
}

// Start this wavefront's share of the copy of BYTES consecutive bytes (a multiple of 16).
template <int BYTES, int NW>
__device__ __forceinline__ void linear_copy(const unsigned char* src, unsigned lds, int wave, int lane)
{
#pragma unroll
    for (int k = 0; k < ((BYTES + 1023) / 1024 + NW - 1) / NW; ++k) {
        const int q = wave + NW * k;
        if (q * 1024 + lane * 16 < BYTES) dma16_off(src + q * 1024, lane * 16u, lds + q * 1024u);
    }
}

// The 8 values of a table at this lane group's tokens 8g .. 8g + 7.
__device__ __forceinline__ void tab_rows(float (&v)[8], unsigned tab, int g)
{
    const f32x4 x = lds_at<f32x4>(tab + 32 * g), y = lds_at<f32x4>(tab + 32 * g + 16);
#pragma unroll
    for (int m = 0; m < 4; ++m) { v[m] = x[m]; v[4 + m] = y[m]; }
}

// ---- what the backward's walk forward keeps -------------------------------------------------------------

template <typename T> struct DeltaKeep {
    const T* dy;
    float* x;                // x = S' k = v - e of every block, head and 16 columns: (2 x 16 tokens) as 64 lanes (4
                             //   columns, token) x 4
    float* ydy;              // (headdim / 16, seqs, nheads, 64 chunks): dy . S' q over 16 columns
    T* S;                    // (seqs, chunks + 1, nheads): the state entering each 64-token chunk, and after the last, as
    T* Slo;                  //   fragments (state_at); for bf16 also what the rounding to T drops
    int64_t chunks;          // 64-token chunks of a row
    __device__ __forceinline__ int64_t frag(int64_t slot, int h, int pt, const DeltaDims& d) const
    {
        return ((slot * d.nheads + h) * (d.headdim / 16) + pt) * 512;
    }
    // where token i of the 32 has its columns 4g .. 4g + 3
    __device__ __forceinline__ static int lane(int i, int g) { return (i >> 4) * 256 + (16 * g + (i & 15)) * 4; }
    // Plane k of a kept state: per 16 rows p and 32 columns n, 64 lanes (g, p) x columns 8g .. 8g + 7, so that
    // a walk's stores and loads are whole lines. kb_stride elements from one 32 columns to the next.
    static constexpr int kb_stride = 512;
    __device__ __forceinline__ static int64_t plane(const DeltaDims& d)
    {
        return d.headdim * ((d.dstate + 31) / 32 * 32);
    }
    __device__ __forceinline__ static int64_t state_at(int64_t plane_index, int pt, int lane_id, const DeltaDims& d)
    {
        return plane_index * plane(d) + (int64_t)pt * ((d.dstate + 31) / 32) * kb_stride + lane_id * 8;
    }
};

// Sums over the four lane groups of two values at once: lane group g returns the sum of a (g < 2) or b (g >= 2) at its
// own r.
__device__ __forceinline__ float sum_groups(float a, float b)
{
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    const float s = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}
// The same of four: lane group g returns the sum of a (0), c (1), b (2), d (3).
__device__ __forceinline__ float sum_groups(float a, float b, float c, float d)
{
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    const auto z = __builtin_amdgcn_permlane32_swap(__float_as_uint(c), __float_as_uint(d), false, false);
    const float s = __uint_as_float(x[0]) + __uint_as_float(x[1]), t = __uint_as_float(z[0]) + __uint_as_float(z[1]);
    const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(t), false, false);
    return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}

template <typename T, bool kBwd>
hipError_t launch_delta_chain(const T* v, const T* k, const T* q, const float* init, const unsigned char* rec, T* y,
                              float* fin, const DeltaKeep<T>& keep, const DeltaDims& d, hipStream_t stream);

}  // namespace ssd
