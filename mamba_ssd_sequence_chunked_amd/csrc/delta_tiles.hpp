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
// Contraction slots (see common.hpp) always stand for indices {4g .. 4g + 3, 16 + 4g .. 16 + 4g + 3} of a block of
// 32: an accumulator tile's rows 4g .. 4g + 3, so that two accumulator tiles are an operand fragment as they are.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace ssd {

constexpr int kDC = 32;      // tokens of a block

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

// What delta_prep leaves for a block and head: 32 x 32 matrices in T as LDS tiles (DTile, so that they can be read
// by rows and by columns), bf16 ones as a hi and a lo plane, and the tables gam, del, beta (32 floats each).
//   forward:  A (hi, lo), M (hi only), tables
//   backward: A, M (both as pairs), tables, B = (I + diag(beta) X)^-1 (pair); the walk forward reads A to the tables,
//             the walk back M to B
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

// A tile of 32 rows of CH 16-byte chunks; chunk c of row r lies at slot c ^ key(r).  It is read in two ways:
// 16 rows (0-15 or 16-31) at one chunk column, and, through the transpose read, 8 consecutive rows at two adjacent
// chunks.  A pass over the 64 banks covers 16 chunks; with the key's upper bits taken from the row's lowest
// (those that share a pass) and its lowest from bit 3, both reads touch 16 different chunk slots of a pass.
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

// Start this wavefront's share of a tile's copies: row r from base + min(r, rmax) * row_bytes, its first `valid`
// chunks only.
template <int CH, int NW>
__device__ __forceinline__ void dtile_copy(const void* base, unsigned row_bytes, int rmax, int valid, unsigned lds,
                                           int wave, int lane)
{
    constexpr int kI = DTile<CH>::kInst;
#pragma unroll
    for (int k = 0; k < (kI + NW - 1) / NW; ++k) {
        const int q = wave + NW * k;
        if (kI % NW != 0 && q >= kI) break;
        const int pos = q * 64 + lane, r = pos / CH, c = (pos % CH) ^ DTile<CH>::key(r);
        if (valid == CH || c < valid)
            dma16_off(base, (unsigned)min(r, rmax) * row_bytes + 16u * c, lds + q * 1024u);
    }
}

// Slots along a row of a tile: elements {32 kb + 4g .. + 3, 32 kb + 16 + 4g .. + 3} of row.
template <int CH>
__device__ __forceinline__ void dtile_row(Vec8<bf16>& f, const unsigned char* tile, int row, int kb, int g)
{
    const int h = (g & 1) * 8, c = 4 * kb + (g >> 1);
    const bf16x4 a = *reinterpret_cast<const bf16x4*>(tile + DTile<CH>::offset(row, c) + h);
    const bf16x4 b = *reinterpret_cast<const bf16x4*>(tile + DTile<CH>::offset(row, c + 2) + h);
    f.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int CH>
__device__ __forceinline__ void dtile_row(Vec8<float>& f, const unsigned char* tile, int row, int kb, int g)
{
    const float4 a = *reinterpret_cast<const float4*>(tile + DTile<CH>::offset(row, 8 * kb + g));
    const float4 b = *reinterpret_cast<const float4*>(tile + DTile<CH>::offset(row, 8 * kb + 4 + g));
    f.v[0] = a.x; f.v[1] = a.y; f.v[2] = a.z; f.v[3] = a.w;
    f.v[4] = b.x; f.v[5] = b.y; f.v[6] = b.z; f.v[7] = b.w;
}

// Slots down the rows of a tile: column c0 + r of rows {4g .. 4g + 3, 16 + 4g .. 16 + 4g + 3}.
template <int CH>
__device__ __forceinline__ void dtile_col(Vec8<bf16>& f, const unsigned char* tile, int c0, int r, int g)
{
    typedef short v4i16 __attribute__((ext_vector_type(4)));
    const int row = 4 * g + (r >> 2), c = (c0 >> 3) + ((r & 3) >> 1), h = (r & 1) * 8;
    const v4i16 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(as_lds<v4i16>(tile + DTile<CH>::offset(row, c) + h));
    const v4i16 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(as_lds<v4i16>(tile + DTile<CH>::offset(row + 16, c) + h));
    f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int CH>
__device__ __forceinline__ void dtile_col(Vec8<float>& f, const unsigned char* tile, int c0, int r, int g)
{
    const int c = (c0 + r) >> 2, h = 4 * (r & 3);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        f.v[m] = *reinterpret_cast<const float*>(tile + DTile<CH>::offset(4 * g + m, c) + h);
        f.v[4 + m] = *reinterpret_cast<const float*>(tile + DTile<CH>::offset(16 + 4 * g + m, c) + h);
    }
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
// a exact, b a pair and the other way round; both pairs: without the product of the two low parts (2^-18)
__device__ __forceinline__ void mma_px(f32x4& acc, const Pair<bf16>& a, const Vec8<bf16>& b) { mma(acc, a.lo, b); mma(acc, a.hi, b); }
__device__ __forceinline__ void mma_px(f32x4& acc, const Pair<float>& a, const Vec8<float>& b) { mma(acc, a.hi, b); }
__device__ __forceinline__ void mma_xp(f32x4& acc, const Vec8<bf16>& a, const Pair<bf16>& b) { mma(acc, a, b.lo); mma(acc, a, b.hi); }
__device__ __forceinline__ void mma_xp(f32x4& acc, const Vec8<float>& a, const Pair<float>& b) { mma(acc, a, b.hi); }
__device__ __forceinline__ void mma_pp(f32x4& acc, const Pair<bf16>& a, const Pair<bf16>& b)
{
    mma(acc, a.lo, b.hi);
    mma(acc, a.hi, b.lo);
    mma(acc, a.hi, b.hi);
}
__device__ __forceinline__ void mma_pp(f32x4& acc, const Pair<float>& a, const Pair<float>& b) { mma(acc, a.hi, b.hi); }

// The matrices of a record: CH of their tiles, and fragments by rows (row tile t) and by columns (column tile t).
template <typename T> constexpr int kRecCH = 32 * (int)sizeof(T) / 16;
__device__ __forceinline__ void rec_rows(Pair<bf16>& f, const unsigned char* m, int t, int r, int g)
{
    dtile_row<4>(f.hi, m, 16 * t + r, 0, g);
    dtile_row<4>(f.lo, m + 2048, 16 * t + r, 0, g);
}
__device__ __forceinline__ void rec_rows(Pair<float>& f, const unsigned char* m, int t, int r, int g)
{
    dtile_row<8>(f.hi, m, 16 * t + r, 0, g);
}
__device__ __forceinline__ void rec_cols(Pair<bf16>& f, const unsigned char* m, int t, int r, int g)
{
    dtile_col<4>(f.hi, m, 16 * t, r, g);
    dtile_col<4>(f.lo, m + 2048, 16 * t, r, g);
}
__device__ __forceinline__ void rec_cols(Pair<float>& f, const unsigned char* m, int t, int r, int g)
{
    dtile_col<8>(f.hi, m, 16 * t, r, g);
}

// Start this wavefront's share of the copy of `bytes` consecutive bytes (a multiple of 16).
template <int BYTES, int NW>
__device__ __forceinline__ void linear_copy(const unsigned char* src, unsigned lds, int wave, int lane)
{
#pragma unroll
    for (int k = 0; k < ((BYTES + 1023) / 1024 + NW - 1) / NW; ++k) {
        const int q = wave + NW * k;
        if (q * 1024 + lane * 16 < BYTES) dma16_off(src, q * 1024u + lane * 16u, lds + q * 1024u);
    }
}

// ---- what the backward's walk forward keeps -------------------------------------------------------------

template <typename T> struct DeltaKeep {
    const T* dy;
    float* e;                // e of every block, head and 16 columns: 2 token tiles x 64 lanes x 4 columns (frag)
    float* ydy;              // (headdim / 16, tokens, nheads): dy . y over 16 columns
    T* S;                    // (seqs, chunks + 1, nheads, headdim, dstate): the state entering each 64-token chunk,
    T* Slo;                  //   and after the last; for bf16 also what the rounding to T drops
    int64_t chunks;          // 64-token chunks of a row
    __device__ __forceinline__ int64_t frag(int64_t slot, int h, int pt, const DeltaDims& d) const
    {
        return ((slot * d.nheads + h) * (d.headdim / 16) + pt) * 512;
    }
};

template <typename T, bool kBwd>
hipError_t launch_delta_chain(const T* v, const T* k, const T* q, const float* init, const unsigned char* rec, T* y,
                              float* fin, const DeltaKeep<T>& keep, const DeltaDims& d, hipStream_t stream);

}  // namespace ssd
