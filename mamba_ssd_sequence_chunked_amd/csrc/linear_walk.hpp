// linear_walk.hpp - the walk over a row's tokens that every call of linear attention with a decay for each head runs on.
//
// With three operands Q, K (rows of Dk) and V (rows of Dv), a state S of Dk x Dv and the head's decay a = exp(g):
//
//   S_t = a S_{t-1} + K_t V_t^T;   O_t = S_t^T Q_t
//
// The forward is (q, k, v); dq is (dy, v, k); dk is (v, dy, q) and dv (k, q, dy), both from the last token to the first.
// In a chunk of C tokens that S enters, with t and s counted in it and G_ts = a^(t - s) for s <= t, else 0:
//
//   O  = diag(a^(t + e)) Q S + (Q K^T o G) V
//   S+ = a^C S + K^T diag(a^(C - s - e)) V
//
// e is 1 forwards, where the entering state decays before the first token; backwards the gradient of the state behind
// the last token does not, and what is carried on includes the step over the chunk's first token: e = 0.
// The weights are powers of one number, so they are tables in registers, worked out once per walk.  Each is at most 1.
//
// The sum's derivative for g (kDg, forwards only) is a second state S' = dS/dg with weights that carry their exponents:
//
//   S'+ = a^C (S' + C S) + K^T diag((C - 1 - s) a^(C - 1 - s)) V
//   dg += sum_t a^(t+1) X_t . ((S' + (t + 1) S)^T Q_t) + sum_{s<t} (t - s) G_ts (Q_t . K_s)(X_t . V_s)
//
// where X is what dL/dO is contracted with: for dq = (dy, v, k) X is q.  No difference of large sums is formed.
//
// Columns of the state do not mix: a wavefront keeps JT x 16 of them for the whole walk as accumulator tiles (rows Dk,
// columns Dv), which are operand fragments as they are (see common.hpp).  The chunk's scores are needed by all of them:
// three make a 16 x 16 tile each, one chunk ahead of the one whose state products run, so that a chunk has one barrier.
// Copies run into a ring of two or three stages of LDS.  (Fewer stages, where the rows are wide: the scores are made in their own
// chunk, with a second barrier.)  Chunks have 32 tokens: with 64 the scores are more than what is saved per
// chunk, and the registers do not hold what is read ahead.
//
// A row may be cut into segments that walk at the same time: a first pass of the same kernel (states only) leaves
// what each adds to the state, linear_join carries the states over, and the walk starts each segment from its own.  Or
// into a chain: one launch in which a segment takes over the state when the one before it is done.
//
// What bounds it, and what it takes (bf16, heads of 64 x 128, 4096 tokens): 320 rows 246 us, 4.1 TB/s, and 512 rows 337, 4.8
// TB/s, where a copy reaches 4.83: HBM, once the CUs are filled evenly.  320 rows towards dq and dg 520: issue, 521
// vector instructions (some 340 of them to split and decay states) and 52 matrix ones a wavefront and chunk, eight
// wavefronts a CU.  480 segments of 256 rows of state (65536 tokens, 80 heads) 1120: issue, 333 and 72, at two wavefronts a
// SIMD, and LDS, 98 of whose 335 cycles a chunk are bank conflicts (see LinearRows).  In fp32 320 rows take 716, the matrix
// products at 58 % of the rate of a large one, with a workgroup a CU.
#pragma once

#include <algorithm>

#include "delta_tiles.hpp"

namespace ssd {

// Operands of a walk: row t of head h at p + t * row + (h / share) * width elements.
template <typename T> struct LinearOperand {
    const T* p;
    int64_t row;             // elements from one token to the next
    int share;               // heads that read the same rows
};

template <typename T> struct LinearWalk {
    LinearOperand<T> q, k, v, x;
    void* o;                 // (tokens, nheads, Dv) in T, or fp32 where of32
    bool of32;
    const float* g;
    const float* enter;      // states that enter, (rows or items, nheads, Dk * Dv), or null (zeros)
    const float* denter;     // the same for S' (by items), or null
    bool by_item;            // enter is by items
    float* fin;              // states at the end: of rows, or of items where only states are wanted; may be null
    float* dfin;             // S' of items
    const float* dlast;      // what the last S' is contracted with, (rows, nheads, Dk * Dv), or null
    float* dpart;            // sums towards dg: (items, nheads, slices, wavefronts)
    int64_t sk, sv;          // state element (i, j) at i * sk + j * sv
    int Dk, Dv;
    bool back;               // from the last token to the first
    DeltaDims d;
    int64_t seg;             // tokens of a segment (a multiple of 64)
    // Segments one after another (chained): a ticket counter and a count of each walk's segments that are done, all zero, and
    // room for each walk's state as fragments.  Null: all segments at once.
    unsigned* ticket;
    unsigned* done;
    float* handed;
    bool alone;              // a chain's workgroups have a CU each
};

// ---- rows and segments ----------------------------------------------------------------------------------

constexpr int64_t kWholeRows = int64_t(1) << 40;      // a segment's length where rows are not cut

// Segments of all rows: a row of n tokens has max(1, ceil(n / seg)).  With offsets, row s's get the numbers
// cu[s] / seg + s on (as blocks in delta_seq); some numbers belong to no row then.
inline int64_t linear_items(const DeltaDims& d, int64_t seg)
{
    if (d.cu) return d.tokens / seg + d.seqs;
    const int64_t n = (d.seqlen + seg - 1) / seg;
    return d.seqs * (n > 0 ? n : 1);
}

struct LinearItem {
    int64_t row, start;      // row, first token
    int len;                 // tokens
    bool first, last;        // of its row, in time
};

__device__ __forceinline__ int64_t linear_offset(const DeltaDims& d, int64_t s)
{
    return min(max((int64_t)d.cu[s], (int64_t)0), d.tokens);
}

__device__ __forceinline__ bool linear_item(const DeltaDims& d, int64_t seg, int64_t item, LinearItem& it)
{
    int64_t begin, n, i;
    if (d.cu) {
        // the last row s with cu[s] / seg + s <= item: 64 rows looked at in a step
        int64_t lo = 0, count = d.seqs;
        while (count > 1) {
            const int64_t step = (count + 63) / 64, at = lo + lane_id() * step;
            const bool ok = at < lo + count && linear_offset(d, at) / seg + at <= item;
            const int steps = max((int)__popcll(__ballot(ok)) - 1, 0);
            const int64_t end = lo + count;
            lo += steps * step;
            count = min(step, end - lo);
        }
        lo = __builtin_amdgcn_readfirstlane((int)lo);
        it.row = lo;
        begin = linear_offset(d, lo);
        n = min(max((int64_t)d.cu[lo + 1], begin), d.tokens) - begin;
        i = item - (begin / seg + lo);
        if (i < 0) return false;
    } else {
        const int64_t per = max((d.seqlen + seg - 1) / seg, (int64_t)1);
        it.row = item / per;
        i = item % per;
        begin = it.row * d.seqlen;
        n = d.seqlen;
    }
    if (i > 0 && i * seg >= n) return false;
    it.start = begin + i * seg;
    it.len = (int)min(n - i * seg, seg);
    it.first = i == 0;
    it.last = (i + 1) * seg >= n;
    return true;
}

// Sum over the 64 lanes, the same in all.
__device__ __forceinline__ int linear_sum(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);          // rows of 16: shifted right by 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);         // lane 15 of a row into the next, lane 31 into
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);         // the upper half
    return __builtin_amdgcn_readlane(v, 63);
}

// A chain's task j in the order first segments of all rows, second segments, ...: its row and which segment of that it is.
// At most kChainRows rows of different lengths, four to a lane; false where there is no such task.
//
// Before turn t there are sum over rows of min(t, the row's segments) tasks, so a task's turn is found by doubling and
// halving: one row of 2^20 tokens has 1024 turns, and trying them one after another took its segments longer than walking
// them (300 heads of 16 x 16: 201 ms, now 41; 131072 tokens 7.3, now 5.0; 9 rows of up to 4096 the same).
constexpr int kChainRows = 256;
__device__ __forceinline__ bool linear_task(const DeltaDims& d, int64_t seg, int j, LinearItem& it, unsigned& turn)
{
    constexpr int kK = kChainRows / 64;
    int segs[kK];                                                  // (a row without tokens has one segment, without tokens)
#pragma unroll
    for (int k = 0; k < kK; ++k) {
        const int64_t s = 64 * k + lane_id();
        segs[k] = 0;
        if (s < d.seqs) {
            const int64_t begin = linear_offset(d, s), n = max(linear_offset(d, s + 1), begin) - begin;
            segs[k] = max((int)((unsigned)(n + seg - 1) / (unsigned)seg), 1);
        }
    }
    auto before = [&](int t) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < kK; ++k) n += min(t, segs[k]);
        return linear_sum(n);
    };
    int t = 0, at = 0;                                             // before(t) = at <= j
    if (j >= d.seqs) {
        const int most = (int)(d.tokens / seg) + 1;                // no row has more segments
        int end = 1, past = (int)d.seqs;
        while (past <= j) {
            if (end >= most) return false;
            t = end;
            at = past;
            end = min(2 * end, most);
            past = before(end);
        }
        while (end - t > 1) {                                      // before(end) > j
            const int mid = (t + end) >> 1, n = before(mid);
            if (n <= j) { t = mid; at = n; }
            else end = mid;
        }
    }
    j -= at;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
        const uint64_t has = __ballot(segs[k] > t);
        const int count = __popcll(has);
        if (j < count) {
            const uint64_t mine = __ballot((has >> lane_id() & 1) && __popcll(has & ((uint64_t(1) << lane_id()) - 1)) == j);
            it.row = 64 * k + __builtin_ctzll(mine);
            const int64_t begin = linear_offset(d, it.row), n = max(linear_offset(d, it.row + 1), begin) - begin;
            const int64_t from = t * seg;
            turn = (unsigned)t;
            it.start = begin + from;
            it.len = (int)min(n - from, seg);
            it.first = t == 0;
            it.last = from + seg >= n;
            return true;
        }
        j -= count;
    }
    return false;
}

// exp(g n) to an ulp or two.  g n is rounded, and an exponent that is off by half a step of up to 64 takes the power off by 64
// of its own half steps (a token whose successors are zeros had its state 3.5e-6 off); what the rounding took is put back.
__device__ __forceinline__ float linear_power(float g, float n)
{
    const float x = g * n, w = expf(x);
    return fmaf(w, fmaf(g, n, -x), w);
}

// A power a^n that a state is multiplied by again and again.  Rounded to fp32 it would be off by the same part every
// time, which adds up where the decay is slow; so the fp32 neighbours below and above it take turns such that their
// product stays within one rounding of the power's.
struct LinearDecay {
    float low, high, share, sum;             // share: of the turns that are high's
    __device__ __forceinline__ void set(float g, int n)
    {
        const double exact = exp((double)g * n);
        low = (float)exact;
        if (low > exact) low = __uint_as_float(__float_as_uint(low) - 1);
        if (exact < 1.1754943508222875e-38) low = 0.f;
        high = low > 0.f ? __uint_as_float(__float_as_uint(low) + 1) : 0.f;
        share = low > 0.f ? (float)((exact - low) / ((double)high - low)) : 0.f;
        sum = 0.5f;
    }
    __device__ __forceinline__ float next()
    {
        sum += share;
        const bool up = sum >= 1.f;
        sum = up ? sum - 1.f : sum;
        return up ? high : low;
    }
};

// ---- copies ---------------------------------------------------------------------------------------------

// One wavefront's share of the copies of a tile of 32 rows: row r from base + r * row_bytes (back: (31 - r) *
// row_bytes), its first `valid` chunks; rows from `rows` on are written as zeros.
template <int CH, int NW>
struct LinearCopy {
    static constexpr int kI = DTile<CH>::kInst, kK = (kI + NW - 1) / NW;
    unsigned off[kK];
    __device__ __forceinline__ static void place(int q, int lane, int& r, int& c)
    {
        const int pos = q * 64 + lane;
        r = pos / CH;
        c = (pos % CH) ^ DTile<CH>::key(r);
    }
    __device__ __forceinline__ void plan(unsigned row_bytes, bool back, int wave, int lane)
    {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            int r, c;
            place(wave + NW * k, lane, r, c);
            off[k] = (unsigned)(back ? 31 - r : r) * row_bytes + 16u * c;
        }
    }
    __device__ __forceinline__ void issue(const void* base, int rows, int valid, unsigned lds, int wave, int lane) const
    {
        if (rows >= 32 && valid == CH) {
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                const int q = wave + NW * k;
                if (kI % NW != 0 && q >= kI) break;
                dma16_off(base, off[k], lds + q * 1024u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                const int q = wave + NW * k;
                if (q >= kI) break;
                int r, c;
                place(q, lane, r, c);
                if (c < valid) {
                    if (r < rows)
                        dma16_off(base, off[k], lds + q * 1024u);
                    else
                        *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(lds + q * 1024u + lane * 16u) = u32x4{0, 0, 0, 0};
                }
            }
        }
    }
};

// ---- the walk -------------------------------------------------------------------------------------------

constexpr int kLC = 32;      // tokens of a chunk

template <typename T, int KB, int NW, int JT, int kBudget, bool kOut, bool kDg> struct LinearShape {
    static constexpr int kEs = (int)sizeof(T);
    static constexpr int CHk = KB * 32 * kEs / 16, CHv = NW * JT * 16 * kEs / 16;
    static constexpr int kQK = kLC * CHk * 16, kV = kLC * CHv * 16;   // bytes of a tile
    static constexpr int kAtK = kOut ? kQK : 0;
    static constexpr int kAtV = kAtK + kQK;
    static constexpr int kAtX = kAtV + kV;
    // (two stages of the widest fp32 rows leave no room for X: it is read from memory)
    static constexpr bool kHasX = kOut && kDg && !(kEs == 4 && KB == 8);
    static constexpr int kStage = kAtX + (kHasX ? kV : 0);
    // three 16 x 16 tiles of decayed scores as operand quads
    static constexpr int kScores = kOut ? 3 * 64 * 4 * kEs : 0;
    static constexpr int kFit = (kBudget - 2 * kScores) / kStage;
    static constexpr int kStages = kFit < 2 ? 2 : kFit > 3 ? 3 : kFit;
    static constexpr bool kPipe = kOut && kStages > 2;                // a chunk's scores are made while the one before is read
    static constexpr int kLds = kStages * kStage + (kPipe ? 2 : 1) * kScores;
    // what every wavefront issues at least: copies for a chunk, stores of a chunk's outputs
    static constexpr int kCopies = (kOut ? 2 : 1) * (DTile<CHk>::kInst / NW) + (kHasX ? 2 : 1) * (DTile<CHv>::kInst / NW);
    static constexpr int kStores = kOut ? 2 * JT : 0;
    // wavefronts a SIMD that the registers are shared out for: two, unless the states alone take half of what they would have
    // (and a workgroup of eight wavefronts puts two on each SIMD in any case)
    static constexpr int kWaves = NW > 4 || KB * 8 * JT * (kDg ? 2 : 1) <= (sizeof(T) == 2 ? 127 : 63) ? 2 : 1;
    static_assert(4 * kWaves >= NW, "a workgroup fits a CU");
};

// Operand fragments of a stage.  What changes with the stage is added to the lane's addresses once a chunk (at), the
// rest are constants.
template <typename T, int CH> struct LinearRows;
template <int CH> struct LinearRows<bf16, CH> {
    static constexpr int kPer = DRows<bf16, CH>::kPer;
    const DRows<bf16, CH> d;
    unsigned b[2][kPer][2];
    __device__ __forceinline__ LinearRows(int r, int g) : d(r, g) {}
    // (rows 16 on have addresses of their own: from one, the compiler would read both rows' quads in one instruction, and
    // move them to their fragments after.  Where a row has 256 elements it still joins blocks kb and kb + 4, 256 bytes apart, in
    // the scores' reads; the halves of such a read fall on the same banks)
    __device__ __forceinline__ void at(unsigned stage)
    {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                b[0][k][x] = b[1][k][x] = d.a[k][x] + stage;
                asm("" : "+v"(b[1][k][x]));
            }
    }
    // row 16 t + r of the tile `tile` bytes into the stage, block kb of 32 elements
    __device__ __forceinline__ void load(Vec8<bf16>& f, int tile, int t, int kb) const
    {
        const int o = tile + t * (16 * CH * 16) + (kb / kPer) * 256;
        const bf16x4 x = lds_at<bf16x4>(b[t][kb % kPer][0] + o), y = lds_at<bf16x4>(b[t][kb % kPer][1] + o);
        f.v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};
template <int CH> struct LinearRows<float, CH> {
    const DRows<float, CH> d;
    unsigned stage;
    __device__ __forceinline__ LinearRows(int r, int g) : d(r, g) {}
    __device__ __forceinline__ void at(unsigned s) { stage = s; }
    __device__ __forceinline__ void load(Vec8<float>& f, int tile, int t, int kb) const { d.load(f, stage + tile, t, kb); }
};
template <typename T, int CH> struct LinearCols;
template <int CH> struct LinearCols<bf16, CH> {
    static constexpr int kPer = DCols<bf16, CH>::kPer;
    const DCols<bf16, CH> d;
    unsigned b[kPer];
    __device__ __forceinline__ LinearCols(int r, int g) : d(r, g) {}
    __device__ __forceinline__ void at(unsigned stage)
    {
#pragma unroll
        for (int k = 0; k < kPer; ++k) b[k] = d.a[k] + stage;
    }
    __device__ __forceinline__ void load(Vec8<bf16>& f, int tile, int t) const
    {
        typedef short v4i16 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4i16* P;
        const unsigned o = b[t % kPer] + (tile + (t / kPer) * 256);
        const v4i16 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)o);
        const v4i16 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)(o + 16 * CH * 16));
        f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};
template <int CH> struct LinearCols<float, CH> {
    const DCols<float, CH> d;
    unsigned stage;
    __device__ __forceinline__ LinearCols(int r, int g) : d(r, g) {}
    __device__ __forceinline__ void at(unsigned s) { stage = s; }
    __device__ __forceinline__ void load(Vec8<float>& f, int tile, int t) const { d.load(f, stage + tile, t); }
};

// An fp32 operand whose product keeps all of fp32: three bf16 values, hi + mid + lo, the value to 2^-24.
template <typename T> struct LinearExact {
    Pair<T> p;
    Vec8<T> lo;
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        p.set(v);
        if constexpr (sizeof(T) == 2) {
            float left[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) left[i] = v[i] - p.hi.get(i) - p.lo.get(i);
            pack8(lo, left);
        }
    }
};
// a exact and b in T, and the other way round
template <typename T>
__device__ __forceinline__ void mma_ex(f32x4& acc, const LinearExact<T>& a, const Vec8<T>& b)
{
    if constexpr (sizeof(T) == 2) mma(acc, a.lo, b);
    mma_px(acc, a.p, b);
}
template <typename T>
__device__ __forceinline__ void mma_xe(f32x4& acc, const Vec8<T>& a, const LinearExact<T>& b)
{
    if constexpr (sizeof(T) == 2) mma(acc, a, b.lo);
    mma_xp(acc, a, b.p);
}

// the 4 values of a T quad at an LDS address, as floats
__device__ __forceinline__ f32x4 lds_quad(unsigned a, bf16)
{
    const bf16x4 q = lds_at<bf16x4>(a);
    return f32x4{(float)q[0], (float)q[1], (float)q[2], (float)q[3]};
}
__device__ __forceinline__ f32x4 lds_quad(unsigned a, float) { return lds_at<f32x4>(a); }
// and put there
__device__ __forceinline__ void lds_put(unsigned a, const f32x4& v, bf16)
{
    *(__attribute__((address_space(3))) u32x2*)(uintptr_t)a = __builtin_bit_cast(u32x2, pack4_bf16(v));
}
__device__ __forceinline__ void lds_put(unsigned a, const f32x4& v, float)
{
    *(__attribute__((address_space(3))) f32x4*)(uintptr_t)a = v;
}
// a fragment of two quads side by side, and one with zeros in its upper half
__device__ __forceinline__ void lds_frag(Vec8<bf16>& f, unsigned a) { f.v = lds_at<bf16x8>(a); }
__device__ __forceinline__ void lds_frag(Vec8<float>& f, unsigned a)
{
    const f32x4 x = lds_at<f32x4>(a), y = lds_at<f32x4>(a + 16);
#pragma unroll
    for (int m = 0; m < 4; ++m) { f.v[m] = x[m]; f.v[4 + m] = y[m]; }
}
__device__ __forceinline__ void lds_half(Vec8<bf16>& f, unsigned a)
{
    f.zero();
    const bf16x4 q = lds_at<bf16x4>(a);
#pragma unroll
    for (int m = 0; m < 4; ++m) f.v[m] = q[m];
}
__device__ __forceinline__ void lds_half(Vec8<float>& f, unsigned a)
{
    const f32x4 x = lds_at<f32x4>(a);
#pragma unroll
    for (int m = 0; m < 4; ++m) { f.v[m] = x[m]; f.v[4 + m] = 0.f; }
}

// Workgroup `block` of the `blocks` of a walk.
template <typename T, int KB, int NW, int JT, int kBudget, bool kOut, bool kDg>
__device__ __forceinline__ void linear_walk_run(const LinearWalk<T>& p, int block, int blocks)
{
    using S = LinearShape<T, KB, NW, JT, kBudget, kOut, kDg>;
    constexpr int CHk = S::CHk, CHv = S::CHv, kNT = 2 * KB, kStages = S::kStages;
    static_assert(NW >= 3, "three wavefronts make a chunk's scores");
    extern __shared__ __attribute__((aligned(1024))) unsigned char lds_raw[];
    const unsigned lds = lds_addr(lds_raw);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
    const int r = lane & 15, g4 = lane >> 4;

    const int slices = (p.Dv + NW * JT * 16 - 1) / (NW * JT * 16);
    const int H = (int)p.d.nheads;
    const bool chained = kOut && p.ticket;
    LinearItem it;
    int at;
    unsigned walk = 0, turn = 0;                                  // a segment's place in its chain
    if (chained) {
        // Workgroups take the segments in the order in which they start: all rows' first ones, all second ones and so on.  The
        // one that a segment waits for was taken before, so its workgroup runs: no wait is for one that has not started.
        if (threadIdx.x == 0) *(__attribute__((address_space(3))) unsigned*)(uintptr_t)lds = atomicAdd(p.ticket, 1u);
        __syncthreads();
        const unsigned mine = __builtin_amdgcn_readfirstlane(lds_at<unsigned>(lds));
        __syncthreads();
        const unsigned of_row = H * slices;
        if (p.d.cu) {
            const unsigned j = __builtin_amdgcn_readfirstlane(mine / of_row);
            if (!linear_task(p.d, p.seg, (int)j, it, turn)) return;
            turn = __builtin_amdgcn_readfirstlane(turn);
            it.row = __builtin_amdgcn_readfirstlane((int)it.row);
            it.start = __builtin_amdgcn_readfirstlane((int)it.start);
            it.len = __builtin_amdgcn_readfirstlane(it.len);
            walk = (unsigned)it.row * of_row + xcd_logical_block((int)(mine - j * of_row), (int)of_row);
            at = walk;
        } else {
            const unsigned walks = (unsigned)p.d.seqs * of_row;
            turn = __builtin_amdgcn_readfirstlane(mine / walks);
            walk = __builtin_amdgcn_readfirstlane(xcd_logical_block((int)(mine - turn * walks), (int)walks));
            const unsigned per = __builtin_amdgcn_readfirstlane((unsigned)blocks / walks), row = walk / of_row;
            at = (row * per + (p.back ? per - 1 - turn : turn)) * of_row + (walk - row * of_row);
        }
    } else {
        at = xcd_logical_block(block, blocks);
    }
    at = __builtin_amdgcn_readfirstlane(at);                      // (fewer than 2^24 workgroups)
    const int slice = at % slices, h = at / slices % H;
    const int64_t item = at / slices / H;
    if (!(chained && p.d.cu) && !linear_item(p.d, p.seg, item, it)) return;
    const bool ends = p.back ? it.first : it.last;                // no segment of the row walks on from this one
    if (!kOut && ends) return;

    // where the walk's own columns of the state lie
    const int col0 = slice * NW * JT * 16;
    const int validk = p.Dk * S::kEs / 16, validv = min(CHv, (p.Dv - col0) * S::kEs / 16);
    const float gl = linear_rate(p.g[h]);
    if constexpr (!kOut) {
        // What a token adds to the state n tokens later is 0 in fp32 where a^n is below e^-200, whatever finite values it
        // has (their product is below e^89, and 0 begins at e^-103): the walk starts where something is left.
        const float reach = -200.f / gl;
        if (gl < 0.f && reach < (float)it.len) {
            const int skip = (it.len - 1 - (int)reach) / kLC * kLC;
            it.len -= skip;
            if (!p.back) it.start += skip;
        }
    }

    // sources: the head's first column, the walk's first token; from there 32 tokens on with every chunk
    const char* src[4];
    int64_t step[4];
    LinearCopy<CHk, NW> copyq, copyk;
    LinearCopy<CHv, NW> copyv, copyx;
    {
        const LinearOperand<T>* ops[4] = {&p.q, &p.k, &p.v, &p.x};
        unsigned row_bytes[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            row_bytes[i] = (unsigned)(ops[i]->row * S::kEs);
            step[i] = p.back ? -(int64_t)kLC * row_bytes[i] : (int64_t)kLC * row_bytes[i];
            const int64_t tok = p.back ? it.start + it.len - kLC : it.start;
            src[i] = (const char*)ops[i]->p + tok * (int64_t)row_bytes[i] +
                     ((int64_t)(h / max(ops[i]->share, 1)) * (i < 2 ? p.Dk : p.Dv) + (i < 2 ? 0 : col0)) * S::kEs;
        }
        if constexpr (kOut) copyq.plan(row_bytes[0], p.back, wave, lane);
        copyk.plan(row_bytes[1], p.back, wave, lane);
        copyv.plan(row_bytes[2], p.back, wave, lane);
        if constexpr (S::kHasX) copyx.plan(row_bytes[3], p.back, wave, lane);
    }
    [[maybe_unused]] const char* xrows = src[3];                  // X of the chunk, where it is not in LDS
    int left = it.len;
    auto issue = [&](unsigned stage) {
        if constexpr (kOut) copyq.issue(src[0], left, validk, stage, wave, lane);
        copyk.issue(src[1], left, validk, stage + S::kAtK, wave, lane);
        copyv.issue(src[2], left, validv, stage + S::kAtV, wave, lane);
        if constexpr (S::kHasX) copyx.issue(src[3], left, validv, stage + S::kAtX, wave, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) src[i] += step[i];
        left -= kLC;
    };

    if (validk < CHk || validv < CHv) {
        // columns that no copy writes hold zeros
        for (int i = threadIdx.x * 16; i < kStages * S::kStage; i += NW * 64 * 16)
            *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(lds + i) = u32x4{0, 0, 0, 0};
        __syncthreads();
    }
    const int nchunks = (it.len + kLC - 1) / kLC;
    for (int c = 0; c < kStages - 1 && c < nchunks; ++c) issue(lds + c * S::kStage);

    // ---- tables of powers
    const int e = p.back ? 0 : 1;
    const float a16 = linear_power(gl, 16.f);
    const float into0 = linear_power(gl, (float)(r + e)), into1 = into0 * a16;  // a^(t + e)
    // the tile of scores that this wavefront makes: t, s = (0, 0), (1, 0), (1, 1); its weights, and t - s times those
    const int tile_t = wave > 0, tile_s = wave == 2;
    float tilew[4];
    [[maybe_unused]] float tiled[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int gap = 16 * (tile_t - tile_s) + r - 4 * g4 - m;
        tilew[m] = gap >= 0 ? linear_power(gl, (float)gap) : 0.f;
        tiled[m] = gap > 0 ? tilew[m] * gap : 0.f;
    }
    float outw[8];
    LinearDecay decay;
    decay.set(gl, kLC);
    auto weights = [&](int rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) outw[i] = linear_power(gl, (float)max(rows - ((i >> 2) * 16 + 4 * g4 + (i & 3)) - e, 0));
    };
    weights(kLC);

    // ---- the entering state
    f32x4 st[kNT][JT], dst[kDg ? kNT : 1][kDg ? JT : 1];
    const int64_t PN = (int64_t)p.Dk * p.Dv;
    auto load_state = [&](const float* base, f32x4& v, int nt, int j) {
        const int col = col0 + (wave * JT + j) * 16 + r, row = 16 * nt + 4 * g4;
        v = f32x4{0.f, 0.f, 0.f, 0.f};
        if (base && row < p.Dk && col < p.Dv) {
            const float* at = base + row * p.sk + col * p.sv;
            if (p.sk == 1) v = *reinterpret_cast<const f32x4*>(at);
            else {
#pragma unroll
                for (int m = 0; m < 4; ++m) v[m] = at[m * p.sk];
            }
        }
    };
    auto store_state = [&](float* base, const f32x4& v, int nt, int j) {
        const int col = col0 + (wave * JT + j) * 16 + r, row = 16 * nt + 4 * g4;
        if (row < p.Dk && col < p.Dv) {
            float* at = base + row * p.sk + col * p.sv;
            if (p.sk == 1) *reinterpret_cast<f32x4*>(at) = v;
            else {
#pragma unroll
                for (int m = 0; m < 4; ++m) at[m * p.sk] = v[m];
            }
        }
    };
    // the state between two segments of a chain, as fragments, written and read past the caches of one XCD
    constexpr int kFrag = NW * 64 * 4;
    float* const handed = p.handed + (int64_t)walk * ((kDg ? 2 : 1) * kNT * JT * kFrag) + threadIdx.x * 4;
    auto take = [&](int i) {
        f32x4 v;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint64_t w = __hip_atomic_load(reinterpret_cast<const uint64_t*>(handed + (int64_t)i * kFrag) + x, __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT);
            v[2 * x] = __uint_as_float((unsigned)w);
            v[2 * x + 1] = __uint_as_float((unsigned)(w >> 32));
        }
        return v;
    };
    auto hand = [&](int i, const f32x4& v) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
            __hip_atomic_store(reinterpret_cast<uint64_t*>(handed + (int64_t)i * kFrag) + x,
                               (uint64_t)__float_as_uint(v[2 * x + 1]) << 32 | __float_as_uint(v[2 * x]), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    };
    if (chained && turn > 0) {
        if (threadIdx.x == 0)
            while (__hip_atomic_load(p.done + walk, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < turn)
                __builtin_amdgcn_s_sleep(8);
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                st[nt][j] = take(nt * JT + j);
                if constexpr (kDg) dst[nt][j] = take((kNT + nt) * JT + j);
            }
    } else {
        const float* in = kOut && p.enter ? p.enter + ((p.by_item ? item : it.row) * H + h) * PN : nullptr;
        const float* din = kOut && kDg && p.denter ? p.denter + (item * H + h) * PN : nullptr;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                load_state(in, st[nt][j], nt, j);
                if constexpr (kDg) load_state(din, dst[nt][j], nt, j);
            }
    }

    // ---- outputs: 4 neighbouring elements of a token a lane, in a buffer of 32 rows that goes along with the chunks
    [[maybe_unused]] const int orow = H * p.Dv * (p.of32 ? 4 : S::kEs);
    [[maybe_unused]] char* out = nullptr;
    [[maybe_unused]] int to[2][JT];
    if constexpr (kOut) {
        out = static_cast<char*>(p.o) + (p.back ? it.start + it.len - kLC : it.start) * (int64_t)orow;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                const int col = col0 + (wave * JT + j) * 16, row = 16 * t + r;
                to[t][j] = col < p.Dv ? (p.back ? kLC - 1 - row : row) * orow + (h * p.Dv + col + 4 * g4) * (p.of32 ? 4 : S::kEs)
                                      : kDropped;
            }
    }

    LinearRows<T, CHk> rowsk(r, g4);
    LinearCols<T, CHk> colsk(r, g4);
    // this wavefront's columns of V (and X): down the rows, and quads along them
    unsigned colv[JT];
#pragma unroll
    for (int j = 0; j < JT; ++j)
        colv[j] = S::kAtV + DTile<CHv>::offset(4 * g4 + (r >> 2), 2 * (wave * JT + j) + ((r & 3) >> 1)) + (r & 1) * 8;
    const unsigned scores = lds + kStages * S::kStage;
    [[maybe_unused]] float dg = 0.f;

    // Three wavefronts make the decayed scores of the chunk at `stage`, a 16 x 16 tile each (rows s, columns t), and leave
    // them as operand quads.
    auto x_quad = [&](unsigned stage, int row, int col, int rows) {
        const int byte = col * S::kEs;
        if constexpr (S::kHasX) {
            return lds_quad(stage + S::kAtX + DTile<CHv>::offset(row, byte >> 4) + (byte & 15), T());
        } else {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            if (row < rows && col0 + col < p.Dv) v = *reinterpret_cast<const f32x4*>(xrows + row * p.x.row * S::kEs + byte);
            return v;
        }
    };
    auto make_scores = [&](unsigned stage, unsigned to_lds, int rows) {
        if (wave >= 3) return;
        f32x4 sc = {0.f, 0.f, 0.f, 0.f};
        LinearRows<T, CHk> rq(r, g4), rk(r, g4);
        rq.at(stage + tile_t * (16 * CHk * 16));
        rk.at(stage + S::kAtK + tile_s * (16 * CHk * 16));
        #pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            Vec8<T> qf, kf;
            rq.load(qf, 0, 0, kb);
            rk.load(kf, 0, 0, kb);
            mma(sc, kf, qf);
        }
        if constexpr (kDg) {
            // the pairs of tokens of this tile towards dg: X . V over this workgroup's columns, Q . K complete
            f32x4 xv = {0.f, 0.f, 0.f, 0.f};
            LinearRows<T, CHv> rx(r, g4), rv(r, g4);
            rx.at(stage + S::kAtX + tile_t * (16 * CHv * 16));
            rv.at(stage + S::kAtV + tile_s * (16 * CHv * 16));
#pragma unroll
            for (int kb = 0; kb < NW * JT / 2; ++kb) {
                Vec8<T> xf, wf;
                if constexpr (S::kHasX) {
                    rx.load(xf, 0, 0, kb);
                } else {
                    const f32x4 x0 = x_quad(stage, 16 * tile_t + r, 32 * kb + 4 * g4, rows);
                    const f32x4 x1 = x_quad(stage, 16 * tile_t + r, 32 * kb + 16 + 4 * g4, rows);
#pragma unroll
                    for (int m = 0; m < 4; ++m) { xf.set(m, x0[m]); xf.set(4 + m, x1[m]); }
                }
                rv.load(wf, 0, 0, kb);
                mma(xv, wf, xf);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) dg = fmaf(xv[m] * sc[m], tiled[m], dg);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) sc[m] *= tilew[m];
        // With bf16 inputs decayed scores are rounded to bf16, and so is the state where outputs are read from it: bf16 outputs are
        // 2.35e-3 of their norm off, 1.66e-3 of it their own rounding.  As pairs both would leave that alone; 320 rows then take
        // 286 us, now 250, 65536 tokens 1738, now 1520, the backward of 320 rows 932, now 880.
        // tile (0, 0) alone, then (1, 0) and (1, 1) side by side
        lds_put(to_lds + (wave == 0 ? lane * 4 * S::kEs : (256 + lane * 8 + tile_s * 4) * S::kEs), sc, T());
    };

    wait_vmem();                                                  // the state's loads: not again in every chunk
    if constexpr (S::kPipe) {
        __syncthreads();
        if (nchunks > 0) make_scores(lds, scores, kLC);
    }
    // the ring's offsets of this chunk and of the one whose copies start now
    unsigned now = 0, next = (kStages - 1) * S::kStage, score = 0;
    for (int c = 0; c < nchunks; ++c) {
        // Memory operations complete in their order, so what was issued behind the copies that are needed may be outstanding:
        // whole chunks' copies and, once as many have gone by, the stores of the chunks since.  Near the end, where
        // copies are fewer, everything is waited for.
        //   kPipe: chunk c + 1 (its scores are made now), issued kStages - 2 chunks ago; else chunk c, kStages - 1 ago
        constexpr int kAgo = S::kPipe ? kStages - 2 : kStages - 1;
        constexpr int kAhead = (kAgo - 1) * S::kCopies, kAll = kAhead + kAgo * S::kStores;
        static_assert(kAll < 64, "vmcnt range");
        if (c + kStages > nchunks) wait_vmem();
        else if (c < kStages) wait_vmem_below<kAhead>();
        else wait_vmem_below<kAll>();
        __syncthreads();
        const unsigned stage = lds + now;
        now = now + S::kStage == kStages * S::kStage ? 0 : now + S::kStage;
        if (c + kStages - 1 < nchunks) issue(lds + next);
        next = stage - lds;
        const int rows = min(kLC, it.len - c * kLC);
        if (rows < kLC) weights(rows);
        unsigned made = scores;
        if constexpr (S::kPipe) {
            made += score;
            score = S::kScores - score;
            if (c + 1 < nchunks) make_scores(lds + now, scores + score, kLC);
        } else if constexpr (kOut) {
            make_scores(stage, scores, rows);
            __syncthreads();
        }
        rowsk.at(stage);
        colsk.at(stage);

        Vec8<T> vf[JT];
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            if constexpr (sizeof(T) == 2) {
                typedef short v4i16 __attribute__((ext_vector_type(4)));
                typedef __attribute__((address_space(3))) v4i16* P;
                const unsigned o = colv[j] + stage;
                const v4i16 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)o);
                const v4i16 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(uintptr_t)(o + 16 * CHv * 16));
                vf[j].v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
            } else {
                DCols<T, CHv>::load_any(vf[j], stage + S::kAtV, wave * JT + j, r, g4);
            }
        }

        // operands of the state's products, kAheadK at a time before they are needed
        constexpr int kAheadK = sizeof(T) == 2 ? (kNT < 4 ? kNT : 4) : 1;
        Vec8<T> kt[kAheadK];
        auto load_first = [&]() {
#pragma unroll
            for (int i = 0; i < kAheadK; ++i) colsk.load(kt[i], S::kAtK, i);
        };

        if constexpr (kOut) {
            f32x4 acc[2][JT], dacc[kDg ? 2 : 1][kDg ? JT : 1];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if constexpr (kDg) dacc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            // against the entering state
            Vec8<T> qf[2][2], sf[2];
            rowsk.load(qf[0][0], 0, 0, 0);
            rowsk.load(qf[0][1], 0, 1, 0);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                if (kb + 1 < KB) {
                    rowsk.load(qf[(kb + 1) & 1][0], 0, 0, kb + 1);
                    rowsk.load(qf[(kb + 1) & 1][1], 0, 1, kb + 1);
                } else {
                    lds_half(sf[0], made + lane * 4 * S::kEs);
                    lds_frag(sf[1], made + (256 + lane * 8) * S::kEs);
                }
                __builtin_amdgcn_sched_barrier(0);                // the next operands are on the way
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    float s8[8];
#pragma unroll
                    for (int m = 0; m < 4; ++m) { s8[m] = st[2 * kb][j][m]; s8[4 + m] = st[2 * kb + 1][j][m]; }
                    if constexpr (kDg) {
                        // dg is an fp32 sum in which much cancels, and takes its terms from here
                        LinearExact<T> f, df;
                        f.set(s8);
#pragma unroll
                        for (int m = 0; m < 4; ++m) { s8[m] = dst[2 * kb][j][m]; s8[4 + m] = dst[2 * kb + 1][j][m]; }
                        df.set(s8);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            mma_ex(acc[t][j], f, qf[kb & 1][t]);
                            mma_ex(dacc[t][j], df, qf[kb & 1][t]);
                        }
                    } else {
                        Vec8<T> f;                                 // (rounded to bf16: see make_scores)
                        pack8(f, s8);
#pragma unroll
                        for (int t = 0; t < 2; ++t) mma(acc[t][j], f, qf[kb & 1][t]);
                    }
                }
            }
            load_first();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    if constexpr (kDg) {
                        const f32x4 x = x_quad(stage, 16 * t + r, (wave * JT + j) * 16 + 4 * g4, rows);
                        float sum = 0.f;
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            sum = fmaf(x[m], fmaf((float)(16 * t + r + 1), acc[t][j][m], dacc[t][j][m]), sum);
                        dg = fmaf(t ? into1 : into0, sum, dg);
                    }
                    acc[t][j] *= t ? into1 : into0;
                    mma(acc[t][j], vf[j], sf[t]);                  // the chunk's own scores
                }
            {
                const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc(out, 0, kLC * orow, kBufferDword3);
                auto store = [&](auto type) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int j = 0; j < JT; ++j)           // (rows behind the walk's end are dropped: always as many stores)
                            buffer_store4(buf, 16 * t + r < rows ? to[t][j] : kDropped, 0, acc[t][j], type);
                };
                if (p.of32) store(0.f);
                else store(T());
                out += p.back ? -(int64_t)kLC * orow : (int64_t)kLC * orow;
            }
            if constexpr (kDg && !S::kHasX) xrows += step[3];
        } else {
            load_first();
        }

        // The state behind the chunk is an fp32 result: its weighted values are three bf16 values each, the state then as exact as
        // fp32 sums are (4e-8 to 4e-7 of its norm).  Pairs left 2.4e-6, and where dg cancels up to 3e-5 of that; they take
        // 2 % off the forward of 320 rows and its backward, 9 % off 65536 tokens' with 256 rows of state.  So are the ones of S'
        // and, where they are read, both states: dg is then as exact as an fp32 sum; with pairs for S and for what a chunk adds
        // to S' the backward takes 4 to 6 % less, and dg is 3e-6 off, or in one head of 22 tokens 2.5e-5.
        LinearExact<T> vw[JT], dvw[kDg ? JT : 1];
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            float w8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w8[i] = vf[j].get(i) * outw[i];
            vw[j].set(w8);
            if constexpr (kDg) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w8[i] = vf[j].get(i) * (outw[i] * (float)(rows - 1 - ((i >> 2) * 16 + 4 * g4 + (i & 3))));
                dvw[j].set(w8);
            }
        }
        const float a = rows < kLC ? linear_power(gl, (float)rows) : decay.next();
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                if constexpr (kDg) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) dst[nt][j][m] = fmaf((float)rows, st[nt][j][m], dst[nt][j][m]) * a;
                }
                st[nt][j] *= a;
                mma_xe(st[nt][j], kt[nt % kAheadK], vw[j]);
                if constexpr (kDg) mma_xe(dst[nt][j], kt[nt % kAheadK], dvw[j]);
            }
            if (nt + kAheadK < kNT) colsk.load(kt[nt % kAheadK], S::kAtK, nt + kAheadK);
        }
    }
    settle();

    // ---- the state at the end
    if constexpr (kOut) {
        if (chained && !ends) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    hand(nt * JT + j, st[nt][j]);
                    if constexpr (kDg) hand((kNT + nt) * JT + j, dst[nt][j]);
                }
            wait_vmem();                                          // every wavefront's part has arrived
            __syncthreads();
            if (threadIdx.x == 0)
                __hip_atomic_store(p.done + walk, turn + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (ends) {
            if (p.fin) {
                float* at = p.fin + (it.row * H + h) * PN;
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int j = 0; j < JT; ++j) store_state(at, st[nt][j], nt, j);
            }
            if constexpr (kDg) {
                const float* last = p.dlast ? p.dlast + (it.row * H + h) * PN : nullptr;
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int j = 0; j < JT; ++j) {
                        f32x4 f;
                        load_state(last, f, nt, j);
                        // (columns and rows that do not exist hold zeros in both)
                        if (last) dg += f[0] * dst[nt][j][0] + f[1] * dst[nt][j][1] + f[2] * dst[nt][j][2] + f[3] * dst[nt][j][3];
                    }
            }
        }
        if constexpr (kDg) {
            const float sum = group_sum<64>(dg);
            if (lane == 0) p.dpart[((item * H + h) * slices + slice) * NW + wave] = sum;
        }
    } else {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                store_state(p.fin + (item * H + h) * PN, st[nt][j], nt, j);
                if constexpr (kDg) store_state(p.dfin + (item * H + h) * PN, dst[nt][j], nt, j);
            }
    }
}

template <typename T, int KB, int NW, int JT, int kBudget, bool kOut, bool kDg>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(
    LinearShape<T, KB, NW, JT, kBudget, kOut, kDg>::kWaves, LinearShape<T, KB, NW, JT, kBudget, kOut, kDg>::kWaves)))
void linear_walk_kernel(LinearWalk<T> p)
{
    linear_walk_run<T, KB, NW, JT, kBudget, kOut, kDg>(p, blockIdx.x, gridDim.x);
}

// Two walks in one launch: dk's and dv's, whose rows and columns of the state are each other's.
template <typename T, int KB, int KB2, int kBudget, bool kOut> struct LinearTwin {
    static constexpr int JT = sizeof(T) == 2 && KB2 > 2 ? 2 : 1, JT2 = sizeof(T) == 2 && KB > 2 ? 2 : 1;
    using A = LinearShape<T, KB, 4, JT, kBudget, kOut, false>;
    using B = LinearShape<T, KB2, 4, JT2, kBudget, kOut, false>;
    static constexpr int kWaves = A::kWaves < B::kWaves ? A::kWaves : B::kWaves;
    static constexpr int kLds = A::kLds > B::kLds ? A::kLds : B::kLds;
};
template <typename T, int KB, int KB2, int kBudget, bool kOut>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(LinearTwin<T, KB, KB2, kBudget, kOut>::kWaves,
                                                                     LinearTwin<T, KB, KB2, kBudget, kOut>::kWaves)))
void linear_twin_kernel(LinearWalk<T> a, LinearWalk<T> b, int blocks_a)
{
    using W = LinearTwin<T, KB, KB2, kBudget, kOut>;
    // eight of one (a workgroup for each XCD), eight of the other: segments that wait in a chain start behind both's first ones
    const int blocks_b = gridDim.x - blocks_a, pairs = min(blocks_a, blocks_b) & ~7, block = blockIdx.x;
    bool second;
    int at;
    if (block < 2 * pairs) {
        second = block >> 3 & 1;
        at = (block >> 4) * 8 + (block & 7);
    } else {
        at = block - pairs;
        second = at >= blocks_a;
        if (second) at -= blocks_a - pairs;
    }
    if (!second) linear_walk_run<T, KB, 4, W::JT, kBudget, kOut, false>(a, at, blocks_a);
    else linear_walk_run<T, KB2, 4, W::JT2, kBudget, kOut, false>(b, at, blocks_b);
}

// ---- launches -------------------------------------------------------------------------------------------

template <typename T> int64_t walk_blocks(const LinearWalk<T>& p, int columns)
{
    return linear_items(p.d, p.seg) * p.d.nheads * ((p.Dv + columns - 1) / columns);
}

// LDS of a launch: more than half of what there is where a second workgroup is not wanted on the CU.
template <typename T> int walk_lds(const LinearWalk<T>& p, int need) { return p.ticket && p.alone ? std::max(need, 84 * 1024) : need; }

template <typename T, int KB, int NW, int JT, int kBudget, bool kOut, bool kDg>
hipError_t launch_walk(const LinearWalk<T>& p, hipStream_t stream)
{
    using S = LinearShape<T, KB, NW, JT, kBudget, kOut, kDg>;
    static_assert(S::kLds <= 160 * 1024, "the ring fits LDS");
    const int64_t blocks = walk_blocks(p, NW * JT * 16);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((linear_walk_kernel<T, KB, NW, JT, kBudget, kOut, kDg>), dim3((unsigned)blocks), dim3(NW * 64),
                       walk_lds(p, S::kLds), stream, p);
    return hipGetLastError();
}

template <typename T, int KB, int KB2, int kBudget, bool kOut>
hipError_t launch_twin(const LinearWalk<T>& a, const LinearWalk<T>& b, hipStream_t stream)
{
    using W = LinearTwin<T, KB, KB2, kBudget, kOut>;
    static_assert(W::kLds <= 160 * 1024, "the rings fit LDS");
    const int64_t first = walk_blocks(a, 64 * W::JT), blocks = first + walk_blocks(b, 64 * W::JT2);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((linear_twin_kernel<T, KB, KB2, kBudget, kOut>), dim3((unsigned)blocks), dim3(256),
                       walk_lds(a, W::kLds), stream, a, b, (int)first);
    return hipGetLastError();
}

// Columns of the state that a workgroup of a walk holds (kDg: of a walk towards dg), and wavefronts it has.
constexpr int linear_columns(int elem_bytes, int Dv) { return elem_bytes == 2 && Dv > 64 ? 128 : 64; }
constexpr int linear_waves(int elem_bytes, bool dg, int Dv) { return dg ? linear_columns(elem_bytes, Dv) / 16 : 4; }

// Floats of the state that a walk hands on (kDg: of both), its rows and columns rounded up to what a workgroup holds.
constexpr int64_t linear_handed(int elem_bytes, bool dg, int64_t Dk, int64_t Dv)
{
    const int64_t rows = Dk <= 32 ? 32 : Dk <= 64 ? 64 : Dk <= 128 ? 128 : 256, columns = linear_columns(elem_bytes, (int)Dv);
    return (dg ? 2 : 1) * rows * ((Dv + columns - 1) / columns * columns);
}

template <typename T, bool kOut, bool kDg>
hipError_t launch_linear_walk(const LinearWalk<T>& p, hipStream_t stream);

// Two walks, a's rows and columns b's columns and rows, at most 128 of each.
template <typename T, bool kOut>
hipError_t launch_linear_twin(const LinearWalk<T>& a, const LinearWalk<T>& b, hipStream_t stream);

}  // namespace ssd
