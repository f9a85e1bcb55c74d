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
// columns Dv), which are operand fragments as they are (see common.hpp).  It works out all scores of a chunk by itself:
// the K and Q fragments are read for the state's products in any case, and in return the wavefronts exchange nothing and
// a chunk has one barrier, behind the copies.  Two stages of LDS: a chunk's copies run while the one before it is
// worked on.
//
// A row may be cut into segments that walk at the same time: a first pass of the same kernel (states only) leaves
// what each adds to the state, linear_join carries the states over, and the walk starts each segment from its own.
#pragma once

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

template <typename T, int KB, int NW, int JT, int C, bool kOut, bool kDg> struct LinearShape {
    static constexpr int kEs = (int)sizeof(T);
    static constexpr int CHk = KB * 32 * kEs / 16, CHv = NW * JT * 16 * kEs / 16;
    static constexpr int kSB = C / 32;
    static constexpr int kQK = 32 * CHk * 16, kV = 32 * CHv * 16;     // bytes of a tile of 32 rows
    static constexpr int kAtK = kOut ? kSB * kQK : 0;
    static constexpr int kAtV = kAtK + kSB * kQK;
    static constexpr int kAtX = kAtV + kSB * kV;
    static constexpr int kStage = kAtX + (kOut && kDg ? kSB * kV : 0);
};

// A DTile's fragment along row 16 t + r (the slots of DRows), for a block of 32 elements that is not a constant.
template <typename T, int CH>
__device__ __forceinline__ void linear_rows_any(Vec8<T>& f, unsigned tile, int t, int kb, int r, int g)
{
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int byte = (32 * kb + 16 * x + 4 * g) * (int)sizeof(T);
        const unsigned at = tile + DTile<CH>::offset(16 * t + r, byte >> 4) + (byte & 15);
        if constexpr (sizeof(T) == 2) {
            const bf16x4 q = lds_at<bf16x4>(at);
#pragma unroll
            for (int m = 0; m < 4; ++m) f.v[4 * x + m] = q[m];
        } else {
            const f32x4 q = lds_at<f32x4>(at);
#pragma unroll
            for (int m = 0; m < 4; ++m) f.v[4 * x + m] = q[m];
        }
    }
}

// the 4 values of a T quad at an LDS address as floats
__device__ __forceinline__ f32x4 lds_quad(unsigned a, bf16)
{
    const bf16x4 q = lds_at<bf16x4>(a);
    return f32x4{(float)q[0], (float)q[1], (float)q[2], (float)q[3]};
}
__device__ __forceinline__ f32x4 lds_quad(unsigned a, float) { return lds_at<f32x4>(a); }

template <typename T, int KB, int NW, int JT, int C, bool kOut, bool kDg>
__global__ __launch_bounds__(NW * 64) void linear_walk_kernel(LinearWalk<T> p)
{
    using S = LinearShape<T, KB, NW, JT, C, kOut, kDg>;
    constexpr int CHk = S::CHk, CHv = S::CHv, kSB = S::kSB, kTT = C / 16, kNT = 2 * KB;
    extern __shared__ __attribute__((aligned(1024))) unsigned char lds_raw[];
    const unsigned lds = lds_addr(lds_raw);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
    const int r = lane & 15, g4 = lane >> 4;

    const int slices = (p.Dv + NW * JT * 16 - 1) / (NW * JT * 16);
    int64_t n = xcd_logical_block(blockIdx.x, gridDim.x);
    const int slice = (int)(n % slices);
    n /= slices;
    const int H = (int)p.d.nheads, h = (int)(n % H);
    const int64_t item = n / H;
    LinearItem it;
    if (!linear_item(p.d, p.seg, item, it)) return;
    const bool ends = p.back ? it.first : it.last;                // no segment of the row walks on from this one
    if (!kOut && ends) return;

    // where the walk's own columns of the state lie
    const int col0 = slice * NW * JT * 16;
    const int validk = p.Dk * S::kEs / 16, validv = min(CHv, (p.Dv - col0) * S::kEs / 16);
    const float gl = fmaxf(p.g[h], -1000.f);

    // sources: head's first column, the walk's first token
    const char* src[4];
    unsigned row_bytes[4];
    {
        const LinearOperand<T>* ops[4] = {&p.q, &p.k, &p.v, &p.x};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int width = i < 2 ? p.Dk : p.Dv;
            row_bytes[i] = (unsigned)(ops[i]->row * S::kEs);
            const int64_t tok = p.back ? it.start + it.len - 32 : it.start;
            src[i] = (const char*)ops[i]->p + tok * (int64_t)row_bytes[i] +
                     ((int64_t)(h / max(ops[i]->share, 1)) * width + (i < 2 ? 0 : col0)) * S::kEs;
        }
    }
    LinearCopy<CHk, NW> copyq, copyk;
    LinearCopy<CHv, NW> copyv, copyx;
    if constexpr (kOut) copyq.plan(row_bytes[0], p.back, wave, lane);
    copyk.plan(row_bytes[1], p.back, wave, lane);
    copyv.plan(row_bytes[2], p.back, wave, lane);
    if constexpr (kOut && kDg) copyx.plan(row_bytes[3], p.back, wave, lane);

    auto issue = [&](int c, unsigned stage) {
#pragma unroll
        for (int sb = 0; sb < kSB; ++sb) {
            const int t0 = c * C + 32 * sb, rows = it.len - t0;
            const int64_t step = p.back ? -(int64_t)t0 : (int64_t)t0;
            if constexpr (kOut) copyq.issue(src[0] + step * row_bytes[0], rows, validk, stage + sb * S::kQK, wave, lane);
            copyk.issue(src[1] + step * row_bytes[1], rows, validk, stage + S::kAtK + sb * S::kQK, wave, lane);
            copyv.issue(src[2] + step * row_bytes[2], rows, validv, stage + S::kAtV + sb * S::kV, wave, lane);
            if constexpr (kOut && kDg)
                copyx.issue(src[3] + step * row_bytes[3], rows, validv, stage + S::kAtX + sb * S::kV, wave, lane);
        }
    };

    if (validk < CHk || validv < CHv) {
        // columns that no copy writes hold zeros
        for (int i = threadIdx.x * 16; i < 2 * S::kStage; i += NW * 64 * 16)
            *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(lds + i) = u32x4{0, 0, 0, 0};
        __syncthreads();
    }
    const int nchunks = (it.len + C - 1) / C;
    if (nchunks > 0) issue(0, lds);

    // ---- tables of powers
    const int e = p.back ? 0 : 1;
    float diag[4], off[4], outw[kSB][8];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int gap = r - 4 * g4 - m;                           // t - s within a 16 x 16 tile
        diag[m] = gap >= 0 ? expf(gl * gap) : 0.f;
        off[m] = expf(gl * (16 + gap));
    }
    const float a16 = expf(gl * 16.f);
    const float into = expf(gl * (r + e));
    float grow;                                                   // a^C - 1: the state's own share stays exact
    auto weights = [&](int rows) {
#pragma unroll
        for (int sb = 0; sb < kSB; ++sb)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = 32 * sb + (i >> 2) * 16 + 4 * g4 + (i & 3);
                outw[sb][i] = expf(gl * max(rows - s - e, 0));
            }
        grow = expm1f(gl * rows);
    };
    weights(C);

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
    {
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

    const DRows<T, CHk> rowsk(r, g4);
    const DCols<T, CHk> colsk(r, g4);
    [[maybe_unused]] float dg = 0.f;

    for (int c = 0; c < nchunks; ++c) {
        const unsigned stage = lds + (c & 1) * S::kStage;
        wait_vmem();
        __syncthreads();
        if (c + 1 < nchunks) issue(c + 1, lds + ((c + 1) & 1) * S::kStage);
        const int rows = min(C, it.len - c * C);
        if (rows < C) weights(rows);

        Vec8<T> vf[kSB][JT];
#pragma unroll
        for (int sb = 0; sb < kSB; ++sb)
#pragma unroll
            for (int j = 0; j < JT; ++j)
                DCols<T, CHv>::load_any(vf[sb][j], stage + S::kAtV + sb * S::kV, wave * JT + j, r, g4);

        if constexpr (kOut) {
            f32x4 acc[kTT][JT], sc[kTT * (kTT + 1) / 2], dacc[kDg ? kTT : 1][kDg ? JT : 1];
#pragma unroll
            for (int t = 0; t < kTT; ++t)
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if constexpr (kDg) dacc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
#pragma unroll
            for (int i = 0; i < kTT * (kTT + 1) / 2; ++i) sc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            // against the entering state, and the scores (rows s, columns t)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                Vec8<T> qf[kTT], kf[kTT];
#pragma unroll
                for (int t = 0; t < kTT; ++t) {
                    rowsk.load(qf[t], stage + (t >> 1) * S::kQK, t & 1, kb);
                    rowsk.load(kf[t], stage + S::kAtK + (t >> 1) * S::kQK, t & 1, kb);
                }
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    float s8[8];
#pragma unroll
                    for (int m = 0; m < 4; ++m) { s8[m] = st[2 * kb][j][m]; s8[4 + m] = st[2 * kb + 1][j][m]; }
                    if constexpr (kDg) {
                        // dg is fp32 and takes its terms from here: pairs
                        Pair<T> f, df;
                        f.set(s8);
#pragma unroll
                        for (int m = 0; m < 4; ++m) { s8[m] = dst[2 * kb][j][m]; s8[4 + m] = dst[2 * kb + 1][j][m]; }
                        df.set(s8);
#pragma unroll
                        for (int t = 0; t < kTT; ++t) {
                            mma_px(acc[t][j], f, qf[t]);
                            mma_px(dacc[t][j], df, qf[t]);
                        }
                    } else {
                        Vec8<T> f;
                        pack8(f, s8);
#pragma unroll
                        for (int t = 0; t < kTT; ++t) mma(acc[t][j], f, qf[t]);
                    }
                }
#pragma unroll
                for (int t = 0; t < kTT; ++t)
#pragma unroll
                    for (int s = 0; s <= t; ++s) mma(sc[t * (t + 1) / 2 + s], kf[s], qf[t]);
            }
            float at = into;                                      // a^(t + e), 16 tokens on with every tile
#pragma unroll
            for (int t = 0; t < kTT; ++t) {
                if constexpr (kDg) {
#pragma unroll
                    for (int j = 0; j < JT; ++j) {
                        const int tile = wave * JT + j;
                        const f32x4 x = lds_quad(stage + S::kAtX + (t >> 1) * S::kV +
                                                     DTile<CHv>::offset((t & 1) * 16 + r, (tile * 16 + 4 * g4) * S::kEs / 16) +
                                                     ((tile * 16 + 4 * g4) * S::kEs & 15), T());
                        float sum = 0.f;
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            sum = fmaf(x[m], fmaf((float)(16 * t + r + 1), acc[t][j][m], dacc[t][j][m]), sum);
                        dg = fmaf(at, sum, dg);
                    }
                }
#pragma unroll
                for (int j = 0; j < JT; ++j) acc[t][j] *= at;
                at *= a16;
            }
            if constexpr (kDg) {
                // the chunk's own pairs: X . V over this wavefront's 32 columns, Q . K complete
                static_assert(JT == 2, "a wavefront's columns are one contraction block");
                Vec8<T> xf[kTT], wf[kTT];
#pragma unroll
                for (int t = 0; t < kTT; ++t) {
                    linear_rows_any<T, CHv>(xf[t], stage + S::kAtX + (t >> 1) * S::kV, t & 1, wave, r, g4);
                    linear_rows_any<T, CHv>(wf[t], stage + S::kAtV + (t >> 1) * S::kV, t & 1, wave, r, g4);
                }
#pragma unroll
                for (int t = 0; t < kTT; ++t) {
                    float far = 1.f;
#pragma unroll
                    for (int s = t; s >= 0; --s) {
                        f32x4 xv = {0.f, 0.f, 0.f, 0.f};
                        mma(xv, wf[s], xf[t]);
                        const f32x4 qk = sc[t * (t + 1) / 2 + s];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const int gap = 16 * (t - s) + r - 4 * g4 - m;
                            const float w = s == t ? diag[m] : off[m] * far;
                            const float term = xv[m] * qk[m] * (w * gap);
                            dg += s == t ? select(gap > 0, term, 0.f) : term;
                        }
                        if (s < t) far *= a16;
                    }
                }
            }
            // the chunk's own scores, decayed
#pragma unroll
            for (int t = 0; t < kTT; ++t) {
#pragma unroll
                for (int sb = 0; sb <= t / 2; ++sb) {
                    float w8[8];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int s = 2 * sb + x;
                        float far = 1.f;
#pragma unroll
                        for (int i = s + 1; i < t; ++i) far *= a16;
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            if (s > t) w8[4 * x + m] = 0.f;
                            else if (s == t) w8[4 * x + m] = select(r >= 4 * g4 + m, sc[t * (t + 1) / 2 + min(s, t)][m] * diag[m], 0.f);
                            else w8[4 * x + m] = sc[t * (t + 1) / 2 + min(s, t)][m] * (off[m] * far);
                        }
                    }
                    Vec8<T> f;
                    pack8(f, w8);
#pragma unroll
                    for (int j = 0; j < JT; ++j) mma(acc[t][j], vf[sb][j], f);
                }
            }
            // rows Dv, columns t: 4 neighbouring elements of a token a lane
#pragma unroll
            for (int t = 0; t < kTT; ++t) {
                const int row = 16 * t + r;
                const int64_t tok = p.back ? it.start + it.len - 1 - (c * C + row) : it.start + c * C + row;
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    const int col = col0 + (wave * JT + j) * 16 + 4 * g4;
                    if (row < rows && col < p.Dv) {
                        const int64_t to = (tok * H + h) * p.Dv + col;
                        if (p.of32) store4((float*)p.o + to, acc[t][j][0], acc[t][j][1], acc[t][j][2], acc[t][j][3]);
                        else store4((T*)p.o + to, acc[t][j][0], acc[t][j][1], acc[t][j][2], acc[t][j][3]);
                    }
                }
            }
        }

        // the state behind the chunk: fp32 results, so the weighted values are pairs
        Pair<T> vw[kSB][JT], dvw[kDg ? kSB : 1][kDg ? JT : 1];
#pragma unroll
        for (int sb = 0; sb < kSB; ++sb)
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                float w8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w8[i] = vf[sb][j].get(i) * outw[sb][i];
                vw[sb][j].set(w8);
                if constexpr (kDg) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w8[i] = vf[sb][j].get(i) * (outw[sb][i] * (float)(rows - 1 - (32 * sb + (i >> 2) * 16 + 4 * g4 + (i & 3))));
                    dvw[sb][j].set(w8);
                }
            }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                if constexpr (kDg) {
                    const f32x4 both = dst[nt][j] + (float)rows * st[nt][j];
#pragma unroll
                    for (int m = 0; m < 4; ++m) dst[nt][j][m] = fmaf(both[m], grow, both[m]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) st[nt][j][m] = fmaf(st[nt][j][m], grow, st[nt][j][m]);
            }
#pragma unroll
            for (int sb = 0; sb < kSB; ++sb) {
                Vec8<T> kf;
                colsk.load(kf, stage + S::kAtK + sb * S::kQK, nt);
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    mma_xp(st[nt][j], kf, vw[sb][j]);
                    if constexpr (kDg) mma_xp(dst[nt][j], kf, dvw[sb][j]);
                }
            }
        }
        settle();
    }

    // ---- the state at the end
    if constexpr (kOut) {
        if (ends) {
            if (p.fin) {
                float* to = p.fin + (it.row * H + h) * PN;
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int j = 0; j < JT; ++j) store_state(to, st[nt][j], nt, j);
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

// ---- launches -------------------------------------------------------------------------------------------

template <typename T, int KB, int NW, int JT, int C, bool kOut, bool kDg>
hipError_t launch_walk(const LinearWalk<T>& p, hipStream_t stream)
{
    using S = LinearShape<T, KB, NW, JT, C, kOut, kDg>;
    static_assert(2 * S::kStage <= 160 * 1024, "two stages of LDS");
    const int64_t slices = (p.Dv + NW * JT * 16 - 1) / (NW * JT * 16);
    const int64_t blocks = linear_items(p.d, p.seg) * p.d.nheads * slices;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((linear_walk_kernel<T, KB, NW, JT, C, kOut, kDg>), dim3((unsigned)blocks), dim3(NW * 64),
                       2 * S::kStage, stream, p);
    return hipGetLastError();
}

// Columns of the state that a workgroup of a walk holds (kDg: of a walk towards dg), and wavefronts it has.
constexpr int linear_columns(int elem_bytes, bool dg, int Dv) { return elem_bytes == 2 && Dv > 64 ? 128 : 64; }
constexpr int linear_waves(int elem_bytes, bool dg, int Dv) { return dg ? linear_columns(elem_bytes, dg, Dv) / 32 : 4; }

template <typename T, bool kOut, bool kDg>
hipError_t launch_linear_walk(const LinearWalk<T>& p, hipStream_t stream);

}  // namespace ssd
