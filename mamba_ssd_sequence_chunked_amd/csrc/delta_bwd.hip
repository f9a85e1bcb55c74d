// delta_bwd.hip - gradients of the gated delta rule.
//
// With H = dL/dS after a block of 32 tokens (notation of delta_tiles.hpp; B = (I + diag(beta) X)^-1):
//
//   dU = M^T dY + diag(del) K H^T       w = B^T dU        dV = diag(beta) w       dbeta_i = w_i . e_i
//   dL/dS before = gam_last H + dY^T diag(gam) Q - w^T diag(beta gam) K
//   W = (dY U^T) o G (j <= i)           Z = -(w U^T) o diag(beta) G (j < i)
//   dQ = diag(gam) dY S + W K           dK = W^T Q + (Z + Z^T) K + diag(del) U H - diag(beta gam) w S
//
// and for the log decay, whose gradient is <dL/dS'_t, S'_t>, the identity
//
//   dg_t = dg_{t+1} + dy_t . y_t - dv_t . v_t,     dg after a block's last token = <H, S>
//
// so it needs row sums only, and the inner product of the two states at the ends of every 64-token chunk: a longer
// sum's rounding errors would outgrow the gradient, which the decay keeps to a few tokens' size. The sum from a
// chunk's end misses the value at its start by the errors of its 64 terms; the difference is spread evenly over them
// (the error left at a token then is that of a bridge between two known ends, a third of the walk's variance).
//
// Four steps: the records (delta_prep); the walk forward again (delta_fwd.hip), keeping e, dy . y and the state
// at every 64th token; the walk back (below), the same form with H in the state's place; and, for all chunks of 64
// tokens at once, dq and dk, summed over the heads that share them inside a workgroup, in a fixed order.
// Everything that leads to H, dbeta and dg is computed on pairs (fp32's accuracy for bf16 inputs); dq and dk,
// which are rounded to T themselves, on T.
#include "delta_tiles.hpp"

namespace ssd {

namespace {

constexpr int kChunk = 64;       // tokens of a chunk of the dq, dk step

// What the walk back keeps, beside DeltaKeep.
template <typename T> struct DeltaBack {
    T* w;                    // as e: w of every block, head and 16 columns
    float* vdv;              // (headdim / 16, tokens, nheads): dv . v over 16 columns
    float* we;               // the same of w . e
    T* H;                    // (seqs, chunks, nheads, headdim, dstate): dL/d(state after each 64-token chunk)
    float* hs;               // (headdim / 16, seqs, chunks + 1, nheads): <H, S> over 16 rows at the chunks' ends
};

// ---- the walk back ------------------------------------------------------------------------------------------

template <typename T, int NB, int NW>
struct RevCfg {
    using R = DeltaRec<T, true>;
    static constexpr int kCH = NB * 32 * (int)sizeof(T) / 16, kCV = 16 * NW * (int)sizeof(T) / 16;
    static constexpr int kK = 0, kQ = DTile<kCH>::kBytes, kY = 2 * DTile<kCH>::kBytes, kR = kY + DTile<kCV>::kBytes;
    static constexpr int kStage = kR + R::kRevBytes;
};

template <typename T, int NB, int NW>
__global__ __launch_bounds__(64 * NW) void delta_rev_kernel(
    const T* __restrict__ v, const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ dfinal,
    const unsigned char* __restrict__ recs, T* __restrict__ dv, float* __restrict__ dinit, DeltaKeep<T> keep,
    DeltaBack<T> back, DeltaDims d, int nslice)
{
    using C = RevCfg<T, NB, NW>;
    using R = DeltaRec<T, true>;
    constexpr int kBuf = 2;
    static_assert(kBuf * C::kStage <= 160 * 1024, "ring");
    __shared__ __attribute__((aligned(1024))) unsigned char ring[kBuf * C::kStage];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int bid = xcd_logical_block(blockIdx.x, gridDim.x);
    const int slice = bid % nslice;
    const int64_t sh = bid / nslice, s = sh / d.nheads;
    const int h = (int)(sh % d.nheads);
    const DeltaSeq sq = delta_seq(d, s);
    const int grp = h / (int)(d.nheads / d.ngroups);
    const int N = (int)d.dstate, P = (int)d.headdim;
    const int pw = 16 * NW * slice, pt = pw / 16 + wave;
    const int p = 16 * pt + r;
    const int nblk = (sq.len + kDC - 1) / kDC;
    const int valid = N * (int)sizeof(T) / 16;
    const unsigned krow = (unsigned)(d.ngroups * N * sizeof(T)), vrow = (unsigned)(d.nheads * P * sizeof(T));
    const T* kbase = Km + (sq.start * d.ngroups + grp) * N;
    const T* qbase = Qm + (sq.start * d.ngroups + grp) * N;
    const T* ybase = keep.dy + (sq.start * d.nheads + h) * P + pw;
    const unsigned char* rbase = recs + (sq.slot * d.nheads + h) * (int64_t)R::kBytes + R::kM;
    const unsigned lds0 = lds_addr(&ring[0]);

    if (valid < C::kCH) {
        for (int i = threadIdx.x; i < kBuf * 32 * C::kCH; i += 64 * NW) {
            const int row = (i / C::kCH) % 32, b = i / (32 * C::kCH), c = i % C::kCH;
            if (c >= valid) {
                unsigned char* st = ring + b * C::kStage + DTile<C::kCH>::offset(row, c);
                *reinterpret_cast<uint4*>(st + C::kK) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(st + C::kQ) = make_uint4(0, 0, 0, 0);
            }
        }
        __syncthreads();
    }
    auto issue = [&](int c) {
        const unsigned st = lds0 + (unsigned)(c % kBuf) * C::kStage;
        const int rmax = min(kDC, sq.len - c * kDC) - 1;
        const int64_t tok = (int64_t)c * kDC;
        dtile_copy<C::kCH, NW>(reinterpret_cast<const unsigned char*>(kbase) + tok * krow, krow, rmax, valid,
                               st + C::kK, wave, lane);
        dtile_copy<C::kCH, NW>(reinterpret_cast<const unsigned char*>(qbase) + tok * krow, krow, rmax, valid,
                               st + C::kQ, wave, lane);
        dtile_copy<C::kCV, NW>(reinterpret_cast<const unsigned char*>(ybase) + tok * vrow, vrow, rmax, C::kCV,
                               st + C::kY, wave, lane);
        linear_copy<R::kRevBytes, NW>(rbase + (int64_t)c * d.nheads * R::kBytes, st + C::kR, wave, lane);
    };

    f32x4 H[2 * NB];
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) {
        H[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (dfinal && 16 * t < N) {
            const float4 a = *reinterpret_cast<const float4*>(dfinal + (sh * P + p) * N + 16 * t + 4 * g);
            H[t] = f32x4{a.x, a.y, a.z, a.w};
        }
    }
    // <H, S> over this wavefront's rows at the start of chunk k (or the end)
    auto put_inner = [&](int k) {
        const int64_t as = ((s * (keep.chunks + 1) + k) * d.nheads + h) * (int64_t)P * N + (int64_t)p * N;
        float dot = 0.f;
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            if (16 * t < N) {
                const float4 a = load4f(keep.S + as + 16 * t + 4 * g);
                dot += H[t][0] * a.x + H[t][1] * a.y + H[t][2] * a.z + H[t][3] * a.w;
                if (sizeof(T) == 2) {
                    const float4 l = load4f(keep.Slo + as + 16 * t + 4 * g);
                    dot += H[t][0] * l.x + H[t][1] * l.y + H[t][2] * l.z + H[t][3] * l.w;
                }
            }
        }
        dot = group_sum<64>(dot);
        if (lane == 0) back.hs[((pt * d.seqs + s) * (keep.chunks + 1) + k) * d.nheads + h] = dot;
    };
    wait_vmem();
    if (nblk > 0) issue(nblk - 1);

    for (int c = nblk - 1; c >= 0; --c) {
        wait_vmem();
        __syncthreads();
        // this block's rows of v and its e, in the form lane = token, 4 columns
        float4 vv[2], ev[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int64_t tok = sq.start + min(c * kDC + 16 * t + r, sq.len - 1);
            vv[t] = load4f(v + (tok * d.nheads + h) * P + 16 * pt + 4 * g);
            ev[t] = load4f(keep.e + keep.frag(sq.slot + c, h, pt, d) + t * 256 + lane * 4);
        }
        if (c % 2 == 1 || c == nblk - 1) {
            const int k = c / 2;
            const int64_t at = ((s * keep.chunks + k) * d.nheads + h) * (int64_t)P * N + (int64_t)p * N;
#pragma unroll
            for (int t = 0; t < 2 * NB; ++t)
                if (16 * t < N) store4(back.H + at + 16 * t + 4 * g, H[t][0], H[t][1], H[t][2], H[t][3]);
            put_inner(k + 1);
        }
        if (c > 0) issue(c - 1);
        const unsigned char* st = ring + (c % kBuf) * C::kStage;
        const unsigned char* rec = st + C::kR - R::kM;
        const float* tab = reinterpret_cast<const float*>(rec + R::kTab);
        const int rows = min(kDC, sq.len - c * kDC);

        // dU = M^T dY + del K H^T (rows tokens, columns p)
        f32x4 kh[2], du[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) kh[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            Pair<T> hp;
            const float hv[8] = {H[2 * kb][0], H[2 * kb][1], H[2 * kb][2], H[2 * kb][3],
                                 H[2 * kb + 1][0], H[2 * kb + 1][1], H[2 * kb + 1][2], H[2 * kb + 1][3]};
            hp.set(hv);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Vec8<T> kf;
                dtile_row<C::kCH>(kf, st + C::kK, 16 * t + r, kb, g);
                mma_xp(kh[t], kf, hp);
            }
        }
        Vec8<T> yf;
        dtile_col<C::kCV>(yf, st + C::kY, 16 * wave, r, g);
        if (rows < kDC) {
            // the copies repeat the last row: rows past the sequence carry no gradient
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((i & 3) + 4 * g + (i >> 2) * 16 >= rows) yf.set(i, 0.f);
        }
        float dU[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int row = 16 * t + 4 * g + m;
                du[t][m] = row < rows ? kh[t][m] * tab[32 + row] : 0.f;
            }
            Pair<T> mt;
            rec_cols(mt, rec + R::kM, t, r, g);
            mma_px(du[t], mt, yf);
#pragma unroll
            for (int m = 0; m < 4; ++m) dU[4 * t + m] = du[t][m];
        }
        Pair<T> dup;
        dup.set(dU);
        // w = B^T dU in both forms: rows tokens (to go on with) and columns tokens (to hand out)
        float bw[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            Pair<T> bt;
            rec_cols(bt, rec + R::kB, t, r, g);
            f32x4 w = {0.f, 0.f, 0.f, 0.f}, wt = w;
            mma_pp(w, bt, dup);
            mma_pp(wt, dup, bt);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int row = 16 * t + 4 * g + m;
                bw[4 * t + m] = -tab[row] * tab[64 + row] * w[m];
            }
            store4(back.w + keep.frag(sq.slot + c, h, pt, d) + t * 256 + lane * 4, wt[0], wt[1], wt[2], wt[3]);
            float we = wt[0] * ev[t].x + wt[1] * ev[t].y + wt[2] * ev[t].z + wt[3] * ev[t].w;
            const float be = tab[64 + 16 * t + r];
            wt *= be;
            float vd = wt[0] * vv[t].x + wt[1] * vv[t].y + wt[2] * vv[t].z + wt[3] * vv[t].w;
            we += __shfl_xor(we, 16, kWave);
            vd += __shfl_xor(vd, 16, kWave);
            we += __shfl_xor(we, 32, kWave);
            vd += __shfl_xor(vd, 32, kWave);
            if (16 * t + r < rows) {
                const int64_t th = (sq.start + c * kDC + 16 * t + r) * d.nheads + h;
                store4(dv + th * P + 16 * pt + 4 * g, wt[0], wt[1], wt[2], wt[3]);
                if (g == 0) {
                    back.vdv[pt * d.tokens * d.nheads + th] = vd;
                    back.we[pt * d.tokens * d.nheads + th] = we;
                }
            }
        }
        // H before the block = gam_last H + Q^T (gam dY) - K^T (beta gam w)
        float gy[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) gy[i] = tab[(i & 3) + 4 * g + (i >> 2) * 16] * yf.get(i);
        Pair<T> gyp, bwp;
        gyp.set(gy);
        bwp.set(bw);
        const float gl = tab[31];
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            H[t] *= gl;
            Vec8<T> qf, kf;
            dtile_col<C::kCH>(qf, st + C::kQ, 16 * t, r, g);
            mma_xp(H[t], qf, gyp);
            dtile_col<C::kCH>(kf, st + C::kK, 16 * t, r, g);
            mma_xp(H[t], kf, bwp);
        }
    }
    put_inner(0);
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
        if (16 * t < N) store4(dinit + (sh * P + p) * N + 16 * t + 4 * g, H[t][0], H[t][1], H[t][2], H[t][3]);
}

// ---- dbeta and dg ---------------------------------------------------------------------------------------------

// A workgroup = two 64-token chunks x 64 heads: a wavefront sums 32 tokens, a lane one head.
__global__ __launch_bounds__(256) void delta_scalar_kernel(
    const float* __restrict__ ydy, const float* __restrict__ vdv, const float* __restrict__ we,
    const float* __restrict__ hs, float* __restrict__ dg, float* __restrict__ dbeta, DeltaDims d, int64_t chunks,
    int nseg, int hblocks, int zero_first)
{
    __shared__ double part[4][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int hb = blockIdx.x % hblocks;
    const int seg = (blockIdx.x / hblocks) % nseg;
    const int64_t s = blockIdx.x / hblocks / nseg;
    const int h = hb * 64 + lane;
    const bool live = h < d.nheads;
    const int npt = (int)d.headdim / 16;
    const int64_t TH = d.tokens * d.nheads;
    const int t0 = seg * 128 + 32 * wave;
    float loc[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        loc[i] = 0.f;
        if (live && t0 + i < d.seqlen) {
            const int64_t th = (s * d.seqlen + t0 + i) * d.nheads + h;
            float b = 0.f;
            for (int pt = 0; pt < npt; ++pt) {
                loc[i] += ydy[pt * TH + th] - vdv[pt * TH + th];
                b += we[pt * TH + th];
            }
            dbeta[th] = b;
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += loc[i];
    part[wave][lane] = sum;
    __syncthreads();
    if (!live) return;
    const int64_t k = 2 * seg + (wave >> 1);
    const int left = (int)d.seqlen - 64 * (int)k;           // tokens from the chunk's start on
    if (left <= 0) return;
    double run = 0.0, start = 0.0;
    for (int pt = 0; pt < npt; ++pt) {
        const float* at = hs + ((pt * d.seqs + s) * (chunks + 1) + k) * d.nheads + h;
        start += at[0];
        run += at[d.nheads];
    }
    const double miss = (start - run - part[wave & 2][lane] - part[(wave & 2) + 1][lane]) / min(left, 64);
    if (!(wave & 1)) {
        run += part[wave + 1][lane];
        if (left > 32) run += miss * (min(left, 64) - 32);
    }
#pragma unroll
    for (int i = 31; i >= 0; --i) {
        if (t0 + i < d.seqlen) {
            run += loc[i] + miss;
            // without an initial state nothing decays into the first token
            dg[(s * d.seqlen + t0 + i) * d.nheads + h] = zero_first && t0 + i == 0 ? 0.f : (float)run;
        }
    }
}

// ---- dq and dk ------------------------------------------------------------------------------------------------

template <typename T, int NB>
struct KqCfg {
    static constexpr int kCH = NB * 32 * (int)sizeof(T) / 16;
    static constexpr int kTile = DTile<kCH>::kBytes;               // 32 rows of S, H, K or Q
    static constexpr int kStage = 2 * kTile;
    static constexpr int kCW = kChunk * (int)sizeof(T) / 16;       // chunks of a row of W or Z
    static constexpr int kWz = 2 * DTile<kCW>::kBytes;             // W or Z: 64 rows
    static constexpr int kEpi = 2 * kTile + 2 * kWz;
    static constexpr int kRing = 2 * kStage > kEpi ? 2 * kStage : kEpi;
    static constexpr int kU = 4 * 64 * 8 * (int)sizeof(T);         // U of 64 tokens x 32 columns as fragments
};

// A workgroup = one 64-token chunk of one (row, group) and a range of the group's heads; a wavefront = 16 of the
// tokens and all N columns of dq and dk (as rows n, columns = tokens).
template <typename T, int NB>
__global__ __launch_bounds__(256) void delta_kq_kernel(
    const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ gv, const float* __restrict__ bv,
    DeltaKeep<T> keep, DeltaBack<T> back, T* __restrict__ dq, T* __restrict__ dk, float* __restrict__ partial,
    DeltaDims d, int nslice)
{
    using C = KqCfg<T, NB>;
    __shared__ __attribute__((aligned(1024))) unsigned char ring[C::kRing];
    __shared__ __attribute__((aligned(16))) unsigned char ub[2][C::kU];
    __shared__ double cst[4][64];
    __shared__ float bet[4][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int slice = blockIdx.x % nslice;
    const int grp = (blockIdx.x / nslice) % d.ngroups;
    const int64_t sk = blockIdx.x / nslice / d.ngroups, s = sk / keep.chunks;
    const int k = (int)(sk % keep.chunks);
    const int N = (int)d.dstate, P = (int)d.headdim, L = (int)d.seqlen;
    const int hpg = (int)(d.nheads / d.ngroups);
    const int h0 = grp * hpg + hpg * slice / nslice, h1 = grp * hpg + hpg * (slice + 1) / nslice;
    const int rows = min(kChunk, L - k * kChunk);
    const int nkb = (P + 31) / 32, nst = (h1 - h0) * nkb;
    const int valid = N * (int)sizeof(T) / 16;
    const int64_t t0 = s * d.seqlen + (int64_t)k * kChunk;
    const int nc32 = (L + kDC - 1) / kDC;
    const int64_t slot = s * nc32 + 2 * k + (wave >> 1);
    const bool blk = 2 * k + (wave >> 1) < nc32;              // this wavefront's block of 32 exists
    const int mine = 16 * wave + r;                           // this lane's token in operand fragments
    const bool tok = mine < rows;
    const unsigned lds0 = lds_addr(&ring[0]);

    auto zero_pad = [&](int tiles) {
        for (int i = threadIdx.x; i < tiles * 32 * C::kCH; i += 256) {
            const int c = i % C::kCH;
            if (c >= valid)
                *reinterpret_cast<uint4*>(ring + (i / (32 * C::kCH)) * C::kTile +
                                          DTile<C::kCH>::offset((i / C::kCH) % 32, c)) = make_uint4(0, 0, 0, 0);
        }
    };
    if (valid < C::kCH) {
        zero_pad(4);
        __syncthreads();
    }
    auto issue = [&](int i) {
        const int h = h0 + i / nkb, kb = i % nkb;
        const unsigned st = lds0 + (unsigned)(i & 1) * C::kStage;
        const int rmax = min(32, P - 32 * kb) - 1;
        const int64_t pn = (int64_t)P * N, off = (int64_t)32 * kb * N;
        dtile_copy<C::kCH, 4>(keep.S + ((s * (keep.chunks + 1) + k) * d.nheads + h) * pn + off,
                              (unsigned)(N * sizeof(T)), rmax, valid, st, wave, lane);
        dtile_copy<C::kCH, 4>(back.H + ((s * keep.chunks + k) * d.nheads + h) * pn + off, (unsigned)(N * sizeof(T)),
                              rmax, valid, st + C::kTile, wave, lane);
    };
    // the operands of a stage in registers: lane = token, slots = columns {4g .., 16 + 4g ..} of 32
    struct Ops { float4 y[2], e[2], w[2]; float gr, be; };
    auto fetch = [&](int i) {
        Ops o;
        const int h = h0 + i / nkb, kb = i % nkb;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            o.y[t] = o.e[t] = o.w[t] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (tok && blk && 32 * kb + 16 * t < P) {
                o.y[t] = load4f(keep.dy + ((t0 + mine) * d.nheads + h) * P + 32 * kb + 16 * t + 4 * g);
                const int64_t f = keep.frag(slot, h, 2 * kb + t, d) + (wave & 1) * 256 + lane * 4;
                o.e[t] = load4f(keep.e + f);
                o.w[t] = load4f(back.w + f);
            }
        }
        const int64_t at = (t0 + min(lane, rows - 1)) * d.nheads + h;
        o.gr = gv[at];
        o.be = bv[at];
        return o;
    };

    f32x4 aq[2 * NB], ak[2 * NB], Ws[4], Zs[4], wa[4], za[4];
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) aq[t] = ak[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t) Ws[t] = Zs[t] = wa[t] = za[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    issue(0);
    Ops cur = fetch(0);
    for (int i = 0; i < nst; ++i) {
        const int kb = i % nkb;
        if (kb == 0) {
            // the head's decays: every wavefront sums the 64 tokens' for itself, lane = token
            double cs = lane < rows ? (double)(cur.gr < -1000.f ? -1000.f : cur.gr) : 0.0;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double up = __shfl_up(cs, m, kWave);
                if (lane >= m) cs += up;
            }
            cst[wave][lane] = cs;
            bet[wave][lane] = lane < rows ? cur.be : 0.f;
        }
        const double ci = cst[wave][mine];
        const float gam = __expf((float)ci), del = __expf((float)(cst[wave][63] - ci)), be = bet[wave][mine];
        float f[8];
        const float yv[8] = {cur.y[0].x, cur.y[0].y, cur.y[0].z, cur.y[0].w, cur.y[1].x, cur.y[1].y, cur.y[1].z, cur.y[1].w};
        const float ev[8] = {cur.e[0].x, cur.e[0].y, cur.e[0].z, cur.e[0].w, cur.e[1].x, cur.e[1].y, cur.e[1].z, cur.e[1].w};
        const float wv[8] = {cur.w[0].x, cur.w[0].y, cur.w[0].z, cur.w[0].w, cur.w[1].x, cur.w[1].y, cur.w[1].z, cur.w[1].w};
        Vec8<T> yf, wf, gy, du, bw, uf;
        pack8(yf, yv);
        pack8(wf, wv);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] = gam * yv[m];
        pack8(gy, f);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] = be * ev[m];
        pack8(uf, f);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] *= del;
        pack8(du, f);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] = -be * gam * wv[m];
        pack8(bw, f);
        T* un = reinterpret_cast<T*>(ub[i & 1]) + (wave * 64 + lane) * 8;
        store8(un, uf);
        wait_vmem();
        __syncthreads();
        if (i + 1 < nst) {
            issue(i + 1);
            cur = fetch(i + 1);
        }
        const unsigned char* st = ring + (i & 1) * C::kStage;
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            Vec8<T> sf, hf;
            dtile_col<C::kCH>(sf, st, 16 * t, r, g);
            dtile_col<C::kCH>(hf, st + C::kTile, 16 * t, r, g);
            mma(aq[t], sf, gy);
            mma(ak[t], hf, du);
            mma(ak[t], sf, bw);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t <= wave) {
                Vec8<T> u;
                load8(u, reinterpret_cast<const T*>(ub[i & 1]) + (t * 64 + lane) * 8);
                mma(wa[t], yf, u);
                mma(za[t], wf, u);
            }
        }
        if (kb == nkb - 1) {
            // the head's W and Z, rows i = 16 wave + 4g + m, columns j = 16 t + r
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (t <= wave) {
                    const double cj = cst[wave][16 * t + r];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const int ri = 16 * wave + 4 * g + m, rj = 16 * t + r;
                        const float G = rj <= ri ? __expf((float)(cst[wave][ri] - cj)) : 0.f;
                        Ws[t][m] = fmaf(G, wa[t][m], Ws[t][m]);
                        Zs[t][m] = fmaf(rj < ri ? -G * bet[wave][ri] : 0.f, za[t][m], Zs[t][m]);
                    }
                    wa[t] = za[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            }
        }
    }
    __syncthreads();
    // W and Z to LDS behind the place of K's two tiles (whose pad columns are zero still): dq += W K, dk += (Z + Z^T) K, then Q in K's place: dk += W^T Q
    unsigned char* const wl = ring + 2 * C::kTile;
    unsigned char* const zl = wl + C::kWz;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int row = 16 * (wave & 1) + 4 * g + m, col = 16 * t + r;
            constexpr int kPer = 16 / (int)sizeof(T);
            const int o = (wave >> 1) * DTile<C::kCW>::kBytes + DTile<C::kCW>::offset(row, col / kPer) +
                          (col % kPer) * (int)sizeof(T);
            *reinterpret_cast<T*>(wl + o) = from_f32<T>(Ws[t][m]);
            *reinterpret_cast<T*>(zl + o) = from_f32<T>(Zs[t][m]);
        }
    }
    auto load_rows = [&](const T* m) {
        for (int b = 0; b < 2; ++b) {
            // a second half past the sequence reads the first half's last row (its weights are zero)
            const int first = min(32 * b, rows - 1), rmax = min(32, rows - first) - 1;
            dtile_copy<C::kCH, 4>(m + ((t0 + first) * d.ngroups + grp) * N, (unsigned)(d.ngroups * N * sizeof(T)), rmax,
                                  valid, lds0 + b * C::kTile, wave, lane);
        }
        wait_vmem();
        __syncthreads();
    };
    load_rows(Km);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        Vec8<T> wr, zr, zc;
        dtile_row<C::kCW>(wr, wl + (wave >> 1) * DTile<C::kCW>::kBytes, 16 * (wave & 1) + r, b, g);
        dtile_row<C::kCW>(zr, zl + (wave >> 1) * DTile<C::kCW>::kBytes, 16 * (wave & 1) + r, b, g);
        dtile_col<C::kCW>(zc, zl + b * DTile<C::kCW>::kBytes, 16 * wave, r, g);
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            Vec8<T> kf;
            dtile_col<C::kCH>(kf, ring + b * C::kTile, 16 * t, r, g);
            mma(aq[t], kf, wr);
            mma(ak[t], kf, zr);
            mma(ak[t], kf, zc);
        }
    }
    __syncthreads();
    load_rows(Qm);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        Vec8<T> wc;
        dtile_col<C::kCW>(wc, wl + b * DTile<C::kCW>::kBytes, 16 * wave, r, g);
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            Vec8<T> qf;
            dtile_col<C::kCH>(qf, ring + b * C::kTile, 16 * t, r, g);
            mma(ak[t], qf, wc);
        }
    }
    if (!tok) return;
    const int64_t at = ((t0 + mine) * d.ngroups + grp) * N + 4 * g;
    const int64_t all = d.tokens * d.ngroups * N;
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) {
        if (16 * t < N) {
            if (nslice == 1) {
                store4(dq + at + 16 * t, aq[t][0], aq[t][1], aq[t][2], aq[t][3]);
                store4(dk + at + 16 * t, ak[t][0], ak[t][1], ak[t][2], ak[t][3]);
            } else {
                float* o = partial + slice * 2 * all + at + 16 * t;
                store4(o, aq[t][0], aq[t][1], aq[t][2], aq[t][3]);
                store4(o + all, ak[t][0], ak[t][1], ak[t][2], ak[t][3]);
            }
        }
    }
}

// dq and dk from the slices' partial sums, 4 elements a thread (n4 = elements / 4 of one of the two)
template <typename T>
__global__ __launch_bounds__(256) void delta_kq_sum_kernel(const float* __restrict__ partial, T* __restrict__ dq,
                                                           T* __restrict__ dk, int64_t n4, int nslice)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < 2 * n4; i += (int64_t)gridDim.x * 256) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < nslice; ++s) {
            const float4 b = reinterpret_cast<const float4*>(partial)[s * 2 * n4 + i];
            a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
        }
        T* o = i < n4 ? dq + 4 * i : dk + 4 * (i - n4);
        store4(o, a.x, a.y, a.z, a.w);
    }
}

// ---- host -----------------------------------------------------------------------------------------------------

// Head slices of the dq, dk step: enough workgroups to fill the GPU twice, at least 2 heads each.
int kq_slices(const DeltaDims& d)
{
    const int64_t wgs = d.seqs * ((d.seqlen + kChunk - 1) / kChunk) * d.ngroups, hpg = d.nheads / d.ngroups;
    if (wgs == 0) return 1;
    const int64_t want = (512 + wgs - 1) / wgs;
    return (int)(want < hpg / 2 ? want : hpg / 2 > 1 ? hpg / 2 : 1);
}

struct BwdSpace { size_t rec, e, w, ydy, vdv, we, S, Slo, H, hs, part, total; };

BwdSpace bwd_space(const DeltaDims& d, size_t es)
{
    const size_t chunks = (d.seqlen + kChunk - 1) / kChunk, slots = delta_slots(d), heads = d.nheads;
    const size_t npt = d.headdim / 16, pn = d.headdim * d.dstate, th = (size_t)d.tokens * heads;
    const int ns = kq_slices(d);
    BwdSpace b;
    size_t at = 0;
    auto put = [&](size_t bytes) { const size_t here = at; at += (bytes + 255) / 256 * 256; return here; };
    b.rec = put(slots * heads * (es == 2 ? DeltaRec<bf16, true>::kBytes : DeltaRec<float, true>::kBytes));
    b.e = put(slots * heads * npt * 512 * 4);
    b.w = put(slots * heads * npt * 512 * es);
    b.ydy = put(npt * th * 4);
    b.vdv = put(npt * th * 4);
    b.we = put(npt * th * 4);
    b.S = put((size_t)d.seqs * (chunks + 1) * heads * pn * es);
    b.Slo = put(es == 2 ? (size_t)d.seqs * (chunks + 1) * heads * pn * es : 0);
    b.H = put((size_t)d.seqs * chunks * heads * pn * es);
    b.hs = put(npt * (size_t)d.seqs * (chunks + 1) * heads * 4);
    b.part = put(ns > 1 ? (size_t)ns * 2 * d.tokens * d.ngroups * d.dstate * 4 : 0);
    b.total = at < 256 ? 256 : at;
    return b;
}

template <typename T, int NB, int NW>
hipError_t launch_rev(const T* v, const T* k, const T* q, const float* dfinal, const unsigned char* rec, T* dv,
                      float* dinit, const DeltaKeep<T>& keep, const DeltaBack<T>& back, const DeltaDims& d,
                      hipStream_t stream)
{
    const int nslice = (int)d.headdim / (16 * NW);
    hipLaunchKernelGGL((delta_rev_kernel<T, NB, NW>), dim3((unsigned)(d.seqs * d.nheads * nslice)), dim3(64 * NW), 0,
                       stream, v, k, q, dfinal, rec, dv, dinit, keep, back, d, nslice);
    return hipGetLastError();
}

template <typename T, int NB>
hipError_t launch_nb(const T* v, const float* g, const float* beta, const T* k, const T* q, const float* dfinal,
                     const unsigned char* rec, T* dv, T* dk, T* dq, float* dinit, float* partial,
                     const DeltaKeep<T>& keep, const DeltaBack<T>& back, const DeltaDims& d, hipStream_t stream)
{
    hipError_t e;
    if (d.headdim == 16) e = launch_rev<T, NB, 1>(v, k, q, dfinal, rec, dv, dinit, keep, back, d, stream);
    else if (d.headdim == 32 || sizeof(T) * NB == 32)
        e = launch_rev<T, NB, 2>(v, k, q, dfinal, rec, dv, dinit, keep, back, d, stream);
    else if constexpr (sizeof(T) * NB < 32)
        e = launch_rev<T, NB, 4>(v, k, q, dfinal, rec, dv, dinit, keep, back, d, stream);
    else e = hipErrorInvalidValue;
    if (e != hipSuccess || d.seqlen == 0) return e;
    const int ns = kq_slices(d);
    hipLaunchKernelGGL((delta_kq_kernel<T, NB>), dim3((unsigned)(d.seqs * keep.chunks * d.ngroups * ns)), dim3(256), 0,
                       stream, k, q, g, beta, keep, back, dq, dk, partial, d, ns);
    e = hipGetLastError();
    if (e != hipSuccess || ns == 1) return e;
    const int64_t n4 = d.tokens * d.ngroups * d.dstate / 4;
    hipLaunchKernelGGL((delta_kq_sum_kernel<T>), dim3((unsigned)(2 * n4 < (1 << 22) ? (2 * n4 + 255) / 256 : 1 << 14)),
                       dim3(256), 0, stream, partial,
                       dq, dk, n4, ns);
    return hipGetLastError();
}

}  // namespace

size_t delta_backward_workspace(const DeltaDims& d, int elem_bytes) { return bwd_space(d, (size_t)elem_bytes).total; }

template <typename T>
hipError_t launch_delta_backward(const T* v, const float* g, const float* beta, const T* k, const T* q,
                                 const float* init, const T* dy, const float* dfinal, T* dv, float* dg, float* dbeta,
                                 T* dk, T* dq, float* dinit, const DeltaDims& d, void* workspace, hipStream_t stream)
{
    if (d.seqs == 0) return hipSuccess;
    const BwdSpace b = bwd_space(d, sizeof(T));
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    auto f = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    auto t = [&](size_t at) { return reinterpret_cast<T*>(ws + at); };
    const int64_t chunks = (d.seqlen + kChunk - 1) / kChunk;
    const DeltaKeep<T> keep{dy, f(b.e), f(b.ydy), t(b.S), t(b.Slo), chunks};
    const DeltaBack<T> back{t(b.w), f(b.vdv), f(b.we), t(b.H), f(b.hs)};
    hipError_t e = launch_delta_prep<T, true>(k, q, g, beta, ws + b.rec, d, stream);
    if (e == hipSuccess)
        e = launch_delta_chain<T, true>(v, k, q, init, ws + b.rec, nullptr, nullptr, keep, d, stream);
    if (e != hipSuccess) return e;
    if (d.dstate <= 32)
        e = launch_nb<T, 1>(v, g, beta, k, q, dfinal, ws + b.rec, dv, dk, dq, dinit, f(b.part), keep, back, d, stream);
    else if (d.dstate <= 64)
        e = launch_nb<T, 2>(v, g, beta, k, q, dfinal, ws + b.rec, dv, dk, dq, dinit, f(b.part), keep, back, d, stream);
    else if (d.dstate <= 128)
        e = launch_nb<T, 4>(v, g, beta, k, q, dfinal, ws + b.rec, dv, dk, dq, dinit, f(b.part), keep, back, d, stream);
    else
        e = launch_nb<T, 8>(v, g, beta, k, q, dfinal, ws + b.rec, dv, dk, dq, dinit, f(b.part), keep, back, d, stream);
    if (e != hipSuccess || d.seqlen == 0) return e;
    const int nseg = (int)((d.seqlen + 127) / 128), hblocks = (int)((d.nheads + 63) / 64);
    hipLaunchKernelGGL(delta_scalar_kernel, dim3((unsigned)(d.seqs * nseg * hblocks)), dim3(256), 0, stream, keep.ydy,
                       back.vdv, back.we, back.hs, dg, dbeta, d, chunks, nseg, hblocks, init == nullptr ? 1 : 0);
    return hipGetLastError();
}

template hipError_t launch_delta_backward<float>(const float*, const float*, const float*, const float*, const float*,
                                                 const float*, const float*, const float*, float*, float*, float*,
                                                 float*, float*, float*, const DeltaDims&, void*, hipStream_t);
template hipError_t launch_delta_backward<bf16>(const bf16*, const float*, const float*, const bf16*, const bf16*,
                                                const float*, const bf16*, const float*, bf16*, float*, float*,
                                                bf16*, bf16*, float*, const DeltaDims&, void*, hipStream_t);

}  // namespace ssd
