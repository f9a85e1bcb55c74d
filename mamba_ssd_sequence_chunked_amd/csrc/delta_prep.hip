// delta_prep.hip - the gated delta rule's per-block matrices: for every (block of 32 tokens, head)
//
//   A = (I + X diag(beta))^-1,  X_ij = G_ij (k_i . k_j) below the diagonal,  M_ij = G_ij (q_i . k_j) on and below
//
// (for the backward also B = (I + diag(beta) X)^-1) and the decay tables, written as the walks over the blocks
// read them (DeltaRec).
//
// K K^T and Q K^T are products of the group, made once per workgroup on the matrix cores. A wavefront then takes
// two heads at a time. With 16 x 16 blocks, (I + L)^-1 = [[A1, 0], [-A2 L21 A1, A2]]: the diagonal blocks by back
// substitution, a lane one row y (y_j = [j = row] - sum_{k>j} y_k L_kj; 2 heads x 2 blocks x 16 rows fill the
// wavefront), the corner by eight fp32 matrix instructions.  (Not by powers of L: for a block of like keys their
// entries grow to binomials and cancel.)  The log decays are summed and subtracted in 64 bits, so that a strong
// decay early in a block costs later pairs no digits.
//
// Bound by the records' bytes and by the substitutions' chain of 16 dependent rows: 4 x 4096 tokens, 80 heads
// (bf16, N = 128) 85 us for 273 MB of records, 145 us for the backward's 524 MB. Forward substitution of whole 32 x 32
// matrices took 140 us and 370.
#include "delta_tiles.hpp"

namespace ssd {

namespace {

constexpr int kHeads = 16;               // heads of a workgroup (of one group): 4 wavefronts x 2 x 2
constexpr int kLd = 36;                  // row pitch (floats) of a 32 x 32 matrix in LDS: 16 rows at a column of 4
                                         //   fall in different banks

template <typename T>
__device__ __forceinline__ Vec8<T> load_row(const T* p, bool ok)
{
    Vec8<T> f;
    f.zero();
    if (ok) load8(f, p);
    return f;
}

// Row i's columns j0 .. j0 + 3 (j0 a multiple of 4) or j0 .. j0 + 15 (of 16) of a record's matrix; kPairs: hi and lo.
template <bool kPairs>
__device__ __forceinline__ void put4(unsigned char* m, int i, int j0, const float (&v)[4], bf16)
{
    unsigned char* at = m + WTile<4>::offset(i, j0 >> 3) + 2 * (j0 & 7);
    store4(reinterpret_cast<bf16*>(at), v[0], v[1], v[2], v[3]);
    if constexpr (kPairs) {
        float lo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) lo[q] = v[q] - static_cast<float>(static_cast<bf16>(v[q]));
        store4(reinterpret_cast<bf16*>(at + 2048), lo[0], lo[1], lo[2], lo[3]);
    }
}
template <bool kPairs>
__device__ __forceinline__ void put4(unsigned char* m, int i, int j0, const float (&v)[4], float)
{
    store4(reinterpret_cast<float*>(m + WTile<8>::offset(i, j0 >> 2)), v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void put16(unsigned char* m, int i, int j0, const float (&v)[16], bf16)
{
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float e[8] = {v[8 * c], v[8 * c + 1], v[8 * c + 2], v[8 * c + 3], v[8 * c + 4], v[8 * c + 5], v[8 * c + 6], v[8 * c + 7]};
        Pair<bf16> f;
        f.set(e);
        unsigned char* at = m + WTile<4>::offset(i, (j0 >> 3) + c);
        store8(reinterpret_cast<bf16*>(at), f.hi);
        store8(reinterpret_cast<bf16*>(at + 2048), f.lo);
    }
}
__device__ __forceinline__ void put16(unsigned char* m, int i, int j0, const float (&v)[16], float)
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
        store4(reinterpret_cast<float*>(m + WTile<8>::offset(i, (j0 >> 2) + c)), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

// (I + L)^-1 - I of two heads into their records' matrix m0 / m1 (null: not wanted). lt: L^T of both (32 x kLd each),
// of which the diagonal blocks are overwritten.
template <typename T>
__device__ __forceinline__ void unit_lower_inverse(float* lt, unsigned char* m0, unsigned char* m1, int lane)
{
    const int g = lane >> 4, r = lane & 15, hh = lane >> 5, blk = g & 1;
    float* d = lt + hh * 32 * kLd + 16 * blk * kLd + 16 * blk;       // this lane's diagonal block
    float y[16];
#pragma unroll
    for (int j = 15; j >= 0; --j) {
        float s = j == r ? 1.f : 0.f;
#pragma unroll
        for (int k4 = (j + 1) & ~3; k4 < 16; k4 += 4) {
            const f32x4 l = *reinterpret_cast<const f32x4*>(d + j * kLd + k4);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (k4 + q > j) s = fmaf(-l[q], y[k4 + q], s);
        }
        y[j] = s;
    }
    // (a wavefront's LDS accesses are served in order)
#pragma unroll
    for (int c = 0; c < 4; ++c) *reinterpret_cast<f32x4*>(d + r * kLd + 4 * c) = f32x4{y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]};
    unsigned char* const m = hh ? m1 : m0;
    if (m) {
        float z[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = j == r ? 0.f : y[j];
        put16(m, 16 * blk + r, 16 * blk, z, T());
        if (blk == 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = 0.f;
            put16(m, r, 16, z, T());
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        // (A2 L21)^T (rows j, columns i), then (A2 L21 A1)^T; contraction index 4g + q in both
        const float* t = lt + e * 32 * kLd;
        const f32x4 l21 = *reinterpret_cast<const f32x4*>(t + r * kLd + 16 + 4 * g);
        const f32x4 a2 = *reinterpret_cast<const f32x4*>(t + (16 + r) * kLd + 16 + 4 * g);
        f32x4 w = {0.f, 0.f, 0.f, 0.f}, x = w;
#pragma unroll
        for (int q = 0; q < 4; ++q) w = __builtin_amdgcn_mfma_f32_16x16x4f32(l21[q], a2[q], w, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) x = __builtin_amdgcn_mfma_f32_16x16x4f32(t[(4 * g + q) * kLd + r], w[q], x, 0, 0, 0);
        settle();
        const float v[4] = {-x[0], -x[1], -x[2], -x[3]};
        unsigned char* const me = e ? m1 : m0;
        if (me) put4<true>(me, 16 + r, 4 * g, v, T());
    }
}

template <typename T, bool kBwd>
__global__ __launch_bounds__(256) void delta_prep_kernel(
    const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ gv, const float* __restrict__ bv,
    unsigned char* __restrict__ rec, DeltaDims d, int hblocks)
{
    using R = DeltaRec<T, kBwd>;
    __shared__ __attribute__((aligned(16))) float kk[32 * kLd], qk[32 * kLd];
    __shared__ __attribute__((aligned(16))) float lts[4][2 * 32 * kLd];
    __shared__ __attribute__((aligned(16))) double css[4][2][32];
    __shared__ __attribute__((aligned(16))) float bes[4][2][32];
    const int64_t slot = blockIdx.x / hblocks;
    const int hpg = (int)(d.nheads / d.ngroups), bpg = (hpg + kHeads - 1) / kHeads;    // head blocks of a group
    const int hb = (int)(blockIdx.x % hblocks), grp = hb / bpg, hin = (hb % bpg) * kHeads;
    const int N = (int)d.dstate;
    DeltaSeq sq;
    int blk;
    if (!delta_slot(d, slot, sq, blk)) return;
    const int rows = min(kDC, sq.len - blk * kDC);
    const int64_t t0 = sq.start + (int64_t)blk * kDC;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;

    // K K^T and Q K^T: wavefront w makes 16 x 16 tile (w / 2, w % 2) of both
    {
        const int ti = wave >> 1, tj = wave & 1;
        f32x4 ak = {0.f, 0.f, 0.f, 0.f}, aq = ak;
        if (tj <= ti) {
            const int64_t pitch = d.ngroups * N;
            const T* ki = Km + (t0 + min(16 * ti + r, rows - 1)) * pitch + grp * N;
            const T* qi = Qm + (t0 + min(16 * ti + r, rows - 1)) * pitch + grp * N;
            const T* kj = Km + (t0 + min(16 * tj + r, rows - 1)) * pitch + grp * N;
            for (int n = 8 * g; n < ((N + 31) & ~31); n += 32) {
                const bool ok = n < N;
                const Vec8<T> a = load_row(ki + n, ok), q = load_row(qi + n, ok), b = load_row(kj + n, ok);
                mma(ak, a, b);
                mma(aq, q, b);
            }
            settle();                                     // they are read behind the branch
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            kk[(16 * ti + 4 * g + m) * kLd + 16 * tj + r] = ak[m];
            qk[(16 * ti + 4 * g + m) * kLd + 16 * tj + r] = aq[m];
        }
    }
    __syncthreads();

    float* const lt = lts[wave];
    for (int pair = wave; 2 * pair < kHeads && hin + 2 * pair < hpg; pair += 4) {
        const int h0 = grp * hpg + hin + 2 * pair;
        const bool second = hin + 2 * pair + 1 < hpg;
        unsigned char* const out0 = rec + (slot * d.nheads + h0) * (int64_t)R::kBytes;
        unsigned char* const out1 = second ? out0 + R::kBytes : nullptr;
        {
            // the two heads' decays, a half-wavefront each, lane c = token
            const int hh = lane >> 5, c = lane & 31;
            const bool tok = c < rows;
            const int64_t at = (t0 + min(c, rows - 1)) * d.nheads + h0 + (second ? hh : 0);
            const float gr = gv[at];
            const float be = tok ? bv[at] : 0.f;
            double cs = tok ? (double)(gr < -1000.f ? -1000.f : gr) * 1.4426950408889634 : 0.0;     // base 2 from here
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const double up = __shfl_up(cs, s, 32);
                if (c >= s) cs += up;
            }
            css[wave][hh][c] = cs;
            bes[wave][hh][c] = be;
            unsigned char* const out = hh ? out1 : out0;
            if (out) {
                float* tab = reinterpret_cast<float*>(out + R::kTab);
                tab[c] = __builtin_amdgcn_exp2f((float)cs);
                tab[32 + c] = __builtin_amdgcn_exp2f((float)(css[wave][hh][31] - cs)) * (kBwd ? 1.f : be);
                tab[64 + c] = be;
            }
        }
        // X of both heads (columns i = 16 I + r a lane, rows j = 16 J + 4g + m), L^T to LDS, M out
        float X[2][3][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            unsigned char* const out = e ? out1 : out0;
#pragma unroll
            for (int J = 0; J < 2; ++J) {
                double cj[4];
                f32x4 bj = *reinterpret_cast<const f32x4*>(&bes[wave][e][16 * J + 4 * g]);
#pragma unroll
                for (int m = 0; m < 4; ++m) cj[m] = css[wave][e][16 * J + 4 * g + m];
#pragma unroll
                for (int I = 0; I < 2; ++I) {
                    const int i = 16 * I + r;
                    float M[4] = {0.f, 0.f, 0.f, 0.f};
                    if (I >= J) {
                        const double ci = css[wave][e][i];
                        const f32x4 k4 = *reinterpret_cast<const f32x4*>(&kk[i * kLd + 16 * J + 4 * g]);
                        const f32x4 q4 = *reinterpret_cast<const f32x4*>(&qk[i * kLd + 16 * J + 4 * g]);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const int j = 16 * J + 4 * g + m;
                            const float G = __builtin_amdgcn_exp2f((float)(ci - cj[m]));
                            const bool in = i < rows && j < rows;
                            M[m] = in && (kBwd ? i > j : i >= j) ? G * q4[m] * (kBwd ? 1.f : bj[m]) : 0.f;
                            if constexpr (kBwd) {
                                if (i == j && out) reinterpret_cast<float*>(out + R::kTab)[96 + i] = in ? q4[m] : 0.f;
                            }
                            X[e][I + J][m] = in && i > j ? G * k4[m] : 0.f;
                            lt[e * 32 * kLd + j * kLd + i] = X[e][I + J][m] * bj[m];
                        }
                    }
                    if (out) put4<kBwd>(out + R::kM, i, 16 * J + 4 * g, M, T());
                }
            }
        }
        unit_lower_inverse<T>(lt, out0 + R::kA, out1 ? out1 + R::kA : nullptr, lane);
        if constexpr (kBwd) {
            // the rows scaled instead of the columns
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const int I = (t + 1) / 2, J = t / 2, i = 16 * I + r;
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        lt[e * 32 * kLd + (16 * J + 4 * g + m) * kLd + i] = X[e][t][m] * bes[wave][e][i];
                }
            }
            unit_lower_inverse<T>(lt, out0 + R::kB, out1 ? out1 + R::kB : nullptr, lane);
        }
    }
}

}  // namespace

template <typename T, bool kBwd>
hipError_t launch_delta_prep(const T* k, const T* q, const float* g, const float* beta, unsigned char* rec,
                             const DeltaDims& d, hipStream_t stream)
{
    const int64_t hpg = d.nheads / d.ngroups, hblocks = d.ngroups * ((hpg + kHeads - 1) / kHeads);
    const int64_t nblocks = delta_slots(d) * hblocks;
    if (nblocks == 0) return hipSuccess;
    hipLaunchKernelGGL((delta_prep_kernel<T, kBwd>), dim3((unsigned)nblocks), dim3(256), 0, stream, k, q, g, beta, rec,
                       d, (int)hblocks);
    return hipGetLastError();
}

#define SSD_DELTA_PREP(T, BWD)                                                                                       \
    template hipError_t launch_delta_prep<T, BWD>(const T*, const T*, const float*, const float*, unsigned char*,    \
                                                  const DeltaDims&, hipStream_t);
SSD_DELTA_PREP(float, false)
SSD_DELTA_PREP(float, true)
SSD_DELTA_PREP(bf16, false)
SSD_DELTA_PREP(bf16, true)
#undef SSD_DELTA_PREP

}  // namespace ssd
