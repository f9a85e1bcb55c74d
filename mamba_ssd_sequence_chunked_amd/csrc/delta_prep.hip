// delta_prep.hip - the gated delta rule's per-block matrices: for every (block of 32 tokens, head)
//
//   A = (I + X diag(beta))^-1,  X_ij = G_ij (k_i . k_j) below the diagonal,  M_ij = G_ij (q_i . k_j) on and below
//
// (for the backward also B = (I + diag(beta) X)^-1) and the decay tables, written as the walks over the blocks
// read them (DeltaRec).  K K^T and Q K^T are products
// of the group, made once per workgroup on the matrix cores; a half-wavefront then does a head, lane c its
// column c.  A is found by forward substitution, row by row: x_i = [i = c] - sum_{j<i} L_ij x_j.  (Not by powers of
// L: for a block of like keys their entries grow to binomials and cancel.)  The log decays are summed and
// subtracted in 64 bits, so that a strong decay early in a block costs later pairs no digits.
#include "delta_tiles.hpp"

namespace ssd {

namespace {

constexpr int kLd = 36;                  // row pitch (floats) of a 32 x 32 matrix in LDS: rows 16-byte aligned

template <typename T>
__device__ __forceinline__ Vec8<T> load_row(const T* p, bool ok)
{
    Vec8<T> f;
    f.zero();
    if (ok) load8(f, p);
    return f;
}

// Column c of (I + L)^-1 - I, for strictly lower L in LDS (pitch kLd)
__device__ __forceinline__ void unit_lower_column(float (&x)[32], const float* L, int c)
{
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float s = i == c ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) s = fmaf(-L[i * kLd + j], x[j], s);
        x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i == c ? 0.f : x[i];
}

// Column c of a 32 x 32 matrix into a record's tile(s): T, or with kPairs a hi and a lo plane.
template <bool kPairs>
__device__ __forceinline__ void put_column(unsigned char* m, const float (&x)[32], int c, bf16)
{
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        unsigned char* at = m + WTile<4>::offset(i, c >> 3) + 2 * (c & 7);
        const bf16 hi = static_cast<bf16>(x[i]);
        *reinterpret_cast<bf16*>(at) = hi;
        if constexpr (kPairs) *reinterpret_cast<bf16*>(at + 2048) = static_cast<bf16>(x[i] - static_cast<float>(hi));
    }
}
template <bool kPairs>
__device__ __forceinline__ void put_column(unsigned char* m, const float (&x)[32], int c, float)
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        *reinterpret_cast<float*>(m + WTile<8>::offset(i, c >> 2) + 4 * (c & 3)) = x[i];
}

// kHeads heads of one group and block: a wavefront for every two
template <typename T, bool kBwd, int kHeads>
__global__ __launch_bounds__(256) void delta_prep_kernel(
    const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ gv, const float* __restrict__ bv,
    unsigned char* __restrict__ rec, DeltaDims d, int hblocks)
{
    __shared__ __attribute__((aligned(16))) float kk[32 * kLd], qk[32 * kLd];
    using R = DeltaRec<T, kBwd>;
    constexpr int kL = 32 * kLd * 4;                 // L's bytes; its place is the record's, or behind it
    constexpr int kBufBytes = kBwd ? R::kBytes + kL : R::kBytes;
    static_assert(R::kTab >= kL && kHeads == 8, "L fits in the record's matrices; four wavefronts");
    __shared__ __attribute__((aligned(16))) unsigned char buf[kHeads][kBufBytes];
    __shared__ double css[kHeads][32];
    __shared__ float tabs[kHeads][32];               // beta
    const int64_t slot = blockIdx.x / hblocks;
    const int hpg = (int)(d.nheads / d.ngroups), bpg = (hpg + kHeads - 1) / kHeads;    // head blocks of a group
    const int hb = (int)(blockIdx.x % hblocks), grp = hb / bpg, hin = (hb % bpg) * kHeads;
    const int N = (int)d.dstate;
    DeltaSeq sq;
    int blk;
    if (!delta_slot(d, slot, sq, blk)) return;
    const int rows = min(kDC, sq.len - blk * kDC);
    const int64_t t0 = sq.start + (int64_t)blk * kDC;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;

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
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            kk[(16 * ti + 4 * g + m) * kLd + 16 * tj + r] = ak[m];
            qk[(16 * ti + 4 * g + m) * kLd + 16 * tj + r] = aq[m];
        }
    }
    __syncthreads();

    const int hw = 2 * wave + (lane >> 5);       // this half-wavefront's head within the workgroup
    const int c = lane & 31;
    const bool live = hin + hw < hpg;
    const int h = grp * hpg + min(hin + hw, hpg - 1);
    unsigned char* B = buf[hw];
    float* L = reinterpret_cast<float*>(B + (kBwd ? R::kBytes : 0));
    const bool tok = c < rows;
    const int64_t at = (t0 + min(c, rows - 1)) * d.nheads + h;
    const float gr = gv[at];
    const float be = tok ? bv[at] : 0.f;
    double cs = tok ? (double)(gr < -1000.f ? -1000.f : gr) : 0.0;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const double up = __shfl_up(cs, s, 32);
        if (c >= s) cs += up;
    }
    css[hw][c] = cs;
    tabs[hw][c] = be;
    float M[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float G = __expf((float)(css[hw][i] - cs));
        const bool ok = tok && i < rows;
        M[i] = ok && i >= c ? G * qk[i * kLd + c] * (kBwd ? 1.f : be) : 0.f;
        L[i * kLd + c] = ok && i > c ? G * kk[i * kLd + c] * be : 0.f;
    }
    float x[32];
    unit_lower_column(x, L, c);
    // where L's place is the record's, its element type changes here: keep the compiler from moving accesses across
    asm volatile("" ::: "memory");
    put_column<true>(B + R::kA, x, c, T());
    put_column<kBwd>(B + R::kM, M, c, T());
    if constexpr (kBwd) {
        asm volatile("" ::: "memory");
        // rows scaled instead of columns
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float G = __expf((float)(css[hw][i] - cs));
            L[i * kLd + c] = tok && i < rows && i > c ? G * kk[i * kLd + c] * tabs[hw][i] : 0.f;
        }
        asm volatile("" ::: "memory");
        unit_lower_column(x, L, c);
        put_column<true>(B + R::kB, x, c, T());
    }
    float* tab = reinterpret_cast<float*>(B + R::kTab);
    tab[c] = __expf((float)cs);
    tab[32 + c] = __expf((float)(css[hw][31] - cs)) * (kBwd ? 1.f : be);
    tab[64 + c] = be;
    tab[96 + c] = 0.f;
    asm volatile("" ::: "memory");
    if (live) {
        unsigned char* out = rec + (slot * d.nheads + h) * (int64_t)R::kBytes;
#pragma unroll
        for (int o = 0; o < R::kBytes; o += 512)
            *reinterpret_cast<uint4*>(out + o + 16 * c) = *reinterpret_cast<const uint4*>(B + o + 16 * c);
    }
}

}  // namespace

template <typename T, bool kBwd>
hipError_t launch_delta_prep(const T* k, const T* q, const float* g, const float* beta, unsigned char* rec,
                             const DeltaDims& d, hipStream_t stream)
{
    constexpr int kHeads = 8;
    const int64_t hpg = d.nheads / d.ngroups, hblocks = d.ngroups * ((hpg + kHeads - 1) / kHeads);
    const int64_t nblocks = delta_slots(d) * hblocks;
    if (nblocks == 0) return hipSuccess;
    hipLaunchKernelGGL((delta_prep_kernel<T, kBwd, kHeads>), dim3((unsigned)nblocks), dim3(256), 0, stream, k, q, g,
                       beta, rec, d, (int)hblocks);
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
