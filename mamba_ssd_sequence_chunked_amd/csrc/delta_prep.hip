// delta_prep.hip - the gated delta rule's per-block matrices: for every (block of 32 tokens, head)
//
//   A = (I + X diag(beta))^-1,  X_ij = G_ij (k_i . k_j) below the diagonal,  M_ij = G_ij (q_i . k_j) on and below
//
// and the decay tables, written as the walk over the blocks reads them (DeltaRec).  K K^T and Q K^T are products
// of the group, made once per workgroup on the matrix cores; a half-wavefront then does a head, lane c its
// column c.  A is found by forward substitution, row by row: x_i = [i = c] - sum_{j<i} L_ij x_j.  (Not by powers of
// L: for a block of like keys their entries grow to binomials and cancel.)  The log decays are summed and
// subtracted in 64 bits, so that a strong decay early in a block costs later pairs no digits.
#include "delta_tiles.hpp"

namespace ssd {

namespace {

constexpr int kHeads = 8;                // heads of a workgroup: 4 wavefronts, 2 heads each
constexpr int kLd = 36;                  // row pitch (floats) of a 32 x 32 matrix in LDS: rows 16-byte aligned

template <typename T>
__device__ __forceinline__ Vec8<T> load_row(const T* p, bool ok)
{
    Vec8<T> f;
    f.zero();
    if (ok) load8(f, p);
    return f;
}

template <typename T>
__global__ __launch_bounds__(256) void delta_prep_kernel(
    const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ gv, const float* __restrict__ bv,
    unsigned char* __restrict__ rec, DeltaDims d, int hblocks)
{
    __shared__ __attribute__((aligned(16))) float kk[32 * kLd], qk[32 * kLd];
    __shared__ __attribute__((aligned(16))) unsigned char buf[kHeads][DeltaRec<T>::kTab];
    __shared__ double css[kHeads][32];
    static_assert(DeltaRec<T>::kTab >= 32 * kLd * 4, "L shares the record's buffer");
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
    float* L = reinterpret_cast<float*>(buf[hw]);
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
    float M[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float G = __expf((float)(css[hw][i] - cs));
        const bool ok = tok && i < rows;
        M[i] = ok && i >= c ? G * qk[i * kLd + c] : 0.f;
        L[i * kLd + c] = ok && i > c ? G * kk[i * kLd + c] * be : 0.f;
    }
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float s = i == c ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) s = fmaf(-L[i * kLd + j], x[j], s);
        x[i] = s;
    }
    // the buffer changes its element type here and below: keep the compiler from moving accesses across
    asm volatile("" ::: "memory");
    // into the record's fragments: row i = 16 t + r', column c = slot s of lane group g'
    const int gc = (c & 15) >> 2, sc = (c & 3) + (c >= 16 ? 4 : 0);
    unsigned char* B = buf[hw];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int ln = (i >> 4) * 64 + 16 * gc + (i & 15);
        if constexpr (sizeof(T) == 2) {
            const bf16 hi = static_cast<bf16>(x[i]);
            reinterpret_cast<bf16*>(B)[ln * 8 + sc] = hi;
            reinterpret_cast<bf16*>(B + 2048)[ln * 8 + sc] = static_cast<bf16>(x[i] - static_cast<float>(hi));
            reinterpret_cast<bf16*>(B + 4096)[ln * 8 + sc] = static_cast<bf16>(M[i]);
        } else {
            reinterpret_cast<float*>(B + (sc >> 2) * 2048)[ln * 4 + (sc & 3)] = x[i];
            reinterpret_cast<float*>(B + 4096 + (sc >> 2) * 2048)[ln * 4 + (sc & 3)] = M[i];
        }
    }
    asm volatile("" ::: "memory");
    if (live) {
        unsigned char* out = rec + (slot * d.nheads + h) * (int64_t)DeltaRec<T>::kBytes;
#pragma unroll
        for (int o = 0; o < DeltaRec<T>::kTab; o += 512)
            *reinterpret_cast<uint4*>(out + o + 16 * c) = *reinterpret_cast<const uint4*>(B + o + 16 * c);
        float* tab = reinterpret_cast<float*>(out + DeltaRec<T>::kTab);
        tab[c] = __expf((float)cs);
        tab[32 + c] = __expf((float)(css[hw][31] - cs));
        tab[64 + c] = be;
    }
}

}  // namespace

template <typename T>
hipError_t launch_delta_prep(const T* k, const T* q, const float* g, const float* beta, unsigned char* rec,
                             const DeltaDims& d, hipStream_t stream)
{
    const int64_t hpg = d.nheads / d.ngroups, hblocks = d.ngroups * ((hpg + kHeads - 1) / kHeads);
    const int64_t nblocks = delta_slots(d) * hblocks;
    if (nblocks == 0) return hipSuccess;
    hipLaunchKernelGGL((delta_prep_kernel<T>), dim3((unsigned)nblocks), dim3(256), 0, stream, k, q, g, beta, rec, d,
                       (int)hblocks);
    return hipGetLastError();
}

template hipError_t launch_delta_prep<float>(const float*, const float*, const float*, const float*, unsigned char*,
                                             const DeltaDims&, hipStream_t);
template hipError_t launch_delta_prep<bf16>(const bf16*, const bf16*, const float*, const float*, unsigned char*,
                                            const DeltaDims&, hipStream_t);

}  // namespace ssd
