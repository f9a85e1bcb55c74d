// linear.hip - linear attention with a decay for each head: the forward and the backward as walks (linear_walk.hpp), and
// the small kernels between and behind them.
//
// The forward is one walk.  The backward is three: dq forwards, with the sums of dg; dk and dv backwards, both in one
// launch.  Keys' and values' gradients that heads share are kept of every head in fp32 and added up by a kernel of their own (80
// heads of 64 x 256 in 8 groups, 4 x 4096 tokens: 1.7 GB written and read again, the sums alone 315 of 2060 us).
// Where there are fewer walks than the GPU holds, rows are cut into segments: a first pass leaves what
// every segment but the last adds to the state, linear_join_kernel turns that into the states that enter them, and the
// walk runs over all segments at once.  Where there are a few too many, segments follow each other in a chain (see
// linear_cut).
#include <algorithm>

#include "linear_walk.hpp"

namespace ssd {

namespace {

// What enters every segment, from what each adds (loc, in place; with dloc the derivative for g too; loc2 where two
// walks are joined).  A thread has 4 elements of a row and head and goes along the row.
//   S_0 = init;  S_{i+1} = a^len S_i + loc_i;   S'_0 = 0;  S'_{i+1} = a^len (S'_i + len S_i) + dloc_i
template <bool kDg>
__global__ __launch_bounds__(256) void linear_join_kernel(float* __restrict__ loc, float* __restrict__ loc2,
                                                          float* __restrict__ dloc, const float* __restrict__ init,
                                                          const float* __restrict__ g, DeltaDims d, int64_t seg,
                                                          bool back, int64_t PN)
{
    if (blockIdx.y > 0) loc = loc2;
    const int64_t quads = PN / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= d.seqs * d.nheads * quads) return;
    const int64_t at = 4 * (i % quads), rh = i / quads, h = rh % d.nheads, row = rh / d.nheads;
    int64_t first, n;
    if (d.cu) {
        const int64_t begin = linear_offset(d, row), end = max(linear_offset(d, row + 1), begin);
        first = begin / seg + row;
        n = end - begin;
    } else {
        first = row * max((d.seqlen + seg - 1) / seg, (int64_t)1);
        n = d.seqlen;
    }
    const int64_t count = max((n + seg - 1) / seg, (int64_t)1);
    const float gl = linear_rate(g[h]);
    LinearDecay decay;
    decay.set(gl, (int)min(seg, n));
    f32x4 s = {0.f, 0.f, 0.f, 0.f}, ds = {0.f, 0.f, 0.f, 0.f};
    if (init) s = *reinterpret_cast<const f32x4*>(init + rh * PN + at);
    // (a few segments' loads at a time, since one after another each waits for memory: 4096 tokens of 4 heads of 64 x 128,
    // 16 segments, 32 us, 35 one by one; of 80 heads, 6 segments, 83 and 82)
    constexpr int kAhead = 4;
    for (int64_t c0 = 0; c0 < count; c0 += kAhead) {
        f32x4 add[kAhead], dadd[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t c = c0 + i, to = ((first + (back ? count - 1 - c : c)) * d.nheads + h) * PN + at;
            add[i] = dadd[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (c + 1 < count) {                                   // (nothing is left there for the last)
                add[i] = *reinterpret_cast<const f32x4*>(loc + to);
                if constexpr (kDg) dadd[i] = *reinterpret_cast<const f32x4*>(dloc + to);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t c = c0 + i, k = back ? count - 1 - c : c, len = min(seg, n - k * seg);
            const int64_t to = ((first + k) * d.nheads + h) * PN + at;
            if (c < count) {
                *reinterpret_cast<f32x4*>(loc + to) = s;
                if constexpr (kDg) *reinterpret_cast<f32x4*>(dloc + to) = ds;
            }
            const float a = len == min(seg, n) ? decay.next() : linear_power(gl, (float)len);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if constexpr (kDg) ds[m] = fmaf(fmaf((float)len, s[m], ds[m]), a, dadd[i][m]);
                s[m] = fmaf(s[m], a, add[i][m]);
            }
        }
    }
}

// dg of a head: the walks' sums in a fixed order, in 64 bits.
__global__ __launch_bounds__(256) void linear_dg_kernel(const float* __restrict__ part, float* __restrict__ dg,
                                                        int64_t items, int64_t nheads, int parts)
{
    __shared__ double sums[256];
    const int64_t h = blockIdx.x;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < items * parts; i += 256) s += part[((i / parts) * nheads + h) * parts + i % parts];
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int n = 128; n > 0; n >>= 1) {
        if ((int)threadIdx.x < n) sums[threadIdx.x] += sums[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0) dg[h] = (float)sums[0];
}

// The gradient of a shared key or value: the sum of its heads' in their order, rounded once.
template <typename T>
__global__ __launch_bounds__(256) void linear_group_kernel(const float* __restrict__ part, T* __restrict__ out,
                                                           int64_t rows, int share, int width)
{
    const int64_t quads = width / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * quads) return;
    const int64_t row = i / quads, at = 4 * (i % quads);
    const float* from = part + row * share * width + at;
    f32x4 s = *reinterpret_cast<const f32x4*>(from);
    for (int m = 1; m < share; ++m) s += *reinterpret_cast<const f32x4*>(from + (int64_t)m * width);
    store4(out + row * width + at, s[0], s[1], s[2], s[3]);
}

unsigned blocks_of(int64_t threads) { return (unsigned)((threads + 255) / 256); }

size_t bytes_up(int64_t floats) { return ((size_t)floats * 4 + 255) / 256 * 256; }

int64_t state_floats(const DeltaDims& d, int64_t items) { return items * d.nheads * d.headdim * d.dstate; }

// How the rows of a walk are run: whole, cut into segments that walk at once (with a pass before), or in a chain.
struct Cut {
    int64_t seg;
    bool chain, alone;       // alone: the chain's workgroups have a CU each
};

__global__ __launch_bounds__(256) void linear_zero_kernel(unsigned* p, int64_t n, unsigned* p2, int64_t n2)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0;
    else if (i - n < n2) p2[i - n] = 0;
}

// Bytes of workspace for one walk: the items' states (dg: twice that), or a chain's counters and states.
size_t walk_bytes(const DeltaDims& d, const Cut& c, int elem_bytes, bool dg, int64_t Dk, int64_t Dv)
{
    if (c.seg == kWholeRows) return 0;
    const int64_t columns = linear_columns(elem_bytes, (int)Dv), walks = d.seqs * d.nheads * ((Dv + columns - 1) / columns);
    if (c.chain) return bytes_up(walks + 1) + bytes_up(d.seqs * d.nheads * linear_handed(elem_bytes, dg, Dk, Dv));
    return (dg ? 2 : 1) * bytes_up(state_floats(d, linear_items(d, c.seg)));
}

template <bool kOut, bool kDg, typename T> hipError_t launch(LinearWalk<T> (&p)[1], hipStream_t stream)
{
    return launch_linear_walk<T, kOut, kDg>(p[0], stream);
}
template <bool kOut, bool kDg, typename T> hipError_t launch(LinearWalk<T> (&p)[2], hipStream_t stream)
{
    static_assert(!kDg);
    return launch_linear_twin<T, kOut>(p[0], p[1], stream);
}

// The walk, or two that the same states enter, or where rows are cut their steps.
template <bool kDg, typename T, int N>
hipError_t walk(LinearWalk<T> (&p)[N], const Cut& c, const float* enter, float* const (&room)[N], hipStream_t stream)
{
    for (LinearWalk<T>& w : p) {
        w.seg = c.seg;
        w.enter = enter;
        w.denter = nullptr;
        w.by_item = false;
        w.ticket = nullptr;
    }
    const DeltaDims& d = p[0].d;
    if (c.seg != kWholeRows && c.chain) {
        int64_t words[2] = {0, 0};
        for (int i = 0; i < N; ++i) {
            const int64_t columns = linear_columns(sizeof(T), p[i].Dv);
            words[i] = d.seqs * d.nheads * ((p[i].Dv + columns - 1) / columns) + 1;
            p[i].ticket = reinterpret_cast<unsigned*>(room[i]);
            p[i].done = p[i].ticket + 1;
            p[i].handed = room[i] + bytes_up(words[i]) / 4;
            p[i].alone = c.alone;
        }
        hipLaunchKernelGGL(linear_zero_kernel, dim3(blocks_of(words[0] + words[1])), dim3(256), 0, stream, p[0].ticket, words[0],
                           p[N - 1].ticket, words[1]);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    } else if (c.seg != kWholeRows) {
        const int64_t PN = d.headdim * d.dstate;
        LinearWalk<T> first[N];
        for (int i = 0; i < N; ++i) {
            first[i] = p[i];
            first[i].fin = room[i];
            first[i].dfin = kDg ? room[i] + bytes_up(state_floats(d, linear_items(d, c.seg))) / 4 : nullptr;
            p[i].enter = first[i].fin;
            p[i].denter = first[i].dfin;
            p[i].by_item = true;
        }
        hipError_t e = launch<false, kDg>(first, stream);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((linear_join_kernel<kDg>), dim3(blocks_of(d.seqs * d.nheads * PN / 4), N), dim3(256), 0, stream,
                           first[0].fin, first[N - 1].fin, first[0].dfin, enter, p[0].g, d, c.seg, p[0].back, PN);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return launch<true, kDg>(p, stream);
}

// A workgroup walks one slice of a row and head.  Measured with heads of 64 x 128 over 4096 tokens in bf16, where one row
// alone takes a CU 175 us, two on one 332:
//  - fewer walks than CUs: rows are cut into segments that walk at once, for a pass over K and V and two launches more, if
//    that is less than a whole row's chunks take one after another (128 walks: 117 us, whole 139).
//  - some more than CUs: a few CUs would have one more than the others from the first token to the last. In a chain
//    a row's segments go to whichever CU is free (forward of 320 walks 240 us, whole 274; 384: 264, 282; 640: 442, 513; 768:
//    525, 558; a backward of three launches of 320: 855, 1056). Not where nearly all CUs have two (448: 330, 305), nor for
//    fewer tokens than the starts are worth. Two workgroups share a CU from 512 walks on (heads of 64 x 256, 640 walks: 575, alone
//    683; the backward's two launches together 843, 854, then with pairs towards dg); fewer rows do not keep two busy, since segments behind their row's
//    first one wait (the backward of 160 heads of 128 x 128: 787, not alone 843). As many segments as leave the fewest
//    CUs idle at the end (288 walks: 2 take 243, 3 229, 4 229; 352: 256, 287, 277; 576: 430, 414, 412). Towards dg, where two on a
//    CU take as long as one after the other, a CU counts once (the backward of 640: 2 take 1594, 4 1645), and in fp32.
//  - rows of different lengths: the same, in pieces of 1024 tokens (20 of up to 1000, 13 heads of 128 x 128: 59 us, cut at
//    once 102; 7 of 64 to 4096, 80 heads: 230, 346; only 336 walks of 4096 tokens and 256 rows of state are slower, 318, 286).
//    Whole where they are short, 384 tokens on average: a chain's workgroups have a CU each, and so little to walk is
//    mostly waiting for a first chunk, which two on a CU share (37 of up to 150, 16 heads of 128 x 128: 34 us, in a chain
//    45; averages of 300 70, 78; of 500 111, 105). In fp32, where one fills a CU, 192 (400 walks of 150 on average: 72, 81; of
//    300 166, 147). With many walks all CUs are busy in any case (2048: 141, whole 128).
//    Few walks are cut at once, since one long row would walk alone, but into three at least, as above.
constexpr double kStartsUs = 9;      // what two launches more take
constexpr double kStartChunks = 3;   // a segment's start in a chain, in chunks
Cut linear_cut(const DeltaDims& d, int64_t slices, double chunk_us, int64_t least_chunks, int64_t brief, bool one)
{
    constexpr int64_t kCUs = 256, kLeast = 256;
    const int64_t walks = d.seqs * d.nheads * slices, over = walks % (2 * kCUs);
    Cut c{kWholeRows, false, false};
    if (d.cu) {
        if (walks >= 4 * kCUs || (d.tokens <= brief * d.seqs && walks > kCUs)) return c;
        c.chain = c.alone = walks > kCUs && d.seqs <= kChainRows;
        c.seg = c.chain ? 1024 : std::max<int64_t>(2 * kLeast, d.tokens * d.nheads * slices / (4 * kCUs));
    } else if (walks < kCUs) {
        const int64_t chunks = (d.seqlen + kLC - 1) / kLC;
        const int64_t n = walks > 0 ? std::min<int64_t>(2 * kCUs / walks, chunks / least_chunks) : 1;
        if (n <= 2 || chunks * chunk_us * (n - 2) / n < kStartsUs) return c;
        c.seg = (d.seqlen + n - 1) / n;
    } else if (walks > kCUs && walks < 4 * kCUs && over > 0 && over <= 3 * kCUs / 2 && d.seqlen >= 8 * kLeast) {
        c.chain = true;
        c.alone = walks < 2 * kCUs;
        const int64_t slots = c.alone || one ? kCUs : 2 * kCUs;
        int64_t n = 2;
        double least = 0;
        for (int64_t i = 2; i <= 4; ++i) {
            const double took = (double)((walks * i + slots - 1) / slots) * (1. / i + kStartChunks * kLC / d.seqlen);
            if (i == 2 || took < least) { least = took; n = i; }
        }
        c.seg = (d.seqlen + n - 1) / n;
    } else {
        return c;
    }
    c.seg = (c.seg + 63) / 64 * 64;
    if (d.cu ? d.tokens <= (c.chain ? 1 : 2) * c.seg : d.seqlen <= c.seg) return Cut{kWholeRows, false, false};
    return c;
}

// What a chunk takes a walk that runs alone: fp32's matrix products are a sixteenth of bf16's rate, and take it per 32
// rows of the state.
double chunk_us(int elem_bytes, bool dg, int64_t Dk) { return (elem_bytes == 2 ? 0.8 + Dk / 512. : 1 + Dk / 34.) * (dg ? 1.6 : 1); }
int64_t least_chunks(int elem_bytes) { return elem_bytes == 2 ? 8 : 2; }
int64_t brief_tokens(int elem_bytes) { return elem_bytes == 2 ? 384 : 192; }

Cut walk_cut(const DeltaDims& d, int elem_bytes, bool dg, int64_t Dk, int64_t Dv)
{
    const int columns = linear_columns(elem_bytes, (int)Dv);
    return linear_cut(d, (Dv + columns - 1) / columns, chunk_us(elem_bytes, dg, Dk), least_chunks(elem_bytes),
                      brief_tokens(elem_bytes), dg || elem_bytes == 4);
}

// dk's and dv's walks in one launch, where each has a workgroup for all columns: the GPU is filled as by one walk of twice as
// many rows, and where rows are cut there are half the launches. (Of what both read, a third comes from an XCD's cache the
// second time: in a chain a row goes with a ticket, and tickets with the order in which the atomics arrive.) The
// backward of 320 rows of 64 x 128 over 4096 tokens took 873 us when this was done, with two launches 936; of 192 540, 602; of 160 heads of
// 128 x 128 807, 949; of 12 rows of 32 x 48 over 501 tokens in fp32 57, 77. None of 22 sizes was slower.
bool walk_twin(const DeltaDims& d, int elem_bytes, Cut& c)
{
    if (d.headdim > 128 || d.dstate > 128) return false;
    const int cv = linear_columns(elem_bytes, (int)d.headdim), ck = linear_columns(elem_bytes, (int)d.dstate);
    const int64_t slices = (d.headdim + cv - 1) / cv + (d.dstate + ck - 1) / ck;
    c = linear_cut(d, slices, chunk_us(elem_bytes, false, std::max(d.headdim, d.dstate)), least_chunks(elem_bytes),
                   brief_tokens(elem_bytes), elem_bytes == 4);
    return linear_items(d, c.seg) * d.nheads * slices < (int64_t(1) << 24);
}

struct GradLayout {
    Cut cq, ck, cv;
    bool twin;               // dk and dv together
    int64_t items;           // of the walk for dq
    int parts;
    size_t second, dpart, dk, dv, total;
};

GradLayout grad_layout(const DeltaDims& d, int elem_bytes)
{
    GradLayout l;
    l.cq = walk_cut(d, elem_bytes, true, d.headdim, d.dstate);
    l.ck = walk_cut(d, elem_bytes, false, d.headdim, d.dstate);
    l.cv = walk_cut(d, elem_bytes, false, d.dstate, d.headdim);
    Cut both;
    l.twin = walk_twin(d, elem_bytes, both);
    if (l.twin) l.ck = l.cv = both;
    l.items = linear_items(d, l.cq.seg);
    const int columns = linear_columns(elem_bytes, (int)d.dstate);
    l.parts = (int)((d.dstate + columns - 1) / columns) * linear_waves(elem_bytes, true, (int)d.dstate);
    // (walks that run one after another share a room for their states)
    const size_t bk = walk_bytes(d, l.ck, elem_bytes, false, d.headdim, d.dstate),
                 bv = walk_bytes(d, l.cv, elem_bytes, false, d.dstate, d.headdim);
    l.second = l.twin ? bk : 0;
    l.dpart = std::max({walk_bytes(d, l.cq, elem_bytes, true, d.headdim, d.dstate), bk, l.second + bv});
    l.dk = l.dpart + bytes_up(l.items * d.nheads * l.parts);
    const bool shared = d.nheads != d.ngroups;
    l.dv = l.dk + (shared ? bytes_up(d.tokens * d.nheads * d.dstate) : 0);
    l.total = l.dv + (shared ? bytes_up(d.tokens * d.nheads * d.headdim) : 0) + 256;
    return l;
}

}  // namespace

size_t linear_forward_workspace(const DeltaDims& d, int elem_bytes)
{
    return 256 + walk_bytes(d, walk_cut(d, elem_bytes, false, d.dstate, d.headdim), elem_bytes, false, d.dstate, d.headdim);
}

size_t linear_backward_workspace(const DeltaDims& d, int elem_bytes) { return grad_layout(d, elem_bytes).total; }

int64_t linear_blocks(const DeltaDims& d, int elem_bytes)
{
    int64_t most = 0;
    for (const bool dg : {false, true})
        for (const int64_t Dv : {d.headdim, d.dstate}) {
            const int columns = linear_columns(elem_bytes, (int)Dv);
            most = std::max(most, linear_items(d, walk_cut(d, elem_bytes, dg, d.headdim + d.dstate - Dv, Dv).seg) * d.nheads * ((Dv + columns - 1) / columns) *
                                      (linear_waves(elem_bytes, dg, (int)Dv) > 4 ? 2 : 1));
        }
    return most;
}

template <typename T>
hipError_t launch_linear_forward(const T* v, const float* g, const T* k, const T* q, const float* init, T* y,
                                 float* fin, const DeltaDims& d, void* workspace, hipStream_t stream)
{
    const int share = (int)(d.nheads / d.ngroups);
    LinearWalk<T> w[1]{};
    LinearWalk<T>& p = w[0];
    p.q = {q, d.nheads * d.dstate, 1};
    p.k = {k, d.ngroups * d.dstate, share};
    p.v = {v, d.ngroups * d.headdim, share};
    p.o = y;
    p.g = g;
    p.fin = fin;
    p.sk = 1;
    p.sv = d.dstate;
    p.Dk = (int)d.dstate;
    p.Dv = (int)d.headdim;
    p.d = d;
    return walk<false>(w, walk_cut(d, sizeof(T), false, d.dstate, d.headdim), init, {static_cast<float*>(workspace)}, stream);
}

template <typename T>
hipError_t launch_linear_backward(const T* v, const float* g, const T* k, const T* q, const float* init, const T* dy,
                                  const float* dfinal, T* dv, float* dg, T* dk, T* dq, float* dinit, const DeltaDims& d,
                                  void* workspace, hipStream_t stream)
{
    const GradLayout l = grad_layout(d, sizeof(T));
    char* ws = static_cast<char*>(workspace);
    float* states = reinterpret_cast<float*>(ws);
    float* dpart = reinterpret_cast<float*>(ws + l.dpart);
    const int share = (int)(d.nheads / d.ngroups);
    const bool shared = share > 1;
    const LinearOperand<T> oq = {q, d.nheads * d.dstate, 1}, ok = {k, d.ngroups * d.dstate, share},
                           ov = {v, d.ngroups * d.headdim, share}, od = {dy, d.nheads * d.headdim, 1};
    LinearWalk<T> wq[1]{};
    LinearWalk<T>& p = wq[0];
    p.g = g;
    p.d = d;
    // dq: the rows of the walk's state are the state's rows, its columns the columns
    p.q = od;
    p.k = ov;
    p.v = ok;
    p.x = oq;
    p.o = dq;
    p.sk = d.dstate;
    p.sv = 1;
    p.Dk = (int)d.headdim;
    p.Dv = (int)d.dstate;
    p.dlast = dfinal;
    p.dpart = dpart;
    hipError_t e = walk<true>(wq, l.cq, init, {states}, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(linear_dg_kernel, dim3((unsigned)d.nheads), dim3(256), 0, stream, dpart, dg, l.items, d.nheads,
                       l.parts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    // dk
    LinearWalk<T> wk{};
    wk.g = g;
    wk.d = d;
    wk.q = ov;
    wk.k = od;
    wk.v = oq;
    wk.back = true;
    wk.of32 = shared;
    wk.o = shared ? static_cast<void*>(ws + l.dk) : dk;
    wk.sk = d.dstate;
    wk.sv = 1;
    wk.Dk = (int)d.headdim;
    wk.Dv = (int)d.dstate;
    // dv, and the gradient of the state before the first token
    LinearWalk<T> wv = wk;
    wv.q = ok;
    wv.k = oq;
    wv.v = od;
    wv.o = shared ? static_cast<void*>(ws + l.dv) : dv;
    wv.sk = 1;
    wv.sv = d.dstate;
    wv.Dk = (int)d.dstate;
    wv.Dv = (int)d.headdim;
    wv.fin = dinit;
    if (l.twin) {
        LinearWalk<T> w[2] = {wk, wv};
        if ((e = walk<false>(w, l.ck, dfinal, {states, states + l.second / 4}, stream)) != hipSuccess) return e;
    } else {
        LinearWalk<T> w[1] = {wk};
        if ((e = walk<false>(w, l.ck, dfinal, {states}, stream)) != hipSuccess) return e;
        w[0] = wv;
        if ((e = walk<false>(w, l.cv, dfinal, {states}, stream)) != hipSuccess) return e;
    }
    if (shared && d.tokens > 0) {
        const int64_t rows = d.tokens * d.ngroups;
        hipLaunchKernelGGL((linear_group_kernel<T>), dim3(blocks_of(rows * d.dstate / 4)), dim3(256), 0, stream,
                           reinterpret_cast<const float*>(ws + l.dk), dk, rows, share, (int)d.dstate);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL((linear_group_kernel<T>), dim3(blocks_of(rows * d.headdim / 4)), dim3(256), 0, stream,
                           reinterpret_cast<const float*>(ws + l.dv), dv, rows, share, (int)d.headdim);
        e = hipGetLastError();
    }
    return e;
}

#define SSD_LINEAR(T)                                                                                                  \
    template hipError_t launch_linear_forward<T>(const T*, const float*, const T*, const T*, const float*, T*, float*,  \
                                                 const DeltaDims&, void*, hipStream_t);                                \
    template hipError_t launch_linear_backward<T>(const T*, const float*, const T*, const T*, const float*, const T*,  \
                                                  const float*, T*, float*, T*, T*, float*, const DeltaDims&, void*,   \
                                                  hipStream_t);
SSD_LINEAR(float)
SSD_LINEAR(bf16)
#undef SSD_LINEAR

}  // namespace ssd
