// ortho.hip -- orthogonalisation of an update by Newton-Schulz products.
//
//   X = G / max(|G|_F, eps);  repeat: P = X X^T, Q = b P + c P P, X = a X + Q X        (rows <= cols)
//   and with P = X^T X, X = a X + X Q for rows > cols, so that P is the smaller square.
//
// All products run on k_gemm16 in float16 with float32 accumulation.  P and Q are symmetric: only tiles on and above
// the diagonal are computed and each writes its mirror image; with few tiles and many k the sums are split along k.  Every singular value of X stays below 1.2 after the
// normalisation, so X is held as 2^12 X and P, Q as 2^13 P, 2^13 Q: far from float16's overflow (|Q| <= 5) and, for
// the entries that matter, above its subnormals.  float16 keeps 11 bits; in bfloat16 the same steps lose 8 times as
// much.  For a float32 result each of X, P, Q is a pair hi + lo of float16 (22 bits) and a product is
// lo hi + hi lo + hi hi.
#include "gsr_internal.hpp"
#include "gemm16.hpp"

namespace gsr {

namespace {

constexpr float kXScale = 4096.f;     // X is stored as 2^12 X
constexpr float kPScale = 8192.f;     // P and Q as 2^13 P, 2^13 Q
constexpr int kNormBlocks = 256;      // partial sums of squares per matrix

template <int PL>
__device__ __forceinline__ void put_planes(uint16_t* p, int64_t plane, f32x4 v0, f32x4 v1) {
    const u16x4 h0 = to16<_Float16>(v0), h1 = to16<_Float16>(v1);
    *(u16x8*)p = pack8(h0, h1);
    if constexpr (PL == 2)
        *(u16x8*)(p + plane) =
            pack8(to16<_Float16>(v0 - from16<_Float16>(h0)), to16<_Float16>(v1 - from16<_Float16>(h1)));
}
// 16 stored values, fetched ahead
template <int PL>
struct Planes16 {
    u16x8 v[PL][2];
    __device__ __forceinline__ void fetch(const uint16_t* p, int64_t plane, int n, int64_t ld) {
#pragma unroll
        for (int k = 0; k < PL; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (n + h * 8 < ld) v[k][h] = *(const u16x8*)(p + k * plane + h * 8);
    }
    __device__ __forceinline__ f32x4 get(int q) const {
        f32x4 r = from16<_Float16>(half8(v[0][q >> 1], q & 1));
        if constexpr (PL == 2) r += from16<_Float16>(half8(v[1][q >> 1], q & 1));
        return r;
    }
};

template <class E>
__device__ __forceinline__ float load_value(const E* p);
template <>
__device__ __forceinline__ float load_value<float>(const float* p) {
    return *p;
}
template <>
__device__ __forceinline__ float load_value<__bf16>(const __bf16* p) {
    return (float)*p;
}

// Partial sums of squares in float64: block j of matrix b sums groups j, j + kNormBlocks, ... of 1024 elements, four
// (neighbouring where the address allows) a thread.
template <class E>
__global__ __launch_bounds__(256) void k_norm(const E* g, int64_t n, double* part) {
    typedef E E4 __attribute__((ext_vector_type(4)));
    const E* p = g + blockIdx.y * n;
    const bool vec = (uintptr_t)p % sizeof(E4) == 0;
    double s = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x * 4; i < n; i += 1024 * kNormBlocks) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (vec && i + 4 <= n) {
            const E4 q = *(const E4*)(p + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)q[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < n) v[e] = (float)p[i + e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s += (double)v[e] * (double)v[e];
    }
    __shared__ double red[256];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int w = 128; w > 0; w >>= 1) {
        if ((int)threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
        __syncthreads();
    }
    if (threadIdx.x == 0) part[blockIdx.y * kNormBlocks + blockIdx.x] = red[0];
}

// X = 2^12 G / max(|G|, eps) into padded float16 planes
template <class E, int PL>
__global__ __launch_bounds__(256) void k_normalise(const E* g, int64_t rows, int64_t cols, const double* part,
                                                   float eps, uint16_t* x, int64_t plane) {
    const int64_t c8 = (cols + 7) / 8 * 8, n = rows * c8 / 8;
    const int64_t b = blockIdx.y;
    __shared__ double red[kNormBlocks];
    static_assert(kNormBlocks == 256, "one partial sum a thread");
    red[threadIdx.x] = part[b * kNormBlocks + threadIdx.x];
    __syncthreads();
    for (int w = 128; w > 0; w >>= 1) {
        if ((int)threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
        __syncthreads();
    }
    const double norm = sqrt(red[0]);
    const double inv = (double)kXScale / (norm < (double)eps ? (double)eps : norm);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i * 8 / c8, c = i * 8 - r * c8;
        const E* p = g + (b * rows + r) * cols + c;
        f32x4 v[2];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = c + e < cols ? (float)((double)load_value(p + e) * inv) : 0.f;
        put_planes<PL>(x + b * rows * c8 + i * 8, plane, v[0], v[1]);
    }
}

// C = alpha acc + beta S on and above the diagonal, mirrored below (S: null for P, the stored P for Q)
template <int PL>
struct EpiSymmetric {
    static constexpr bool kDual = false, kSymmetric = true;
    static constexpr int kAhead = 2;
    using Pre = Planes16<PL>;
    uint16_t* c;
    const uint16_t* s;
    int64_t plane, ld, batch_stride;
    int n;
    float alpha, beta;
    int bm;  // tile size, to tell diagonal tiles
    __device__ __forceinline__ Pre fetch(int batch, int m, int col) const {
        Pre r;
        if (s && m < n) r.fetch(s + batch * batch_stride + m * ld + col, plane, col, ld);
        return r;
    }
    __device__ __forceinline__ void row(int batch, int, int m, int col, const f32x4 (&acc)[4], const Pre& pre) const {
        if (m >= n) return;
        const int64_t base = batch * batch_stride;
        const bool mirror = m / bm != col / bm;  // a diagonal tile holds both halves already
        f32x4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = acc[q] * alpha;
            if (s) v[q] += beta * pre.get(q);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (col + h * 8 < ld) put_planes<PL>(c + base + m * ld + col + h * 8, plane, v[h * 2], v[h * 2 + 1]);
        if (!mirror) return;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if (col + e >= n) continue;
            uint16_t* d = c + base + (int64_t)(col + e) * ld + m;
            const float x = v[e >> 2][e & 3];
            const _Float16 hi = (_Float16)x;
            *d = __builtin_bit_cast(uint16_t, hi);
            if constexpr (PL == 2) d[plane] = __builtin_bit_cast(uint16_t, (_Float16)(x - (float)hi));
        }
    }
};

// X' = a X + alpha acc, stored again in float16 planes, or in the result's type after the last step
template <int PL, class Out>
struct EpiUpdate {
    static constexpr bool kDual = false, kSymmetric = false;
    static constexpr int kAhead = 2;
    using Pre = Planes16<PL>;
    const uint16_t* x;
    uint16_t* xn;
    int64_t plane, ld, batch_stride;
    Out* out;  // null: another step follows
    int M, N;  // rows, columns of the matrix
    float a, alpha;
    int vec;
    __device__ __forceinline__ Pre fetch(int batch, int m, int n) const {
        Pre r;
        if (m < M) r.fetch(x + batch * batch_stride + (int64_t)m * ld + n, plane, n, ld);
        return r;
    }
    __device__ __forceinline__ void row(int batch, int, int m, int n, const f32x4 (&acc)[4], const Pre& pre) const {
        if (m >= M) return;
        f32x4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = a * pre.get(q) + alpha * acc[q];
        if (!out) {
            uint16_t* d = xn + batch * batch_stride + (int64_t)m * ld + n;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (n + h * 8 < ld) put_planes<PL>(d + h * 8, plane, v[h * 2], v[h * 2 + 1]);
            return;
        }
        Out* d = out + ((int64_t)batch * M + m) * N + n;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] *= 1.f / kXScale;
            if (vec >= 4 && n + q * 4 + 4 <= N) {
                if constexpr (sizeof(Out) == 4)
                    *(f32x4*)(d + q * 4) = v[q];
                else
                    *(u16x4*)(d + q * 4) = to16<Out>(v[q]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + q * 4 + e < N) d[q * 4 + e] = (Out)v[q][e];
            }
        }
    }
};

template <int PL>
void ortho_segments(GemmArgs& g, const uint16_t* a, int64_t pa, const uint16_t* b, int64_t pb) {
    if (PL == 2) {
        g.a[g.nseg] = a + pa, g.b[g.nseg] = b, ++g.nseg;
        g.a[g.nseg] = a, g.b[g.nseg] = b + pb, ++g.nseg;
    }
    g.a[g.nseg] = a, g.b[g.nseg] = b, ++g.nseg;
}

// float32 partial sums of a symmetric product split along k: part[split][batch][tile][256 or 128]^2, one tile after
// another, since only those on and above the diagonal exist
struct EpiSymPartial {
    static constexpr bool kDual = false, kSymmetric = true;
    static constexpr int kAhead = 0;
    using Pre = NoPre;
    float* part;
    int64_t split_stride, batch_stride;
    int shift;  // log2 of the tile size
    __device__ __forceinline__ Pre fetch(int, int, int) const { return {}; }
    __device__ __forceinline__ void row(int batch, int split, int m, int n, const f32x4 (&v)[4], const Pre&) const {
        const int tm = m >> shift, tn = n >> shift, mask = (1 << shift) - 1;
        float* p = part + split * split_stride + batch * batch_stride +
                   (((int64_t)(tn * (tn + 1) / 2 + tm)) << (2 * shift)) + ((m & mask) << shift) + (n & mask);
#pragma unroll
        for (int q = 0; q < 4; ++q) *(f32x4*)(p + q * 4) = v[q];
    }
};

// Sum of those in split order, handed to the symmetric epilogue; a thread takes 16 columns of a row.
template <int PL>
__global__ __launch_bounds__(256) void k_sym_reduce(EpiSymPartial ep, int splits, int tiles, EpiSymmetric<PL> epi) {
    const int side = 1 << ep.shift, per = side * side / 16;
    const int batch = blockIdx.y;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)tiles * per; i += (int64_t)gridDim.x * 256) {
        const int tile = (int)(i / per), in = (int)(i - (int64_t)tile * per);
        // neighbouring threads take neighbouring rows: the mirrored half is written along them
        const int r = in & (side - 1), c = (in >> ep.shift) * 16;
        int tm, tn;
        symmetric_tile(tile, tm, tn);
        const float* p = ep.part + batch * ep.batch_stride + ((int64_t)tile << (2 * ep.shift)) + (r << ep.shift) + c;
        f32x4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = *(const f32x4*)(p + q * 4);
        for (int s = 1; s < splits; ++s)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += *(const f32x4*)(p + s * ep.split_stride + q * 4);
        const int m = tm * side + r, col = tn * side + c;
        epi.row(batch, 0, m, col, v, epi.fetch(batch, m, col));
    }
}

constexpr int kMaxSymSplits = 16;
GemmPlan sym_plan(int64_t n, int64_t batch, int64_t ktiles) {
    return plan_gemm(n, n, batch, ktiles, false, true, kMaxSymSplits);
}
int64_t sym_part_elems(int64_t n, int64_t batch, int64_t ktiles) {
    const GemmPlan p = sym_plan(n, batch, ktiles);
    const int t = p.big ? 256 : 128;
    return p.splits > 1 ? p.splits * batch * tile_count(n, n, t, true) * t * t : 0;
}

template <int PL, bool KC>
hipError_t launch_symmetric(const GemmArgs& p, EpiSymmetric<PL> epi, float* part, hipStream_t st) {
    const GemmPlan plan = sym_plan(p.N, p.batch, k_tiles(p));
    const int t = plan.big ? 256 : 128;
    epi.bm = t;
    if (plan.splits == 1) return launch_planned<_Float16, KC, KC>(p, plan, epi, st);
    const int64_t tiles = tile_count(p.N, p.N, t, true);
    EpiSymPartial ep{part, p.batch * tiles * t * t, tiles * t * t, plan.big ? 8 : 7};
    GSR_TRY((launch_planned<_Float16, KC, KC>(p, plan, ep, st)));
    int64_t bx = (tiles * t * t / 16 + 255) / 256;
    if (bx > 4096) bx = 4096;
    k_sym_reduce<PL><<<dim3((unsigned)bx, (unsigned)p.batch), 256, 0, st>>>(ep, plan.splits, (int)tiles, epi);
    return hipGetLastError();
}

struct OrthoLayout {
    int64_t B, R, C, lo, C8, lo8, x_plane, p_plane;
    int planes;
    explicit OrthoLayout(const gs_ortho_dims& d)
        : B(d.batch), R(d.rows), C(d.cols), lo(d.rows < d.cols ? d.rows : d.cols), C8(round8(C)), lo8(round8(lo)),
          x_plane(B * R * C8), p_plane(B * lo * lo8), planes(d.out_dtype == GS_F32 ? 2 : 1) {}
    // float32 partial sums of X X^T and P P
    int64_t part_elems() const {
        const int64_t seg = planes == 2 ? 3 : 1, hi = R < C ? C : R, side = R > C ? lo8 : lo;
        const int64_t a = sym_part_elems(side, B, seg * ((hi + kGemmBK - 1) / kGemmBK));
        const int64_t b = sym_part_elems(lo, B, seg * ((lo + kGemmBK - 1) / kGemmBK));
        return a > b ? a : b;
    }
};

template <class In, class Out, int PL>
hipError_t ortho_impl(const gs_ortho_dims& d, const void* gin, void* out, char* ws, hipStream_t st) {
    const OrthoLayout L(d);
    Carver cv{ws};
    double* part = cv.take<double>(L.B * kNormBlocks);
    uint16_t* x = cv.take<uint16_t>(L.x_plane * PL);
    uint16_t* xn = cv.take<uint16_t>(L.x_plane * PL);
    uint16_t* P = cv.take<uint16_t>(L.p_plane * PL);
    uint16_t* Q = cv.take<uint16_t>(L.p_plane * PL);
    float* sums = cv.take<float>(L.part_elems());
    const In* g = (const In*)gin;
    k_norm<In><<<dim3(kNormBlocks, (unsigned)L.B), 256, 0, st>>>(g, L.R * L.C, part);
    GSR_TRY(hipGetLastError());
    int64_t bx = (L.R * L.C8 / 8 + 255) / 256;
    if (bx > 2048) bx = 2048;
    k_normalise<In, PL><<<dim3((unsigned)bx, (unsigned)L.B), 256, 0, st>>>(g, L.R, L.C, part, d.eps, x, L.x_plane);
    GSR_TRY(hipGetLastError());
    const bool tall = d.rows > d.cols;
    for (int step = 0; step < d.steps; ++step) {
        EpiSymmetric<PL> es{P, nullptr, L.p_plane, L.lo8, L.lo * L.lo8, (int)L.lo, kPScale / (kXScale * kXScale), 0.f,
                            128};
        GemmArgs gp = make_args(L.lo, L.lo, tall ? L.R : L.C);
        gp.batch = (int)L.B;
        gp.lda = gp.ldb = L.C8;
        gp.batch_a = gp.batch_b = L.R * L.C8;
        ortho_segments<PL>(gp, x, L.x_plane, x, L.x_plane);
        if (tall) {
            gp.M = gp.N = (int)L.lo8;  // columns of X: the padded ones are zero
            GSR_TRY((launch_symmetric<PL, false>(gp, es, sums, st)));
        } else {
            GSR_TRY((launch_symmetric<PL, true>(gp, es, sums, st)));
        }
        EpiSymmetric<PL> eq{Q, P, L.p_plane, L.lo8, L.lo * L.lo8, (int)L.lo, d.c / kPScale, d.b, 128};
        GemmArgs gq = make_args(L.lo, L.lo, L.lo);
        gq.batch = (int)L.B;
        gq.lda = gq.ldb = L.lo8;
        gq.batch_a = gq.batch_b = L.lo * L.lo8;
        ortho_segments<PL>(gq, P, L.p_plane, P, L.p_plane);
        GSR_TRY((launch_symmetric<PL, true>(gq, eq, sums, st)));
        const bool last = step + 1 == d.steps;
        EpiUpdate<PL, Out> eu{x, xn, L.x_plane, L.C8, L.R * L.C8, last ? (Out*)out : nullptr, (int)L.R, (int)L.C,
                              d.a, 1.f / kPScale, vec_width(out, L.C, sizeof(Out))};
        GemmArgs gu = make_args(L.R, L.C8, L.lo);
        gu.batch = (int)L.B;
        if (tall) {  // X Q, Q symmetric
            gu.N = (int)L.C;
            gu.lda = L.C8, gu.ldb = L.lo8;
            gu.batch_a = L.R * L.C8, gu.batch_b = L.lo * L.lo8;
            ortho_segments<PL>(gu, x, L.x_plane, Q, L.p_plane);
            GSR_TRY((launch_gemm<_Float16, true, true>(gu, eu, st)));
        } else {  // Q X
            gu.lda = L.lo8, gu.ldb = L.C8;
            gu.batch_a = L.lo * L.lo8, gu.batch_b = L.R * L.C8;
            ortho_segments<PL>(gu, Q, L.p_plane, x, L.x_plane);
            GSR_TRY((launch_gemm<_Float16, true, false>(gu, eu, st)));
        }
        uint16_t* t = x;
        x = xn;
        xn = t;
    }
    return hipSuccess;
}

}  // namespace

size_t ortho_workspace(const gs_ortho_dims& d) {
    const OrthoLayout L(d);
    return (size_t)(round_up(L.B * kNormBlocks * 8, kAlign) + 2 * round_up(L.x_plane * L.planes * 2, kAlign) +
                    2 * round_up(L.p_plane * L.planes * 2, kAlign) + round_up(L.part_elems() * 4, kAlign));
}

hipError_t launch_ortho(const gs_ortho_dims& d, const void* g, void* out, void* ws, hipStream_t st) {
    char* b = (char*)ws;
    if (d.dtype == GS_F32)
        return d.out_dtype == GS_F32 ? ortho_impl<float, float, 2>(d, g, out, b, st)
                                     : ortho_impl<float, __bf16, 1>(d, g, out, b, st);
    return d.out_dtype == GS_F32 ? ortho_impl<__bf16, float, 2>(d, g, out, b, st)
                                 : ortho_impl<__bf16, __bf16, 1>(d, g, out, b, st);
}

}  // namespace gsr
