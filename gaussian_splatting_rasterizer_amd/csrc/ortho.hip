// ortho.hip -- orthogonalisation of an update by Newton-Schulz products.
//
//   X = G / max(|G|_F, eps);  repeat: P = X X^T, Q = b P + c P P, X = a X + Q X        (rows <= cols)
//   and with P = X^T X, X = a X + X Q for rows > cols, so that P is the smaller square.
//
// computed as Q = (a - 1) I + b P + c P P, X = X + Q X: a X and Q X of the first form nearly cancel where a singular
// value has arrived near 1, and what float16 loses of Q then counts several times (12 x 128 x 512: error 1.34 times that
// of the result's own bfloat16 rounding, 1.15 in this form; 40 x 77: 1.57 and 1.33).
//
// All products run on k_gemm16 in float16 with float32 accumulation.  P and Q are symmetric: only tiles on and above
// the diagonal are computed and each writes its mirror image; with few tiles and many k the sums are split along k.
// The singular values of X start in [0, 1] and the default coefficients keep them below 1.3, so X is held as 2^12 X and
// P, Q as 2^13 P, 2^13 Q: below float16's overflow (|P| <= 1.6, |Q| <= 2.5) and, for the entries that matter, above its
// subnormals.  Coefficients that let them grow take smaller powers of two (ortho_scales).  float16 keeps 11 bits; in
// bfloat16 the same steps lose 8 times as much.  For a float32 result each of X, P, Q is a pair hi + lo of
// float16 (22 bits) and a product is lo hi + hi lo + hi hi.
//
// Measured: 2048 x 5632 bfloat16 640 us, of each step's 147 us P 44 + 12 (its split sums), Q 25, X 64 (740 TFLOP/s on
// 176 of 256 CUs; tiles of 192 x 256 on 242 CUs gained 1 %, the power limit lowers the clock instead).  Two matrices of
// 1366 x 500 float32: 250 us, of each step's 50 us P 13 + 7, Q 14, X 16; these products have 11 to 24 k tiles in 72 to
// 432 workgroups and wait for LDS and barriers (a ring of four tiles in LDS instead of two changed nothing).
#include <algorithm>
#include <cmath>

#include "gsr_internal.hpp"
#include "gemm16.hpp"

namespace gsr {

namespace {

// X is stored as x X, P and Q as p P, p Q: powers of two, so that the scaling is exact.
struct Scales {
    float x, p;
};
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

// scale G / max(|G|, eps) into padded float16 planes
template <class E, int PL>
__global__ __launch_bounds__(256) void k_normalise(const E* g, int64_t rows, int64_t cols, const double* part,
                                                   float eps, float scale, uint16_t* x, int64_t plane) {
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
    const double inv = (double)scale / (norm < (double)eps ? (double)eps : norm);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i * 8 / c8, c = i * 8 - r * c8;
        const E* p = g + (b * rows + r) * cols + c;
        f32x4 v[2];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = c + e < cols ? (float)((double)load_value(p + e) * inv) : 0.f;
        put_planes<PL>(x + b * rows * c8 + i * 8, plane, v[0], v[1]);
    }
}

// C = alpha acc + beta S + diag I on and above the diagonal, mirrored below (S: null for P, the stored P for Q)
template <int PL>
struct EpiSymmetric {
    static constexpr bool kDual = false, kSymmetric = true;
    static constexpr int kAhead = 2;
    using Pre = Planes16<PL>;
    uint16_t* c;
    const uint16_t* s;
    int64_t plane, ld, batch_stride;
    int n;
    float alpha, beta, diag;
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
            if (s) {
                v[q] += beta * pre.get(q);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[q][e] += m == col + q * 4 + e ? diag : 0.f;
            }
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

// X' = X + alpha acc, stored again in float16 planes, or in the result's type after the last step
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
    float alpha, inv_scale;  // inv_scale times what is stored is the result
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
        for (int q = 0; q < 4; ++q) v[q] = pre.get(q) + alpha * acc[q];
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
            v[q] *= inv_scale;
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
        g.a[g.nseg] = (const char*)(a + pa), g.b[g.nseg] = (const char*)b, ++g.nseg;
        g.a[g.nseg] = (const char*)a, g.b[g.nseg] = (const char*)(b + pb), ++g.nseg;
    }
    g.a[g.nseg] = (const char*)a, g.b[g.nseg] = (const char*)b, ++g.nseg;
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
    const int t = p.tile;
    return p.splits > 1 ? p.splits * batch * tile_count(n, n, t, true) * t * t : 0;
}

template <int PL, bool KC>
hipError_t launch_symmetric(const GemmArgs& p, EpiSymmetric<PL> epi, float* part, hipStream_t st) {
    const GemmPlan plan = sym_plan(p.N, p.batch, k_tiles<_Float16>(p));
    const int t = plan.tile;
    epi.bm = t;
    if (plan.splits == 1) return launch_planned<_Float16, KC, KC>(p, plan, epi, st);
    const int64_t tiles = tile_count(p.N, p.N, t, true);
    EpiSymPartial ep{part, p.batch * tiles * t * t, tiles * t * t, t == 256 ? 8 : t == 128 ? 7 : 6};
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
        const int64_t a = sym_part_elems(side, B, seg * ((hi + kTileK<_Float16> - 1) / kTileK<_Float16>));
        const int64_t b = sym_part_elems(lo, B, seg * ((lo + kTileK<_Float16> - 1) / kTileK<_Float16>));
        return a > b ? a : b;
    }
};

template <class In, class Out, int PL>
hipError_t ortho_impl(const gs_ortho_dims& d, const void* gin, void* out, char* ws, hipStream_t st) {
    const OrthoLayout L(d);
    Scales sc;
    if (!ortho_scales(d, &sc.x, &sc.p)) return hipErrorInvalidValue;
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
    k_normalise<In, PL><<<dim3((unsigned)bx, (unsigned)L.B), 256, 0, st>>>(g, L.R, L.C, part, d.eps, sc.x, x,
                                                                              L.x_plane);
    GSR_TRY(hipGetLastError());
    const bool tall = d.rows > d.cols;
    for (int step = 0; step < d.steps; ++step) {
        EpiSymmetric<PL> es{P, nullptr, L.p_plane, L.lo8, L.lo * L.lo8, (int)L.lo, sc.p / (sc.x * sc.x), 0.f, 0.f, 128};
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
        EpiSymmetric<PL> eq{Q, P, L.p_plane, L.lo8, L.lo * L.lo8, (int)L.lo, d.c / sc.p, d.b,
                            (float)(((double)d.a - 1.0) * sc.p), 128};
        GemmArgs gq = make_args(L.lo, L.lo, L.lo);
        gq.batch = (int)L.B;
        gq.lda = gq.ldb = L.lo8;
        gq.batch_a = gq.batch_b = L.lo * L.lo8;
        ortho_segments<PL>(gq, P, L.p_plane, P, L.p_plane);
        GSR_TRY((launch_symmetric<PL, true>(gq, eq, sums, st)));
        const bool last = step + 1 == d.steps;
        EpiUpdate<PL, Out> eu{x, xn, L.x_plane, L.C8, L.R * L.C8, last ? (Out*)out : nullptr, (int)L.R, (int)L.C,
                              1.f / sc.p, 1.f / sc.x, vec_width(out, L.C, sizeof(Out))};
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

// ---- small matrices ------------------------------------------------------------------------------------

// A matrix whose padded X and P fit in LDS takes one workgroup and one launch for all steps (12 matrices of 128 x 512:
// 72 us, 17 launches took 123; 11 us a step, the rest for reading, norm and result).  X lies as m rows of n (m the
// smaller side) with n contiguous, rows of a multiple of 128 bytes (see at); P and then Q share a second buffer of the
// same form.
//   P: every wave takes a 32 x 64 block of X X^T and keeps it in registers;
//   Q: the same block of P P (P from LDS), plus b P and (a - 1) I; then Q replaces P;
//   X: every wave takes strips of 32 columns, which depend on nothing but themselves and Q, in place.
// LDS reads bound it: a block needs six 16-byte fragments a lane for eight products, 7 us of the 11.  Reading the next
// fragments during the products gained nothing, strips of 64 columns did not fit the registers.
constexpr int kSmallWaves = 8;
constexpr int kSmallLds = 160 * 1024;  // all of a CU's: the kernel has no other shared memory
constexpr int kSmallSide = 128;

template <int PL>
struct SmallView {
    char* base;
    int pitch, plane;  // bytes of a row, of a plane
    // chunk c8 of row r: any 8 consecutive rows differ (fragments along k), and the 4 rows of a transpose read differ by
    // whole pairs of chunks
    __device__ __forceinline__ int at(int r, int c8) const {
        return r * pitch + ((c8 ^ ((r & 3) << 1 | (r >> 2 & 1))) << 4);
    }
    // 16 rows from r0 (lane: row l % 16), k (l / 16) * 8 .. + 8 from k0
    __device__ __forceinline__ s16x8 rows(int pl, int r0, int k0, int lane) const {
        return *(const s16x8*)(base + pl * plane + at(r0 + (lane & 15), (k0 >> 3) + (lane >> 4)));
    }
    // the same with rows running along n: 16 columns from c0 (lane: column l % 16), k the row
    __device__ __forceinline__ s16x8 cols(int pl, int c0, int k0, int lane) const {
        s16x8 v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = k0 + (lane >> 4) * 8 + h * 4 + ((lane & 15) >> 2), c = c0 + (lane & 3) * 4;
            const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(base + pl * plane + at(k, c >> 3) + (c & 4) * 2));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h * 4 + e] = t[e];
        }
        return v;
    }
    // four values of row r from column c (a multiple of 4)
    __device__ __forceinline__ f32x4 get(int r, int c) const {
        const int o = at(r, c >> 3) + (c & 4) * 2;
        f32x4 v = from16<_Float16>(*(const u16x4*)(base + o));
        if constexpr (PL == 2) v += from16<_Float16>(*(const u16x4*)(base + plane + o));
        return v;
    }
    __device__ __forceinline__ void put(int r, int c, f32x4 v) const {
        const int o = at(r, c >> 3) + (c & 4) * 2;
        const u16x4 hi = to16<_Float16>(v);
        *(u16x4*)(base + o) = hi;
        if constexpr (PL == 2) *(u16x4*)(base + plane + o) = to16<_Float16>(v - from16<_Float16>(hi));
    }
    __device__ __forceinline__ float get1(int r, int c) const {
        const int o = at(r, c >> 3) + (c & 7) * 2;
        float v = (float)*(const _Float16*)(base + o);
        if constexpr (PL == 2) v += (float)*(const _Float16*)(base + plane + o);
        return v;
    }
    __device__ __forceinline__ void put1(int r, int c, float v) const {
        const int o = at(r, c >> 3) + (c & 7) * 2;
        const _Float16 hi = (_Float16)v;
        *(_Float16*)(base + o) = hi;
        if constexpr (PL == 2) *(_Float16*)(base + plane + o) = (_Float16)(v - (float)hi);
    }
};

template <int PL>
__device__ __forceinline__ f32x4 small_product(const s16x8 (&a)[PL], const s16x8 (&b)[PL], f32x4 acc) {
    if constexpr (PL == 2) {
        acc = Mfma<_Float16>::run(a[1], b[0], acc);
        acc = Mfma<_Float16>::run(a[0], b[1], acc);
    }
    return Mfma<_Float16>::run(a[0], b[0], acc);
}

// A value as the planes hold it.  b P takes the rounded P that P P is made of: with the unrounded one the two terms'
// errors no longer cancel in part (one 1 x 40 row: worst of 200 seeds 0.9 % off instead of 0.5 %).
template <int PL>
__device__ __forceinline__ f32x4 rounded(f32x4 v) {
    const f32x4 hi = from16<_Float16>(to16<_Float16>(v));
    if constexpr (PL == 1) return hi;
    return hi + from16<_Float16>(to16<_Float16>(v - hi));
}

// X = X + Q X for 32 columns from c0, in place
template <int PL>
__device__ __forceinline__ void small_update(const SmallView<PL>& X, const SmallView<PL>& Q, int c0, int mp,
                                             float inv_p, int lane) {
    constexpr int kTiles = kSmallSide / 16, J = 2;
    const int row = lane & 15, col = (lane >> 4) * 4;
    f32x4 x[kTiles][J];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) x[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < mp; k += 32) {
        s16x8 fb[J][PL];
#pragma unroll
        for (int q = 0; q < PL; ++q)
#pragma unroll
            for (int j = 0; j < J; ++j) fb[j][q] = X.cols(q, c0 + j * 16, k, lane);
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
            if (i * 16 < mp) {
                s16x8 fa[PL];
#pragma unroll
                for (int q = 0; q < PL; ++q) fa[q] = Q.rows(q, i * 16, k, lane);
#pragma unroll
                for (int j = 0; j < J; ++j) x[i][j] = small_product<PL>(fb[j], fa, x[i][j]);
            }
    }
    // the columns are read before they are written: other waves read other columns
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
        if (i * 16 < mp) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                x[i][j] = X.get(i * 16 + row, c0 + j * 16 + col) + x[i][j] * inv_p;
        }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
        if (i * 16 < mp) {
#pragma unroll
            for (int j = 0; j < J; ++j) X.put(i * 16 + row, c0 + j * 16 + col, x[i][j]);
        }
}

struct SmallArgs {
    const void* g;
    void* out;
    int rows, cols, m, n, mp, np, steps;  // m, n: smaller and larger side; mp, np: padded
    float diag, b, c_p, eps;  // (a - 1) p scale, b, c / p scale
    float x_scale, to_p, inv_p, inv_x;
};

// Row and column of every NT-th four elements of a matrix with `cols` columns, without a division for each.
struct Walk {
    int cols, dr, dc, r, c;
    __device__ __forceinline__ Walk(int cols, int first, int step) : cols(cols) {
        dr = step / cols, dc = step - dr * cols;
        r = first / cols, c = first - r * cols;
    }
    __device__ __forceinline__ void next() {
        r += dr, c += dc;
        if (c >= cols) c -= cols, ++r;
    }
};

template <class In, class Out, int PL>
__global__ __launch_bounds__(kSmallWaves * 64) void k_ortho_small(const SmallArgs p) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    constexpr int NT = kSmallWaves * 64;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const SmallView<PL> X{lds, p.np * 2, p.mp * p.np * 2};
    const SmallView<PL> P{lds + PL * X.plane, p.mp * 2, p.mp * p.mp * 2};
    const int64_t size = (int64_t)p.rows * p.cols;
    const In* g = (const In*)p.g + blockIdx.x * size;
    Out* out = (Out*)p.out + blockIdx.x * size;

    // Four consecutive values a thread, up to 32 times: the matrix is read once and stays in registers until its norm
    // is known; what is left of a larger one is read again.
    typedef In In4 __attribute__((ext_vector_type(4)));
    constexpr int kHeld = 32;
    const int n = (int)size;
    const bool vec = (uintptr_t)g % sizeof(In4) == 0;
    auto four = [&](int i) {
        f32x4 v{0.f, 0.f, 0.f, 0.f};
        if (vec && i + 4 <= n) {
            const In4 q = *(const In4*)(g + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)q[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < n) v[e] = load_value(g + i + e);
        }
        return v;
    };
    f32x4 held[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) held[k] = four((k * NT + tid) * 4);
    double s = 0.0;
    auto square = [&](const f32x4& v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s += (double)v[e] * (double)v[e];
    };
    // zero everything meanwhile: the padding stays zero
    for (int i = tid; i < PL * (X.plane + P.plane) / 16; i += NT) *(u32x4*)(lds + i * 16) = u32x4{0, 0, 0, 0};
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kHeld; ++k) square(held[k]);
    for (int i = (kHeld * NT + tid) * 4; i < n; i += NT * 4) square(four(i));
#pragma unroll
    for (int w = 32; w > 0; w >>= 1) s += __shfl_xor(s, w, 64);
    double* red = (double*)P.base;
    if (lane == 0) red[wave] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) s += red[w];
    __syncthreads();
    if (tid < kSmallWaves) red[tid] = 0.0;  // P's padding again
    // the factor as a power of two and a rest in [1/2, 1): neither over- nor underflows float32
    const double norm = sqrt(s);
    int ex;
    const float rest = (float)frexp((double)p.x_scale / (norm < (double)p.eps ? (double)p.eps : norm), &ex);
    const bool tall = p.rows > p.cols;
    Walk at(p.cols, tid * 4, NT * 4);
    auto place = [&](int i, f32x4 v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ldexpf(v[e], ex) * rest;
        if (!tall && p.cols % 4 == 0) {
            if (i < n) X.put(at.r, at.c, v);
        } else {
            int r = at.r, c = at.c;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (i + e < n) X.put1(tall ? c : r, tall ? r : c, v[e]);
                if (++c == p.cols) c = 0, ++r;
            }
        }
        at.next();
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k) place((k * NT + tid) * 4, held[k]);
    for (int i = (kHeld * NT + tid) * 4; i < n; i += NT * 4) place(i, four(i));
    __syncthreads();

    const int across = p.mp / 64, blocks = p.mp / 32 * across;
    const int row = lane & 15, col = (lane >> 4) * 4;  // of the lane's four results in a 16 x 16 tile
    const bool mine = wave < blocks;                   // at most 4 x 2 blocks
    const int r0 = mine ? wave / across * 32 : 0, c0 = mine ? wave % across * 64 : 0;
    for (int step = 0; step < p.steps; ++step) {
        f32x4 pv[2][4], acc[2][4];
        auto block = [&](const SmallView<PL>& v, int depth) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < depth; k += 32) {
                s16x8 fa[2][PL], fb[4][PL];
#pragma unroll
                for (int q = 0; q < PL; ++q) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) fa[i][q] = v.rows(q, r0 + i * 16, k, lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j) fb[j][q] = v.rows(q, c0 + j * 16, k, lane);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = small_product<PL>(fb[j], fa[i], acc[i][j]);
            }
        };
        auto keep = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) P.put(r0 + i * 16 + row, c0 + j * 16 + col, pv[i][j]);
        };
        if (mine) {
            block(X, p.np);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) pv[i][j] = rounded<PL>(acc[i][j] * p.to_p);
            keep();
        }
        __syncthreads();
        if (mine) {
            block(P, p.mp);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    pv[i][j] = p.b * pv[i][j] + p.c_p * acc[i][j];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        pv[i][j][e] += r0 + i * 16 + row == c0 + j * 16 + col + e ? p.diag : 0.f;
                }
        }
        __syncthreads();
        if (mine) keep();
        __syncthreads();
        for (int t = wave; t < p.np / 32; t += kSmallWaves) small_update<PL>(X, P, t * 32, p.mp, p.inv_p, lane);
        __syncthreads();
    }
    typedef Out Out4 __attribute__((ext_vector_type(4)));
    const bool vec_out = (uintptr_t)out % sizeof(Out4) == 0;
    Walk to(p.cols, tid * 4, NT * 4);
#pragma unroll 4
    for (int i = tid * 4; i < n; i += NT * 4) {
        f32x4 v;
        if (!tall && p.cols % 4 == 0) {
            v = X.get(to.r, to.c);
        } else {
            int r = to.r, c = to.c;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = i + e < n ? X.get1(tall ? c : r, tall ? r : c) : 0.f;
                if (++c == p.cols) c = 0, ++r;
            }
        }
        to.next();
        Out4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (Out)(v[e] * p.inv_x);
        if (vec_out && i + 4 <= n) {
            *(Out4*)(out + i) = o;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < n) out[i + e] = o[e];
        }
    }
}

// LDS of the one-workgroup form, 0 where it does not apply.
int small_lds(const gs_ortho_dims& d) {
    const int64_t m = d.rows < d.cols ? d.rows : d.cols, n = d.rows < d.cols ? d.cols : d.rows;
    const int64_t mp = round_up(m, 64), np = round_up(n, 64), pl = d.out_dtype == GS_F32 ? 2 : 1;
    const int64_t bytes = pl * mp * (np + mp) * 2;
    return mp <= kSmallSide && bytes <= kSmallLds ? (int)bytes : 0;
}

template <class In, class Out, int PL>
hipError_t ortho_small(const gs_ortho_dims& d, const void* g, void* out, hipStream_t st) {
    const int bytes = small_lds(d);
    SmallArgs p{};
    p.g = g, p.out = out;
    p.rows = (int)d.rows, p.cols = (int)d.cols;
    p.m = d.rows < d.cols ? p.rows : p.cols, p.n = d.rows < d.cols ? p.cols : p.rows;
    p.mp = (int)round_up(p.m, 64), p.np = (int)round_up(p.n, 64);
    p.steps = d.steps, p.b = d.b, p.eps = d.eps;
    Scales sc;
    if (!ortho_scales(d, &sc.x, &sc.p)) return hipErrorInvalidValue;
    p.x_scale = sc.x, p.to_p = sc.p / (sc.x * sc.x), p.c_p = d.c / sc.p;
    p.diag = (float)(((double)d.a - 1.0) * sc.p), p.inv_p = 1.f / sc.p, p.inv_x = 1.f / sc.x;
    GSR_TRY(hipFuncSetAttribute((const void*)k_ortho_small<In, Out, PL>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                kSmallLds));
    k_ortho_small<In, Out, PL><<<dim3((unsigned)d.batch), kSmallWaves * 64, bytes, st>>>(p);
    return hipGetLastError();
}

template <class In, class Out, int PL>
hipError_t ortho_any(const gs_ortho_dims& d, const void* g, void* out, char* ws, hipStream_t st) {
    return small_lds(d) ? ortho_small<In, Out, PL>(d, g, out, st) : ortho_impl<In, Out, PL>(d, g, out, ws, st);
}

}  // namespace

// Follows the interval [0, 1] of the singular values through the steps: P reaches s^2, Q the largest
// |a - 1 + b s^2 + c s^4| and X the largest |a s + b s^3 + c s^5| for s in it (at its ends or where the derivative is
// zero), and no entry of a matrix exceeds its largest singular value.  2 % a step cover the float16 roundings.  The scales
// are the largest powers of two, up to 2^12 and 2^13, that keep these below float16's 65504.  Below 2^8 the entries that
// matter come near float16's subnormals: false.
bool ortho_scales(const gs_ortho_dims& d, float* x_scale, float* p_scale) {
    const double a = d.a, b = d.b, c = d.c, slack = 1.02, most = 65504.0, least_scale = 256.0;
    double s = slack, top_x = s, top_p = 0.0;
    for (int step = 0; step < d.steps; ++step) {
        const double s2 = s * s;
        double q = std::max(std::fabs(a - 1.0), std::fabs(a - 1.0 + b * s2 + c * s2 * s2));
        double next = std::fabs(s * (a + b * s2 + c * s2 * s2));
        if (c != 0.0) {
            const double at = -b / (2.0 * c);
            if (at > 0.0 && at < s2) q = std::max(q, std::fabs(a - 1.0 + b * at + c * at * at));
        }
        // a + 3 b t + 5 c t^2 = 0 in t = s^2
        double roots[2] = {-1.0, -1.0};
        const double disc = 9.0 * b * b - 20.0 * a * c;
        if (c != 0.0 && disc >= 0.0) {
            roots[0] = (-3.0 * b + std::sqrt(disc)) / (10.0 * c);
            roots[1] = (-3.0 * b - std::sqrt(disc)) / (10.0 * c);
        } else if (c == 0.0 && b != 0.0) {
            roots[0] = -a / (3.0 * b);
        }
        for (double t : roots)
            if (t > 0.0 && t < s2) next = std::max(next, std::fabs(std::sqrt(t) * (a + b * t + c * t * t)));
        top_p = std::max(top_p, std::max(s2, q * slack));
        s = next * slack;
        top_x = std::max(top_x, s);
        if (!(top_p * least_scale < most) || !(top_x * least_scale < most)) return false;
    }
    *x_scale = 4096.f;
    *p_scale = 8192.f;
    while (top_x * *x_scale >= most) *x_scale *= 0.5f;
    while (top_p * *p_scale >= most) *p_scale *= 0.5f;
    return true;
}

size_t ortho_workspace(const gs_ortho_dims& d) {
    if (small_lds(d)) return 0;
    const OrthoLayout L(d);
    return (size_t)(round_up(L.B * kNormBlocks * 8, kAlign) + 2 * round_up(L.x_plane * L.planes * 2, kAlign) +
                    2 * round_up(L.p_plane * L.planes * 2, kAlign) + round_up(L.part_elems() * 4, kAlign));
}

hipError_t launch_ortho(const gs_ortho_dims& d, const void* g, void* out, void* ws, hipStream_t st) {
    char* b = (char*)ws;
    if (d.dtype == GS_F32)
        return d.out_dtype == GS_F32 ? ortho_any<float, float, 2>(d, g, out, b, st)
                                     : ortho_any<float, __bf16, 1>(d, g, out, b, st);
    return d.out_dtype == GS_F32 ? ortho_any<__bf16, float, 2>(d, g, out, b, st)
                                 : ortho_any<__bf16, __bf16, 1>(d, g, out, b, st);
}

}  // namespace gsr
