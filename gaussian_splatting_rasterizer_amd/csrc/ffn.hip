// ffn.hip -- gated feed-forward block of the learned updater and its gradients.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T                                  (forward)
//   dh = dy Wd, dg = dh u act'(g), du = dh act(g),
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h                      (backward)
//
// Every product runs on k_gemm16: both projections share one pass over x, the activation and the gating are in the
// first product's epilogue, their derivatives in the epilogue of dh, and dx sums its two products in one
// accumulator.  float32 runs on the float32 matrix instructions (FmtF32) or, for large products, with operands split
// into three bfloat16 parts and multiplied in six partial products (FmtF32Split), which keeps 24 bits (the parts left
// out are below 2^-24) at the bfloat16 matrix rate / 6; see split_f32.
//
// Rows that are not 16-byte aligned, or whose length is not a multiple of 8 elements, are copied once into a
// zero-padded layout in the workspace (k_pack); other operands are read in place.
//
// Roundings of the 16-bit types: the matrix instructions take 16-bit operands, so h, dg and du are rounded to the type
// once before their products (for float16 they have to stay within its range).  With the result's own rounding, every
// result carries two.  g and u are kept for the backward pass with 4 (bfloat16) or 5 (float16) bits more than the type
// has, and with float32's range (KeepHigh): kept in the type they doubled the variance of dx, dWg and dWu, and in
// float16 the infinite g of a closed gate made NaN of its gradients.  131072 rows of 512 x 2048 x 512 bfloat16 took 3.00
// ms, 2.82 with g and u in the type, 3.11 with 24 bits of each.  Everything else is float32.
//
// Measured, bfloat16 SiLU, 131072 rows of 512 x 2048 x 512, forward and backward 2.93 ms (840 TFLOP/s; the power limit
// lowers the shader clock to 1.9 GHz); in a kernel trace, us:
//   g, u, h  860  1.9 GB of results (370 at a copy's rate) and products (360) alternate in a workgroup
//   y        285  products, 970 TFLOP/s
//   dg, du   750  2.5 GB read and written (490) after the products (180)
//   dx       470  products, 1170 TFLOP/s
//   dWg, dWu 440, dWd 245: products split along the rows, 1250 and 1120 TFLOP/s; the sums of the parts 13 each
// Asking for the tile's g and u during its products made the third 80 us slower: the lines arrive, but the fetches of
// operands wait behind them.
#include <algorithm>

#include "gsr_internal.hpp"
#include "gemm16.hpp"

namespace gsr {

namespace {

// ---- packing -------------------------------------------------------------------------------------------

struct PackJob {
    const void* src;
    void* dst;
    int64_t rows, cols, ld, plane;  // dst rows are round8(cols) long, planes `plane` elements apart
};
struct PackJobs {
    PackJob j[5];
};

// [rows][cols] -> planes of [rows][round8(cols)], zero padded; one thread per 8 destination elements.
template <class F>
__global__ __launch_bounds__(256) void k_pack(const PackJobs jobs) {
    const PackJob& jb = jobs.j[blockIdx.y];
    const int64_t c8 = (jb.cols + 7) / 8, n = jb.rows * c8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / c8, c = (i - r * c8) * 8;
        const typename F::Elem* s = (const typename F::Elem*)jb.src + r * jb.ld + c;
        OperandElem<F>* d = (OperandElem<F>*)jb.dst + i * 8;
        const int64_t left = jb.cols - c;
        if constexpr (sizeof(typename F::Elem) == 2) {
            u16x8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < left ? s[e] : (uint16_t)0;
            *(u16x8*)d = v;
        } else {
            f32x4 v[2];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = e < left ? s[e] : 0.f;
            put_operand8<F>(d, jb.plane, v[0], v[1]);
        }
    }
}

// ---- activations ---------------------------------------------------------------------------------------

// act(g) and its derivative.  The sigmoid is one exponential and one reciprocal (1 ulp): a correctly rounded division
// took a third of the gradient product's epilogue.  For g < -88 the exponential is inf and the sigmoid 0.
// Phi(-|g|) = 1/2 exp(-x^2) erfcx(x), x = |g| / sqrt 2, with erfcx(x) = exp(x^2) erfc(x) as t times a polynomial in
// t = 1 / (1 + p x): the relative error stays the same into the far tail (1/2 (1 + erf) has no digits left at -6).
// The polynomials are least maximum relative error fits: 7 terms 4.3e-6 for the 16-bit types, 10 terms 3.2e-8 for
// float32, where 8 2^-24 + 2^-24 g^2 come from the roundings, the second part from that of g^2.
template <bool WIDE>
__device__ __forceinline__ float erfcx_poly(float t) {
    constexpr float c10[10] = {0.253885321f,   0.253883149f, 0.228271938f,  0.17524937f,  0.119964137f,
                               -0.0223974529f, 0.142469072f, -0.300651575f, 0.190725904f, -0.0413998491f};
    constexpr float c7[7] = {0.310304171f, 0.310187702f,  0.266718943f, 0.138616215f,
                             0.177182023f, -0.301853708f, 0.0988489167f};
    constexpr int n = WIDE ? 10 : 7;
    float q = WIDE ? c10[9] : c7[6];
#pragma unroll
    for (int i = n - 2; i >= 0; --i) q = __builtin_fmaf(t, q, WIDE ? c10[i] : c7[i]);
    return q * t;
}

template <class F, int ACT>
__device__ __forceinline__ void activation(float g, float& a, float& da) {
    if constexpr (ACT == GS_ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.f + __expf(-g));
        a = g * s;
        da = s * (1.f + g * (1.f - s));
    } else {
        const float e = __expf(-0.5f * g * g);
        constexpr bool kWide = sizeof(typename F::Elem) == 4;
        constexpr float p = (kWide ? 0.45f : 0.55f) * 0.70710678118654752f;
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(p, __builtin_fabsf(g), 1.f));
        const float q = 0.5f * e * erfcx_poly<kWide>(t);
        const float cdf = g < 0.f ? q : 1.f - q;
        a = g * cdf;
        da = __builtin_fmaf(g * 0.39894228040143268f, e, cdf);
    }
}

// ---- epilogues -----------------------------------------------------------------------------------------

// h = act(g) u, with g and u kept for the backward pass when asked for
template <class F, int ACT>
struct EpiGate {
    static constexpr bool kDual = true, kSymmetric = false;
    static constexpr int kAhead = 0;
    OperandElem<F>* h;
    int64_t h_plane;
    Kept gu;  // of F::Keep; p null: not kept
    int64_t f8;
    int M;
    __device__ __forceinline__ void row(int m, int n, f32x4 g0, f32x4 g1, f32x4 u0, f32x4 u1) const {
        if (m >= M || n >= f8) return;
        if (gu.p) F::Keep::put(gu, m, n, g0, g1, u0, u1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, da;
            activation<F, ACT>(g0[e], a, da);
            u0[e] *= a;
            activation<F, ACT>(g1[e], a, da);
            u1[e] *= a;
        }
        put_operand8<F>(h + (int64_t)m * f8 + n, h_plane, u0, u1);
    }
};

// The same for few rows: h is also the next product's input, which takes the block's type as it is; split planes are
// written only for the backward pass.
template <class F, int ACT>
struct EpiGateFew {
    static constexpr bool kDual = true;
    EpiGate<F, ACT> all;        // all.h null: nothing is kept
    typename F::Elem* h;        // [M][f8]
    __device__ __forceinline__ void row(int m, int n, f32x4 g0, f32x4 g1, f32x4 u0, f32x4 u1) const {
        if (m >= all.M || n >= all.f8) return;
        if (all.h) all.row(m, n, g0, g1, u0, u1);
        if ((const void*)h == (const void*)all.h) return;
        f32x4 a0, a1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, da;
            activation<F, ACT>(g0[e], a, da);
            a0[e] = a * u0[e];
            activation<F, ACT>(g1[e], a, da);
            a1[e] = a * u1[e];
        }
        F::put8(h + (int64_t)m * all.f8 + n, a0, a1);
    }
};

// dg and du from dh and the saved g and u.  The saved values are fetched ahead: read where they are used, each row of
// products waited for its own (131072 x 2048 x 512: 1050 us).
template <class F, int ACT>
struct EpiGateGrad {
    static constexpr bool kDual = false, kSymmetric = false;
    using K = typename F::Keep;
    static constexpr int kAhead = K::kAhead;
    Kept gu;
    OperandElem<F>* dgu;  // [M][2 F8]
    int64_t plane;
    int64_t f8;
    int M;
    struct Pre {
        typename K::Raw gu[2];
    };
    __device__ __forceinline__ Pre fetch(int, int m, int n) const {
        Pre r;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (m < M && n + h * 8 < f8) r.gu[h] = K::get(gu, m, n + h * 8);
        return r;
    }
    __device__ __forceinline__ void row(int, int, int m, int n, const f32x4 (&dh)[4], const Pre& pre) const {
        const int64_t at = (int64_t)m * 2 * f8 + n;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (m >= M || n + h * 8 >= f8) continue;
            f32x4 dg[2], du[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const f32x4 g = K::g(pre.gu[h], q), u = K::u(pre.gu[h], q), d = dh[h * 2 + q];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float a, da;
                    activation<F, ACT>(g[e], a, da);
                    du[q][e] = d[e] * a;
                    dg[q][e] = d[e] * u[e] * da;
                }
            }
            put_operand8<F>(dgu + at + h * 8, plane, dg[0], dg[1]);
            put_operand8<F>(dgu + at + f8 + h * 8, plane, du[0], du[1]);
        }
    }
};

// Plain store.  Rows [0, rows0) go to c0; rows [off1, off1 + rows0) to c1 (the two halves of a joint gradient).
template <class F>
struct EpiStore {
    static constexpr bool kDual = false, kSymmetric = false;
    static constexpr int kAhead = 0;
    using Pre = NoPre;
    typename F::Elem* c0;
    typename F::Elem* c1;
    int64_t ld;
    int rows0, off1, N;
    int vec;  // elements a store may take: 8, 4 or 1
    __device__ __forceinline__ Pre fetch(int, int, int) const { return {}; }
    __device__ __forceinline__ typename F::Elem* row_of(int m) const {
        if (m < rows0) return c0 ? c0 + (int64_t)m * ld : nullptr;
        const int r = m - off1;
        return c1 && r >= 0 && r < rows0 ? c1 + (int64_t)r * ld : nullptr;
    }
    __device__ __forceinline__ void put4(typename F::Elem* c, int n, f32x4 v) const {
        if (vec >= 4 && n + 4 <= N) {
            F::put(c + n, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < N) F::put1(c + n + e, v[e]);
        }
    }
    __device__ __forceinline__ void row(int, int, int m, int n, const f32x4 (&v)[4], const Pre&) const {
        row8(m, n, v[0], v[1]);
        row8(m, n + 8, v[2], v[3]);
    }
    __device__ __forceinline__ void row8(int m, int n, f32x4 v0, f32x4 v1) const {
        typename F::Elem* c = row_of(m);
        if (!c) return;
        if (vec == 8 && n + 8 <= N) {
            F::put8(c + n, v0, v1);
        } else {
            put4(c, n, v0);
            put4(c, n + 4, v1);
        }
    }
};

// float32 partial sums of a product split along k: part[split][M][n4]
struct EpiPartial {
    static constexpr bool kDual = false, kSymmetric = false;
    static constexpr int kAhead = 0;
    using Pre = NoPre;
    float* part;
    int64_t n4;
    int M;
    __device__ __forceinline__ Pre fetch(int, int, int) const { return {}; }
    __device__ __forceinline__ void row(int, int split, int m, int n, const f32x4 (&v)[4], const Pre&) const {
        if (m >= M) return;
        float* p = part + ((int64_t)split * M + m) * n4;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (n + q * 4 < n4) *(f32x4*)(p + n + q * 4) = v[q];
    }
};

// Sum of the partials, stored like EpiStore.  Eight threads share four columns' splits and their sums are joined in a
// fixed order (the result does not depend on scheduling); with one thread for all splits the many small loads in a
// row took 18 us for 64 splits of 512 x 57.
template <class F>
__global__ __launch_bounds__(256) void k_reduce(const float* part, int splits, int M, int64_t n4, EpiStore<F> st) {
    __shared__ f32x4 s_sum[8][32];
    const int64_t q4 = n4 / 4, n = (int64_t)M * q4;
    const int li = threadIdx.x & 31, g = threadIdx.x >> 5;
    for (int64_t i0 = (int64_t)blockIdx.x * 32; i0 < n; i0 += (int64_t)gridDim.x * 32) {
        const int64_t i = i0 + li;
        f32x4 s{0.f, 0.f, 0.f, 0.f};
        if (i < n) {
#pragma unroll 4
            for (int k = g; k < splits; k += 8) s += *(const f32x4*)(part + (int64_t)k * M * n4 + i * 4);
        }
        s_sum[g][li] = s;
        __syncthreads();
        if (g == 0 && i < n) {
#pragma unroll
            for (int k = 1; k < 8; ++k) s += s_sum[k][li];
            const int64_t m = i / q4;
            typename F::Elem* c = st.row_of((int)m);
            if (c) st.put4(c, (int)(i - m * q4) * 4, s);
        }
        __syncthreads();
    }
}

// ---- few rows ------------------------------------------------------------------------------------------

// At most 64 rows: the weights are read once, straight into the matrix instructions' operands, and that is all the
// work there is.  A workgroup takes 16 or 8 columns (of both projections) and splits k over its waves; the partial sums
// meet in LDS.  Every wave's loads are independent, so the whole weight matrix is in flight at once.  One row of 1024 x
// 4096 x 1024 bfloat16: 6.2 + 6.3 us for 16.8 and 8.4 MB, half of it the launch and the first load's latency.  48 rows
// of 1024 x 2816 x 1024: 9.0 + 12.8 us; the second is bound by its rows, which every workgroup reads in full (393 KB a
// CU).
// 16-bit: lane l holds row l % 16, k (l / 16) * 8 .. + 8 of a 16x16x32 product.  float32: k (l / 16) * 4 + j for the
// j-th of four 16x16x4 products (both operands permute k alike).  WIDE: rows allow 16-byte loads; otherwise
// elements are read one by one.
constexpr int kFewRows = 64;

template <class F>
struct FewRows {
    static constexpr uint32_t kElem = sizeof(typename F::Elem);
    static constexpr int kStep = 64 / kElem;   // k of one set of fragments
    static constexpr int kLane = kStep / 4;    // elements of a lane

    // the lane's elements of one row, k0 .. of K; `row` is the byte offset of the row or kOobOffset
    template <bool WIDE>
    static __device__ __forceinline__ u32x4 load(__amdgpu_buffer_rsrc_t rs, uint32_t row, int k0, int K) {
        if constexpr (WIDE) {
            const uint32_t off = k0 < K ? row + k0 * kElem : kOobOffset;
            return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
        } else if constexpr (kElem == 4) {
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = __builtin_amdgcn_raw_buffer_load_b32(rs, k0 + e < K ? row + (k0 + e) * 4u : kOobOffset, 0, 0);
            return v;
        } else {
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = k0 + e * 2;
                const uint32_t lo =
                    (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, k < K ? row + k * 2u : kOobOffset, 0, 0);
                const uint32_t hi =
                    (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, k + 1 < K ? row + k * 2u + 2u : kOobOffset, 0, 0);
                v[e] = lo | (hi << 16);
            }
            return v;
        }
    }
    static __device__ __forceinline__ f32x4 multiply(u32x4 w, u32x4 x, f32x4 acc) {
        using T = std::conditional_t<kElem == 4, float, typename F::Mma>;
        return Mfma<T>::run(__builtin_bit_cast(s16x8, w), __builtin_bit_cast(s16x8, x), acc);
    }
};

struct FewArgs {
    const void* x;
    const void* w;
    const void* w2;  // the second projection of a dual product
    int M, N, K;
    int cols;    // columns of a workgroup: 16 or 8
    int64_t ldx, ldw;
};

// MT tiles of 16 rows, NW waves
template <class F, int MT, int NW, bool WIDE, class Epi>
__global__ __launch_bounds__(NW * 64) void k_few_rows(const FewArgs p, const Epi epi) {
    using R = FewRows<F>;
    using E = typename F::Elem;
    constexpr int ND = Epi::kDual ? 2 : 1;
    // steps of weights that are fetched together, and of rows, one fetch ahead of the products (48 rows, 2816 -> 1024:
    // 12.8 us, 14.1 with all of four steps at a time)
    constexpr int kAhead = MT == 1 ? 8 : ND == 2 ? 4 : 6, kRows = 2;
    __shared__ __attribute__((aligned(16))) float red[NW][MT * 16][ND * 16 + 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * p.cols, li = lane & 15;
    const int steps = (p.K + R::kStep - 1) / R::kStep, per = (steps + NW - 1) / NW;
    const int s0 = wave * per, s1 = min(steps, s0 + per);
    const E* w0 = (const E*)p.w + (int64_t)n0 * p.ldw;
    const E* w1 = (const E*)(Epi::kDual ? p.w2 : p.w) + (int64_t)n0 * p.ldw;
    const __amdgpu_buffer_rsrc_t rw[2] = {gemm_rsrc(w0), gemm_rsrc(w1)};
    const __amdgpu_buffer_rsrc_t rx = gemm_rsrc(p.x);
    const uint32_t wrow = li < p.cols && n0 + li < p.N ? (uint32_t)li * (uint32_t)p.ldw * R::kElem : kOobOffset;
    uint32_t xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        xrow[m] = m * 16 + li < p.M ? (uint32_t)(m * 16 + li) * (uint32_t)p.ldx * R::kElem : kOobOffset;
    f32x4 acc[MT][ND];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = s0; s < s1; s += kAhead) {
        u32x4 wf[kAhead][ND], xf[2][kRows][MT];
        // past the wave's share: out of range, zero
        auto k_of = [&](int i) { return s + i < s1 ? (s + i) * R::kStep + (lane >> 4) * R::kLane : p.K; };
        auto fetch = [&](int i) {
#pragma unroll
            for (int q = 0; q < kRows; ++q)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    xf[i / kRows & 1][q][m] =
                        R::template load<WIDE>(rx, xrow[m], xrow[m] == kOobOffset ? p.K : k_of(i + q), p.K);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int d = 0; d < ND; ++d)
                wf[i][d] = R::template load<WIDE>(rw[d], wrow, wrow == kOobOffset ? p.K : k_of(i), p.K);
        fetch(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kAhead; i += kRows) {
            if (i + kRows < kAhead) fetch(i + kRows);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < kRows; ++q)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int d = 0; d < ND; ++d)
                        acc[m][d] = R::multiply(wf[i + q][d], xf[i / kRows & 1][q][m], acc[m][d]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int d = 0; d < ND; ++d)
            *(f32x4*)&red[wave][m * 16 + li][d * 16 + (lane >> 4) * 4] = acc[m][d];
    __syncthreads();
    // eight columns of one row (dual: of both products) a thread, the waves' sums in order
    for (int t = threadIdx.x; t < MT * 32; t += NW * 64) {
        const int m = t >> 1, c = (t & 1) * 8;
        if (c >= p.cols) continue;
        f32x4 v[2 * ND];
#pragma unroll
        for (int q = 0; q < 2 * ND; ++q) {
            const int at = (q >> 1) * 16 + c + (q & 1) * 4;
            v[q] = *(const f32x4*)&red[0][m][at];
#pragma unroll 4
            for (int w = 1; w < NW; ++w) v[q] += *(const f32x4*)&red[w][m][at];
        }
        if constexpr (Epi::kDual)
            epi.row(m, n0 + c, v[0], v[1], v[2], v[3]);
        else
            epi.row8(m, n0 + c, v[0], v[1]);
    }
}

// ---- launchers -----------------------------------------------------------------------------------------

// Segments of one product: one, or the six partial products of split operands, the smallest first.
template <class F>
void add_segments(GemmArgs& g, const Operand& a, const Operand& b, const Operand* b2, int64_t a_off = 0) {
    static const int pa[6] = {2, 0, 1, 1, 0, 0}, pb[6] = {0, 2, 1, 0, 1, 0};
    const int n = F::kPlanes == 1 ? 1 : 6;
    for (int i = 0; i < n; ++i) {
        const int ia = F::kPlanes == 1 ? 0 : pa[i], ib = F::kPlanes == 1 ? 0 : pb[i];
        using E = OperandElem<F>;
        g.a[g.nseg] = (const char*)((const E*)a.p + ia * a.plane + a_off);
        g.b[g.nseg] = (const char*)((const E*)b.p + ib * b.plane);
        g.b2[g.nseg] = b2 ? (const char*)((const E*)b2->p + ib * b2->plane) : nullptr;
        ++g.nseg;
    }
    g.lda = a.ld;
    g.ldb = b.ld;
}

// Weight gradients may be split along the rows they sum over.
constexpr int kMaxSplits = 128;
template <class F>
GemmPlan grad_plan(int64_t M, int64_t N, int64_t K) {
    constexpr int bk = kTileK<typename F::Mma>;
    return plan_gemm(M, N, 1, (K + bk - 1) / bk * (F::kPlanes == 1 ? 1 : 6), false, false, kMaxSplits,
                     sizeof(typename F::Mma) == 4);
}

template <class F>
struct Layout {
    int64_t M, D, H, O, D8, H8, O8;
    explicit Layout(const gs_ffn_dims& d)
        : M(d.rows), D(d.d_in), H(d.d_hidden), O(d.d_out), D8(round8(D)), H8(round8(H)), O8(round8(O)) {}
    int64_t saved_gu_bytes() const { return round_up(F::Keep::bytes(M * H8), kAlign); }
    Kept kept(const void* saved) const { return {(char*)saved, H8, M * H8}; }
    int64_t h_elems() const { return M * H8 * F::kPlanes; }
    int64_t h_bytes() const { return round_up(h_elems() * (int64_t)sizeof(OperandElem<F>), kAlign); }
};

// An operand is read in place when its rows are 16-byte aligned and a multiple of 8 elements long: the backward products
// run over row lengths rounded up to 8, which an unpadded array does not have.
template <class F>
bool direct(const void* p, int64_t cols, int64_t ld) {
    constexpr int64_t e = 16 / (int64_t)sizeof(OperandElem<F>);
    return F::kPlanes == 1 && cols % 8 == 0 && ld % e == 0 && ((uintptr_t)p % 16) == 0;
}

struct Packer {
    PackJobs jobs{};
    int n = 0;
    int64_t most = 0;
    template <class F>
    Operand add(Carver& cv, const void* src, int64_t rows, int64_t cols, int64_t ld,
                bool always = false) {
        if (!always && direct<F>(src, cols, ld)) return {src, 0, ld};
        const int64_t c8 = round8(cols);
        OperandElem<F>* d = cv.take<OperandElem<F>>(rows * c8 * F::kPlanes);
        jobs.j[n++] = {src, d, rows, cols, ld, rows * c8};
        if (rows * c8 / 8 > most) most = rows * c8 / 8;
        return {d, rows * c8, c8};
    }
    template <class F>
    hipError_t launch(hipStream_t st) const {
        if (!n || !most) return hipSuccess;
        int64_t bx = (most + 255) / 256;
        if (bx > 4096) bx = 4096;
        k_pack<F><<<dim3((unsigned)bx, (unsigned)n), 256, 0, st>>>(jobs);
        return hipGetLastError();
    }
};

template <class F, int NW, bool WIDE, class Epi>
hipError_t launch_few(FewArgs p, const Epi& epi, hipStream_t st) {
    // Eight columns a workgroup as long as that makes at most one workgroup a CU, else 16.  The whole forward pass in us
    // with 8 and with 16 columns in the product named, bfloat16, the other product small and the same:
    //   projections, 1024 wide         1 row          16 rows        48 rows
    //     1024 columns             10.2 / 10.8    11.5 / 12.1    15.9 / 16.5
    //     2048 columns             10.5 / 11.1    12.6 / 13.1    18.4 / 18.8
    //     2816 columns             12.6 / 11.2    15.8 / 13.8    24.4 / 20.4
    //   down product, 2816 wide
    //     1024 columns              9.7 / 10.4    11.8 / 12.4    17.8 / 18.5
    //     2048 columns              9.9 / 10.6    12.0 / 12.6    18.2 / 18.8
    //     2816 columns             12.3 / 10.6    16.2 / 12.7    29.0 / 18.9
    // (float32 alike: one row of 2816 to 2048 15.9 / 16.9, to 2816 22.0 / 18.0.)
    constexpr int kCus = 256;
    p.cols = p.N <= 8 * kCus ? 8 : 16;
    const dim3 gd((unsigned)((p.N + p.cols - 1) / p.cols)), bd(NW * 64);
    if (p.M <= 16)
        k_few_rows<F, 1, NW, WIDE, Epi><<<gd, bd, 0, st>>>(p, epi);
    else if (p.M <= 32)
        k_few_rows<F, 2, NW, WIDE, Epi><<<gd, bd, 0, st>>>(p, epi);
    else
        k_few_rows<F, 4, NW, WIDE, Epi><<<gd, bd, 0, st>>>(p, epi);
    return hipGetLastError();
}

// 16-byte loads: rows of 16-byte multiples on 16-byte boundaries
template <class F>
bool wide_rows(const void* p, int64_t cols, int64_t ld) {
    const int64_t e = 16 / (int64_t)sizeof(typename F::Elem);
    return cols % e == 0 && ld % e == 0 && ((uintptr_t)p % 16) == 0;
}

template <class F, int ACT>
hipError_t forward_few(const gs_ffn_dims& d, const void* x, int64_t ldx, const gs_ffn_weights& w, void* y,
                       int64_t ldy, void* saved, char* ws, hipStream_t st) {
    using E = typename F::Elem;
    const Layout<F> L(d);
    Carver cv{ws};
    EpiGateFew<F, ACT> e1{{nullptr, L.M * L.H8, L.kept(nullptr), L.H8, (int)L.M}, nullptr};
    if (saved) {
        e1.all.gu = L.kept(saved);
        e1.all.h = (OperandElem<F>*)((char*)saved + L.saved_gu_bytes());
    }
    // the 16-bit h that is kept is the next product's input too
    e1.h = saved && F::kPlanes == 1 ? (E*)e1.all.h : cv.take<E>(L.M * L.H8);
    FewArgs a{x, w.gate, w.up, (int)L.M, (int)L.H, (int)L.D, 16, ldx, L.D};
    if (wide_rows<F>(x, L.D, ldx) && wide_rows<F>(w.gate, L.D, L.D) && wide_rows<F>(w.up, L.D, L.D))
        GSR_TRY((launch_few<F, 8, true>(a, e1, st)));
    else
        GSR_TRY((launch_few<F, 8, false>(a, e1, st)));
    FewArgs b{e1.h, w.down, nullptr, (int)L.M, (int)L.O, (int)L.H, 16, L.H8, L.H};
    EpiStore<F> e2{(E*)y, nullptr, ldy, (int)L.M, 0, (int)L.O, vec_width(y, ldy, sizeof(E))};
    if (wide_rows<F>(w.down, L.H, L.H)) return launch_few<F, 16, true>(b, e2, st);
    return launch_few<F, 16, false>(b, e2, st);
}

template <class F, int ACT>
hipError_t forward_impl(const gs_ffn_dims& d, const void* x, int64_t ldx, const gs_ffn_weights& w, void* y,
                        int64_t ldy, void* saved, char* ws, hipStream_t st) {
    using E = typename F::Elem;
    const Layout<F> L(d);
    if (L.M <= kFewRows) return forward_few<F, ACT>(d, x, ldx, w, y, ldy, saved, ws, st);
    Carver cv{ws};
    Packer pk;
    const Operand ox = pk.add<F>(cv, x, L.M, L.D, ldx);
    const bool wdir = direct<F>(w.gate, L.D, L.D) && direct<F>(w.up, L.D, L.D);
    Operand og, ou;
    if (wdir) {
        og = {w.gate, 0, L.D};
        ou = {w.up, 0, L.D};
    } else {  // the dual product reads both with one row length
        og = pk.add<F>(cv, w.gate, L.H, L.D, L.D, true);
        ou = pk.add<F>(cv, w.up, L.H, L.D, L.D, true);
    }
    const Operand od = pk.add<F>(cv, w.down, L.O, L.H, L.H);
    GSR_TRY(pk.launch<F>(st));
    OperandElem<F>* h;
    if (saved) {
        h = (OperandElem<F>*)((char*)saved + L.saved_gu_bytes());
    } else {
        h = cv.take<OperandElem<F>>(L.h_elems());
    }
    const int64_t h_plane = L.M * L.H8;
    GemmArgs g1 = make_args(L.M, L.H, L.D);
    add_segments<F>(g1, ox, og, &ou);
    EpiGate<F, ACT> e1{h, h_plane, L.kept(saved), L.H8, (int)L.M};
    GSR_TRY((launch_gemm<typename F::Mma, true, true>(g1, e1, st)));
    GemmArgs g2 = make_args(L.M, L.O, L.H8);
    add_segments<F>(g2, Operand{h, h_plane, L.H8}, od, nullptr);
    g2.K = (int)L.H;
    EpiStore<F> e2{(E*)y, nullptr, ldy, (int)L.M, 0, (int)L.O, vec_width(y, ldy, sizeof(E))};
    return launch_gemm<typename F::Mma, true, true>(g2, e2, st);
}

template <class F>
hipError_t weight_grad(const Operand& a, int64_t a_cols, const Operand& b, int64_t b_cols, int64_t rows,
                       EpiStore<F> store, float* part, hipStream_t st) {
    GemmArgs g = make_args(a_cols, b_cols, rows);
    add_segments<F>(g, a, b, nullptr);
    const GemmPlan plan = grad_plan<F>(a_cols, b_cols, rows);
    if (plan.splits == 1) return launch_planned<typename F::Mma, false, false>(g, plan, store, st);
    const int64_t n4 = (store.N + 3) / 4 * 4;
    EpiPartial ep{part, n4, (int)a_cols};
    GSR_TRY((launch_planned<typename F::Mma, false, false>(g, plan, ep, st)));
    int64_t bx = (a_cols * n4 / 4 + 31) / 32;
    if (bx > 8192) bx = 8192;
    k_reduce<F><<<dim3((unsigned)bx), 256, 0, st>>>(part, plan.splits, (int)a_cols, n4, store);
    return hipGetLastError();
}

template <class F>
int64_t part_elems(const Layout<F>& L) {
    const int64_t s1 = grad_plan<F>(2 * L.H8, L.D8, L.M).splits, s2 = grad_plan<F>(L.O8, L.H8, L.M).splits;
    const int64_t p1 = s1 > 1 ? s1 * 2 * L.H8 * L.D8 : 0, p2 = s2 > 1 ? s2 * L.O8 * L.H8 : 0;
    return p1 > p2 ? p1 : p2;
}

template <class F, int ACT>
hipError_t backward_impl(const gs_ffn_dims& d, const void* x, int64_t ldx, const gs_ffn_weights& w,
                         const void* saved, const void* dy, int64_t lddy, const gs_ffn_grads& out, int64_t lddx,
                         char* ws, hipStream_t st) {
    using E = typename F::Elem;
    using T = typename F::Mma;
    const Layout<F> L(d);
    Carver cv{ws};
    float* part = cv.take<float>(part_elems<F>(L));
    const int64_t plane = L.M * 2 * L.H8;
    OperandElem<F>* dgu = cv.take<OperandElem<F>>(plane * F::kPlanes);
    const OperandElem<F>* h = (const OperandElem<F>*)((const char*)saved + L.saved_gu_bytes());
    const int64_t h_plane = L.M * L.H8;
    Packer pk;
    const Operand ody = pk.add<F>(cv, dy, L.M, L.O, lddy);
    const Operand od = pk.add<F>(cv, w.down, L.O, L.H, L.H);
    const Operand ox = pk.add<F>(cv, x, L.M, L.D, ldx);
    // one row length for both weight matrices of dx
    const bool wpack = !(direct<F>(w.gate, L.D, L.D) && direct<F>(w.up, L.D, L.D));
    const Operand og = pk.add<F>(cv, w.gate, L.H, L.D, L.D, wpack);
    const Operand ou = pk.add<F>(cv, w.up, L.H, L.D, L.D, wpack);
    GSR_TRY(pk.launch<F>(st));

    GemmArgs g1 = make_args(L.M, L.H8, L.O);
    add_segments<F>(g1, ody, od, nullptr);
    EpiGateGrad<F, ACT> e1{L.kept(saved), dgu, plane, L.H8, (int)L.M};
    GSR_TRY((launch_gemm<T, true, false>(g1, e1, st)));
    const Operand odgu{dgu, plane, 2 * L.H8};
    if (out.x) {
        GemmArgs g2 = make_args(L.M, L.D8, L.H);
        add_segments<F>(g2, odgu, og, nullptr, 0);
        add_segments<F>(g2, odgu, ou, nullptr, L.H8);
        EpiStore<F> e2{(E*)out.x, nullptr, lddx, (int)L.M, 0, (int)L.D, vec_width(out.x, lddx, sizeof(E))};
        GSR_TRY((launch_gemm<T, true, false>(g2, e2, st)));
    }
    if (out.gate || out.up) {
        EpiStore<F> e3{(E*)out.gate, (E*)out.up, L.D, (int)L.H, (int)L.H8, (int)L.D,
                       std::min(vec_width(out.gate, L.D, sizeof(E)), vec_width(out.up, L.D, sizeof(E)))};
        GSR_TRY(weight_grad<F>(odgu, 2 * L.H8, ox, L.D8, L.M, e3, part, st));
    }
    if (out.down) {
        EpiStore<F> e4{(E*)out.down, nullptr, L.H, (int)L.O, 0, (int)L.H, vec_width(out.down, L.H, sizeof(E))};
        GSR_TRY(weight_grad<F>(ody, L.O8, Operand{h, h_plane, L.H8}, L.H8, L.M, e4, part, st));
    }
    return hipSuccess;
}

template <class F>
void sizes_impl(const gs_ffn_dims& d, size_t* saved, size_t* fwd, size_t* bwd) {
    const Layout<F> L(d);
    auto pad = [](int64_t rows, int64_t c8) {
        return round_up(rows * c8 * F::kPlanes * (int64_t)sizeof(OperandElem<F>), kAlign);
    };
    *saved = (size_t)(L.saved_gu_bytes() + L.h_bytes());
    // every operand counted as copied: whether one is depends on its address and stride
    const int64_t weights = 2 * pad(L.H, L.D8) + pad(L.O, L.H8) + pad(L.M, L.D8);
    *fwd = (size_t)(weights + std::max(L.h_bytes(), round_up(L.M * L.H8 * (int64_t)sizeof(typename F::Elem), kAlign)));
    *bwd = (size_t)(weights + pad(L.M, L.O8) + pad(L.M, 2 * L.H8) + round_up(part_elems<F>(L) * 4, kAlign));
}

}  // namespace

namespace {

// Whether float32 operands are split.  Six products at the bfloat16 rate take half the time of one at the float32
// rate, but move 6 bytes per value instead of 4, convert every operand, and want large tiles.  Measured, forward and
// backward together in us:
//   rows x in x hidden x out       f32    split      rows x in x hidden x out       f32    split
//   23040 x 57 x 256 x 128         176      204      23040 x 256 x 512 x 256        602      559
//   131072 x 64 x 256 x 64         604      932      65536 x 192 x 768 x 192       1897     1563
//   131072 x 128 x 512 x 128      1668     1919      8192 x 512 x 2048 x 512       1331     1176
//   2048 x 512 x 2048 x 512        419      518      4000 x 2048 x 4096 x 2048     4626     3187
//   1000 x 1000 x 2731 x 1000      609      798      16384 x 1024 x 4096 x 1024    9381     6148
// (4000 x 512 x 2048 x 512 and 16384 x 256 x 1024 x 256 are within 4 %.)  So: rows of at least 192 values and
// enough work.
bool split_f32(const gs_ffn_dims& d) {
    return d.d_in >= 192 && d.d_out >= 192 &&
           (double)d.rows * d.d_hidden * (2.0 * d.d_in + d.d_out) >= 8589934592.0;  // 2^33 multiplications
}

}  // namespace

void ffn_sizes(const gs_ffn_dims& d, size_t* saved, size_t* fwd, size_t* bwd) {
    if (d.dtype == GS_F32 && split_f32(d)) return sizes_impl<FmtF32Split>(d, saved, fwd, bwd);
    if (d.dtype == GS_F32) return sizes_impl<FmtF32>(d, saved, fwd, bwd);
    if (d.dtype == GS_F16) return sizes_impl<FmtF16>(d, saved, fwd, bwd);
    return sizes_impl<FmtBf16>(d, saved, fwd, bwd);
}

hipError_t launch_ffn_forward(const gs_ffn_dims& d, const void* x, int64_t ldx, const gs_ffn_weights& w, void* y,
                              int64_t ldy, void* saved, void* ws, hipStream_t st) {
    char* b = (char*)ws;
    const bool silu = d.activation == GS_ACT_SILU;
    if (d.dtype == GS_BF16)
        return silu ? forward_impl<FmtBf16, GS_ACT_SILU>(d, x, ldx, w, y, ldy, saved, b, st)
                    : forward_impl<FmtBf16, GS_ACT_GELU>(d, x, ldx, w, y, ldy, saved, b, st);
    if (d.dtype == GS_F16)
        return silu ? forward_impl<FmtF16, GS_ACT_SILU>(d, x, ldx, w, y, ldy, saved, b, st)
                    : forward_impl<FmtF16, GS_ACT_GELU>(d, x, ldx, w, y, ldy, saved, b, st);
    if (split_f32(d))
        return silu ? forward_impl<FmtF32Split, GS_ACT_SILU>(d, x, ldx, w, y, ldy, saved, b, st)
                    : forward_impl<FmtF32Split, GS_ACT_GELU>(d, x, ldx, w, y, ldy, saved, b, st);
    return silu ? forward_impl<FmtF32, GS_ACT_SILU>(d, x, ldx, w, y, ldy, saved, b, st)
                : forward_impl<FmtF32, GS_ACT_GELU>(d, x, ldx, w, y, ldy, saved, b, st);
}

hipError_t launch_ffn_backward(const gs_ffn_dims& d, const void* x, int64_t ldx, const gs_ffn_weights& w,
                               const void* saved, const void* dy, int64_t lddy, const gs_ffn_grads& out,
                               int64_t lddx, void* ws, hipStream_t st) {
    char* b = (char*)ws;
    const bool silu = d.activation == GS_ACT_SILU;
    if (d.dtype == GS_BF16)
        return silu ? backward_impl<FmtBf16, GS_ACT_SILU>(d, x, ldx, w, saved, dy, lddy, out, lddx, b, st)
                    : backward_impl<FmtBf16, GS_ACT_GELU>(d, x, ldx, w, saved, dy, lddy, out, lddx, b, st);
    if (d.dtype == GS_F16)
        return silu ? backward_impl<FmtF16, GS_ACT_SILU>(d, x, ldx, w, saved, dy, lddy, out, lddx, b, st)
                    : backward_impl<FmtF16, GS_ACT_GELU>(d, x, ldx, w, saved, dy, lddy, out, lddx, b, st);
    if (split_f32(d))
        return silu ? backward_impl<FmtF32Split, GS_ACT_SILU>(d, x, ldx, w, saved, dy, lddy, out, lddx, b, st)
                    : backward_impl<FmtF32Split, GS_ACT_GELU>(d, x, ldx, w, saved, dy, lddy, out, lddx, b, st);
    return silu ? backward_impl<FmtF32, GS_ACT_SILU>(d, x, ldx, w, saved, dy, lddy, out, lddx, b, st)
                : backward_impl<FmtF32, GS_ACT_GELU>(d, x, ldx, w, saved, dy, lddy, out, lddx, b, st);
}

}  // namespace gsr
