// gemm16.hpp -- the matrix-core product of the updater's operators (device code and its launcher).
//
//   C[m][n] = sum over segments s, k of A_s(m, k) B_s(n, k),   16-bit operands, float32 accumulation.
//
// Each operand is stored either with k contiguous ([rows][k], "KC") or with its rows contiguous ([k][rows]); the
// four products of a block's forward and backward pass then need no transposed copies.  A list of segments adds up
// several products in one accumulator: two weight matrices of one gradient, or the six (three) partial products
// that make a float32 product out of operands split into bfloat16 (float16) parts.
//
// Tile BM x BN x 64 per workgroup, split over WM x WN waves of 16x16x32 matrix instructions.  Tiles go from global
// memory to LDS directly (16 bytes per lane, no registers), double buffered.  A row of a KC tile is 128 bytes = 8
// chunks; chunk c of row r lies at chunk position c ^ (r & 7), so the 16-byte fragment reads of 8 consecutive rows
// cover all banks.  A tile with rows contiguous keeps its [k][row] order and is read with the LDS transpose read
// (4 k x 16 rows per 16 lanes); chunk position c ^ f(k) spreads the four k rows over the banks.
// Out-of-range rows and k read as zero through the buffer descriptor's range check.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

namespace gsr {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kGemmSegs = 12;
constexpr int kGemmBK = 64;

struct GemmArgs {
    const uint16_t* a[kGemmSegs];
    const uint16_t* b[kGemmSegs];
    const uint16_t* b2[kGemmSegs];  // second matrix of a dual product (same layout as b)
    int nseg;
    int M, N, K;
    int64_t lda, ldb;                  // elements between rows of the stored arrays
    int64_t batch_a, batch_b;          // elements between the batch's matrices
    int tiles_m, tiles_n, batch;
    int splits;                        // workgroups along k (1: none)
    int tiles_per_split;               // k tiles of one split
};

template <class T>
struct Mfma;
template <>
struct Mfma<__bf16> {
    static __device__ __forceinline__ f32x4 run(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16> {
    static __device__ __forceinline__ f32x4 run(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b),
                                                      c, 0, 0, 0);
    }
};

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// An offset past every descriptor's range: the lane reads zero.
constexpr uint32_t kOobOffset = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t gemm_rsrc(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, 0x7fffffff, 0x00020000);
}

// Loader of one operand's tiles: R rows x 64 k by NT threads.
template <bool KC, int R, int NT, bool DUAL, int WROWS>
struct TileLoader {
    static constexpr int kLoads = R * 8 / NT;
    static constexpr int kBytes = R * 128;
    uint32_t off[kLoads];  // byte offset within the tile, kOobOffset for rows out of range
    int kk[kLoads];        // k within the tile of the chunk (its first k for KC)

    __device__ __forceinline__ void init(int tid, int row0, int rows, int64_t ld) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = i * NT + tid;
            if (KC) {
                int r = q >> 3;
                const int c = (q & 7) ^ (r & 7);
                // dual: the wave's WROWS rows are WROWS/2 of the first matrix, then the same rows of the second
                if (DUAL) r = (r / WROWS) * (WROWS / 2) + (r % (WROWS / 2));
                kk[i] = c * 8;
                off[i] = row0 + r < rows ? (uint32_t)(r * (uint32_t)ld * 2u + c * 16u) : kOobOffset;
            } else {
                constexpr int CH = R / 8;
                const int k = q / CH;
                const int c = (q % CH) ^ swz(k);
                kk[i] = k;
                off[i] = row0 + c * 8 < rows ? (uint32_t)(k * (uint32_t)ld * 2u + c * 16u) : kOobOffset;
            }
        }
    }
    static __device__ __forceinline__ int swz(int k) { return 2 * ((k & 3) | ((k >> 1) & 4)); }

    // first / second: the tile's first element in the (two) matrices; krem: k left from the tile's start
    __device__ __forceinline__ void load(const uint16_t* first, const uint16_t* second, int krem, char* lds,
                                         int tid) const {
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const __amdgpu_buffer_rsrc_t ra = gemm_rsrc(first);
        const __amdgpu_buffer_rsrc_t rb = DUAL ? gemm_rsrc(second) : ra;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t o = kk[i] < krem ? off[i] : kOobOffset;
            // dual: the 8 rows of one instruction belong to one matrix
            const bool up = DUAL && (((i * NT + wave * 64) >> 3) % WROWS) >= WROWS / 2;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? rb : ra, (lds_void*)(lds + (i * NT + wave * 64) * 16), 16, o,
                                                     0, 0, 0);
        }
    }
    // fragment of 16 rows from row r0, k from kk0 (0 or 32): lane l holds row l % 16, k (l / 16) * 8 .. + 8
    static __device__ __forceinline__ s16x8 frag(const char* lds, int r0, int kk0, int lane) {
        if (KC) {
            const int r = r0 + (lane & 15);
            const int c = ((kk0 >> 3) + (lane >> 4)) ^ (r & 7);
            return *reinterpret_cast<const s16x8*>(lds + r * 128 + c * 16);
        } else {
            s16x8 v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kk0 + (lane >> 4) * 8 + h * 4 + ((lane & 15) >> 2);
                const int col = r0 + (lane & 3) * 4;
                const char* p = lds + k * (R * 2) + (((col >> 3) ^ swz(k)) << 4) + (col & 4) * 2;
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[h * 4 + e] = t[e];
            }
            return v;
        }
    }
};

// Tile of a workgroup: workgroups are dealt to the 8 XCDs in turn, so each XCD gets a contiguous run of tiles; in
// the run, groups of 8 tile rows are walked column by column so that neighbours share operand tiles in the XCD's L2.
__device__ __forceinline__ void gemm_tile(const GemmArgs& p, int id, int& tm, int& tn) {
    constexpr int kGroup = 8;
    const int per = kGroup * p.tiles_n;
    const int g = id / per;
    const int rows = min(kGroup, p.tiles_m - g * kGroup);
    const int in = id - g * per;
    tm = g * kGroup + in % rows;
    tn = in / rows;
}

__device__ __forceinline__ int xcd_order(int bid, int n) {
    const int x = bid & 7, l = bid >> 3;
    const int q = n >> 3, r = n & 7;
    return x * q + min(x, r) + l;
}

template <class T, bool AKC, bool BKC, int BM, int BN, int WM, int WN, class Epi>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_gemm16(const GemmArgs p,
                                                                                         const Epi epi) {
    constexpr int NT = WM * WN * 64;
    constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    using LA = TileLoader<AKC, BM, NT, false, BM>;
    using LB = TileLoader<BKC, BN, NT, Epi::kDual, BN / WN>;
    constexpr int kStage = LA::kBytes + LB::kBytes;
    __shared__ __attribute__((aligned(1024))) char smem[2 * kStage];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int tiles = p.tiles_m * p.tiles_n;
    int id = xcd_order(blockIdx.x, gridDim.x);
    const int batch = id / (tiles * p.splits);
    id -= batch * (tiles * p.splits);
    const int split = id / tiles;
    int tm, tn;
    gemm_tile(p, id - split * tiles, tm, tn);
    if (Epi::kSymmetric && tm > tn) return;  // the mirrored tile writes both

    constexpr int BNR = Epi::kDual ? BN / 2 : BN;  // output columns of a tile
    const int m0 = tm * BM, n0 = tn * BNR;
    LA la;
    LB lb;
    la.init(tid, m0, p.M, p.lda);
    lb.init(tid, n0, p.N, p.ldb);

    const int ktiles = (p.K + kGemmBK - 1) / kGemmBK;
    const int total = ktiles * p.nseg;
    const int t_begin = split * p.tiles_per_split;
    const int t_end = min(total, t_begin + p.tiles_per_split);
    const int64_t a0 = batch * p.batch_a + (AKC ? (int64_t)m0 * p.lda : m0);
    const int64_t b0 = batch * p.batch_b + (BKC ? (int64_t)n0 * p.ldb : n0);
    const int64_t astep = AKC ? kGemmBK : kGemmBK * p.lda;
    const int64_t bstep = BKC ? kGemmBK : kGemmBK * p.ldb;

    f32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto issue = [&](int t, char* buf) {
        const int s = t / ktiles, kt = t - s * ktiles;
        const int krem = p.K - kt * kGemmBK;
        la.load(p.a[s] + a0 + kt * astep, nullptr, krem, buf, tid);
        lb.load(p.b[s] + b0 + kt * bstep, Epi::kDual ? p.b2[s] + b0 + kt * bstep : nullptr, krem, buf + LA::kBytes,
                tid);
    };
    if (t_begin < t_end) issue(t_begin, smem);
    for (int t = t_begin; t < t_end; ++t) {
        char* cur = smem + ((t - t_begin) & 1) * kStage;
        char* nxt = smem + ((t - t_begin + 1) & 1) * kStage;
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (t + 1 < t_end) issue(t + 1, nxt);
#pragma unroll
        for (int kk = 0; kk < kGemmBK; kk += 32) {
            s16x8 fa[MI], fb[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j) fb[j] = LB::frag(cur + LA::kBytes, wn * (BN / WN) + j * 16, kk, lane);
#pragma unroll
            for (int i = 0; i < MI; ++i) fa[i] = LA::frag(cur, wm * (BM / WM) + i * 16, kk, lane);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[i][j] = Mfma<T>::run(fb[j], fa[i], acc[i][j]);
        }
    }
    // lane: row m, four consecutive columns
    const int mb = m0 + wm * (BM / WM) + (lane & 15);
    const int nb = n0 + wn * (BNR / WN) + (lane >> 4) * 4;
    if constexpr (Epi::kDual) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI / 2; ++j) epi.pair(mb + i * 16, nb + j * 16, acc[i][j], acc[i][j + NI / 2]);
    } else {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) epi.one(batch, split, mb + i * 16, nb + j * 16, acc[i][j]);
    }
}

// ---- values in and out -------------------------------------------------------------------------------

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

template <class T>
__device__ __forceinline__ u16x4 to16(f32x4 v) {
    u16x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __builtin_bit_cast(uint16_t, (T)v[e]);
    return o;
}
template <class T>
__device__ __forceinline__ f32x4 from16(u16x4 v) {
    f32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (float)__builtin_bit_cast(T, (uint16_t)v[e]);
    return o;
}

// float32 as the sum of three bfloat16: hi + mid + lo carries 24 bits, each part rounded to nearest.  A value whose
// hi is not finite keeps zero remainders.
__device__ __forceinline__ void split3(float v, uint16_t& hi, uint16_t& mid, uint16_t& lo) {
    const __bf16 h = (__bf16)v;
    const float hf = (float)h;
    const bool fin = __builtin_fabsf(hf) < __builtin_inff();
    const float r1 = fin ? v - hf : 0.f;
    const __bf16 m = (__bf16)r1;
    const __bf16 l = (__bf16)(r1 - (float)m);
    hi = __builtin_bit_cast(uint16_t, h);
    mid = __builtin_bit_cast(uint16_t, m);
    lo = __builtin_bit_cast(uint16_t, l);
}

// Element formats of the block: what a stored 16-bit matrix operand and a value array look like for each type.
struct FmtBf16 {
    using Mma = __bf16;
    using Elem = uint16_t;  // value arrays (inputs, outputs, saved pre-activations)
    static constexpr int kPlanes = 1;
    static __device__ __forceinline__ f32x4 get(const Elem* p) { return from16<__bf16>(*(const u16x4*)p); }
    static __device__ __forceinline__ void put(Elem* p, f32x4 v) { *(u16x4*)p = to16<__bf16>(v); }
    static __device__ __forceinline__ float get1(const Elem* p) { return (float)__builtin_bit_cast(__bf16, *p); }
    static __device__ __forceinline__ void put1(Elem* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }
};
struct FmtF16 {
    using Mma = _Float16;
    using Elem = uint16_t;
    static constexpr int kPlanes = 1;
    static __device__ __forceinline__ f32x4 get(const Elem* p) { return from16<_Float16>(*(const u16x4*)p); }
    static __device__ __forceinline__ void put(Elem* p, f32x4 v) { *(u16x4*)p = to16<_Float16>(v); }
    static __device__ __forceinline__ float get1(const Elem* p) { return (float)__builtin_bit_cast(_Float16, *p); }
    static __device__ __forceinline__ void put1(Elem* p, float v) { *p = __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct FmtF32 {
    using Mma = __bf16;
    using Elem = float;
    static constexpr int kPlanes = 3;  // matrix operands are split into three bfloat16 planes
    static __device__ __forceinline__ f32x4 get(const Elem* p) { return *(const f32x4*)p; }
    static __device__ __forceinline__ void put(Elem* p, f32x4 v) { *(f32x4*)p = v; }
    static __device__ __forceinline__ float get1(const Elem* p) { return *p; }
    static __device__ __forceinline__ void put1(Elem* p, float v) { *p = v; }
};

// Four consecutive values of a matrix operand (one or three planes).
template <class F>
__device__ __forceinline__ void put_operand(uint16_t* p, int64_t plane, f32x4 v) {
    if constexpr (F::kPlanes == 1) {
        *(u16x4*)p = to16<typename F::Mma>(v);
    } else {
        u16x4 h, m, l;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint16_t a, b, c;
            split3(v[e], a, b, c);
            h[e] = a, m[e] = b, l[e] = c;
        }
        *(u16x4*)p = h;
        *(u16x4*)(p + plane) = m;
        *(u16x4*)(p + 2 * plane) = l;
    }
}

// ---- launchers -----------------------------------------------------------------------------------------

template <class T, bool AKC, bool BKC, int BM, int BN, int WM, int WN, class Epi>
inline hipError_t launch_tiles(GemmArgs p, const Epi& epi, hipStream_t st) {
    constexpr int BNR = Epi::kDual ? BN / 2 : BN;
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_n = (p.N + BNR - 1) / BNR;
    const int64_t n = (int64_t)p.tiles_m * p.tiles_n * p.batch * p.splits;
    if (n <= 0) return hipSuccess;
    if (n > 0x7fffffff) return hipErrorInvalidValue;
    k_gemm16<T, AKC, BKC, BM, BN, WM, WN, Epi><<<dim3((unsigned)n), dim3(WM * WN * 64), 0, st>>>(p, epi);
    return hipGetLastError();
}

inline int64_t tile_count(const GemmArgs& p, int bm, int bnr) {
    return (int64_t)((p.M + bm - 1) / bm) * ((p.N + bnr - 1) / bnr) * p.batch * p.splits;
}

// 256x256 tiles read each operand half as often as 128x128 ones but leave CUs idle below one tile per CU.
constexpr int64_t kBigTiles = 192;

template <class T, bool AKC, bool BKC, class Epi>
inline hipError_t launch_gemm(const GemmArgs& p, const Epi& epi, hipStream_t st) {
    if (tile_count(p, 256, Epi::kDual ? 128 : 256) >= kBigTiles)
        return launch_tiles<T, AKC, BKC, 256, 256, 2, 4, Epi>(p, epi, st);
    return launch_tiles<T, AKC, BKC, 128, 128, 2, 2, Epi>(p, epi, st);
}

// One stored matrix operand: planes (split operands) `plane` elements apart, rows of `ld` elements.
struct Operand {
    const uint16_t* p;
    int64_t plane, ld;
};

inline GemmArgs make_args(int64_t M, int64_t N, int64_t K) {
    GemmArgs g{};
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.batch = 1;
    g.splits = 1;
    return g;
}

// all k tiles in one workgroup per output tile
inline void one_split(GemmArgs& g) {
    g.splits = 1;
    g.tiles_per_split = g.nseg * ((g.K + kGemmBK - 1) / kGemmBK);
}

// ---- workspace -----------------------------------------------------------------------------------------

constexpr int64_t kAlign = 256;
inline int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }
inline int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

struct Carver {
    char* base;
    int64_t used = 0;
    template <class P>
    P* take(int64_t n) {
        P* p = base ? (P*)(base + used) : nullptr;
        used += round_up(n * (int64_t)sizeof(P), kAlign);
        return p;
    }
};

inline bool vec_ok(const void* p, int64_t ld, size_t elem) { return ld % 4 == 0 && ((uintptr_t)p % (4 * elem)) == 0; }

#define GSR_TRY(x)                          \
    do {                                    \
        hipError_t e_ = (x);                \
        if (e_ != hipSuccess) return e_;    \
    } while (0)

}  // namespace gsr
