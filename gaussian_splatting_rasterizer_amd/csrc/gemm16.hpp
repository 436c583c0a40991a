// gemm16.hpp -- the matrix-core product of the updater's operators (device code and its launcher).
//
//   C[m][n] = sum over segments s, k of A_s(m, k) B_s(n, k),   16-bit or float32 operands, float32 accumulation.
//
// Each operand is stored either with k contiguous ([rows][k], "KC") or with its rows contiguous ([k][rows]); the
// four products of a block's forward and backward pass then need no transposed copies.  A list of segments adds up
// several products in one accumulator: two weight matrices of one gradient, or the six (three) partial products
// that make a float32 product out of operands split into bfloat16 (float16) parts.
//
// Tile BM x BN x 64 (float32: 32) per workgroup, split over WM x WN waves of 16x16x32 (16x16x4) matrix instructions.
// Tiles go from global memory to LDS directly (16 bytes per lane, no registers), double buffered.  A row of a KC tile is 128 bytes = 8
// chunks; chunk c of row r lies at chunk position c ^ f(r), so the 16-byte fragment reads of 8 lanes cover all 32
// banks (no conflicts measured).  A tile with rows contiguous keeps its [k][row] order and is read with the LDS
// transpose read (4 k x 16 rows per 16 lanes); chunk position c ^ f(k) spreads the four k rows over the banks.
// Out-of-range rows and k read as zero through the buffer descriptor's range check.
//
// There is no such read for 32 bits: float32 tiles of this order are read element by element, four rows of 16
// consecutive floats at a time on different banks.
//
// The loop keeps one half of a tile (64 bytes of k) in registers while it multiplies the other: the second half is read
// during the first half's products, the next tile's first half during the second's, and the tile after it is fetched
// there too, all pinned between rows of products.  There is one barrier per tile, in front of which the wave already
// holds the operands of its next 32 products.  The fetches are asm because the compiler, not knowing which half of
// LDS they write, puts a wait for all of them in front of every later transpose read.
//
// 8192^3 in bfloat16: 938 us with both operands KC, 941 with one, 955 with none (1172, 1168, 1151 TFLOP/s); fetches
// at the top of a tile 1005, 1209, 1214 us; reads and fetches left to the compiler's order 978, 1005, 1022 us.  On
// zeros the same kernel reaches 1600 TFLOP/s: on real data the card's power limit sets the clock (1.9 GHz here), which
// is not all of it: a library's product reaches 1511 TFLOP/s on such data.
// 32x32x16 instructions (995 us), four waves of 128x128 (1031 us), 32-k tiles in rings of three to five (1005 us) and
// waves taking turns between reading and multiplying (1092 us) were measured slower.
//
// Fragments of the column operand take their 16 rows four apart, so that a lane ends up with 16 (dual: 8 + 8)
// consecutive columns of a row and the epilogue reads and writes 16 bytes at a time.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <type_traits>

namespace gsr {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kGemmSegs = 12;
// k of a tile: 128 bytes of an operand's row
template <class T>
constexpr int kTileK = 128 / (int)sizeof(T);

struct GemmArgs {
    const char* a[kGemmSegs];
    const char* b[kGemmSegs];
    const char* b2[kGemmSegs];  // second matrix of a dual product (same layout as b)
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

// float32: four 16x16x4 products, the j-th with element j of the lanes' four (both operands permute k alike)
template <>
struct Mfma<float> {
    static __device__ __forceinline__ f32x4 run(s16x8 a, s16x8 b, f32x4 c) {
        const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[j], fb[j], c, 0, 0, 0);
        return c;
    }
};

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// An offset past every descriptor's range: the lane reads zero.
constexpr uint32_t kOobOffset = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t gemm_rsrc(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, 0x7fffffff, 0x00020000);
}

// Loader of one operand's tiles: R rows x 128 bytes of k by NT threads, elements of ES bytes.  SPREAD: 0, fragment j
// holds rows 16 j + i; otherwise rows 4 SPREAD (i >> 2) + 4 (j % SPREAD) + (i & 3) of its group of 16 SPREAD rows
// (i: the lane's row, 0..15).
// DUAL: each group of 64 rows is 32 rows of the first matrix and the same 32 of the second.
template <bool KC, int R, int NT, int SPREAD, bool DUAL, int ES>
struct TileLoader {
    static constexpr int kChunk = 16 / ES;  // elements of a 16-byte chunk
    static constexpr int kLoads = R * 8 / NT;
    static constexpr int kBytes = R * 128;
    uint32_t off[kLoads];  // byte offset within the tile, kOobOffset for rows out of range
    int kk[kLoads];        // k within the tile of the chunk (its first k for KC)

    static __device__ __forceinline__ int row_swizzle(int r) {
        if (SPREAD == 4) return (r & 3) | ((r >> 2) & 4);
        if (SPREAD == 2) return (r & 3) | ((r >> 1) & 4);
        return r & 7;
    }
    static __device__ __forceinline__ int k_swizzle(int k) {
        if (ES == 4) return ((k >> 2) & 1) * (SPREAD ? 2 : 4);
        if (R == 64) return SPREAD ? k & 1 : 2 * (k & 3);  // 8 chunks a row
        return SPREAD ? (k & 1) | ((k & 2) << 2) : 2 * ((k & 3) | ((k >> 1) & 4));
    }
    static __device__ __forceinline__ int frag_row(int j, int i) {
        if (SPREAD) return (j / SPREAD) * 16 * SPREAD + (i >> 2) * 4 * SPREAD + (j % SPREAD) * 4 + (i & 3);
        return j * 16 + i;
    }
    __device__ __forceinline__ void init(int tid, int row0, int rows, int64_t ld) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = i * NT + tid;
            if (KC) {
                int r = q >> 3;
                const int c = (q & 7) ^ row_swizzle(r);
                if (DUAL) r = (r / 64) * 32 + (r % 32);
                kk[i] = c * kChunk;
                off[i] = row0 + r < rows ? (uint32_t)(r * (uint32_t)ld * ES + c * 16u) : kOobOffset;
            } else {
                constexpr int CH = R / kChunk;
                const int k = q / CH;
                const int c = (q % CH) ^ k_swizzle(k);
                kk[i] = k;
                off[i] = row0 + c * kChunk < rows ? (uint32_t)(k * (uint32_t)ld * ES + c * 16u) : kOobOffset;
            }
        }
    }
    // The i-th load of a tile.  first / second: the tile's first element in the (two) matrices; krem: k left from the
    // tile's start.  The asm has no register outputs; what it writes in LDS is waited for with vmcnt before it is read.
    __device__ __forceinline__ void load(int i, const char* first, const char* second, int krem, char* lds,
                                         int wave) const {
        const uint32_t o = kk[i] < krem ? off[i] : kOobOffset;
        // dual: the 8 rows of one instruction belong to one matrix
        const bool up = DUAL && (((i * NT + wave * 64) >> 3) % 64) >= 32;
        const uint64_t base = (uint64_t)(up ? second : first);
        const u32x4 rs = {(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, 0x7fffffffu, 0x00020000u};
        const uint32_t dst = (uint32_t)(uintptr_t)(lds_void*)(lds + (i * NT + wave * 64) * 16);
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved register; it is clobbered all the same
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(o), "s"(rs), "s"(dst)
                     : "memory", "m0");
#pragma clang diagnostic pop
    }
    // fragment j of the wave's rows from r0, first or second half of the tile's k: lane l holds row i = l % 16 and
    // 16 bytes of k from chunk l / 16 of the half
    static __device__ __forceinline__ s16x8 frag(const char* lds, int r0, int j, int half, int lane) {
        if constexpr (KC) {
            const int r = r0 + frag_row(j, lane & 15);
            const int c = (half * 4 + (lane >> 4)) ^ row_swizzle(r);
            return *reinterpret_cast<const s16x8*>(lds + r * 128 + c * 16);
        } else if constexpr (ES == 4) {  // no transpose read for 32 bits: one element at a time
            f32x4 v;
            const int col = r0 + frag_row(j, lane & 15);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = half * 16 + (lane >> 4) * 4 + e;
                v[e] = *reinterpret_cast<const float*>(lds + k * (R * 4) + (((col >> 2) ^ k_swizzle(k)) << 4) +
                                                       (col & 3) * 4);
            }
            return __builtin_bit_cast(s16x8, v);
        } else {
            s16x8 v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = half * 32 + (lane >> 4) * 8 + h * 4 + ((lane & 15) >> 2);
                const int col = r0 + frag_row(j, (lane & 3) * 4);
                const char* p = lds + k * (R * 2) + (((col >> 3) ^ k_swizzle(k)) << 4) + (col & 4) * 2;
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

// On and above the diagonal, column by column (the mirrored tile is written too).
__device__ __forceinline__ void symmetric_tile(int id, int& tm, int& tn) {
    tn = (int)((__builtin_sqrtf(8.f * (float)id + 1.f) - 1.f) * 0.5f);
    while (tn * (tn + 1) / 2 > id) --tn;
    while ((tn + 1) * (tn + 2) / 2 <= id) ++tn;
    tm = id - tn * (tn + 1) / 2;
}

__device__ __forceinline__ int xcd_order(int bid, int n) {
    const int x = bid & 7, l = bid >> 3;
    const int q = n >> 3, r = n & 7;
    return x * q + min(x, r) + l;
}

// k tiles after which a float32 product's sums go over to a second accumulator.  The error of a sum of K terms in one
// float32 accumulator grows like sqrt(K); in chains of 256 it stays at a chain's, about 12 roundings (K = 2575: 1.0e-6 of
// the result in one chain, 0.4e-6 so).  The 16-bit instructions round once in 32 terms and need no second accumulator,
// for which a 256 x 256 tile has no registers.
constexpr int kChainTiles = 8;

template <class T, bool AKC, bool BKC, int BM, int BN, int WM, int WN, class Epi>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_gemm16(const GemmArgs p, const Epi epi) {
    constexpr int NT = WM * WN * 64;
    constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    static_assert(NI == 4, "a wave covers 64 columns");
    constexpr int ES = (int)sizeof(T), BK = kTileK<T>;
    using LA = TileLoader<AKC, BM, NT, 0, false, ES>;
    using LB = TileLoader<BKC, BN, NT, Epi::kDual ? 2 : 4, Epi::kDual, ES>;
    constexpr int kStage = LA::kBytes + LB::kBytes;
    constexpr int kLoads = LA::kLoads + LB::kLoads;
    __shared__ __attribute__((aligned(1024))) char smem[2 * kStage];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int tiles = Epi::kSymmetric ? p.tiles_n * (p.tiles_n + 1) / 2 : p.tiles_m * p.tiles_n;
    int id = xcd_order(blockIdx.x, gridDim.x);
    const int batch = id / (tiles * p.splits);
    id -= batch * (tiles * p.splits);
    const int split = id / tiles;
    int tm, tn;
    if (Epi::kSymmetric)
        symmetric_tile(id - split * tiles, tm, tn);
    else
        gemm_tile(p, id - split * tiles, tm, tn);

    constexpr int BNR = Epi::kDual ? BN / 2 : BN;  // output columns of a tile
    const int m0 = tm * BM, n0 = tn * BNR;
    LA la;
    LB lb;
    la.init(tid, m0, p.M, p.lda);
    lb.init(tid, n0, p.N, p.ldb);

    const int ktiles = (p.K + BK - 1) / BK;
    const int t_begin = split * p.tiles_per_split;
    const int t_end = min(ktiles * p.nseg, t_begin + p.tiles_per_split);
    const int64_t a0 = (batch * p.batch_a + (AKC ? (int64_t)m0 * p.lda : m0)) * ES;  // bytes, like the steps
    const int64_t b0 = (batch * p.batch_b + (BKC ? (int64_t)n0 * p.ldb : n0)) * ES;
    const int64_t astep = AKC ? 128 : 128 * p.lda;
    const int64_t bstep = BKC ? 128 : 128 * p.ldb;

    constexpr bool kChains = sizeof(T) == 4 && BM < 256;
    f32x4 acc[MI][NI], total[kChains ? MI : 1][kChains ? NI : 1];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (kChains) total[i][j] = acc[i][j];
        }

    if (t_begin < t_end) {
        // the tile to fetch; past the last one nothing is read (krem 0: every lane is out of range)
        int s = t_begin / ktiles, kt = t_begin - s * ktiles, left = t_end - t_begin, krem = 0;
        const char* na = p.a[s] + a0 + kt * astep;
        const char* nb = p.b[s] + b0 + kt * bstep;
        const char* nb2 = Epi::kDual ? p.b2[s] + b0 + kt * bstep : nullptr;
        const char *fa0 = na, *fb0 = nb, *fb2 = nb2;
        auto next = [&]() {
            krem = left > 0 ? p.K - kt * BK : 0;
            fa0 = na, fb0 = nb, fb2 = nb2;
            --left;
            na += astep, nb += bstep;
            if (Epi::kDual) nb2 += bstep;
            if (++kt == ktiles) {
                kt = 0;
                if (s + 1 < p.nseg) ++s;
                na = p.a[s] + a0, nb = p.b[s] + b0;
                if (Epi::kDual) nb2 = p.b2[s] + b0;
            }
        };
        auto fetch = [&](int i, char* buf) {
            if (i < LA::kLoads)
                la.load(i, fa0, nullptr, krem, buf, wave);
            else
                lb.load(i - LA::kLoads, fb0, fb2, krem, buf + LA::kBytes, wave);
        };
        s16x8 fa[2][MI], fb[2][NI];
        auto read = [&](int half, int f, const char* buf) {
            if (f < NI)
                fb[half][f] = LB::frag(buf + LA::kBytes, wn * (BN / WN), f, half, lane);
            else
                fa[half][f - NI] = LA::frag(buf, wm * (BM / WM), f - NI, half, lane);
        };
        // fragments and fetches per row of products; the last rows read nothing, so nothing is waited for after them
        constexpr int kFrags = MI + NI, kReadRows = MI > 1 ? MI * 3 / 4 : 1;
        constexpr int kReads = (kFrags + kReadRows - 1) / kReadRows;
        constexpr int kFetches = (kLoads + MI - 1) / MI;
        // one half of a tile: NI products of each of the MI rows
        auto multiply = [&](int half, const char* from, bool fetching, char* to) {
#pragma unroll
            for (int g = 0; g < MI; ++g) {
#pragma unroll
                for (int f = g * kReads; f < (g + 1) * kReads && f < kFrags; ++f) read(half ^ 1, f, from);
                if (fetching) {
#pragma unroll
                    for (int i = g * kFetches; i < (g + 1) * kFetches && i < kLoads; ++i) fetch(i, to);
                }
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[g][j] = Mfma<T>::run(fb[half][j], fa[half][g], acc[g][j]);
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        next();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) fetch(i, smem);
        next();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) fetch(i, smem + kStage);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int f = 0; f < kFrags; ++f) read(0, f, smem);
        for (int t = t_begin; t < t_end; ++t) {
            char* cur = smem + ((t - t_begin) & 1) * kStage;
            char* nxt = smem + ((t - t_begin + 1) & 1) * kStage;
            multiply(0, cur, false, nullptr);
            next();
            // the wave has read all of cur, and its share of nxt has landed; after the barrier everyone's has
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            multiply(1, nxt, true, cur);
            if constexpr (kChains)
                if ((t - t_begin) % kChainTiles == kChainTiles - 1) {
#pragma unroll
                    for (int i = 0; i < MI; ++i)
#pragma unroll
                        for (int j = 0; j < NI; ++j) {
                            total[i][j] += acc[i][j];
                            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                        }
                }
        }
        if constexpr (kChains) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[i][j] += total[i][j];
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no fetch outlives the workgroup's LDS
    }

    // lane: row m, 16 consecutive columns (dual: 8 of each product); what the epilogue reads is fetched ahead
    const int mb = m0 + wm * (BM / WM) + (lane & 15);
    constexpr int kAhead = Epi::kAhead;
    if constexpr (Epi::kDual) {
        const int nb = n0 + wn * (BNR / WN) + (lane >> 4) * 8;
#pragma unroll
        for (int i = 0; i < MI; ++i) epi.row(mb + i * 16, nb, acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    } else {
        const int nb = n0 + wn * (BN / WN) + (lane >> 4) * 16;
        typename Epi::Pre pre[kAhead + 1];
#pragma unroll
        for (int i = 0; i < kAhead && i < MI; ++i) pre[i] = epi.fetch(batch, mb + i * 16, nb);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if (i + kAhead < MI) pre[(i + kAhead) % (kAhead + 1)] = epi.fetch(batch, mb + (i + kAhead) * 16, nb);
            epi.row(batch, split, mb + i * 16, nb, acc[i], pre[i % (kAhead + 1)]);
        }
    }
}

// ---- values in and out -------------------------------------------------------------------------------

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

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

__device__ __forceinline__ u16x8 pack8(u16x4 a, u16x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
__device__ __forceinline__ u16x4 half8(u16x8 v, int h) {
    return h ? __builtin_shufflevector(v, v, 4, 5, 6, 7) : __builtin_shufflevector(v, v, 0, 1, 2, 3);
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

// Pre-activations kept for the backward pass: g and u of rows x cols (cols a multiple of 8), eight of each at a time.
struct Kept {
    char* p;
    int64_t cols, n;  // n = rows * cols
};

// Float32 as it is: [rows][2][cols].
struct Keep32 {
    static constexpr int64_t bytes(int64_t n) { return n * 8; }
    static constexpr int kAhead = 1;  // rows whose values fit the registers ahead of their use
    struct Raw {
        f32x4 v[4];
    };
    static __device__ __forceinline__ void put(const Kept& k, int64_t row, int col, f32x4 g0, f32x4 g1, f32x4 u0,
                                               f32x4 u1) {
        f32x4* g = (f32x4*)((float*)k.p + row * 2 * k.cols + col);
        f32x4* u = (f32x4*)((float*)k.p + (row * 2 + 1) * k.cols + col);
        g[0] = g0, g[1] = g1, u[0] = u0, u[1] = u1;
    }
    static __device__ __forceinline__ Raw get(const Kept& k, int64_t row, int col) {
        const f32x4* g = (const f32x4*)((const float*)k.p + row * 2 * k.cols + col);
        const f32x4* u = (const f32x4*)((const float*)k.p + (row * 2 + 1) * k.cols + col);
        return {{g[0], g[1], u[0], u[1]}};
    }
    static __device__ __forceinline__ f32x4 g(const Raw& r, int h) { return r.v[h]; }
    static __device__ __forceinline__ f32x4 u(const Raw& r, int h) { return r.v[2 + h]; }
};
// The upper 16 + LO bits of a float32, rounded: float32's range and 8 + LO significant bits.  First the upper 16 bits of
// all values, [rows][2][cols], then the lower bits, LO / 4 words for eight g and as many for the eight u beside them.
// Records of all bits of eight g and u one after another were slower (lines are written in more parts).
template <int LO>
struct KeepHigh {
    static_assert(LO == 4 || LO == 8);
    static constexpr int kWords = LO / 4;
    static constexpr int64_t bytes(int64_t n) { return n * 4 + n / 4 * LO; }
    static constexpr int kAhead = 2;
    typedef uint32_t Low __attribute__((ext_vector_type(2 * kWords)));
    struct Raw {
        u32x4 g, u;
        Low lo;
    };
    // four values: two words of upper halves, and their lower bits into lo from word w
    static __device__ __forceinline__ void pack(f32x4 x, int h, u32x4& hi, Low& lo, int w) {
        uint32_t t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = x[e];  // an element of a vector cannot be cast in place
            t[e] = __builtin_bit_cast(uint32_t, f) + (LO == 8 ? 0x80u : 0x800u);
        }
        hi[h * 2] = __builtin_amdgcn_perm(t[1], t[0], 0x07060302u);
        hi[h * 2 + 1] = __builtin_amdgcn_perm(t[3], t[2], 0x07060302u);
        const uint32_t b = __builtin_amdgcn_perm(__builtin_amdgcn_perm(t[3], t[2], 0x0c0c0501u),
                                                 __builtin_amdgcn_perm(t[1], t[0], 0x0c0c0501u), 0x05040100u);
        if constexpr (LO == 8)
            lo[w + h] = b;
        else if (h == 0)
            lo[w] = (b >> 4) & 0x0f0f0f0fu;
        else
            lo[w] |= b & 0xf0f0f0f0u;
    }
    static __device__ __forceinline__ void put(const Kept& k, int64_t row, int col, f32x4 g0, f32x4 g1, f32x4 u0,
                                               f32x4 u1) {
        Raw r;
        pack(g0, 0, r.g, r.lo, 0);
        pack(g1, 1, r.g, r.lo, 0);
        pack(u0, 0, r.u, r.lo, kWords);
        pack(u1, 1, r.u, r.lo, kWords);
        char* p = k.p + (row * 2 * k.cols + col) * 2;
        *(u32x4*)p = r.g;
        *(u32x4*)(p + k.cols * 2) = r.u;
        *(Low*)(k.p + k.n * 4 + (row * k.cols + col) / 4 * LO) = r.lo;
    }
    static __device__ __forceinline__ Raw get(const Kept& k, int64_t row, int col) {
        const char* p = k.p + (row * 2 * k.cols + col) * 2;
        return {*(const u32x4*)p, *(const u32x4*)(p + k.cols * 2),
                *(const Low*)(k.p + k.n * 4 + (row * k.cols + col) / 4 * LO)};
    }
    static __device__ __forceinline__ f32x4 unpack(u32x4 hi, const Low& lo, int w, int h) {
        const uint32_t b = LO == 8 ? lo[w + (LO == 8 ? h : 0)] : h ? lo[w] & 0xf0f0f0f0u : (lo[w] & 0x0f0f0f0fu) << 4;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = __builtin_bit_cast(
                float, __builtin_amdgcn_perm(hi[h * 2 + (e >> 1)], b, (e & 1 ? 0x0706000cu : 0x0504000cu) | e << 8));
        return v;
    }
    static __device__ __forceinline__ f32x4 g(const Raw& r, int h) { return unpack(r.g, r.lo, 0, h); }
    static __device__ __forceinline__ f32x4 u(const Raw& r, int h) { return unpack(r.u, r.lo, kWords, h); }
};

// Element formats of the block: what a stored 16-bit matrix operand and a value array look like for each type.
struct FmtBf16 {
    using Mma = __bf16;
    using Elem = uint16_t;     // value arrays (inputs, outputs)
    using Keep = KeepHigh<4>;  // saved pre-activations
    static constexpr int kPlanes = 1;
    static __device__ __forceinline__ f32x4 get(const Elem* p) { return from16<__bf16>(*(const u16x4*)p); }
    static __device__ __forceinline__ void put(Elem* p, f32x4 v) { *(u16x4*)p = to16<__bf16>(v); }
    static __device__ __forceinline__ void put8(Elem* p, f32x4 a, f32x4 b) { *(u16x8*)p = pack8(to16<__bf16>(a), to16<__bf16>(b)); }
    static __device__ __forceinline__ float to_float(uint16_t v) { return (float)__builtin_bit_cast(__bf16, v); }
    static __device__ __forceinline__ uint16_t from_float(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
    static __device__ __forceinline__ float get1(const Elem* p) { return to_float(*p); }
    static __device__ __forceinline__ void put1(Elem* p, float v) { *p = from_float(v); }
};
struct FmtF16 {
    using Mma = _Float16;
    using Elem = uint16_t;
    using Keep = KeepHigh<8>;
    static constexpr int kPlanes = 1;
    static __device__ __forceinline__ f32x4 get(const Elem* p) { return from16<_Float16>(*(const u16x4*)p); }
    static __device__ __forceinline__ void put(Elem* p, f32x4 v) { *(u16x4*)p = to16<_Float16>(v); }
    static __device__ __forceinline__ void put8(Elem* p, f32x4 a, f32x4 b) { *(u16x8*)p = pack8(to16<_Float16>(a), to16<_Float16>(b)); }
    static __device__ __forceinline__ float to_float(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ uint16_t from_float(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
    static __device__ __forceinline__ float get1(const Elem* p) { return to_float(*p); }
    static __device__ __forceinline__ void put1(Elem* p, float v) { *p = from_float(v); }
};
struct F32Values {
    using Elem = float;
    using Keep = Keep32;
    static __device__ __forceinline__ f32x4 get(const Elem* p) { return *(const f32x4*)p; }
    static __device__ __forceinline__ void put(Elem* p, f32x4 v) { *(f32x4*)p = v; }
    static __device__ __forceinline__ void put8(Elem* p, f32x4 a, f32x4 b) {
        *(f32x4*)p = a;
        *(f32x4*)(p + 4) = b;
    }
    static __device__ __forceinline__ float get1(const Elem* p) { return *p; }
    static __device__ __forceinline__ void put1(Elem* p, float v) { *p = v; }
};
struct FmtF32 : F32Values {  // float32 matrix instructions
    using Mma = float;
    static constexpr int kPlanes = 1;
};
struct FmtF32Split : F32Values {  // matrix operands split into three bfloat16 planes
    using Mma = __bf16;
    static constexpr int kPlanes = 3;
};

// What a matrix operand is stored as.
template <class F>
using OperandElem = std::conditional_t<sizeof(typename F::Mma) == 4, float, uint16_t>;

// Eight consecutive values of a matrix operand (one or three planes), 16-byte aligned.
template <class F>
__device__ __forceinline__ void put_operand8(OperandElem<F>* p, int64_t plane, f32x4 v0, f32x4 v1) {
    if constexpr (F::kPlanes == 1) {
        F::put8(p, v0, v1);
    } else {
        u16x8 h, m, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint16_t a, b, c;
            split3(e < 4 ? v0[e & 3] : v1[e & 3], a, b, c);
            h[e] = a, m[e] = b, l[e] = c;
        }
        *(u16x8*)p = h;
        *(u16x8*)(p + plane) = m;
        *(u16x8*)(p + 2 * plane) = l;
    }
}

// What an epilogue fetches ahead when it needs nothing.
struct NoPre {};

// ---- launchers -----------------------------------------------------------------------------------------

constexpr int64_t kMaxThreads = (1ll << 32) - 1;  // of a launch

template <class T, bool AKC, bool BKC, int BM, int BN, int WM, int WN, class Epi>
inline hipError_t launch_tiles(GemmArgs p, const Epi& epi, hipStream_t st) {
    constexpr int BNR = Epi::kDual ? BN / 2 : BN;
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_n = (p.N + BNR - 1) / BNR;
    const int64_t tiles = Epi::kSymmetric ? (int64_t)p.tiles_n * (p.tiles_n + 1) / 2 : (int64_t)p.tiles_m * p.tiles_n;
    const int64_t n = tiles * p.batch * p.splits;
    if (n <= 0) return hipSuccess;
    if (n > kMaxThreads / (WM * WN * 64)) return hipErrorInvalidValue;
    k_gemm16<T, AKC, BKC, BM, BN, WM, WN, Epi><<<dim3((unsigned)n), dim3(WM * WN * 64), 0, st>>>(p, epi);
    return hipGetLastError();
}

inline int64_t tile_count(int64_t M, int64_t N, int t, bool symmetric) {
    const int64_t tm = (M + t - 1) / t, tn = (N + t - 1) / t;
    return symmetric ? tn * (tn + 1) / 2 : tm * tn;
}

// Tile size and splits along k of one product, from what the tiles were measured to take (TileTimes).  Small tiles
// read each operand more often but fill the CUs with several workgroups, which hide each other's epilogues and waits:
// 23040 x 256 x 57 in float32 37 us with 64x64 tiles, 44 with 128x128; 1366 x 1366 x 500 float16 (three products)
// 17 and 25 us; a k tile of 256x256 costs 1.75 us a CU, four of 128x128 2.4, sixteen of 64x64 4.2.  A split product's
// float32 partial sums are read again at 4.5 TB/s by one more kernel (symmetric products, whose kernel also mirrors:
// half as fast).  dual: N counts the columns of one of the two matrices.
struct GemmPlan {
    int tile, splits, tiles_per_split;
    double us;
};
// One tile size: workgroups a CU holds, microseconds per k tile of a lone workgroup and with the CU full, and around.
struct TileTimes {
    int tile, per_cu;
    double alone, full, around;
};
inline GemmPlan plan_gemm(int64_t M, int64_t N, int64_t batch, int64_t ktiles, bool dual, bool symmetric,
                          int max_splits, bool f32 = false) {
    static const TileTimes t16[3] = {{256, 1, 1.75, 1.75, 7}, {128, 2, 0.85, 1.2, 4}, {64, 4, 0.5, 1.05, 3}};
    static const TileTimes t32[3] = {{256, 1, 8.4, 8.4, 20}, {128, 2, 2.3, 4.3, 16}, {64, 4, 0.85, 3.2, 3}};
    GemmPlan best{128, 1, (int)ktiles, 1e30};
    // a long float32 sum needs a tile with two accumulators (kChainTiles)
    for (int i = f32 && ktiles > 2 * kChainTiles ? 1 : 0; i < 3; ++i) {
        const TileTimes& tt = f32 ? t32[i] : t16[i];
        const int t = tt.tile;
        const int64_t tiles =
            (dual ? ((M + t - 1) / t) * ((N + t / 2 - 1) / (t / 2)) : tile_count(M, N, t, symmetric)) * batch;
        for (int s = 1; s <= max_splits; s = s < 8 ? s + 1 : s + s / 4) {
            const int64_t per = (ktiles + s - 1) / s, n = tiles * s, slots = 256 * tt.per_cu;
            if (s > 1 && (per < 4 || n > 1024)) break;
            if (n > kMaxThreads / (t == 256 ? 512 : 256)) break;
            const int64_t rounds = (n + slots - 1) / slots;
            const double busy = rounds > 1 ? 1.0 : (double)((n + 255) / 256) / tt.per_cu;
            const double per_k = tt.full * busy > tt.alone ? tt.full * busy : tt.alone;
            const double sums = s > 1 ? (symmetric ? 8 : 4) + (double)tiles * t * t * 4 * s / (symmetric ? 2e6 : 4.5e6) : 0;
            const double us = rounds * (per_k * per + tt.around) + sums;
            if (us < best.us) best = {t, s, (int)per, us};
        }
    }
    return best;
}

template <class T, bool AKC, bool BKC, class Epi>
inline hipError_t launch_planned(GemmArgs p, const GemmPlan& plan, const Epi& epi, hipStream_t st) {
    p.splits = plan.splits;
    p.tiles_per_split = plan.tiles_per_split;
    if (plan.tile == 256) return launch_tiles<T, AKC, BKC, 256, 256, 2, 4, Epi>(p, epi, st);
    if (plan.tile == 128) return launch_tiles<T, AKC, BKC, 128, 128, 2, 2, Epi>(p, epi, st);
    return launch_tiles<T, AKC, BKC, 64, 64, 4, 1, Epi>(p, epi, st);
}
template <class T>
inline int64_t k_tiles(const GemmArgs& p) {
    return (int64_t)p.nseg * ((p.K + kTileK<T> - 1) / kTileK<T>);
}

// One product without splits.
template <class T, bool AKC, bool BKC, class Epi>
inline hipError_t launch_gemm(const GemmArgs& p, const Epi& epi, hipStream_t st) {
    const GemmPlan plan = plan_gemm(p.M, p.N, p.batch, k_tiles<T>(p), Epi::kDual, false, 1, sizeof(T) == 4);
    return launch_planned<T, AKC, BKC>(p, plan, epi, st);
}

// One stored matrix operand: planes (split operands) `plane` elements apart, rows of `ld` elements.
struct Operand {
    const void* p;
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

// widest store the rows of an output allow: 8, 4 or 1 elements
inline int vec_width(const void* p, int64_t ld, size_t elem) {
    if (ld % 8 == 0 && (uintptr_t)p % 16 == 0) return 8;
    return ld % 4 == 0 && (uintptr_t)p % (4 * elem) == 0 ? 4 : 1;
}

#define GSR_TRY(x)                          \
    do {                                    \
        hipError_t e_ = (x);                \
        if (e_ != hipSuccess) return e_;    \
    } while (0)

}  // namespace gsr
