// scan.hip -- gated linear recurrence of the learned updater and its gradient.
//
//   a_t = sigma(z_t), h_t = a_t h_{t-1} + (1 - a_t) x_t              per channel, h_{-1} = h0 of the sequence
//   e_t = a_t G_t,    G_t = dy_t + e_{t+1}                           e past the last row = dh_last
//   dx = (1 - a) G,   dz = a (1 - a) (h_{t-1} - x) G,   dh0 = e_0
//
// Sequences of any length lie one after another in the rows.  One pass over the data: a workgroup takes a chunk of
// rows of some channels into registers, row groups of R rows reduce to (A, H) -- h_out = A h_in + H -- and are joined
// in LDS, the chunk's (A, H) is published, the state that enters the chunk is gathered from the chunks before it,
// and the rows are then run once more from their registers with the true state.  A row that starts a sequence
// replaces the state instead of multiplying it by zero, so nothing of one sequence, NaN included, reaches the next.
//
// The state entering chunk k is joined in a fixed order whatever the timing, so results are reproducible: first the
// (A, H) of the chunks before it in its group of 8, then those of the whole groups before it in its group of 64,
// then the running state of the group of 64 before that, which alone forms a chain along the sequence.  Published
// values are 64-bit words {value, tag} written and read atomically, so a word is either absent or whole.  Chunks are
// taken by ticket, so a workgroup only ever waits for one that has already started.
//
// The forward pass keeps the state entering every chunk in float32; the backward pass reruns the states
// from there, instead of reading back rounded ones, and scans e from the other end in the same way.
#include "gsr_internal.hpp"
#include "gemm16.hpp"

namespace gsr {

namespace {

constexpr int kChunk = 128;     // rows of a chunk
constexpr int kGroupRows = 16;  // rows of a row group (one thread's)
constexpr int kGroups = kChunk / kGroupRows;
constexpr int kFan = 8;         // chunks per level-1 group, level-1 groups per level-2 group
constexpr uint32_t kTagValid = 1u, kTagReset = 2u;

struct ScanArgs {
    const void* z;
    const void* x;
    const void* dy;
    int64_t ldz, ldx, ldy, lddy, lddz, lddx;
    const float* h0;
    const float* dh_last;
    void* y;
    float* h_last;
    float* saved;
    void* dz;
    void* dx;
    float* dh0;
    const int64_t* offsets;
    int64_t n_seq, seq_len, rows;
    int C, ncb;
    int64_t nchunks;
    uint64_t* agg1;    // [chunk][2][C]
    uint64_t* agg2;    // [chunk / 8][2][C]
    uint64_t* run;     // [chunk / 64][C]
    uint32_t* ticket;
};

__device__ __forceinline__ void gate(float z, float& a, float& na) {
    const float e = __expf(-__builtin_fabsf(z));
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    const float er = e * r;
    a = z >= 0.f ? r : er;
    na = z >= 0.f ? er : r;
}

__device__ __forceinline__ uint64_t word(float v, uint32_t tag) {
    return ((uint64_t)tag << 32) | __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void post(uint64_t* p, uint64_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// waits for a word; v holds what a first look found
__device__ __forceinline__ uint64_t await(const uint64_t* p, uint64_t v) {
    while (!(uint32_t)(v >> 32)) {
        __builtin_amdgcn_s_sleep(1);
        v = peek(p);
    }
    return v;
}
__device__ __forceinline__ float value(uint64_t w) { return __builtin_bit_cast(float, (uint32_t)w); }

struct Span {  // h_out = reset ? H : A h_in + H
    float A, H;
    bool reset;
};
__device__ __forceinline__ Span join(const Span& first, const Span& then) {
    if (then.reset) return then;
    return {first.A * then.A, __builtin_fmaf(then.A, first.H, then.H), first.reset};
}
__device__ __forceinline__ float apply(const Span& s, float h) {
    return s.reset ? s.H : __builtin_fmaf(s.A, h, s.H);
}

// State entering chunk k (counted in scan direction) of one channel; publishes the chunk's own span.
__device__ float exchange(const ScanArgs& p, int64_t k, int c, const Span& own) {
    const uint32_t tag = kTagValid | (own.reset ? kTagReset : 0u);
    uint64_t* mine = p.agg1 + k * 2 * p.C + c;
    post(mine, word(own.A, tag));
    post(mine + p.C, word(own.H, tag));
    const int64_t k1 = k / kFan, k2 = k1 / kFan;
    const int n1 = (int)(k - k1 * kFan), n2 = (int)(k1 - k2 * kFan);
    // one look at everything that is needed, so that the latencies overlap
    uint64_t wa[kFan - 1], wh[kFan - 1], va[kFan - 1], vh[kFan - 1], wr = 0;
    const uint64_t* b1 = p.agg1 + k1 * kFan * 2 * p.C + c;
    const uint64_t* b2 = p.agg2 + k2 * kFan * 2 * p.C + c;
    const uint64_t* br = p.run + (k2 - 1) * p.C + c;
#pragma unroll
    for (int j = 0; j < kFan - 1; ++j) {
        wa[j] = j < n1 ? peek(b1 + (int64_t)j * 2 * p.C) : 0;
        wh[j] = j < n1 ? peek(b1 + ((int64_t)j * 2 + 1) * p.C) : 0;
        va[j] = j < n2 ? peek(b2 + (int64_t)j * 2 * p.C) : 0;
        vh[j] = j < n2 ? peek(b2 + ((int64_t)j * 2 + 1) * p.C) : 0;
    }
    if (k2 > 0) wr = peek(br);
    Span s1{1.f, 0.f, false};
#pragma unroll
    for (int j = 0; j < kFan - 1; ++j) {
        if (j < n1) {
            const uint64_t a = await(b1 + (int64_t)j * 2 * p.C, wa[j]);
            const uint64_t h = await(b1 + ((int64_t)j * 2 + 1) * p.C, wh[j]);
            s1 = join(s1, Span{value(a), value(h), ((uint32_t)(a >> 32) & kTagReset) != 0});
        }
    }
    if (n1 == kFan - 1) {
        const Span g = join(s1, own);
        const uint32_t t = kTagValid | (g.reset ? kTagReset : 0u);
        uint64_t* d = p.agg2 + k1 * 2 * p.C + c;
        post(d, word(g.A, t));
        post(d + p.C, word(g.H, t));
    }
    float h = 0.f;
    if (!s1.reset) {
        Span s2{1.f, 0.f, false};
#pragma unroll
        for (int j = 0; j < kFan - 1; ++j) {
            if (j < n2) {
                const uint64_t a = await(b2 + (int64_t)j * 2 * p.C, va[j]);
                const uint64_t v = await(b2 + ((int64_t)j * 2 + 1) * p.C, vh[j]);
                s2 = join(s2, Span{value(a), value(v), ((uint32_t)(a >> 32) & kTagReset) != 0});
            }
        }
        if (!s2.reset && k2 > 0) h = value(await(br, wr));
        h = apply(s2, h);
    }
    h = apply(s1, h);
    if (n1 == kFan - 1 && n2 == kFan - 1) post(p.run + k2 * p.C + c, word(apply(own, h), kTagValid));
    return h;
}

// Sequence starts of a chunk: s_start[i] is the sequence that starts at row row0 + i (the last one, where empty
// sequences share the row), -1 where none does, and the row past the last one counts as a start.  Returns the
// sequence that holds row row0 - 1 or starts at row0.
__device__ int64_t sequence_starts(const ScanArgs& p, int64_t row0, int* s_start, int tid, int nt) {
    if (!p.offsets) {
        for (int i = tid; i <= kChunk; i += nt) {
            const int64_t r = row0 + i;
            s_start[i] = r >= p.rows || r % p.seq_len == 0 ? (int)(r / p.seq_len) : -1;
        }
        __syncthreads();
        return row0 / p.seq_len;
    }
    // first sequence with offsets[s] >= row0
    int64_t lo = 0, hi = p.n_seq;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (p.offsets[mid] < row0)
            lo = mid + 1;
        else
            hi = mid;
    }
    for (int i = tid; i <= kChunk; i += nt) s_start[i] = row0 + i >= p.rows ? (int)p.n_seq : -1;
    __syncthreads();
    for (int64_t s = lo + tid; s <= p.n_seq; s += nt) {
        const int64_t at = p.offsets[s] - row0;
        if (at > kChunk) break;
        if (at >= 0 && row0 + at < p.rows) atomicMax(&s_start[at], (int)s);
    }
    __syncthreads();
    return lo - 1;
}

// sequence that holds row i of the chunk
__device__ __forceinline__ int64_t sequence_of(const int* s_start, int i, int64_t before) {
    for (; i >= 0; --i)
        if (s_start[i] >= 0) return s_start[i];
    return before;
}

template <class F, int VC>
struct Vec;
template <int VC>
struct Vec<FmtF32, VC> {
    typedef float V __attribute__((ext_vector_type(VC)));
};
template <int VC>
struct Vec<FmtBf16, VC> {
    typedef uint16_t V __attribute__((ext_vector_type(VC)));
};
template <int VC>
struct Vec<FmtF16, VC> {
    typedef uint16_t V __attribute__((ext_vector_type(VC)));
};

// LPR lanes x VC channels hold a row; kGroups row groups of kGroupRows rows.
template <class F, int VC, int LPR, bool CARRY>
__global__ __launch_bounds__(LPR* kGroups) void k_scan_forward(const ScanArgs p) {
    using E = typename F::Elem;
    using V = typename Vec<F, VC>::V;
    constexpr int CB = LPR * VC, NT = LPR * kGroups;
    __shared__ int s_start[kChunk + 1];
    __shared__ float s_a[kGroups][CB], s_h[kGroups][CB];
    __shared__ int s_reset[kGroups];
    __shared__ uint32_t s_ticket;
    const int tid = threadIdx.x;
    uint32_t t = blockIdx.x;
    if (CARRY) {
        if (tid == 0) s_ticket = atomicAdd(p.ticket, 1u);
        __syncthreads();
        t = s_ticket;
    }
    const int64_t chunk = t / (uint32_t)p.ncb;
    const int cb = (int)(t - (uint32_t)chunk * (uint32_t)p.ncb);
    const int g = tid / LPR, li = tid % LPR;
    const int c = cb * CB + li * VC;
    const bool live = c < p.C;
    const int64_t row0 = chunk * kChunk, base = row0 + g * kGroupRows;
    const int n = (int)(p.rows - base < kGroupRows ? (p.rows - base < 0 ? 0 : p.rows - base) : kGroupRows);

    V z[kGroupRows], x[kGroupRows];
    const E* pz = (const E*)p.z + base * p.ldz + c;
    const E* px = (const E*)p.x + base * p.ldx + c;
#pragma unroll
    for (int r = 0; r < kGroupRows; ++r) {
        if (live && r < n) {
            z[r] = *(const V*)(pz + r * p.ldz);
            x[r] = *(const V*)(px + r * p.ldx);
        }
    }
    const int64_t before = sequence_starts(p, row0, s_start, tid, NT);
    const int* st = s_start + g * kGroupRows;

    float A[VC], H[VC];
    bool reset = false;
#pragma unroll
    for (int e = 0; e < VC; ++e) A[e] = 1.f, H[e] = 0.f;
    if (live) {
#pragma unroll
        for (int r = 0; r < kGroupRows; ++r) {
            if (r < n) {
                const int s = st[r];
                float h0[VC];
    #pragma unroll
                for (int e = 0; e < VC; ++e) h0[e] = 0.f;
                if (s >= 0) {
                    reset = true;
                    if (p.h0 && s < p.n_seq) {
    #pragma unroll
                        for (int e = 0; e < VC; ++e) h0[e] = p.h0[(int64_t)s * p.C + c + e];
                    }
                }
    #pragma unroll
                for (int e = 0; e < VC; ++e) {
                    float a, na;
                    gate(F::get1((const E*)&z[r] + e), a, na);
                    const float b = na * F::get1((const E*)&x[r] + e);
                    H[e] = __builtin_fmaf(a, s >= 0 ? h0[e] : H[e], b);
                    A[e] *= a;
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        s_a[g][li * VC + e] = A[e];
        s_h[g][li * VC + e] = H[e];
    }
    if (li == 0) s_reset[g] = reset;
    __syncthreads();
    // the chunk's span, the state entering it, and the state entering each row group (left in s_h)
    for (int i = tid; i < CB; i += NT) {
        const int cc = cb * CB + i;
        if (cc >= p.C) break;
        float h = 0.f;
        if (CARRY) {
            Span own{1.f, 0.f, false};
#pragma unroll
            for (int k = 0; k < kGroups; ++k) own = join(own, Span{s_a[k][i], s_h[k][i], s_reset[k] != 0});
            h = exchange(p, chunk, cc, own);
        }
        if (p.saved) p.saved[chunk * p.C + cc] = h;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const Span s{s_a[k][i], s_h[k][i], s_reset[k] != 0};
            s_h[k][i] = h;
            h = apply(s, h);
        }
    }
    __syncthreads();
    if (!live) return;
    float h[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) h[e] = s_h[g][li * VC + e];
    E* py = (E*)p.y + base * p.ldy + c;
#pragma unroll
    for (int r = 0; r < kGroupRows; ++r) {
        if (r < n) {
            const int s = st[r];
            if (s >= 0) {
    #pragma unroll
                for (int e = 0; e < VC; ++e) h[e] = p.h0 && s < p.n_seq ? p.h0[(int64_t)s * p.C + c + e] : 0.f;
            }
            V o;
    #pragma unroll
            for (int e = 0; e < VC; ++e) {
                float a, na;
                gate(F::get1((const E*)&z[r] + e), a, na);
                const float b = na * F::get1((const E*)&x[r] + e);
                h[e] = __builtin_fmaf(a, h[e], b);
                F::put1((E*)&o + e, h[e]);
            }
            *(V*)(py + r * p.ldy) = o;
            if (p.h_last && st[r + 1] >= 0) {
                const int64_t q = sequence_of(s_start, g * kGroupRows + r, before);
                if (q >= 0 && q < p.n_seq) {
    #pragma unroll
                    for (int e = 0; e < VC; ++e) p.h_last[q * p.C + c + e] = h[e];
                }
            }
        }
    }
}

template <class F, int VC, int LPR, bool CARRY>
__global__ __launch_bounds__(LPR* kGroups) void k_scan_backward(const ScanArgs p) {
    using E = typename F::Elem;
    using V = typename Vec<F, VC>::V;
    constexpr int CB = LPR * VC, NT = LPR * kGroups;
    __shared__ int s_start[kChunk + 1];
    // A is the same product in both directions; s_h: states, s_e: the gradient's
    __shared__ float s_a[kGroups][CB], s_h[kGroups][CB], s_e[kGroups][CB];
    __shared__ int s_reset[kGroups], s_end[kGroups];
    __shared__ uint32_t s_ticket;
    const int tid = threadIdx.x;
    uint32_t t = blockIdx.x;
    if (CARRY) {
        if (tid == 0) s_ticket = atomicAdd(p.ticket, 1u);
        __syncthreads();
        t = s_ticket;
    }
    const int64_t order = t / (uint32_t)p.ncb;  // chunks from the last to the first
    const int cb = (int)(t - (uint32_t)order * (uint32_t)p.ncb);
    const int64_t chunk = p.nchunks - 1 - order;
    const int g = tid / LPR, li = tid % LPR;
    const int c = cb * CB + li * VC;
    const bool live = c < p.C;
    const int64_t row0 = chunk * kChunk, base = row0 + g * kGroupRows;
    const int n = (int)(p.rows - base < kGroupRows ? (p.rows - base < 0 ? 0 : p.rows - base) : kGroupRows);

    V z[kGroupRows], x[kGroupRows], dy[kGroupRows];
    const E* pz = (const E*)p.z + base * p.ldz + c;
    const E* px = (const E*)p.x + base * p.ldx + c;
    const E* pd = (const E*)p.dy + base * p.lddy + c;
#pragma unroll
    for (int r = 0; r < kGroupRows; ++r) {
        if (live && r < n) {
            z[r] = *(const V*)(pz + r * p.ldz);
            x[r] = *(const V*)(px + r * p.ldx);
            dy[r] = *(const V*)(pd + r * p.lddy);
        }
    }
    const int64_t before = sequence_starts(p, row0, s_start, tid, NT);
    const int* st = s_start + g * kGroupRows;

    float A[VC], H[VC], Ee[VC];
    bool reset = false, end = false;
#pragma unroll
    for (int e = 0; e < VC; ++e) A[e] = 1.f, H[e] = 0.f, Ee[e] = 0.f;
    if (live) {
#pragma unroll
        for (int r = 0; r < kGroupRows; ++r) {
            if (r < n) {
                const int s = st[r];
                if (s >= 0) {
                    reset = true;
    #pragma unroll
                    for (int e = 0; e < VC; ++e) H[e] = p.h0 && s < p.n_seq ? p.h0[(int64_t)s * p.C + c + e] : 0.f;
                }
    #pragma unroll
                for (int e = 0; e < VC; ++e) {
                    float a, na;
                    gate(F::get1((const E*)&z[r] + e), a, na);
                    H[e] = __builtin_fmaf(a, H[e], na * F::get1((const E*)&x[r] + e));
                    A[e] *= a;
                }
            }
        }
#pragma unroll
        for (int r = kGroupRows - 1; r >= 0; --r) {
            if (r < n) {
                if (st[r + 1] >= 0) {
                    end = true;
                    const int64_t q = sequence_of(s_start, g * kGroupRows + r, before);
    #pragma unroll
                    for (int e = 0; e < VC; ++e)
                        Ee[e] = p.dh_last && q >= 0 && q < p.n_seq ? p.dh_last[q * p.C + c + e] : 0.f;
                }
    #pragma unroll
                for (int e = 0; e < VC; ++e) {
                    float a, na;
                    gate(F::get1((const E*)&z[r] + e), a, na);
                    Ee[e] = a * (F::get1((const E*)&dy[r] + e) + Ee[e]);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        s_a[g][li * VC + e] = A[e];
        s_h[g][li * VC + e] = H[e];
        s_e[g][li * VC + e] = Ee[e];
    }
    if (li == 0) s_reset[g] = reset, s_end[g] = end;
    __syncthreads();
    for (int i = tid; i < CB; i += NT) {
        const int cc = cb * CB + i;
        if (cc >= p.C) break;
        float h = p.saved[chunk * p.C + cc], e = 0.f;
        if (CARRY) {
            Span own{1.f, 0.f, false};
#pragma unroll
            for (int k = kGroups - 1; k >= 0; --k) own = join(own, Span{s_a[k][i], s_e[k][i], s_end[k] != 0});
            e = exchange(p, order, cc, own);
        }
#pragma unroll
        for (int k = kGroups - 1; k >= 0; --k) {
            const Span s{s_a[k][i], s_e[k][i], s_end[k] != 0};
            s_e[k][i] = e;
            e = apply(s, e);
        }
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const Span s{s_a[k][i], s_h[k][i], s_reset[k] != 0};
            s_h[k][i] = h;
            h = apply(s, h);
        }
    }
    __syncthreads();
    if (!live) return;
    float hp[kGroupRows][VC];  // h_{t-1} of every row
    float h[VC], ev[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) h[e] = s_h[g][li * VC + e], ev[e] = s_e[g][li * VC + e];
#pragma unroll
    for (int r = 0; r < kGroupRows; ++r) {
        if (r < n) {
            const int s = st[r];
            if (s >= 0) {
    #pragma unroll
                for (int e = 0; e < VC; ++e) h[e] = p.h0 && s < p.n_seq ? p.h0[(int64_t)s * p.C + c + e] : 0.f;
            }
    #pragma unroll
            for (int e = 0; e < VC; ++e) {
                hp[r][e] = h[e];
                float a, na;
                gate(F::get1((const E*)&z[r] + e), a, na);
                h[e] = __builtin_fmaf(a, h[e], na * F::get1((const E*)&x[r] + e));
            }
        }
    }
    E* oz = (E*)p.dz + base * p.lddz + c;
    E* ox = (E*)p.dx + base * p.lddx + c;
#pragma unroll
    for (int r = kGroupRows - 1; r >= 0; --r) {
        if (r < n) {
            if (st[r + 1] >= 0) {
                const int64_t q = sequence_of(s_start, g * kGroupRows + r, before);
    #pragma unroll
                for (int e = 0; e < VC; ++e)
                    ev[e] = p.dh_last && q >= 0 && q < p.n_seq ? p.dh_last[q * p.C + c + e] : 0.f;
            }
            V vz, vx;
    #pragma unroll
            for (int e = 0; e < VC; ++e) {
                float a, na;
                gate(F::get1((const E*)&z[r] + e), a, na);
                const float G = F::get1((const E*)&dy[r] + e) + ev[e];
                const float gx = na * G;
                F::put1((E*)&vx + e, gx);
                F::put1((E*)&vz + e, a * gx * (hp[r][e] - F::get1((const E*)&x[r] + e)));
                ev[e] = a * G;
            }
            if (p.dz) *(V*)(oz + r * p.lddz) = vz;
            if (p.dx) *(V*)(ox + r * p.lddx) = vx;
            const int s = st[r];
            if (p.dh0 && s >= 0 && s < p.n_seq) {
    #pragma unroll
                for (int e = 0; e < VC; ++e) p.dh0[(int64_t)s * p.C + c + e] = ev[e];
            }
        }
    }
}

// Clears the exchange words and the ticket, and passes the state of empty sequences through.
__global__ __launch_bounds__(256) void k_scan_prepare(uint64_t* words, int64_t n, const int64_t* offsets,
                                                      int64_t n_seq, int C, const float* from, float* to) {
    const int64_t step = (int64_t)gridDim.x * 256;
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t i = i0; i < n; i += step) words[i] = 0;
    if (!offsets || !to) return;
    for (int64_t i = i0; i < n_seq * C; i += step) {
        const int64_t s = i / C;
        if (offsets[s] == offsets[s + 1]) to[i] = from ? from[i] : 0.f;
    }
}

int64_t chunks_of(int64_t rows) { return (rows + kChunk - 1) / kChunk; }
int64_t exchange_words(int64_t rows, int64_t C) {
    const int64_t k = chunks_of(rows), k1 = (k + kFan - 1) / kFan, k2 = (k1 + kFan - 1) / kFan;
    return 1 + (2 * k + 2 * k1 + k2) * C;
}

template <class F, int VC, int LPR, bool BWD>
hipError_t launch_scan(ScanArgs p, bool carry, hipStream_t st) {
    p.ncb = (p.C + LPR * VC - 1) / (LPR * VC);
    const int64_t grid = p.nchunks * p.ncb;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 gd((unsigned)grid), bd(LPR * kGroups);
    if (BWD) {
        if (carry)
            k_scan_backward<F, VC, LPR, true><<<gd, bd, 0, st>>>(p);
        else
            k_scan_backward<F, VC, LPR, false><<<gd, bd, 0, st>>>(p);
    } else {
        if (carry)
            k_scan_forward<F, VC, LPR, true><<<gd, bd, 0, st>>>(p);
        else
            k_scan_forward<F, VC, LPR, false><<<gd, bd, 0, st>>>(p);
    }
    return hipGetLastError();
}

// Widest vector the addresses and strides allow; narrow rows take 32 lanes so that no half wave idles.
template <class F, bool BWD>
hipError_t pick_scan(const ScanArgs& p, bool carry, bool pairs, hipStream_t st) {
    if (pairs) {
        if (p.C <= 64) return launch_scan<F, 2, 32, BWD>(p, carry, st);
        return launch_scan<F, 2, 64, BWD>(p, carry, st);
    }
    if (p.C <= 32) return launch_scan<F, 1, 32, BWD>(p, carry, st);
    return launch_scan<F, 1, 64, BWD>(p, carry, st);
}

size_t elem_size(int dtype) { return dtype == GS_F32 ? 4 : 2; }

bool pairs_ok(const gs_scan_dims& d, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
    if (d.channels % 2) return false;
    for (const void* q : ptrs)
        if ((uintptr_t)q % (2 * elem_size(d.dtype))) return false;
    for (int64_t l : lds)
        if (l % 2) return false;
    return true;
}

// A scan needs no exchange when every chunk starts a sequence, or is the only one.
bool needs_carry(const gs_scan_dims& d, const int64_t* offsets, int64_t nchunks) {
    if (nchunks <= 1) return false;
    if (offsets) return true;
    return kChunk % (d.rows / d.n_seq) != 0;
}

void fill_common(ScanArgs& p, const gs_scan_dims& d, const int64_t* offsets, void* ws) {
    p.offsets = offsets;
    p.n_seq = d.n_seq;
    p.rows = d.rows;
    p.seq_len = !offsets && d.n_seq > 0 ? d.rows / d.n_seq : 1;
    if (p.seq_len < 1) p.seq_len = 1;
    p.C = d.channels;
    p.nchunks = chunks_of(d.rows);
    const int64_t k1 = (p.nchunks + kFan - 1) / kFan;
    uint64_t* w = (uint64_t*)ws;
    p.ticket = (uint32_t*)w;
    p.agg1 = w + 1;
    p.agg2 = p.agg1 + 2 * p.nchunks * p.C;
    p.run = p.agg2 + 2 * k1 * p.C;
}

hipError_t prepare(const ScanArgs& p, bool carry, const float* from, float* to, hipStream_t st) {
    const int64_t n = carry ? exchange_words(p.rows, p.C) : 0;
    const int64_t work = n > p.n_seq * p.C ? n : (p.offsets && to ? p.n_seq * p.C : n);
    if (work <= 0) return hipSuccess;
    int64_t bx = (work + 255) / 256;
    if (bx > 2048) bx = 2048;
    k_scan_prepare<<<dim3((unsigned)bx), 256, 0, st>>>((uint64_t*)p.ticket, n, p.offsets, p.n_seq, p.C, from, to);
    return hipGetLastError();
}

}  // namespace

void scan_sizes(const gs_scan_dims& d, size_t* saved, size_t* ws) {
    *saved = (size_t)round_up(chunks_of(d.rows) * d.channels * 4, kAlign);
    *ws = (size_t)round_up(exchange_words(d.rows, d.channels) * 8, kAlign);
}

hipError_t launch_scan_forward(const gs_scan_dims& d, const int64_t* offsets, const gs_scan_inputs& in, void* y,
                               int64_t ldy, float* h_last, float* saved, void* ws, hipStream_t st) {
    ScanArgs p{};
    fill_common(p, d, offsets, ws);
    p.z = in.gate, p.x = in.x, p.h0 = in.h0, p.ldz = in.ld_gate, p.ldx = in.ld_x;
    p.y = y, p.ldy = ldy, p.h_last = h_last, p.saved = saved;
    const bool carry = needs_carry(d, offsets, p.nchunks);
    GSR_TRY(prepare(p, carry, in.h0, h_last, st));
    if (d.rows == 0) return hipSuccess;
    const bool pairs = pairs_ok(d, {in.gate, in.x, y}, {in.ld_gate, in.ld_x, ldy});
    if (d.dtype == GS_BF16) return pick_scan<FmtBf16, false>(p, carry, pairs, st);
    if (d.dtype == GS_F16) return pick_scan<FmtF16, false>(p, carry, pairs, st);
    return pick_scan<FmtF32, false>(p, carry, pairs, st);
}

hipError_t launch_scan_backward(const gs_scan_dims& d, const int64_t* offsets, const gs_scan_inputs& in,
                                const float* saved, const void* dy, int64_t lddy, const float* dh_last,
                                const gs_scan_grads& out, void* ws, hipStream_t st) {
    ScanArgs p{};
    fill_common(p, d, offsets, ws);
    p.z = in.gate, p.x = in.x, p.h0 = in.h0, p.ldz = in.ld_gate, p.ldx = in.ld_x;
    p.saved = const_cast<float*>(saved);
    p.dy = dy, p.lddy = lddy, p.dh_last = dh_last;
    p.dz = out.gate, p.dx = out.x, p.dh0 = out.h0, p.lddz = out.ld_gate, p.lddx = out.ld_x;
    const bool carry = needs_carry(d, offsets, p.nchunks);
    GSR_TRY(prepare(p, carry, dh_last, out.h0, st));
    if (d.rows == 0) return hipSuccess;
    const bool pairs = pairs_ok(d, {in.gate, in.x, dy, out.gate, out.x},
                                {in.ld_gate, in.ld_x, lddy, out.ld_gate, out.ld_x});
    if (d.dtype == GS_BF16) return pick_scan<FmtBf16, true>(p, carry, pairs, st);
    if (d.dtype == GS_F16) return pick_scan<FmtF16, true>(p, carry, pairs, st);
    return pick_scan<FmtF32, true>(p, carry, pairs, st);
}

}  // namespace gsr
