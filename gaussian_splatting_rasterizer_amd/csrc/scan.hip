// scan.hip -- gated linear recurrence of the learned updater and its gradient.
//
//   a_t = sigma(z_t), h_t = a_t h_{t-1} + (1 - a_t) x_t              per channel, h_{-1} = h0 of the sequence
//   e_t = a_t G_t,    G_t = dy_t + e_{t+1}                           e past the last row = dh_last
//   dx = (1 - a) G,   dz = a (1 - a) (h_{t-1} - x) G,   dh0 = e_0
//
// Sequences of any length lie one after another in the rows.  Rows are cut into spans (one wave's rows) and chunks of
// 8 spans (one workgroup's).  Three kernels: k_scan_spans reduces every span to (A, H) with h_out = A h_in + H, and
// every chunk; k_scan_join runs through the chunks and leaves the state that enters each; k_scan_forward (or
// k_scan_backward) joins the spans before it in the chunk and runs the recurrence.  The second reading of the inputs
// goes backwards through the chunks, so most of it comes from the 256 MB last-level cache.  A span that starts a
// sequence needs no state: where all do (short equal sequences, single steps) the last kernel runs alone.
//
// A row that starts a sequence replaces the state instead of multiplying it by zero, so nothing of one sequence, NaN
// included, reaches the next.  All orders are fixed: results are reproducible.
//
// h_last may be h0 (and dh0 may be dh_last): one wave of the last kernel then writes a sequence's final state where
// another would read its first.  Only the last sequence that starts in a span can end outside of it, so k_scan_spans
// keeps that one's first state beside the span's (A, H) and the last kernel takes it from there.  Every other sequence
// starts and ends in one span, whose wave reads before it writes.
//
// The forward pass keeps the state in front of every 8 rows in float32; the backward pass reruns the states from
// there, instead of reading back rounded ones.
//
// Bound by memory.  311,296 rows x 256 bfloat16 channels in one sequence, us and TB/s: forward spans 88 (3.6), join 21,
// recurrence 91 (5.7, part of it from the last-level cache); backward spans 96 (3.3), join 21, recurrence 174 (4.8); a
// large copy reaches 5.2.  One pass over the data, workgroups waiting for the state of the one before, took 249 us
// forward and 373 backward: the chain through 1216 chunks is longer than the second reading.
#include "gsr_internal.hpp"
#include "gemm16.hpp"

namespace gsr {

namespace {

constexpr int kBatch = 8;   // rows held in registers at a time; the forward pass saves the state in front of each
constexpr int kSpans = 8;   // spans of a chunk
constexpr int kMaxSpan = 128;
constexpr int kJoinLanes = 16, kJoinRuns = 64, kJoinChunks = 16;  // k_scan_join: channels, runs, chunks of a run

struct ScanArgs {
    const void* z;
    const void* x;
    const void* dy;
    int64_t ldz, ldx, ldy, lddy, lddz, lddx;
    const float* h0;
    const float* dh_last;
    void* y;
    float* h_last;
    float* saved;      // [rows / 8][C]
    void* dz;
    void* dx;
    float* dh0;
    const int64_t* offsets;
    int64_t n_seq, seq_len, rows, nchunks;
    int C, ncb, span;  // span: rows of a span
    // [chunk * 8 + span][3][C]: a Span's c and H, and the given state of the last sequence that starts (backward: ends)
    // in the span on the way through it, unwritten where none does.  Null: no state passes between spans.
    float* agg1;
    float* agg2;       // [chunk][2][C]
    float* state;      // [chunk][C] state entering the chunk
};

// A gate is held as the smaller of a = sigma(z) and 1 - a, to its own relative precision, and which of the two it is.
// The larger one, rounded, would be off by 2^-25, and a state that remembers 1 / (1 - a) rows by 2^-25 / (1 - a) of
// itself (z = 10: 1.4e-4), so it is never multiplied by: a v = v - (1 - a) v.
struct Gate {
    float s;
    bool keeps;  // s = 1 - a, else s = a
    __device__ __forceinline__ explicit Gate(float z) {
        const float e = __expf(-__builtin_fabsf(z));
        s = e * __builtin_amdgcn_rcpf(1.f + e);
        keeps = z >= 0.f;
    }
    __device__ __forceinline__ Gate(float s, bool keeps) : s(s), keeps(keeps) {}
    // a h + (1 - a) x; d = x - h
    __device__ __forceinline__ float mix(float h, float x, float d) const {
        return __builtin_fmaf(keeps ? s : -s, d, keeps ? h : x);
    }
    // a v and (1 - a) v
    __device__ __forceinline__ void split(float v, float& kept, float& rest) const {
        const float small = s * v, large = __builtin_fmaf(-s, v, v);
        kept = keeps ? large : small;
        rest = keeps ? small : large;
    }
};

// What a run of rows does to the state: h_out = A h_in + H, or h_out = H where a sequence starts (backward: ends) in
// it.  A product of gates is held like a gate, as A or as -(1 - A), whichever is smaller, in one number; kReset says
// that there is no A.
constexpr float kReset = 2.f;
struct Span {
    float c, H;
    __device__ __forceinline__ bool reset() const { return c > 1.f; }
    __device__ __forceinline__ bool keeps() const { return __builtin_bit_cast(int, c) < 0; }
    // of a product A and its complement, each to its own precision
    static __device__ __forceinline__ float code(float A, float rest) { return A > 0.5f ? -rest : A; }
};
constexpr float kIdentity = -0.f;  // c of the span that changes nothing
__device__ __forceinline__ float apply(const Span& s, float h) {
    const float in = s.reset() ? 0.f : h;
    return (s.keeps() ? in : 0.f) + __builtin_fmaf(s.c, in, s.H);
}
__device__ __forceinline__ Span join(const Span& first, const Span& then) {
    if (then.reset()) return then;
    const float H = apply(then, first.H);
    if (first.reset()) return {kReset, H};
    const float A = (first.keeps() ? 1.f + first.c : first.c) * (then.keeps() ? 1.f + then.c : then.c);
    const float rest = -(first.c + then.c + first.c * then.c);  // where both keep: 1 - (1 + c)(1 + c')
    return {first.keeps() && then.keeps() ? Span::code(A, rest) : A, H};
}

// Sequence starts of a chunk: s_start[i] is the sequence that starts at row row0 + i (the last one, where empty
// sequences share the row), -1 where none does, and the row past the last one counts as a start.  Returns the
// sequence that holds row row0 - 1 or starts at row0.
__device__ int64_t sequence_starts(const ScanArgs& p, int64_t row0, int* s_start, int tid, int nt) {
    const int rows = p.span * kSpans;
    if (!p.offsets) {
        const uint32_t len = (uint32_t)p.seq_len, first = (uint32_t)row0 / len;  // rows stay below 2^31
        for (int i = tid; i <= rows; i += nt) {
            const uint32_t r = (uint32_t)row0 + i, q = r / len;
            s_start[i] = r >= (uint32_t)p.rows || q * len == r ? (int)q : -1;
        }
        __syncthreads();
        return first;
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
    for (int i = tid; i <= rows; i += nt) s_start[i] = row0 + i >= p.rows ? (int)p.n_seq : -1;
    __syncthreads();
    for (int64_t s = lo + tid; s <= p.n_seq; s += nt) {
        const int64_t at = p.offsets[s] - row0;
        if (at > rows) break;
        if (at >= 0 && row0 + at < p.rows) atomicMax(&s_start[at], (int)s);
    }
    __syncthreads();
    return lo - 1;
}

// sequence that starts at / that holds row i of the chunk (i is uniform over the wave)
__device__ __forceinline__ int start_of(const int* st, int i) { return __builtin_amdgcn_readfirstlane(st[i]); }
__device__ __forceinline__ int sequence_of(const int* s_start, int i, int64_t before) {
    for (; i >= 0; --i) {
        const int s = start_of(s_start, i);
        if (s >= 0) return s;
    }
    return (int)before;
}

// One lane's channels of a row in a register: a pair of 16-bit values stays one word, or the compiler splits it.
template <class F, int VC>
struct Cell {
    using E = typename F::Elem;
    E v[VC];
    __device__ __forceinline__ float get(int e) const { return F::get1(v + e); }
    __device__ __forceinline__ void set(int e, float x) { F::put1(v + e, x); }
};
template <class F>
struct Pair16 {
    uint32_t v;
    __device__ __forceinline__ float get(int e) const {
        return F::to_float((uint16_t)(e ? v >> 16 : v & 0xffffu));
    }
    __device__ __forceinline__ void set(int e, float x) {
        const uint32_t h = F::from_float(x);
        v = e ? (v & 0xffffu) | (h << 16) : h;  // element 0 is set first
    }
};
template <>
struct Cell<FmtBf16, 2> : Pair16<FmtBf16> {};
template <>
struct Cell<FmtF16, 2> : Pair16<FmtF16> {};

// Element c of a row that starts at a uniform address: a scalar base and a 32-bit lane offset.
template <class T, class E>
__device__ __forceinline__ T* lane_at(E* row, int c) {
    return (T*)((char*)row + (uint32_t)c * (uint32_t)sizeof(E));
}

// Rows of one array seen from a span: descriptor at the span's first row, this lane's column as the offset.  Rows past
// the end and lanes past the channels go out of the descriptor's range: they read zero and are not written.
struct RowPtr {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t step, col;  // bytes of a row; the lane's column, kOobOffset for a lane without channels
    template <class E>
    static __device__ __forceinline__ RowPtr make(const void* p, int64_t row, int64_t ld, int c, bool live) {
        return {gemm_rsrc((const E*)p + row * ld), (uint32_t)(ld * sizeof(E)),
                live ? (uint32_t)c * (uint32_t)sizeof(E) : kOobOffset};
    }
    __device__ __forceinline__ uint32_t at(int r, int n) const { return r < n ? col : kOobOffset; }
};

// One batch of rows of one lane's channels.
template <class F, int VC>
struct Rows {
    using V = Cell<F, VC>;
    V v[kBatch];
    __device__ __forceinline__ void load(const RowPtr& p, int r0, int n) {
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const uint32_t off = p.at(r0 + r, n), row = (uint32_t)(r0 + r) * p.step;
            if constexpr (sizeof(V) == 8)
                v[r] = __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b64(p.rs, off, row, 0));
            else if constexpr (sizeof(V) == 4)
                v[r] = __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b32(p.rs, off, row, 0));
            else
                v[r] = __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b16(p.rs, off, row, 0));
        }
    }
    __device__ __forceinline__ float get(int r, int e) const { return v[r].get(e); }
};
template <class V>
__device__ __forceinline__ void store_row(const RowPtr& p, int r, int n, const V& v) {
    const uint32_t off = p.at(r, n), row = (uint32_t)r * p.step;
    if constexpr (sizeof(V) == 8)
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, v), p.rs, off, row, 0);
    else if constexpr (sizeof(V) == 4)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), p.rs, off, row, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), p.rs, off, row, 0);
}

// What a wave of the row kernels works on: 64 lanes x VC channels, span g of a chunk.  All but c and live are uniform
// over the wave and kept in scalar registers, so that rows are addressed by a scalar base and a lane offset.
template <int VC>
struct Place {
    int g, li, c0, c, n;
    int64_t chunk, row0, base;
    bool live;
    __device__ __forceinline__ Place(const ScanArgs& p, uint32_t id) {
        const uint32_t k = id / (uint32_t)p.ncb;
        chunk = k;
        c0 = (int)(id - k * (uint32_t)p.ncb) * (64 * VC);
        g = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        li = threadIdx.x & 63;
        c = c0 + li * VC;
        live = c < p.C;
        row0 = chunk * (p.span * kSpans);
        base = row0 + g * p.span;
        const int64_t left = p.rows - base;
        n = (int)(left < 0 ? 0 : left < p.span ? left : p.span);
    }
};

// The span's row with the last mark of st[0 .. n) (backward: the first), -1 where there is none.
template <bool BWD>
__device__ __forceinline__ int outer_mark(const int* st, int n, int lane) {
    int at = -1;
#pragma unroll
    for (int i = 0; i < kMaxSpan; i += 64) {
        const int r = (BWD ? kMaxSpan - 64 - i : i);
        const uint64_t m = __ballot(r + lane < n && st[r + lane] >= 0);
        if (m) at = r + (BWD ? __builtin_ctzll(m) : 63 - __builtin_clzll(m));
    }
    return at;
}

// bit r: a sequence starts at row r of the batch, one of the first n
__device__ __forceinline__ uint32_t start_bits(const int* st, int n) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < kBatch; ++r) m |= st[r] >= 0 ? 1u << r : 0u;
    m = __builtin_amdgcn_readfirstlane(m);
    return n < kBatch ? m & ((1u << n) - 1u) : m;
}

template <class F, int VC, bool BWD>
__global__ __launch_bounds__(64 * kSpans) void k_scan_spans(const ScanArgs p) {
    using E = typename F::Elem;
    constexpr int CB = 64 * VC, NT = 64 * kSpans;
    __shared__ int s_start[kMaxSpan * kSpans + 1];
    __shared__ float s_a[kSpans][CB], s_h[kSpans][CB];
    const Place<VC> at(p, blockIdx.x);
    const int tid = threadIdx.x;
    const int* st = s_start + at.g * p.span;
    const RowPtr pz = RowPtr::make<E>(p.z, at.base, p.ldz, at.c, at.live);
    const RowPtr px = BWD ? RowPtr::make<E>(p.dy, at.base, p.lddy, at.c, at.live)
                          : RowPtr::make<E>(p.x, at.base, p.ldx, at.c, at.live);
    float A[VC], rest[VC], H[VC], given_state[VC];  // A and 1 - A
    bool reset = false;
#pragma unroll
    for (int e = 0; e < VC; ++e) A[e] = 1.f, rest[e] = 0.f, H[e] = 0.f, given_state[e] = 0.f;
    const int nb = (at.n + kBatch - 1) / kBatch;
    Rows<F, VC> z[2], x[2];
    auto fetch = [&](int k, int b) {
        const int r0 = (BWD ? nb - 1 - k : k) * kBatch;
        z[b].load(pz, r0, at.n);
        x[b].load(px, r0, at.n);
    };
    if (nb > 0) fetch(0, 0);
    const int64_t before = sequence_starts(p, at.row0, s_start, tid, NT);
    auto run = [&](int k, int b) {
        const int r0 = (BWD ? nb - 1 - k : k) * kBatch;
        const uint32_t marks = start_bits(st + r0 + (BWD ? 1 : 0), at.n - r0);
        if (marks) reset = true;
        // rows past the end, which read zero, come last (backward: first, and leave the zero gradient zero)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = BWD ? kBatch - 1 - i : i;
            if ((marks >> r) & 1) {
                const float* src = BWD ? p.dh_last : p.h0;
                const int64_t q = BWD ? sequence_of(s_start, at.g * p.span + r0 + r, before) : start_of(st, r0 + r);
                const bool given = src && q >= 0 && q < p.n_seq && at.live;
#pragma unroll
                for (int e = 0; e < VC; ++e)
                    given_state[e] = H[e] = given ? lane_at<const float>(src + q * p.C, at.c)[e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                const Gate a(z[b].get(r, e));
                const float xv = x[b].get(r, e);
                float gone;
                if (BWD)
                    a.split(xv + H[e], H[e], gone);
                else
                    H[e] = a.mix(H[e], xv, xv - H[e]);
                a.split(A[e], A[e], gone);
                rest[e] += gone;
            }
        }
    };
    for (int k = 0; k < nb; k += 2) {
        if (k + 1 < nb) fetch(k + 1, 1);
        run(k, 0);
        if (k + 2 < nb) fetch(k + 2, 0);
        if (k + 1 < nb) run(k + 1, 1);
    }
#pragma unroll
    for (int e = 0; e < VC; ++e) A[e] = reset ? kReset : Span::code(A[e], rest[e]);
    if (at.live && nb > 0) {
        float* d = lane_at<float>(p.agg1 + (at.chunk * kSpans + at.g) * 3 * p.C, at.c);
#pragma unroll
        for (int e = 0; e < VC; ++e) d[e] = A[e], d[p.C + e] = H[e];
        if (reset) {
#pragma unroll
            for (int e = 0; e < VC; ++e) d[2 * p.C + e] = given_state[e];
        }
    }
#pragma unroll
    for (int e = 0; e < VC; ++e) s_a[at.g][at.li * VC + e] = A[e], s_h[at.g][at.li * VC + e] = H[e];
    __syncthreads();
    if (tid < CB && at.c0 + tid < p.C) {
        Span own{kIdentity, 0.f};
#pragma unroll
        for (int i = 0; i < kSpans; ++i) {
            const int k = BWD ? kSpans - 1 - i : i;
            own = join(own, Span{s_a[k][tid], s_h[k][tid]});
        }
        float* d = p.agg2 + at.chunk * 2 * p.C + at.c0 + tid;
        d[0] = own.c;
        d[p.C] = own.H;
    }
    // an empty sequence passes its state through
    if (p.offsets) {
        const float* from = BWD ? p.dh_last : p.h0;
        float* to = BWD ? p.dh0 : p.h_last;
        if (to)
            for (int64_t i = (int64_t)blockIdx.x * NT + tid; i < p.n_seq * p.C; i += (int64_t)gridDim.x * NT) {
                const int64_t s = i / p.C;
                if (p.offsets[s] == p.offsets[s + 1]) to[i] = from ? from[i] : 0.f;
            }
    }
}

// The same for a call without rows.
__global__ __launch_bounds__(256) void k_scan_empty(const float* from, float* to, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        to[i] = from ? from[i] : 0.f;
}

// State entering every chunk.  A workgroup takes 16 channels and splits the chunks into 64 runs of 16: each thread
// reduces its run in registers, all runs are joined through LDS, and the thread walks its run again.  64 channels and
// 16 runs of 32 took 14 us for 512 chunks, nearly all of it waiting for the loads of one wave's run.
template <bool BWD>
__global__ __launch_bounds__(kJoinLanes* kJoinRuns) void k_scan_join(const ScanArgs p) {
    __shared__ float s_a[kJoinRuns][kJoinLanes], s_h[kJoinRuns][kJoinLanes];
    const int lane = threadIdx.x % kJoinLanes, w = threadIdx.x / kJoinLanes;
    const int c = blockIdx.x * kJoinLanes + lane;
    const bool live = c < p.C;
    float run = 0.f;  // state in front of the block of runs
    for (int64_t o = 0; o < p.nchunks; o += kJoinRuns * kJoinChunks) {
        Span v[kJoinChunks];
        const int64_t o0 = o + w * kJoinChunks;
#pragma unroll
        for (int i = 0; i < kJoinChunks; ++i) {
            v[i] = {kIdentity, 0.f};
            if (live && o0 + i < p.nchunks) {
                const float* a = p.agg2 + (BWD ? p.nchunks - 1 - o0 - i : o0 + i) * 2 * p.C + c;
                v[i] = {a[0], a[p.C]};
            }
        }
        Span own{kIdentity, 0.f};
#pragma unroll
        for (int i = 0; i < kJoinChunks; ++i) own = join(own, v[i]);
        s_a[w][lane] = own.c, s_h[w][lane] = own.H;
        __syncthreads();
        float h = run;
#pragma unroll 8
        for (int j = 0; j < kJoinRuns; ++j) {
            if (j == w) h = run;
            run = apply(Span{s_a[j][lane], s_h[j][lane]}, run);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kJoinChunks; ++i) {
            if (live && o0 + i < p.nchunks) p.state[(BWD ? p.nchunks - 1 - o0 - i : o0 + i) * p.C + c] = h;
            h = apply(v[i], h);
        }
    }
}

// State entering the lane's span: the chunk's, then the spans in front of it.
template <int VC, bool BWD>
__device__ __forceinline__ void span_state(const ScanArgs& p, const Place<VC>& at, float (*s_a)[64 * VC],
                                           float (*s_h)[64 * VC], float (&h)[VC]) {
#pragma unroll
    for (int e = 0; e < VC; ++e) h[e] = 0.f;
    if (!p.agg1) return;
    const bool mine = at.live && at.n > 0;
    const float* d = lane_at<const float>(p.agg1 + (at.chunk * kSpans + at.g) * 3 * p.C, at.c);
    const float* s = lane_at<const float>(p.state + at.chunk * p.C, at.c);
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        s_a[at.g][at.li * VC + e] = mine ? d[e] : kIdentity;
        s_h[at.g][at.li * VC + e] = mine ? d[p.C + e] : 0.f;
        if (at.live && p.state) h[e] = s[e];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSpans - 1; ++i) {
        const int j = BWD ? kSpans - 1 - i : i;
        if (BWD ? j > at.g : j < at.g) {
#pragma unroll
            for (int e = 0; e < VC; ++e) h[e] = apply(Span{s_a[j][at.li * VC + e], s_h[j][at.li * VC + e]}, h[e]);
        }
    }
}

template <class F, int VC>
__global__ __launch_bounds__(64 * kSpans) void k_scan_forward(const ScanArgs p) {
    using E = typename F::Elem;
    constexpr int CB = 64 * VC, NT = 64 * kSpans;
    __shared__ int s_start[kMaxSpan * kSpans + 1];
    __shared__ float s_a[kSpans][CB], s_h[kSpans][CB];
    const Place<VC> at(p, gridDim.x - 1 - blockIdx.x);  // what was read last comes first
    const int* st = s_start + at.g * p.span;
    const RowPtr pz = RowPtr::make<E>(p.z, at.base, p.ldz, at.c, at.live);
    const RowPtr px = RowPtr::make<E>(p.x, at.base, p.ldx, at.c, at.live);
    const RowPtr py = RowPtr::make<E>(p.y, at.base, p.ldy, at.c, at.live);
    const int nb = (at.n + kBatch - 1) / kBatch;
    Rows<F, VC> z[2], x[2];
    auto fetch = [&](int k, int b) {
        z[b].load(pz, k * kBatch, at.n);
        x[b].load(px, k * kBatch, at.n);
    };
    if (nb > 0) fetch(0, 0);
    const int64_t before = sequence_starts(p, at.row0, s_start, threadIdx.x, NT);
    float h[VC];
    span_state<VC, false>(p, at, s_a, s_h, h);
    // the row whose first state h_last may overwrite, and that state's copy
    const int kept_row = p.agg1 ? outer_mark<false>(st, at.n, at.li) : -1;
    const float* kept = p.agg1 + ((at.chunk * kSpans + at.g) * 3 + 2) * p.C;
    auto run = [&](int k, int b) {
        const int r0 = k * kBatch;
        const uint32_t starts = start_bits(st + r0, at.n - r0);
        const uint32_t ends = p.h_last ? start_bits(st + r0 + 1, at.n - r0) : 0u;
        if (p.saved && at.live) {
            float* d = lane_at<float>(p.saved + (at.base + r0) / kBatch * p.C, at.c);
#pragma unroll
            for (int e = 0; e < VC; ++e) d[e] = h[e];
        }
        float first[kBatch][VC];
        if (starts) {
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                const int s = (starts >> r) & 1 ? start_of(st, r0 + r) : -1;
                const bool given = p.h0 && s >= 0 && s < p.n_seq && at.live;
                const float* src = r0 + r == kept_row ? kept : p.h0 + (int64_t)s * p.C;
#pragma unroll
                for (int e = 0; e < VC; ++e) first[r][e] = given ? lane_at<const float>(src, at.c)[e] : 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            Cell<F, VC> y;
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                if ((starts >> r) & 1) h[e] = first[r][e];
                const float xv = x[b].get(r, e);
                h[e] = Gate(z[b].get(r, e)).mix(h[e], xv, xv - h[e]);
                y.set(e, h[e]);
            }
            store_row(py, r0 + r, at.n, y);
            if (((ends >> r) & 1) && at.live) {
                const int64_t q = sequence_of(s_start, at.g * p.span + r0 + r, before);
                if (q >= 0 && q < p.n_seq) {
#pragma unroll
                    for (int e = 0; e < VC; ++e) lane_at<float>(p.h_last + q * p.C, at.c)[e] = h[e];
                }
            }
        }
    };
    for (int k = 0; k < nb; k += 2) {
        if (k + 1 < nb) fetch(k + 1, 1);
        run(k, 0);
        if (k + 2 < nb) fetch(k + 2, 0);
        if (k + 1 < nb) run(k + 1, 1);
    }
}

template <class F, int VC>
__global__ __launch_bounds__(64 * kSpans) void k_scan_backward(const ScanArgs p) {
    using E = typename F::Elem;
    constexpr int CB = 64 * VC, NT = 64 * kSpans;
    __shared__ int s_start[kMaxSpan * kSpans + 1];
    __shared__ float s_a[kSpans][CB], s_h[kSpans][CB];
    const Place<VC> at(p, blockIdx.x);  // the spans were read from the last chunk to the first
    const int* st = s_start + at.g * p.span;
    const RowPtr pz = RowPtr::make<E>(p.z, at.base, p.ldz, at.c, at.live);
    const RowPtr px = RowPtr::make<E>(p.x, at.base, p.ldx, at.c, at.live);
    const RowPtr pd = RowPtr::make<E>(p.dy, at.base, p.lddy, at.c, at.live);
    const RowPtr oz = RowPtr::make<E>(p.dz, at.base, p.lddz, at.c, at.live && p.dz);
    const RowPtr ox = RowPtr::make<E>(p.dx, at.base, p.lddx, at.c, at.live && p.dx);
    const int nb = (at.n + kBatch - 1) / kBatch;
    Rows<F, VC> z, x, dy;
    float hs[VC];
    auto fetch = [&](int k) {
        const int r0 = k * kBatch;
        z.load(pz, r0, at.n);
        x.load(px, r0, at.n);
        dy.load(pd, r0, at.n);
        const float* d = lane_at<const float>(p.saved + (at.base + r0) / kBatch * p.C, at.live ? at.c : 0);
#pragma unroll
        for (int e = 0; e < VC; ++e) hs[e] = d[e];
    };
    if (nb > 0) fetch(nb - 1);
    const int64_t before = sequence_starts(p, at.row0, s_start, threadIdx.x, NT);
    float ev[VC];
    span_state<VC, true>(p, at, s_a, s_h, ev);
    // the row whose final gradient dh0 may overwrite, and that gradient's copy
    const int kept_row = p.agg1 ? outer_mark<true>(st + 1, at.n, at.li) : -1;
    const float* kept = p.agg1 + ((at.chunk * kSpans + at.g) * 3 + 2) * p.C;
    for (int k = nb - 1; k >= 0; --k) {
        const int r0 = k * kBatch;
        const uint32_t starts = start_bits(st + r0, at.n - r0), ends = start_bits(st + r0 + 1, at.n - r0);
        // the gate, s negative where it is a; a (1 - a) (h_{t-1} - x)
        float q[kBatch][VC], w[kBatch][VC];
        float h[VC];
#pragma unroll
        for (int e = 0; e < VC; ++e) h[e] = hs[e];
        // states in front of rows that start a sequence, then the gradients that leave those rows
        float first[kBatch][VC];
        if (starts) {
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                const int s = (starts >> r) & 1 ? start_of(st, r0 + r) : -1;
                const bool given = p.h0 && s >= 0 && s < p.n_seq && at.live;
#pragma unroll
                for (int e = 0; e < VC; ++e)
                    first[r][e] = given ? lane_at<const float>(p.h0 + (int64_t)s * p.C, at.c)[e] : 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                if ((starts >> r) & 1) h[e] = first[r][e];
                const Gate a(z.get(r, e));
                const float xv = x.get(r, e), d = xv - h[e];
                q[r][e] = a.keeps ? a.s : -a.s;
                w[r][e] = __builtin_fmaf(a.s, a.s, -a.s) * d;
                h[e] = a.mix(h[e], xv, d);
            }
        }
        const Rows<F, VC> d = dy;
        if (k > 0) fetch(k - 1);
        float last[kBatch][VC];
        if (ends) {
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                const int64_t s = (ends >> r) & 1 ? sequence_of(s_start, at.g * p.span + r0 + r, before) : -1;
                const bool given = p.dh_last && s >= 0 && s < p.n_seq && at.live;
                const float* src = r0 + r == kept_row ? kept : p.dh_last + s * p.C;
#pragma unroll
                for (int e = 0; e < VC; ++e) last[r][e] = given ? lane_at<const float>(src, at.c)[e] : 0.f;
            }
        }
#pragma unroll
        for (int r = kBatch - 1; r >= 0; --r) {
            Cell<F, VC> vz, vx;
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                if ((ends >> r) & 1) ev[e] = last[r][e];
                const Gate a(__builtin_fabsf(q[r][e]), __builtin_bit_cast(int, q[r][e]) >= 0);
                const float G = d.get(r, e) + ev[e];
                float gx;
                a.split(G, ev[e], gx);
                vx.set(e, gx);
                vz.set(e, w[r][e] * G);
                first[r][e] = ev[e];
            }
            store_row(oz, r0 + r, at.n, vz);
            store_row(ox, r0 + r, at.n, vx);
        }
        if (starts && p.dh0 && at.live) {
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                const int s = (starts >> r) & 1 ? start_of(st, r0 + r) : -1;
                if (s >= 0 && s < p.n_seq) {
#pragma unroll
                    for (int e = 0; e < VC; ++e) lane_at<float>(p.dh0 + (int64_t)s * p.C, at.c)[e] = first[r][e];
                }
            }
        }
    }
}

// ---- host ----------------------------------------------------------------------------------------------

// Rows of a span.  Longer spans leave fewer states to join, shorter ones more waves: 16 rows while that gives 4096
// waves (16 a CU), longer ones only from 16384 waves on.  Forward + backward of one sequence of 311,296 rows x 256
// bfloat16 channels took 482 us with spans of 16, 468 with 32, 464 with 64, 607 with 128; 50,021 x 192 float32 161 us
// with spans of 8, 150 with 16, 166 with 32, 215 with 64.
int span_rows(const gs_scan_dims& d) {
    const int64_t waves = d.rows * ((d.channels + 127) / 128);
    int s = kBatch;
    while (s < kMaxSpan && waves / (2 * s) >= (s == kBatch ? 4096 : 16384)) s *= 2;
    return s;
}
int64_t chunks_of(const gs_scan_dims& d) {
    const int64_t c = (int64_t)span_rows(d) * kSpans;
    return (d.rows + c - 1) / c;
}

template <class F, int VC, bool BWD>
hipError_t launch_scan(ScanArgs p, hipStream_t st) {
    p.ncb = (p.C + 64 * VC - 1) / (64 * VC);
    const int64_t grid = p.nchunks * p.ncb;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 gd((unsigned)grid), bd(64 * kSpans);
    if (p.agg1) {
        k_scan_spans<F, VC, BWD><<<gd, bd, 0, st>>>(p);
        GSR_TRY(hipGetLastError());
        if (p.nchunks > 1) {
            const dim3 gj((unsigned)((p.C + kJoinLanes - 1) / kJoinLanes));
            k_scan_join<BWD><<<gj, kJoinLanes * kJoinRuns, 0, st>>>(p);
            GSR_TRY(hipGetLastError());
        } else {
            p.state = nullptr;
        }
    }
    if (BWD)
        k_scan_backward<F, VC><<<gd, bd, 0, st>>>(p);
    else
        k_scan_forward<F, VC><<<gd, bd, 0, st>>>(p);
    return hipGetLastError();
}

// Two channels a lane where addresses and strides allow and there are more than one for every lane.
template <class F, bool BWD>
hipError_t pick_scan(const ScanArgs& p, bool pairs, hipStream_t st) {
    return pairs && p.C > 64 ? launch_scan<F, 2, BWD>(p, st) : launch_scan<F, 1, BWD>(p, st);
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

int64_t carve_scan(const gs_scan_dims& d, char* ws, ScanArgs* p) {
    Carver cv{ws};
    const int64_t n = chunks_of(d), C = d.channels;
    p->agg1 = cv.take<float>(n * kSpans * 3 * C);
    p->agg2 = cv.take<float>(n * 2 * C);
    p->state = cv.take<float>(n * C);
    return cv.used;
}

void fill_common(ScanArgs& p, const gs_scan_dims& d, const int64_t* offsets, const gs_scan_inputs& in, void* ws) {
    carve_scan(d, (char*)ws, &p);
    p.z = in.gate, p.x = in.x, p.h0 = in.h0, p.ldz = in.ld_gate, p.ldx = in.ld_x;
    p.offsets = offsets;
    p.n_seq = d.n_seq;
    p.rows = d.rows;
    p.seq_len = !offsets && d.n_seq > 0 && d.rows > 0 ? d.rows / d.n_seq : 1;
    p.C = d.channels;
    p.span = span_rows(d);
    p.nchunks = chunks_of(d);
    if (!offsets && p.span % p.seq_len == 0) p.agg1 = nullptr;  // every span starts a sequence
}

hipError_t pass_through(const gs_scan_dims& d, const float* from, float* to, hipStream_t st) {
    const int64_t n = d.n_seq * d.channels;
    if (!to || n == 0) return hipSuccess;
    const int64_t bx = (n + 255) / 256;
    k_scan_empty<<<dim3((unsigned)(bx > 2048 ? 2048 : bx)), 256, 0, st>>>(from, to, n);
    return hipGetLastError();
}

}  // namespace

void scan_sizes(const gs_scan_dims& d, size_t* saved, size_t* ws) {
    ScanArgs p{};
    *saved = (size_t)round_up((d.rows + kBatch - 1) / kBatch * d.channels * 4, kAlign);
    *ws = (size_t)carve_scan(d, nullptr, &p);
}

hipError_t launch_scan_forward(const gs_scan_dims& d, const int64_t* offsets, const gs_scan_inputs& in, void* y,
                               int64_t ldy, float* h_last, float* saved, void* ws, hipStream_t st) {
    if (d.rows == 0) return pass_through(d, in.h0, h_last, st);
    ScanArgs p{};
    fill_common(p, d, offsets, in, ws);
    p.y = y, p.ldy = ldy, p.h_last = h_last, p.saved = saved;
    const bool pairs = pairs_ok(d, {in.gate, in.x, y}, {in.ld_gate, in.ld_x, ldy});
    if (d.dtype == GS_BF16) return pick_scan<FmtBf16, false>(p, pairs, st);
    if (d.dtype == GS_F16) return pick_scan<FmtF16, false>(p, pairs, st);
    return pick_scan<FmtF32, false>(p, pairs, st);
}

hipError_t launch_scan_backward(const gs_scan_dims& d, const int64_t* offsets, const gs_scan_inputs& in,
                                const float* saved, const void* dy, int64_t lddy, const float* dh_last,
                                const gs_scan_grads& out, void* ws, hipStream_t st) {
    if (d.rows == 0) return pass_through(d, dh_last, out.h0, st);
    ScanArgs p{};
    fill_common(p, d, offsets, in, ws);
    p.saved = const_cast<float*>(saved);
    p.dy = dy, p.lddy = lddy, p.dh_last = dh_last;
    p.dz = out.gate, p.dx = out.x, p.dh0 = out.h0, p.lddz = out.ld_gate, p.lddx = out.ld_x;
    const bool pairs = pairs_ok(d, {in.gate, in.x, dy, out.gate, out.x},
                                {in.ld_gate, in.ld_x, lddy, out.ld_gate, out.ld_x});
    if (d.dtype == GS_BF16) return pick_scan<FmtBf16, true>(p, pairs, st);
    if (d.dtype == GS_F16) return pick_scan<FmtF16, true>(p, pairs, st);
    return pick_scan<FmtF32, true>(p, pairs, st);
}

}  // namespace gsr
