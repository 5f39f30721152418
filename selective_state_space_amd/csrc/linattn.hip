// linattn.hip -- linear attention with one fixed decay per head: the chunked form
// for prompts and training, its backward, and the step for single tokens.
//
//     S_t = lambda S_{t-1} + k_t (x) v_t,   o_t = scale q_t^T S_t,   lambda = e^{log_decay[h]}
//
// Chunked form, chunk of C = 64 tokens, i and j positions in the chunk, S the state
// entering it:
//     o_i = scale (sum_{j<=i} lambda^{i-j} (q_i . k_j) v_j + lambda^{i+1} q_i^T S)
//     S  <- lambda^C S + sum_j lambda^{C-1-j} k_j (x) v_j
// The decay is fixed, so every weight is a power of one number in the positions'
// difference: no prefix sums, no decay tensor.
//
// The backward is the same chunked form three times, on other operands and, for the
// keys and values, from the last token to the first:
//     dq_i = scale sum_{j<=i} lambda^{i-j} (do_i . v_j) k_j + ...   queries do, keys v, values k
//     dk_j = scale sum_{i>=j} lambda^{i-j} (v_j . do_i) q_i + ...   queries v, keys do, values q, reversed
//     dv_j = scale sum_{i>=j} lambda^{i-j} (k_j . q_i) do_i + ...   queries k, keys q, values do, reversed
// In the reversed runs the state is the adjoint R (entering: the final state's
// gradient), a token's own product meets it undecayed, so its power is i instead of
// i + 1 and C - j instead of C - 1 - j.
//
// A sequence is cut into segments so that the device is full: k_la_state computes
// each segment's own end state, k_la_carry composes them into the states that enter
// the segments, k_la_out walks the chunks of every segment from there.
#include <algorithm>

#include "mb_internal.h"

namespace mb {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));

constexpr int kC = 64;          // tokens of a chunk
constexpr int kV = 64;          // value columns of a workgroup
constexpr int kMaxDim = 128;    // of keys and of values
constexpr int kThreads = 256;

struct __attribute__((aligned(16))) PlanEntry {
    int seq, first, len, idx;         // sequence (-1: none), its first token and length, the segment's place in it
    int state, pad[3];                // where the segment's entering state lies
};

struct LaArgs {
    const void* a;              // query role, key role, value role, output
    const void* b;
    const void* c;
    void* o;
    int64_t a_ts, b_ts, c_ts, o_ts;   // elements between tokens
    int a_rep, b_rep, c_rep;          // heads that share one row of it
    int H, Da, Dv, nv;                // heads, width of a and b, width of c and o, column tiles of c
    const float* log_decay;
    float s_in, s_carry, s_up;        // factors: masked scores, carried state's product, state update
    int shift;                        // a token's own power of lambda on the carried state: 1, reversed 0
    int reversed;
    int n_seq;
    int64_t T, L;                     // tokens in all; of a sequence when they are equal
    int seg_len, nseg;                // segment length, segments launched
    int per_seq;                      // segments of a sequence when lengths are equal, else 0
    const int32_t* cu;
    const struct PlanEntry* plan;     // one for each segment; NULL: by arithmetic
    const int2* seqs;                 // (first state, segments) of a sequence, with plan
    float* states;                    // per (state, head, column tile): a state in fragment order
    const float* h0;
    const uint8_t* has_h0;
    const int32_t* slots;
    int64_t n_slots;
    int transposed;                   // h0 is (H, Dv, Da)
    float* h_out;
};

struct Seg {
    int seq;             // < 0: nothing to do
    int64_t first, len;  // the sequence's first token and length
    int idx;             // the segment's place in it
    int state;           // where its entering state lies
    int64_t p0;          // its first position in walking order
    int n;               // its tokens
    bool last, only;
};

__device__ __forceinline__ Seg segment(const LaArgs& A, int s) {
    Seg g;
    if (A.plan) {
        const PlanEntry e = A.plan[s];
        g.seq = e.seq;
        g.first = e.first;
        g.len = e.len;
        g.idx = e.idx;
        g.state = e.state;
    } else if (A.cu) {   // every sequence is one segment
        const int64_t b = min((int64_t)max(A.cu[s], 0), A.T), e = min((int64_t)max(A.cu[s + 1], 0), A.T);
        g.seq = s;
        g.first = b;
        g.len = max(e - b, (int64_t)0);
        g.idx = 0;
        g.state = 0;
    } else {
        g.seq = s / A.per_seq;
        g.idx = s - g.seq * A.per_seq;
        g.first = g.seq * A.L;
        g.len = A.L;
        g.state = s;
    }
    g.p0 = (int64_t)g.idx * A.seg_len;
    g.n = (int)min((int64_t)A.seg_len, g.len - g.p0);
    g.last = g.p0 + g.n >= g.len;
    g.only = g.last && g.idx == 0;
    return g;
}

// Row of h0 / h_out of a sequence, or -1 where it has none.
__device__ __forceinline__ int64_t state_row(const LaArgs& A, int seq) {
    if (!A.slots) return seq;
    const int64_t r = A.slots[seq];
    return r >= 0 && r < A.n_slots ? r : -1;
}

// log2 of lambda, kept finite so that a power of zero is one at lambda = 0 too.
__device__ __forceinline__ float log2_decay(const LaArgs& A, int h) {
    const float l = A.log_decay[h] * kLog2e;
    return l < -16384.0f ? -16384.0f : l;
}
__device__ __forceinline__ float power(float l2, int64_t n) { return exp2_fast(l2 * (float)n); }

// ------------------------------------------------------------- fragments ----
// A fragment is 16 bytes a lane: bf16 eight values of one 16x16x32 product, fp32
// four values of four 16x16x4 products (lane group g then holds contraction indices
// 4g .. 4g + 3 of 16, the same on both operands, so any order of them is right).
template <typename T> struct Frag;
template <> struct Frag<bf16> {
    static constexpr int K = 32, VE = 8;
    static __device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    }
};
template <> struct Frag<float> {
    static constexpr int K = 16, VE = 4;
    static __device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
        return c;
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));   // nearest even
}

// Four tokens of one column from a row-major tile [token][column]: lane m of a
// 16-lane group gets tokens tok .. tok + 3 of the m-th of the 16 columns that the
// group's addresses name (lane m points at token tok + m / 4 and four columns).
__device__ __forceinline__ u2 tr4(const bf16* p) {
    typedef __attribute__((address_space(3))) s4* lp;
    return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p)));
}

// One row's vector of VE elements from global memory; elements at and behind `n` are zero.
template <typename T, bool VEC>
__device__ __forceinline__ u4 load_row(const T* p, int n) {
    u4 v = {0, 0, 0, 0};
    if constexpr (VEC) {
        if (n > 0) v = *reinterpret_cast<const u4*>(p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) v[e] = __float_as_uint(p[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    return v;
}

// A tile of kC tokens by W columns: its global reads into registers, and from there to LDS.
template <typename T, int W, bool VEC>
struct Tile {
    static constexpr int VE = Frag<T>::VE;
    static constexpr int PER_ROW = W / VE;
    static constexpr int N = kC * PER_ROW / kThreads;
    static constexpr int STRIDE = W + 16 / (int)sizeof(T);   // 16 bytes of padding spread rows over the banks
    static_assert(N * kThreads == kC * PER_ROW, "whole vectors for every thread");
    u4 v[N];

    // base: the tile's first token's row; step: signed elements to the next token's row.
    __device__ __forceinline__ void load(const T* base, int64_t step, int tokens, int width) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = i * kThreads + threadIdx.x;
            const int r = k / PER_ROW, c = (k % PER_ROW) * VE;
            v[i] = load_row<T, VEC>(base + r * step + c, r < tokens ? width - c : 0);
        }
    }
    __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = i * kThreads + threadIdx.x;
            const int r = k / PER_ROW, c = (k % PER_ROW) * VE;
            *reinterpret_cast<u4*>(lds + r * STRIDE + c) = v[i];
        }
    }
};

// ---------------------------------------------------------- state update ----
// S += sum over the chunk's tokens of K (x) (w V): wave w holds value columns
// 16 w .. 16 w + 15 of the tile, all DA rows, as DA / 16 accumulators (rows 16 u +
// 4 g + r, column lane & 15).
//
// bf16: w V does not fit bf16, and one rounding of it would leave 2^-9 in a state that
// is kept in fp32.  It is cut into three bf16 pieces (8 + 8 + 8 bits hold all 24 of the
// product), three products on the exact K.
template <typename T, int DA>
__device__ __forceinline__ void update_state(f4 (&S)[DA / 16], const T* kt, const T* vt, const float* wt, int wave, int lane) {
    constexpr int KS = Tile<T, DA, true>::STRIDE, VS = Tile<T, kV, true>::STRIDE;
    const int m = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int t0 = 32 * s + 8 * g + (m >> 2);
            const u2 v0 = tr4(vt + t0 * VS + 16 * wave + 4 * (m & 3)), v1 = tr4(vt + (t0 + 4) * VS + 16 * wave + 4 * (m & 3));
            const uint32_t raw[4] = {v0[0], v0[1], v1[0], v1[1]};
            const f4 w0 = *reinterpret_cast<const f4*>(wt + 32 * s + 8 * g), w1 = *reinterpret_cast<const f4*>(wt + 32 * s + 8 * g + 4);
            u4 p[3];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = __uint_as_float(raw[e] << 16) * (e < 2 ? w0[2 * e] : w1[2 * e - 4]);
                float y = __uint_as_float(raw[e] & 0xffff0000u) * (e < 2 ? w0[2 * e + 1] : w1[2 * e - 3]);
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    const uint32_t hx = __float_as_uint(x) & 0xffff0000u, hy = __float_as_uint(y) & 0xffff0000u;
                    p[q][e] = (hx >> 16) | hy;
                    x -= __uint_as_float(hx);
                    y -= __uint_as_float(hy);
                }
            }
#pragma unroll
            for (int u = 0; u < DA / 16; ++u) {
                const u2 a0 = tr4(kt + t0 * KS + 16 * u + 4 * (m & 3)), a1 = tr4(kt + (t0 + 4) * KS + 16 * u + 4 * (m & 3));
                const u4 a = {a0[0], a0[1], a1[0], a1[1]};
#pragma unroll
                for (int q = 0; q < 3; ++q) S[u] = Frag<T>::mma(a, p[q], S[u]);
            }
        }
    } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int t0 = 16 * s + 4 * g;
            const f4 w = *reinterpret_cast<const f4*>(wt + t0);
            u4 b;
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(vt[(t0 + e) * VS + 16 * wave + m] * w[e]);
#pragma unroll
            for (int u = 0; u < DA / 16; ++u) {
                u4 a;
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = __float_as_uint(kt[(t0 + e) * KS + 16 * u + m]);
                S[u] = Frag<T>::mma(a, b, S[u]);
            }
        }
    }
}

// Weights of the state update of a chunk of n tokens: s_up lambda^{n - shift - j}; the rows
// behind its tokens are zeros, and their weight too.
__device__ __forceinline__ void fill_weights(float* wt, float l2, int n, int shift, float s_up) {
    if (threadIdx.x < kC) wt[threadIdx.x] = (int)threadIdx.x < n ? s_up * power(l2, n - shift - (int)threadIdx.x) : 0.0f;
}

template <typename T>
__device__ __forceinline__ const T* rows_of(const void* p, const LaArgs& A, const Seg& g, int64_t pos, int64_t ts, int head_off) {
    const int64_t t = A.reversed ? g.first + g.len - 1 - pos : g.first + pos;
    return (const T*)p + t * ts + head_off;
}

__device__ __forceinline__ int64_t state_at(const LaArgs& A, int at, int h, int tile, int da) {
    return (((int64_t)at * A.H + h) * A.nv + tile) * (da * kV);
}

struct Unit { int seg, h, tile; };
__device__ __forceinline__ Unit unit_of(const LaArgs& A) {
    int b = blockIdx.x;
    Unit u;
    u.tile = b % A.nv;
    b /= A.nv;
    u.h = b % A.H;
    u.seg = b / A.H;
    return u;
}

// ------------------------------------------------------------------ plan ----
// Inclusive running sum and maximum over the workgroup's 256 threads.
__device__ __forceinline__ int running(int v, bool sum, int* lds) {
    lds[threadIdx.x] = v;
    __syncthreads();
    for (int o = 1; o < 256; o <<= 1) {
        const int u = (int)threadIdx.x >= o ? lds[threadIdx.x - o] : 0;
        __syncthreads();
        v = sum ? v + u : max(v, u);
        lds[threadIdx.x] = v;
        __syncthreads();
    }
    return v;
}

// Segments of packed sequences.  Offsets that decrease or leave [0, T] are taken as
// empty sequences, so there are never more than T / seg_len + n_seq segments, nor more
// than 2 T / seg_len in sequences of several (each such has at most 2 len / seg_len).
__global__ void __launch_bounds__(256) k_la_plan(const int32_t* cu, int n_seq, int64_t T, int seg_len, int nseg, PlanEntry* plan,
                                                 int2* seqs) {
    __shared__ int lds[256], total[3];
    int base = 0, sbase = 0, reach = 0;          // segments, states, largest offset so far
    for (int s0 = 0; s0 < n_seq; s0 += 256) {
        const int s = s0 + threadIdx.x;
        const bool in = s < n_seq;
        const int b0 = in ? (int)min((int64_t)max(cu[s], 0), T) : 0, e0 = in ? (int)min((int64_t)max(cu[s + 1], 0), T) : 0;
        const int top = max(reach, running(max(b0, e0), false, lds));
        const int before = threadIdx.x ? max(reach, lds[threadIdx.x - 1]) : reach;
        const int b = max(b0, before), len = max(e0 - b, 0);
        const int cnt = in ? max((int)(((int64_t)len + seg_len - 1) / seg_len), 1) : 0, st = cnt > 1 ? cnt : 0;
        __syncthreads();
        const int at = running(cnt, true, lds) - cnt;
        __syncthreads();
        const int sat = running(st, true, lds) - st;
        if (in) {
            seqs[s] = make_int2(sbase + sat, cnt);
            for (int i = 0; i < cnt; ++i)
                if (base + at + i < nseg) plan[base + at + i] = PlanEntry{s, b, len, i, sbase + sat + i, {0, 0, 0}};
        }
        if (threadIdx.x == 255) {
            total[0] = at + cnt;
            total[1] = sat + st;
            total[2] = top;
        }
        __syncthreads();
        base += total[0];
        sbase += total[1];
        reach = total[2];
        __syncthreads();
    }
    for (int i = base + threadIdx.x; i < nseg; i += 256) plan[i] = PlanEntry{-1, 0, 0, 0, 0, {0, 0, 0}};
}

// ---------------------------------------------------------- segment state ----
template <typename T, int DA, bool VEC>
__global__ void __launch_bounds__(kThreads) k_la_state(LaArgs A) {
    using KT = Tile<T, DA, VEC>;
    using VT = Tile<T, kV, VEC>;
    __shared__ __attribute__((aligned(16))) T kt[kC * KT::STRIDE];
    __shared__ __attribute__((aligned(16))) T vt[kC * VT::STRIDE];
    __shared__ __attribute__((aligned(16))) float wt[kC];
    const Unit u = unit_of(A);
    const Seg g = segment(A, u.seg);
    if (g.seq < 0 || g.last) return;             // a last segment's end state is the final state: the walk makes it
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float l2 = log2_decay(A, u.h);
    const int64_t bs = A.reversed ? -A.b_ts : A.b_ts, cs = A.reversed ? -A.c_ts : A.c_ts;
    const T* kp = rows_of<T>(A.b, A, g, g.p0, A.b_ts, (u.h / A.b_rep) * A.Da);
    const T* vp = rows_of<T>(A.c, A, g, g.p0, A.c_ts, (u.h / A.c_rep) * A.Dv + u.tile * kV);
    const int vw = A.Dv - u.tile * kV;
    f4 S[DA / 16];
#pragma unroll
    for (int i = 0; i < DA / 16; ++i) S[i] = f4{0, 0, 0, 0};
    fill_weights(wt, l2, kC, A.shift, A.s_up);
    const float carry = power(l2, kC);
    KT k;
    VT v;
    k.load(kp, bs, min(kC, g.n), A.Da);
    v.load(vp, cs, min(kC, g.n), vw);
    for (int c0 = 0; c0 < g.n; c0 += kC) {       // whole chunks: only a last segment has a ragged one
        __syncthreads();
        k.store(kt);
        v.store(vt);
        __syncthreads();
        if (c0 + kC < g.n) {
            k.load(kp + (c0 + kC) * bs, bs, min(kC, g.n - c0 - kC), A.Da);
            v.load(vp + (c0 + kC) * cs, cs, min(kC, g.n - c0 - kC), vw);
        }
#pragma unroll
        for (int i = 0; i < DA / 16; ++i) S[i] *= carry;
        update_state<T, DA>(S, kt, vt, wt, wave, lane);
    }
    float* out = A.states + state_at(A, g.state, u.h, u.tile, DA);
#pragma unroll
    for (int i = 0; i < DA / 16; ++i)
        *reinterpret_cast<f4*>(out + ((wave * (DA / 16) + i) * 64 + lane) * 4) = S[i];
}

// The four state values of accumulator i of a wave's lane: rows 16 i + 4 g + r, one column.
__device__ __forceinline__ f4 load_h0(const LaArgs& A, int seq, int h, int tile, int wave, int i, int lane) {
    f4 v = {0, 0, 0, 0};
    const int64_t row = state_row(A, seq);
    if (!A.h0 || row < 0 || (A.has_h0 && !A.has_h0[seq])) return v;
    const float* p = A.h0 + (row * A.H + h) * (int64_t)A.Da * A.Dv;
    const int col = tile * kV + 16 * wave + (lane & 15), r0 = 16 * i + 4 * (lane >> 4);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (col < A.Dv && r0 + r < A.Da) v[r] = A.transposed ? p[(int64_t)col * A.Da + r0 + r] : p[(int64_t)(r0 + r) * A.Dv + col];
    return v;
}

// ---------------------------------------------------------------- carry ----
// In place over a sequence's segments: the state that enters each of them.  A workgroup
// takes 1024 values (256 lanes of four) of one (sequence, head, tile).
template <int DA>
__global__ void __launch_bounds__(256) k_la_carry(LaArgs A) {
    constexpr int PER = DA * kV / 1024;
    int b = blockIdx.x;
    const int part = b % PER;
    b /= PER;
    const int tile = b % A.nv;
    b /= A.nv;
    const int h = b % A.H, seq = b / A.H;
    int first, n;
    if (A.plan) {
        const int2 e = A.seqs[seq];
        first = e.x;
        n = e.y;
    } else {
        first = seq * A.per_seq;
        n = A.per_seq;
    }
    if (n <= 1) return;                          // the walk reads h0 itself
    const int frag = part * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    f4 run = load_h0(A, seq, h, tile, frag / (DA / 16), frag % (DA / 16), lane);
    const float f = power(log2_decay(A, h), A.seg_len);
    float* p = A.states + state_at(A, first, h, tile, DA) + (frag * 64 + lane) * 4;
    const int64_t step = state_at(A, 1, 0, 0, DA);
    for (int i = 0; i < n; ++i) {
        f4* q = reinterpret_cast<f4*>(p + i * step);
        f4 own = {0, 0, 0, 0};
        if (i + 1 < n) own = *q;
        *q = run;
        run = run * f + own;
    }
}

// ----------------------------------------------------------------- walk ----
// TO: type of the output (fp32 where several heads' gradients are still to be added up).
template <typename T, typename TO, int DA, bool VEC>
__global__ void __launch_bounds__(kThreads) k_la_out(LaArgs A) {
    using KT = Tile<T, DA, VEC>;
    using VT = Tile<T, kV, VEC>;
    constexpr int SS = KT::STRIDE;               // state copy [value column][row]
    constexpr int NK = DA / Frag<T>::K;
    __shared__ __attribute__((aligned(16))) T kt[kC * KT::STRIDE];
    __shared__ __attribute__((aligned(16))) T vt[kC * VT::STRIDE];
    __shared__ __attribute__((aligned(16))) T st[kV * SS];
    __shared__ __attribute__((aligned(16))) float wt[kC];
    const Unit un = unit_of(A);
    const Seg g = segment(A, un.seg);
    if (g.seq < 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, gr = lane >> 4;
    const float l2 = log2_decay(A, un.h);
    const int64_t as = A.reversed ? -A.a_ts : A.a_ts, bs = A.reversed ? -A.b_ts : A.b_ts, cs = A.reversed ? -A.c_ts : A.c_ts;
    const T* ap = rows_of<T>(A.a, A, g, g.p0, A.a_ts, (un.h / A.a_rep) * A.Da);
    const T* kp = rows_of<T>(A.b, A, g, g.p0, A.b_ts, (un.h / A.b_rep) * A.Da);
    const T* vp = rows_of<T>(A.c, A, g, g.p0, A.c_ts, (un.h / A.c_rep) * A.Dv + un.tile * kV);
    const int64_t os = A.reversed ? -A.o_ts : A.o_ts;
    TO* op = const_cast<TO*>(rows_of<TO>(A.o, A, g, g.p0, A.o_ts, un.h * A.Dv + un.tile * kV));
    const int vw = A.Dv - un.tile * kV;

    f4 S[DA / 16];
    if (g.only) {
#pragma unroll
        for (int i = 0; i < DA / 16; ++i) S[i] = load_h0(A, g.seq, un.h, un.tile, wave, i, lane);
    } else {
        const float* in = A.states + state_at(A, g.state, un.h, un.tile, DA);
#pragma unroll
        for (int i = 0; i < DA / 16; ++i)
            S[i] = *reinterpret_cast<const f4*>(in + ((wave * (DA / 16) + i) * 64 + lane) * 4);
    }
    const int64_t hrow = g.last && A.h_out ? state_row(A, g.seq) : -1;

    const int qi = 16 * wave + m;                // this lane's query position in the chunk
    const float carry = power(l2, kC), at_q = A.s_carry * power(l2, qi + A.shift);
    float dec[4][4];                             // s_in lambda^{i - j}, j = 16 t + 4 gr + r
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = qi - (16 * t + 4 * gr + r);
            dec[t][r] = d >= 0 ? A.s_in * power(l2, d) : 0.0f;
        }
    fill_weights(wt, l2, min(kC, g.n), A.shift, A.s_up);

    KT k;
    VT v;
    u4 q[NK], qn[NK];
    auto load_q = [&](int c0) {
#pragma unroll
        for (int s = 0; s < NK; ++s) {
            const int c = Frag<T>::K * s + Frag<T>::VE * gr;
            qn[s] = load_row<T, VEC>(ap + (c0 + qi) * as + c, c0 + qi < g.n ? A.Da - c : 0);
        }
    };
    if (g.n > 0) {
        k.load(kp, bs, min(kC, g.n), A.Da);
        v.load(vp, cs, min(kC, g.n), vw);
        load_q(0);
    }
    for (int c0 = 0; c0 < g.n; c0 += kC) {
        const int n = min(kC, g.n - c0);
        const bool more = c0 + kC < g.n;
        __syncthreads();                         // the last chunk's reads of the tiles are over
        k.store(kt);
        v.store(vt);
        if (n < kC && c0 > 0) fill_weights(wt, l2, n, A.shift, A.s_up);
#pragma unroll
        for (int i = 0; i < DA / 16; ++i) {      // S^T for this chunk's product
            T* p = st + (16 * wave + m) * SS + 16 * i + 4 * gr;
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<u2*>(p) = u2{pack_bf16(S[i][0], S[i][1]), pack_bf16(S[i][2], S[i][3])};
            } else {
                *reinterpret_cast<f4*>(p) = S[i];
            }
        }
#pragma unroll
        for (int s = 0; s < NK; ++s) q[s] = qn[s];
        __syncthreads();
        if (more) {
            k.load(kp + (c0 + kC) * bs, bs, min(kC, g.n - c0 - kC), A.Da);
            v.load(vp + (c0 + kC) * cs, cs, min(kC, g.n - c0 - kC), vw);
            load_q(c0 + kC);
        }

        // carried part: O^T = S^T Q^T, then lambda^{i + shift} for the lane's token.  Value
        // columns are dealt to accumulators so that a lane ends with 16 neighbours: row
        // 4 g' + r of accumulator tv is column 16 g' + 4 tv + r.
        f4 o[4];
#pragma unroll
        for (int tv = 0; tv < 4; ++tv) {
            o[tv] = f4{0, 0, 0, 0};
            const T* sp = st + (16 * (m >> 2) + 4 * tv + (m & 3)) * SS + Frag<T>::VE * gr;
#pragma unroll
            for (int s = 0; s < NK; ++s)
                o[tv] = Frag<T>::mma(*reinterpret_cast<const u4*>(sp + Frag<T>::K * s), q[s], o[tv]);
            o[tv] *= at_q;
        }
        // masked scores P^T = K Q^T, rows j, column i: what a lane holds is the operand of
        // the product with V as it stands, tokens in the same order on both sides.
        u4 p[sizeof(T) == 2 ? 2 : 4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f4 x = {0, 0, 0, 0};
            if (t <= wave) {
                const T* kr = kt + (16 * t + m) * KT::STRIDE + Frag<T>::VE * gr;
#pragma unroll
                for (int s = 0; s < NK; ++s) x = Frag<T>::mma(*reinterpret_cast<const u4*>(kr + Frag<T>::K * s), q[s], x);
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = 16 * t + 4 * gr + r <= qi ? x[r] * dec[t][r] : 0.0f;
            }
            if constexpr (sizeof(T) == 2) {
                p[t >> 1][2 * (t & 1)] = pack_bf16(x[0], x[1]);
                p[t >> 1][2 * (t & 1) + 1] = pack_bf16(x[2], x[3]);
            } else {
                p[t] = __builtin_bit_cast(u4, x);
            }
        }
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (2 * s > wave) continue;
                const bf16* vr = vt + (32 * s + 4 * gr + (m >> 2)) * VT::STRIDE + 16 * (m & 3);
#pragma unroll
                for (int tv = 0; tv < 4; ++tv) {
                    const u2 v0 = tr4(vr + 4 * tv), v1 = tr4(vr + 16 * VT::STRIDE + 4 * tv);
                    o[tv] = Frag<T>::mma(u4{v0[0], v0[1], v1[0], v1[1]}, p[s], o[tv]);
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (t > wave) continue;
                const float* vr = vt + (16 * t + 4 * gr) * VT::STRIDE + 16 * (m >> 2) + (m & 3);
#pragma unroll
                for (int tv = 0; tv < 4; ++tv) {
                    u4 a;
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = __float_as_uint(vr[e * VT::STRIDE + 4 * tv]);
                    o[tv] = Frag<T>::mma(a, p[t], o[tv]);
                }
            }
        }
        if (qi < n) {
            TO* row = op + (c0 + qi) * os + 16 * gr;
            if constexpr (VEC) {
                if (16 * gr < vw) {
                    if constexpr (sizeof(TO) == 2) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (16 * gr + 8 * e < vw)
                                *reinterpret_cast<u4*>(row + 8 * e) =
                                    u4{pack_bf16(o[2 * e][0], o[2 * e][1]), pack_bf16(o[2 * e][2], o[2 * e][3]),
                                       pack_bf16(o[2 * e + 1][0], o[2 * e + 1][1]), pack_bf16(o[2 * e + 1][2], o[2 * e + 1][3])};
                    } else {
#pragma unroll
                        for (int tv = 0; tv < 4; ++tv)
                            if (16 * gr + 4 * tv < vw) *reinterpret_cast<f4*>(row + 4 * tv) = o[tv];
                    }
                }
            } else {
#pragma unroll
                for (int tv = 0; tv < 4; ++tv)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * gr + 4 * tv + r < vw) store_out(row + 4 * tv + r, o[tv][r]);
            }
        }
        if (more || hrow >= 0) {
            const float f = n == kC ? carry : power(l2, n);
#pragma unroll
            for (int i = 0; i < DA / 16; ++i) S[i] *= f;
            update_state<T, DA>(S, kt, vt, wt, wave, lane);
        }
    }
    if (hrow >= 0) {
        float* p = A.h_out + (hrow * A.H + un.h) * (int64_t)A.Da * A.Dv;
        const int col = un.tile * kV + 16 * wave + m;
#pragma unroll
        for (int i = 0; i < DA / 16; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * gr + r;
                if (col < A.Dv && row < A.Da) p[(int64_t)row * A.Dv + col] = S[i][r];
            }
    }
}

// Gradients of keys or values shared by `rep` heads: (T, H, D) fp32 added up to (T, H / rep, D).
template <typename T>
__global__ void __launch_bounds__(256) k_la_fold(const float* __restrict__ in, T* __restrict__ out, int64_t n, int G, int rep, int D) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t tg = i / D;
        const int d = (int)(i - tg * D);
        const float* p = in + tg * rep * D + d;
        float s = 0.0f;
        for (int k = 0; k < rep; ++k) s += p[(int64_t)k * D];
        store_out(out + i, s);
    }
}

// Gradient rows of tokens in no sequence (in front of the first, behind the last): zero.
template <typename T>
__global__ void __launch_bounds__(256) k_la_clear(const int32_t* cu, int n_seq, int64_t T_, T* dq, int64_t nq, T* dk, int64_t nk, T* dv, int64_t nv) {
    const int64_t b = min((int64_t)max(cu[0], 0), T_), e = min(max((int64_t)cu[n_seq], b), T_);
    const int64_t all = T_ - (e - b);
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    auto clear = [&](T* p, int64_t per) {
        for (int64_t i = i0; i < all * per; i += step) p[i < b * per ? i : i + (e - b) * per] = (T)0;
    };
    clear(dq, nq);
    clear(dk, nk);
    clear(dv, nv);
}

// ----------------------------------------------------------------- step ----
struct StepArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* log_decay;
    const int32_t* slots;
    const float* h_in;
    float* h_out;
    void* o;
    int64_t n, n_slots, q_ts, k_ts, v_ts;
    int H, rep, Dk, Dv, cols, tiles;     // value columns of a workgroup, workgroups of a row's head
    float scale;
};

// A workgroup owns CW = 4 LN value columns of one (row, head): LN lanes side by side hold
// four columns each, the 256 / LN rows of lanes share out the state's rows, and their parts
// of o are added up in LDS.  All its state reads are under way before the first is used.
template <typename T, int LN, bool VEC>
__global__ void __launch_bounds__(256) k_la_step(StepArgs A) {
    constexpr int RG = 256 / LN;                 // state rows at a time
    constexpr int NR = (kMaxDim + RG - 1) / RG;
    constexpr int CPL = VEC ? 4 : 1;             // columns of a lane
    __shared__ float qs[kMaxDim], ks[kMaxDim];
    __shared__ float red[RG][LN * CPL + 1];
    int b = blockIdx.x;
    const int tile = b % A.tiles;
    b /= A.tiles;
    const int h = b % A.H;
    const int64_t row = b / A.H;
    const int ln = threadIdx.x % LN, rg = threadIdx.x / LN;
    const int col = (tile * LN + ln) * CPL;
    int64_t slot = row;
    if (A.slots) {
        slot = A.slots[row];
        if (slot < 0 || slot >= A.n_slots) slot = -1;
    }
    const int64_t at = (slot * A.H + h) * (int64_t)A.Dk * A.Dv + col;
    const bool in = col < A.Dv;
    float s[NR][CPL];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = i * RG + rg;
#pragma unroll
        for (int c = 0; c < CPL; ++c) s[i][c] = 0.0f;
        if (A.h_in && slot >= 0 && in && r < A.Dk) {
            const float* p = A.h_in + at + (int64_t)r * A.Dv;
            if constexpr (VEC) {
                const f4 t = *reinterpret_cast<const f4*>(p);
#pragma unroll
                for (int c = 0; c < 4; ++c) s[i][c] = t[c];
            } else {
                s[i][0] = *p;
            }
        }
    }
    const int hk = h / A.rep;
    for (int i = threadIdx.x; i < A.Dk; i += 256) {
        qs[i] = to_f32(((const T*)A.q)[row * A.q_ts + (int64_t)h * A.Dk + i]);
        ks[i] = to_f32(((const T*)A.k)[row * A.k_ts + (int64_t)hk * A.Dk + i]);
    }
    float v[CPL], o[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        o[c] = 0.0f;
        v[c] = in ? to_f32(((const T*)A.v)[row * A.v_ts + (int64_t)hk * A.Dv + col + c]) : 0.0f;
    }
    const float l2 = A.log_decay[h] * kLog2e, lam = exp2_fast(l2);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = i * RG + rg;
        if (r < A.Dk) {
            const float k = ks[r], q = qs[r];
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                s[i][c] = fmaf(lam, s[i][c], k * v[c]);
                o[c] = fmaf(q, s[i][c], o[c]);
            }
            if (A.h_out && slot >= 0 && in) {
                float* p = A.h_out + at + (int64_t)r * A.Dv;
                if constexpr (VEC) *reinterpret_cast<f4*>(p) = f4{s[i][0], s[i][1], s[i][2], s[i][3]};
                else *p = s[i][0];
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) red[rg][ln * CPL + c] = o[c];
    __syncthreads();
    if (threadIdx.x < LN * CPL && tile * LN * CPL + (int)threadIdx.x < A.Dv) {
        float t = 0.0f;
#pragma unroll 8
        for (int i = 0; i < RG; ++i) t += red[i][threadIdx.x];
        store_out((T*)A.o + (row * A.H + h) * A.Dv + tile * LN * CPL + threadIdx.x, t * A.scale);
    }
}

// ------------------------------------------------------------------ host ----
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }
inline bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Segment length: as many segments as it takes to put about four workgroups on each
// compute unit, no shorter than 256 tokens (a segment costs its state's trip through
// memory).
int plan_seg_len(int64_t n_seq, int64_t T, int64_t H, int64_t Dv) {
    const int64_t units = H * ((Dv + kV - 1) / kV);
    const int64_t want = (4 * (int64_t)device_cu_count() + units - 1) / units;
    int64_t len = (T + want - 1) / want;
    len = (len + kC - 1) / kC * kC;
    if (len < 256) len = 256;
    if (len > 1 << 20) len = 1 << 20;
    return (int)len;
}

struct Plan {
    int seg_len, nseg, per_seq;
    bool table;         // packed sequences of more than one segment
    size_t states, seqs_at, table_bytes;
    int da;
};

Plan make_plan(int64_t n_seq, int64_t T, int64_t H, int64_t Da, int64_t Dv, bool packed) {
    Plan p;
    p.seg_len = plan_seg_len(n_seq, T, H, Dv);
    p.da = Da <= 64 ? 64 : 128;
    const int64_t L = T / n_seq;
    p.table = packed && T > p.seg_len;
    p.per_seq = packed ? 0 : (int)((L + p.seg_len - 1) / p.seg_len);
    if (!packed && p.per_seq < 1) p.per_seq = 1;
    const int64_t nseg = packed ? (p.table ? T / p.seg_len + n_seq : n_seq) : n_seq * p.per_seq;
    p.nseg = (int)nseg;
    const bool states = packed ? p.table : p.per_seq > 1;
    const int64_t nst = packed ? std::min(nseg, 2 * T / p.seg_len) : nseg;
    p.states = states ? (size_t)nst * H * ((Dv + kV - 1) / kV) * p.da * kV * 4 : 0;
    p.seqs_at = up256((size_t)nseg * sizeof(PlanEntry));
    p.table_bytes = p.table ? p.seqs_at + up256((size_t)n_seq * 8) : 0;
    return p;
}

bool sizes_ok(int64_t n_seq, int64_t T, int64_t H, int64_t G, int64_t Dk, int64_t Dv) {
    if (n_seq < 0 || T < 0 || H < 1 || G < 1 || H % G || H > 4096 || Dk < 1 || Dk > kMaxDim || Dv < 1 || Dv > kMaxDim) return false;
    if (n_seq > 1 << 20 || T >= (int64_t)1 << 31) return false;
    return true;
}

template <typename T, typename TO, int DA, bool VEC>
mb_status run_passes(const LaArgs& A, const Plan& p, hipStream_t s) {
    const int64_t units = (int64_t)p.nseg * A.H * A.nv;
    if (p.states) {
        hipLaunchKernelGGL((k_la_state<T, DA, VEC>), dim3((unsigned)units), dim3(kThreads), 0, s, A);
        mb_status st = check_launch();
        if (st != MB_OK) return st;
        hipLaunchKernelGGL(k_la_carry<DA>, dim3((unsigned)((int64_t)A.n_seq * A.H * A.nv * (DA * kV / 1024))), dim3(256), 0, s, A);
        st = check_launch();
        if (st != MB_OK) return st;
    }
    hipLaunchKernelGGL((k_la_out<T, TO, DA, VEC>), dim3((unsigned)units), dim3(kThreads), 0, s, A);
    return check_launch();
}

template <typename T, typename TO>
mb_status run_typed(LaArgs A, const Plan& p, hipStream_t s) {
    constexpr int VE = Frag<T>::VE, VO = 16 / sizeof(TO);
    const bool vec = A.Da % VE == 0 && A.Dv % VE == 0 && A.Dv % VO == 0 && A.a_ts % VE == 0 && A.b_ts % VE == 0 && A.c_ts % VE == 0 &&
                     al16(A.a) && al16(A.b) && al16(A.c) && al16(A.o);
    if (p.da == 64) return vec ? run_passes<T, TO, 64, true>(A, p, s) : run_passes<T, TO, 64, false>(A, p, s);
    return vec ? run_passes<T, TO, 128, true>(A, p, s) : run_passes<T, TO, 128, false>(A, p, s);
}

// One run of the chunked form; `out_f32` where heads' gradients are added up afterwards.
mb_status run(LaArgs A, const Plan& p, mb_dtype dtype, bool out_f32, char* ws, hipStream_t s) {
    A.nv = (A.Dv + kV - 1) / kV;
    A.seg_len = p.seg_len;
    A.nseg = p.nseg;
    A.per_seq = p.per_seq;
    A.plan = p.table ? (const PlanEntry*)ws : nullptr;
    A.seqs = p.table ? (const int2*)(ws + p.seqs_at) : nullptr;
    A.states = p.states ? (float*)(ws + p.table_bytes) : nullptr;
    if (dtype == MB_F32) return run_typed<float, float>(A, p, s);
    return out_f32 ? run_typed<bf16, float>(A, p, s) : run_typed<bf16, bf16>(A, p, s);
}

mb_status launch_plan(const LaArgs& A, const Plan& p, char* ws, hipStream_t s) {
    if (!p.table) return MB_OK;
    hipLaunchKernelGGL(k_la_plan, dim3(1), dim3(256), 0, s, A.cu, A.n_seq, A.T, p.seg_len, p.nseg, (PlanEntry*)ws,
                       (int2*)(ws + p.seqs_at));
    return check_launch();
}

struct BwdPlan {
    Plan q, k, v;          // the three runs
    size_t states, fold;
    size_t total;
};

BwdPlan bwd_plan(int64_t n_seq, int64_t T, int64_t H, int64_t G, int64_t Dk, int64_t Dv, bool packed) {
    BwdPlan b;
    b.q = make_plan(n_seq, T, H, Dv, Dk, packed);
    b.k = b.q;
    b.v = make_plan(n_seq, T, H, Dk, Dv, packed);
    auto most = [](size_t x, size_t y) { return x > y ? x : y; };
    b.states = most(b.q.table_bytes + b.q.states, b.v.table_bytes + b.v.states);
    b.states = up256(b.states);
    b.fold = G < H ? up256((size_t)T * H * most(Dk, Dv) * 4) : 0;
    b.total = b.states + b.fold;
    return b;
}

// Bytes that `tokens` rows of `stride` elements with `row` in use span.
size_t span_of(int64_t tokens, int64_t stride, int64_t row, size_t es) {
    return tokens > 0 ? ((size_t)(tokens - 1) * stride + row) * es : 0;
}

}  // namespace

size_t linear_attn_workspace(int64_t n_seq, int64_t T, int64_t H, int64_t G, int64_t Dk, int64_t Dv) {
    if (!sizes_ok(n_seq, T, H, G, Dk, Dv) || n_seq == 0) return 0;
    // the larger of packed and equal lengths: the size does not depend on how the call is made
    const Plan a = make_plan(n_seq, T, H, Dk, Dv, true), b = make_plan(n_seq, T, H, Dk, Dv, false);
    const size_t x = a.table_bytes + a.states, y = T % n_seq ? 0 : b.states;
    return x > y ? x : y;
}

size_t linear_attn_bwd_workspace(int64_t n_seq, int64_t T, int64_t H, int64_t G, int64_t Dk, int64_t Dv) {
    if (!sizes_ok(n_seq, T, H, G, Dk, Dv) || n_seq == 0) return 0;
    const size_t x = bwd_plan(n_seq, T, H, G, Dk, Dv, true).total, y = T % n_seq ? 0 : bwd_plan(n_seq, T, H, G, Dk, Dv, false).total;
    return x > y ? x : y;
}

}  // namespace mb

extern "C" mb_status mb_linear_attn(const void* q, const void* k, const void* v, const float* log_decay,
                                    const int32_t* cu_seqlens, const float* h0, const uint8_t* has_h0,
                                    const int32_t* slots, void* o, float* h_out, int64_t n_seq, int64_t T, int64_t H,
                                    int64_t G, int64_t Dk, int64_t Dv, int64_t n_slots, int64_t q_stride,
                                    int64_t k_stride, int64_t v_stride, float scale, mb_dtype dtype, void* ws,
                                    size_t ws_bytes, hipStream_t stream) {
    using namespace mb;
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (!sizes_ok(n_seq, T, H, G, Dk, Dv)) return MB_ERR_SHAPE;
    if (q_stride < H * Dk || k_stride < G * Dk || v_stride < G * Dv) return MB_ERR_SHAPE;
    if (slots ? n_slots < 1 : n_slots != 0) return MB_ERR_SHAPE;
    if (n_seq == 0) return MB_OK;
    if (!cu_seqlens && T % n_seq) return MB_ERR_SHAPE;
    if (!log_decay || (T > 0 && (!q || !k || !v || !o))) return MB_ERR_NULL;
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)q % es || (uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)o % es || ((uintptr_t)log_decay & 3) ||
        ((uintptr_t)cu_seqlens & 3) || ((uintptr_t)slots & 3) || ((uintptr_t)h0 & 3) || ((uintptr_t)h_out & 3))
        return MB_ERR_ALIGN;
    const Plan p = make_plan(n_seq, T, H, Dk, Dv, cu_seqlens != nullptr);
    const size_t need = p.table_bytes + p.states;
    if ((int64_t)p.nseg * H * ((Dv + kV - 1) / kV) > 0x7fffffff || n_seq * H * 16 > 0x7fffffff) return MB_ERR_SHAPE;
    if (need && (!ws || ws_bytes < need || ((uintptr_t)ws & 255))) return MB_ERR_WORKSPACE;
    const size_t nh = (size_t)(slots ? n_slots : n_seq) * H * Dk * Dv * 4;
    const Span ins[8] = {{q, span_of(T, q_stride, H * Dk, es)}, {k, span_of(T, k_stride, G * Dk, es)}, {v, span_of(T, v_stride, G * Dv, es)},
                         {log_decay, (size_t)H * 4}, {cu_seqlens, (size_t)(n_seq + 1) * 4}, {has_h0, (size_t)n_seq},
                         {slots, (size_t)n_seq * 4}, {h0, nh}};
    const size_t no = (size_t)T * H * Dv * es;
    if (overlaps_any(o, no, ins, 8) || overlaps_any(h_out, nh, ins, h_out == h0 ? 7 : 8) || overlaps(o, no, h_out, nh)) return MB_ERR_ALIAS;
    if (need && (overlaps_any(ws, need, ins, 8) || overlaps(ws, need, o, no) || overlaps(ws, need, h_out, nh))) return MB_ERR_ALIAS;
    const int rep = (int)(H / G);
    LaArgs A{};
    A.a = q; A.b = k; A.c = v; A.o = o;
    A.a_ts = q_stride; A.b_ts = k_stride; A.c_ts = v_stride; A.o_ts = H * Dv;
    A.a_rep = 1; A.b_rep = A.c_rep = rep;
    A.H = (int)H; A.Da = (int)Dk; A.Dv = (int)Dv;
    A.log_decay = log_decay;
    A.s_in = A.s_carry = scale; A.s_up = 1.0f;
    A.shift = 1; A.reversed = 0;
    A.n_seq = (int)n_seq; A.T = T; A.L = T / n_seq;
    A.cu = cu_seqlens;
    A.h0 = h0; A.has_h0 = has_h0; A.slots = slots; A.n_slots = n_slots;
    A.h_out = h_out;
    mb_status st = launch_plan(A, p, (char*)ws, stream);
    return st != MB_OK ? st : run(A, p, dtype, false, (char*)ws, stream);
}

extern "C" mb_status mb_linear_attn_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                                        const int32_t* cu_seqlens, const float* h0, const void* d_o,
                                        const float* dh_out, void* dq, void* dk, void* dv, float* dh0, int64_t n_seq,
                                        int64_t T, int64_t H, int64_t G, int64_t Dk, int64_t Dv, int64_t q_stride,
                                        int64_t k_stride, int64_t v_stride, float scale, mb_dtype dtype, void* ws,
                                        size_t ws_bytes, hipStream_t stream) {
    using namespace mb;
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (!sizes_ok(n_seq, T, H, G, Dk, Dv)) return MB_ERR_SHAPE;
    if (q_stride < H * Dk || k_stride < G * Dk || v_stride < G * Dv) return MB_ERR_SHAPE;
    if (n_seq == 0) return MB_OK;
    if (!cu_seqlens && T % n_seq) return MB_ERR_SHAPE;
    if (!log_decay || (T > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv))) return MB_ERR_NULL;
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)q % es || (uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)d_o % es || (uintptr_t)dq % es ||
        (uintptr_t)dk % es || (uintptr_t)dv % es || ((uintptr_t)log_decay & 3) || ((uintptr_t)cu_seqlens & 3) ||
        ((uintptr_t)h0 & 3) || ((uintptr_t)dh_out & 3) || ((uintptr_t)dh0 & 3))
        return MB_ERR_ALIGN;
    const BwdPlan bp = bwd_plan(n_seq, T, H, G, Dk, Dv, cu_seqlens != nullptr);
    const int64_t tiles = (std::max(Dk, Dv) + kV - 1) / kV;
    if (std::max(bp.q.nseg, bp.v.nseg) * H * tiles > 0x7fffffff || n_seq * H * 16 > 0x7fffffff) return MB_ERR_SHAPE;
    if (bp.total && (!ws || ws_bytes < bp.total || ((uintptr_t)ws & 255))) return MB_ERR_WORKSPACE;
    const size_t nh = (size_t)n_seq * H * Dk * Dv * 4;
    const Span ins[8] = {{q, span_of(T, q_stride, H * Dk, es)}, {k, span_of(T, k_stride, G * Dk, es)}, {v, span_of(T, v_stride, G * Dv, es)},
                         {log_decay, (size_t)H * 4}, {cu_seqlens, (size_t)(n_seq + 1) * 4}, {h0, nh},
                         {d_o, (size_t)T * H * Dv * es}, {dh_out, nh}};
    const Span outs[5] = {{dq, (size_t)T * H * Dk * es}, {dk, (size_t)T * G * Dk * es}, {dv, (size_t)T * G * Dv * es}, {dh0, nh},
                          {bp.total ? ws : nullptr, bp.total}};
    for (int i = 0; i < 5; ++i) {
        if (overlaps_any(outs[i].p, outs[i].bytes, ins, 8)) return MB_ERR_ALIAS;
        if (overlaps_any(outs[i].p, outs[i].bytes, outs, i)) return MB_ERR_ALIAS;
    }
    const int rep = (int)(H / G);
    char* w = (char*)ws;
    float* fold = (float*)(w + bp.states);
    LaArgs A{};
    A.H = (int)H;
    A.log_decay = log_decay;
    A.n_seq = (int)n_seq; A.T = T; A.L = T / n_seq;
    A.cu = cu_seqlens;
    mb_status st;
    auto add_up = [&](void* out, int64_t D) -> mb_status {
        const int64_t n = T * G * D;
        if (rep == 1 || n == 0) return MB_OK;
        const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 8192);
        if (dtype == MB_F32) hipLaunchKernelGGL(k_la_fold<float>, dim3(blocks), dim3(256), 0, stream, fold, (float*)out, n, (int)G, rep, (int)D);
        else hipLaunchKernelGGL(k_la_fold<bf16>, dim3(blocks), dim3(256), 0, stream, fold, (bf16*)out, n, (int)G, rep, (int)D);
        return check_launch();
    };
    // dq: queries do, keys v, values k, forward; the state is S^T.
    LaArgs Q = A;
    Q.a = d_o; Q.b = v; Q.c = k; Q.o = dq;
    Q.a_ts = H * Dv; Q.b_ts = v_stride; Q.c_ts = k_stride; Q.o_ts = H * Dk;
    Q.a_rep = 1; Q.b_rep = Q.c_rep = rep;
    Q.Da = (int)Dv; Q.Dv = (int)Dk;
    Q.s_in = Q.s_carry = scale; Q.s_up = 1.0f;
    Q.shift = 1; Q.reversed = 0;
    Q.h0 = h0; Q.transposed = 1;
    if ((st = launch_plan(Q, bp.q, w, stream)) != MB_OK || (st = run(Q, bp.q, dtype, false, w, stream)) != MB_OK) return st;
    // dk: queries v, keys do, values q, reversed; the state is R^T and holds the scale.
    LaArgs K = A;
    K.a = v; K.b = d_o; K.c = q; K.o = rep > 1 ? (void*)fold : dk;
    K.a_ts = v_stride; K.b_ts = H * Dv; K.c_ts = q_stride; K.o_ts = H * Dk;
    K.a_rep = rep; K.b_rep = K.c_rep = 1;
    K.Da = (int)Dv; K.Dv = (int)Dk;
    K.s_in = K.s_up = scale; K.s_carry = 1.0f;
    K.shift = 0; K.reversed = 1;
    K.h0 = dh_out; K.transposed = 1;
    if ((st = run(K, bp.k, dtype, rep > 1, w, stream)) != MB_OK || (st = add_up(dk, Dk)) != MB_OK) return st;
    // dv: queries k, keys q, values do, reversed; the state is R, its end the gradient of h0.
    LaArgs V = K;
    V.a = k; V.b = q; V.c = d_o; V.o = rep > 1 ? (void*)fold : dv;
    V.a_ts = k_stride; V.b_ts = q_stride; V.c_ts = H * Dv; V.o_ts = H * Dv;
    V.Da = (int)Dk; V.Dv = (int)Dv;
    V.transposed = 0;
    V.h_out = dh0;
    if ((st = launch_plan(V, bp.v, w, stream)) != MB_OK || (st = run(V, bp.v, dtype, rep > 1, w, stream)) != MB_OK ||
        (st = add_up(dv, Dv)) != MB_OK)
        return st;
    if (cu_seqlens && T > 0) {
        if (dtype == MB_F32)
            hipLaunchKernelGGL(k_la_clear<float>, dim3(256), dim3(256), 0, stream, cu_seqlens, (int)n_seq, T, (float*)dq, H * Dk,
                               (float*)dk, G * Dk, (float*)dv, G * Dv);
        else
            hipLaunchKernelGGL(k_la_clear<bf16>, dim3(256), dim3(256), 0, stream, cu_seqlens, (int)n_seq, T, (bf16*)dq, H * Dk,
                               (bf16*)dk, G * Dk, (bf16*)dv, G * Dv);
        return check_launch();
    }
    return MB_OK;
}

extern "C" mb_status mb_linear_attn_step(const void* q, const void* k, const void* v, const float* log_decay,
                                         const int32_t* slots, const float* h_in, float* h_out, void* o, int64_t n,
                                         int64_t H, int64_t G, int64_t Dk, int64_t Dv, int64_t n_slots,
                                         int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                                         mb_dtype dtype, hipStream_t stream) {
    using namespace mb;
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (!sizes_ok(n, 0, H, G, Dk, Dv)) return MB_ERR_SHAPE;
    if (q_stride < H * Dk || k_stride < G * Dk || v_stride < G * Dv) return MB_ERR_SHAPE;
    if (slots ? n_slots < 1 : n_slots != 0) return MB_ERR_SHAPE;
    if (n == 0) return MB_OK;
    if (!q || !k || !v || !log_decay || !o || !h_out) return MB_ERR_NULL;
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)q % es || (uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)o % es || ((uintptr_t)log_decay & 3) ||
        ((uintptr_t)slots & 3) || ((uintptr_t)h_in & 3) || ((uintptr_t)h_out & 3))
        return MB_ERR_ALIGN;
    const size_t nh = (size_t)(slots ? n_slots : n) * H * Dk * Dv * 4, no = (size_t)n * H * Dv * es;
    const Span ins[6] = {{q, span_of(n, q_stride, H * Dk, es)}, {k, span_of(n, k_stride, G * Dk, es)}, {v, span_of(n, v_stride, G * Dv, es)},
                         {log_decay, (size_t)H * 4}, {slots, (size_t)n * 4}, {h_in, nh}};
    if (overlaps_any(o, no, ins, 6) || overlaps_any(h_out, nh, ins, h_out == h_in ? 5 : 6) || overlaps(o, no, h_out, nh)) return MB_ERR_ALIAS;
    const bool vec = Dv % 4 == 0 && al16(h_in) && al16(h_out);
    StepArgs A{q, k, v, log_decay, slots, h_in, h_out, o, n, n_slots, q_stride, k_stride, v_stride,
               (int)H, (int)(H / G), (int)Dk, (int)Dv, 0, 0, scale};
    // Few rows: narrow column tiles, so that the one token's states are read by more compute
    // units; many rows: a tile as wide as a row of the state.
    const bool few = n * H < 2 * device_cu_count();
    const int ln = few ? 4 : 16, cpl = vec ? 4 : 1;
    A.cols = ln * cpl;
    A.tiles = (int)((Dv + A.cols - 1) / A.cols);
    const int64_t grid = n * H * A.tiles;
    if (grid > 0x7fffffff) return MB_ERR_SHAPE;
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), 0, stream, A); };
    if (dtype == MB_F32) {
        if (vec) few ? go(k_la_step<float, 4, true>) : go(k_la_step<float, 16, true>);
        else few ? go(k_la_step<float, 4, false>) : go(k_la_step<float, 16, false>);
    } else {
        if (vec) few ? go(k_la_step<bf16, 4, true>) : go(k_la_step<bf16, 16, true>);
        else few ? go(k_la_step<bf16, 4, false>) : go(k_la_step<bf16, 16, false>);
    }
    return check_launch();
}
