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
// each segment's own end state (the first one's from h0), and k_la_out walks the chunks of
// every segment from the state that enters it, composed from the end states in front of it: by
// the walk itself where a sequence has few segments, by k_la_carry beforehand where it has many.
// A sequence of n segments has n places for states: end states 0 to n - 2, and in the last, which has
// no end state to hand on, a copy of h0 (h_out may be h0, and the last segment may write it
// before the first one reads it).
//
// bf16 tensors lose nothing beside the rounding of their outputs: what is computed and has to be an operand of a bf16 product
// once more is cut into bf16 pieces, the masked, decayed scores and the state's copy into two (2^-16 of a term is left), the
// weighted values of the state's update into three.  With one piece of the first two the outputs were off from 64 bits by
// 2.3e-3 (root mean square, relative), so by the 1.7e-3 of their own rounding, for twice the products with them: packed prompt
// 85.1 -> 83.1 us and backward 189 -> 191, both with the registers' use mended (forget_lane), seven short prompts 16.5 -> 17.5.
// An infinity in one piece leaves NaN in the next.
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
// Up to these the walk composes its entering state itself.  Measured at 4, 8 and 16: three sequences of 5461 tokens
// 90 us at 8, 87 at 16; fp32 of 2 x 4095 tokens (16 segments each) 67.7 and 65.7; backward 194 us at 4, else 188.
constexpr int kFewSegments = 16;
constexpr int kWalkThreads = 512;
// Packed sequences that every workgroup looks through itself: one look of a wave.  More have their segments in a table, which
// costs a launch and its own looks once.  Looked through and table, 16384 tokens of 16 heads of 128 x 64, bf16: 32 sequences 60.1 and
// 61.4 us (backward 145.0, 143.9), 64 68.0 and 66.7 (161, 153), 128 87 and 79 (211, 180), 256 143 and 111 (344, 242); of 2 heads 9
// sequences 32.4 and 33.4 (71, 74), 64 24.2 and 24.5 (48.7, 50.1), 128 22.1 and 23.2 (46.5, 45.3), 256 27.3 and 25.3 (63, 52).
constexpr int kLookThrough = 64;

// A segment of a sequence.  A sequence of L tokens is cut into ceil(L / target) segments (one if it
// is empty) of equal length, rounded up to whole chunks.
struct __attribute__((aligned(16))) Seg {
    int seq;             // < 0: nothing to do
    int first, len;      // the sequence's first token and length
    int p0, n;           // the segment's first position in walking order, its tokens
    int idx, count;      // its place among the sequence's segments
    int state;           // where its entering state lies
};
__device__ __forceinline__ bool is_last(const Seg& g) { return g.idx + 1 == g.count; }

struct LaArgs {
    const void* a;              // query role, key role, value role, output
    const void* b;
    const void* c;
    void* o;
    int64_t a_ts, b_ts, c_ts, o_ts;   // elements between tokens
    int a_rep, b_rep, c_rep;          // heads that share one row of it
    int H, Da, Dv, nv;                // heads, width of a and b, width of c and o, column tiles of c
    int share;                        // heads side by side that read the same rows of b or c
    const float* log_decay;
    float s_in, s_carry, s_up;        // factors: masked scores, carried state's product, state update
    int shift;                        // a token's own power of lambda on the carried state: 1, reversed 0
    int reversed;
    int n_seq;
    int T, L;                         // tokens in all; of a sequence when they are equal
    int target, seg0, nseg;           // longest segment; segments seg0 to nseg - 1 are launched
    int per_seq;                      // segments of a sequence when lengths are equal, else 0
    int single;                       // packed sequences of one segment each, at most kOneSegment tokens in all
    const int32_t* cu;
    const Seg* plan;                  // segments of many packed sequences; NULL: worked out by every workgroup
    const int2* seqs;                 // (first state, segments) of a sequence, with plan
    float* states;                    // per (state, head, column tile): a state in fragment order
    const float* h0;
    const uint8_t* has_h0;
    const int32_t* slots;
    int64_t n_slots;
    int transposed;                   // h0 is (H, Dv, Da)
    float* h_out;
};

__device__ __forceinline__ int segments_of(int len, int target) { return max((int)(((int64_t)len + target - 1) / target), 1); }

// Tokens of each of a sequence's `count` segments but the last: even parts in whole chunks.  A length and
// the number of its segments may add up to 2^31 and more: unsigned.
__device__ __forceinline__ int segment_tokens(int len, int count) {
    const uint32_t even = ((uint32_t)len + (uint32_t)count - 1) / (uint32_t)count;
    return (int)((even + kC - 1) / kC * kC);
}

// Fills in p0 and n from idx and count.
__device__ __forceinline__ void place(Seg& g) {
    const int each = segment_tokens(g.len, g.count);
    g.p0 = g.idx * each;
    g.n = max(min(each, g.len - g.p0), 0);
}

// 64 packed sequences, one a lane: their tokens, segments, and the sums of segments and states in
// front of them.  Offsets that decrease or leave [0, T] are taken as empty sequences, so that
// the sequences' lengths never add up to more than T, the segments to T / target + n_seq, and those of
// sequences of several (each at most 2 len / target) to 2 T / target.
struct Lane64 {
    int first, len, count, at, state;
    int reach, segs, states;       // running over the groups of 64: largest offset, segments, states

    __device__ __forceinline__ void read(const LaArgs& A, int s0, int lane) {
        const int s = s0 + lane;
        const bool in = s < A.n_seq;
        const int b = in ? min(max(A.cu[s], 0), A.T) : 0, e = in ? min(max(A.cu[s + 1], 0), A.T) : 0;
        int top = max(reach, max(b, e));
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(top, o);
            if (lane >= o) top = max(top, v);
        }
        const int before = __shfl_up(top, 1);
        first = max(b, lane ? before : reach);
        len = max(e - first, 0);
        count = in ? segments_of(len, A.target) : 0;
        const int own = count > 1 ? count : 0;
        int x = count, y = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(x, o), v = __shfl_up(y, o);
            if (lane >= o) {
                x += u;
                y += v;
            }
        }
        at = segs + x - count;
        state = states + y - own;
        reach = __builtin_amdgcn_readlane(top, 63);
        segs += __builtin_amdgcn_readlane(x, 63);
        states += __builtin_amdgcn_readlane(y, 63);
    }
};

// Segment s of the launch, in every wave (uniform).
__device__ __forceinline__ Seg segment(const LaArgs& A, int s) {
    Seg g;
    if (A.plan) return A.plan[s];
    g.seq = -1;
    if (A.single) {
        // Segment s is sequence s, whatever lies in front of it: one look at its own offsets.
        g.seq = s;
        g.first = min(max(A.cu[s], 0), A.T);
        g.len = max(min(max(A.cu[s + 1], 0), A.T) - g.first, 0);
        g.idx = 0;
        g.count = 1;
        g.state = s;
    } else if (A.cu) {
        const int lane = threadIdx.x & 63;
        Lane64 l;
        l.reach = l.segs = l.states = 0;
        l.read(A, 0, lane);
        if (s >= l.segs) return g;
        const uint64_t hit = __ballot(l.count > 0 && l.at <= s && s < l.at + l.count);
        const int k = __ffsll((unsigned long long)hit) - 1;
        g.seq = k;
        g.first = __builtin_amdgcn_readlane(l.first, k);
        g.len = __builtin_amdgcn_readlane(l.len, k);
        g.count = __builtin_amdgcn_readlane(l.count, k);
        g.idx = s - __builtin_amdgcn_readlane(l.at, k);
        g.state = __builtin_amdgcn_readlane(l.state, k) + g.idx;
    } else {
        g.seq = s / A.per_seq;
        g.idx = s - g.seq * A.per_seq;
        g.first = g.seq * A.L;
        g.len = A.L;
        g.count = A.per_seq;
        g.state = s;
    }
    place(g);
    return g;
}

// First state, segments and segment length of a sequence.
__device__ __forceinline__ void sequence(const LaArgs& A, int seq, int& state, int& count, int& len) {
    if (A.plan) {
        state = A.seqs[seq].x;
        count = A.seqs[seq].y;
        len = min(max(A.cu[seq + 1], 0), A.T) - min(max(A.cu[seq], 0), A.T);
    } else if (A.cu) {
        const int lane = threadIdx.x & 63;
        Lane64 l;
        l.reach = l.segs = l.states = 0;
        l.read(A, 0, lane);
        state = __builtin_amdgcn_readlane(l.state, seq);
        count = __builtin_amdgcn_readlane(l.count, seq);
        len = __builtin_amdgcn_readlane(l.len, seq);
    } else {
        state = seq * A.per_seq;
        count = A.per_seq;
        len = A.L;
    }
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

// A barrier for what waves share through LDS: it waits for this wave's LDS operations alone.  The
// ordinary one would also wait for the loads of the next chunk and for the stores of this one's outputs.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);          // lgkmcnt(0), no other counter
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

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

// 16 bytes of LDS on a 16-byte border.  Said once more, since the compiler loses sight of it and reads fp32 in four pieces.
template <typename T>
__device__ __forceinline__ u4 fragment_at(const T* p) {
    return *reinterpret_cast<const u4*>(__builtin_assume_aligned(p, 16));
}

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

// A chunk's tokens of one tensor as a buffer: base at the lowest row, so that rows behind
// the chunk's tokens (and, reversed, in front of them) lie outside its range and read zero.
struct Window {
    __amdgpu_buffer_rsrc_t r;
    int row0, step;      // byte offsets: of the first row in walking order, and to the next one
    const char* base;    // the same range as r, for vectors at any element's address
    uint32_t bytes;
};

// p: the chunk's first token in walking order; ts: elements between tokens; n: tokens; width: elements of a row in use.
template <typename T>
__device__ __forceinline__ Window window(const T* p, int64_t ts, bool reversed, int n, int width) {
    const int b = (int)(ts * (int64_t)sizeof(T));
    Window w;
    w.row0 = reversed ? (n - 1) * b : 0;
    w.step = reversed ? -b : b;
    const char* base = (const char*)p - (reversed && n > 0 ? w.row0 : 0);
    w.base = base;
    w.bytes = n > 0 ? (n - 1) * b + width * (int)sizeof(T) : 0;
    w.r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)w.bytes, 0x00027000);
    return w;
}

// VE elements from column c of row r; columns at and behind `width` are zero.  Without VEC they may start at any
// element's address, which the memory takes in one access; a row's last vector may be cut short (2 x 8192 tokens, 16 heads
// of 128 x 64, bf16, from an odd address on: element by element 199 us and backward 555, so 102 and 254; aligned 78 and 194).
template <typename T, bool VEC>
__device__ __forceinline__ u4 load_row(const Window& w, int r, int c, int width) {
    const uint32_t off = (uint32_t)(w.row0 + r * w.step + c * (int)sizeof(T));
    u4 v;
    if constexpr (VEC) {
        v = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(w.r, c < width ? off : 0x80000000u, 0, 0));
    } else {
        // Strides hold a row's width: an offset inside the range is in one of its rows.
        constexpr int VE = Frag<T>::VE;
        const int left = off < w.bytes ? width - c : 0;
        v = u4{0, 0, 0, 0};
        if (left >= VE) {
            __builtin_memcpy(&v, w.base + off, 16);
        } else if (left > 0) {
            T part[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) part[e] = e < left ? reinterpret_cast<const T*>(w.base + off)[e] : (T)0;
            __builtin_memcpy(&v, part, 16);
        }
    }
    return v;
}

// Where (row, col) of an LDS tile lies, in elements.  bf16: 16-byte pieces of a row change places by
// an exclusive-or with bits of the row, so that the 16 rows of a fragment read, the 8 rows of a
// transposed read and the rows of a store each fall into different banks without padding (rows
// of 128 bytes share the banks in pairs).  fp32: one piece of padding a row.
//
// Readers go from the place of their lane's first (row, col) to the others by `go`, a step whose
// column bits and lane's column bits do not meet (so that adding them is an exclusive-or) and whose
// rows change no bit of the row that the places depend on, but for row bit 2, given as `row4`.
template <typename T, int W>
struct Tiled {
    static constexpr int ROW = sizeof(T) == 2 ? W : W + 4;
    static_assert(W == 64 || W == 128, "tile widths");
    // tokens by columns
    static __device__ __forceinline__ int at(int r, int c) {
        if constexpr (sizeof(T) == 4) return r * ROW + c;
        const int b1 = (r >> 1) & 1, b2 = (r >> 2) & 1, b3 = (r >> 3) & 1;
        const int f = W == 128 ? b2 | (r & 1) << 1 | b1 << 2 | (b2 ^ b3) << 3 : b2 | b1 << 1 | (b2 ^ b3) << 2;
        return r * ROW + ((((c >> 3) ^ f) << 3) | (c & 7));
    }
    static __device__ __forceinline__ int go(int at, int rows, int cols, bool row4 = false) {
        if constexpr (sizeof(T) == 4) return at + (rows + (row4 ? 4 : 0)) * ROW + cols;
        return (at ^ (cols ^ (row4 ? (W == 128 ? 0x48 : 0x28) : 0))) + (rows + (row4 ? 4 : 0)) * ROW;
    }
    // the state's copy: value columns by state rows; the places depend on row bits 0 - 4
    static __device__ __forceinline__ int at_state(int r, int c) {
        if constexpr (sizeof(T) == 4) return r * ROW + c;
        const int b1 = (r >> 1) & 1, b3 = (r >> 3) & 1, b24 = ((r >> 2) ^ (r >> 4)) & 1;
        const int f = W == 128 ? (r & 3) | b3 << 2 | b24 << 3 : b1 | b3 << 1 | b24 << 2;
        return r * ROW + ((((c >> 3) ^ f) << 3) | (c & 7));
    }
    // `flip`: the step changes one of row bits 2 and 4
    static __device__ __forceinline__ int go_state(int at, int rows, int cols, bool flip) {
        if constexpr (sizeof(T) == 4) return at + rows * ROW + cols;
        return (at ^ (cols ^ (flip ? W / 2 : 0))) + rows * ROW;
    }
};

// Hides how a lane's place came about, once a chunk: the places derived from it are then worked out
// where they are used instead of being held in registers over the whole walk.
__device__ __forceinline__ void forget(int& x) { asm volatile("" : "+v"(x)); }
// The lane itself, where a walk's registers do not reach for what follows from it: a reload from scratch also waits for the
// loads of the next chunk.  With and without: packed prompt 82.4 and 86.9 us, backward 190 and 193, 4 groups of heads 274 and
// 283; key width 64 and fp32, which have registers left, lose by it: seven prompts 18.2 and 17.8, fp32 66.0 and 64.8.
template <typename T, int DA>
__device__ __forceinline__ void forget_lane(int& x) {
    if constexpr (sizeof(T) == 2 && DA == 128) forget(x);
}

// A tile of kC tokens by W columns: its global reads into registers, and from there to LDS.
template <typename T, int W, bool VEC, int NT>
struct Tile {
    static constexpr int VE = Frag<T>::VE;
    static constexpr int PER_ROW = W / VE;
    static constexpr int N = kC * PER_ROW / NT;
    static_assert(N > 0 && N * NT == kC * PER_ROW, "whole vectors for every thread");
    u4 v[N];

    __device__ __forceinline__ void load(const Window& w, int width, int thread) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = i * NT + thread;
            v[i] = load_row<T, VEC>(w, k / PER_ROW, (k % PER_ROW) * VE, width);
        }
    }
    // Whether one of this thread's elements is infinite or NaN.
    __device__ __forceinline__ bool odd_values() const {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(T) == 2) {  // an exponent of ones carries into the bit above it
                    any |= ((v[i][e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                } else {
                    any |= ((v[i][e] & 0x7f800000u) + 0x00800000u) & 0x80000000u;
                }
            }
        return any != 0;
    }
    __device__ __forceinline__ void store(T* lds, int thread) const {
        static_assert(NT / PER_ROW % 16 == 0 || sizeof(T) == 4, "steps of 16 rows keep the places' pattern");
        const int at = Tiled<T, W>::at(thread / PER_ROW, (thread % PER_ROW) * VE);
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u4*>(lds + Tiled<T, W>::go(at, i * (NT / PER_ROW), 0)) = v[i];
    }
};

// ---------------------------------------------------------- state update ----
// S += sum over the chunk's tokens of K (x) (w V): wave w holds value columns
// 16 w .. 16 w + 15 of the tile, all DA rows, as DA / 16 accumulators (rows 16 u +
// 4 g + r, column lane & 15).
//
// bf16: w V does not fit bf16, and one rounding of it would leave 2^-8 in a state that
// is kept in fp32.  It is cut into three bf16 pieces (8 + 8 + 8 bits hold all 24 of the
// product), three products on the exact K.
// PARTS = 2: one half of the chunk's tokens, `part`; another wave adds the other half.
template <typename T, int DA, int PARTS = 1>
__device__ __forceinline__ void update_state(f4 (&S)[DA / 16], const T* kt, const T* vt, const float* wt, int wave, int lane, int part = 0) {
    using KL = Tiled<T, DA>;
    using VL = Tiled<T, kV>;
    const int m = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
        int ka = KL::at(8 * g + (m >> 2), 4 * (m & 3)) + part * 32 * KL::ROW;
        int va = VL::at(8 * g + (m >> 2), 16 * wave + 4 * (m & 3)) + part * 32 * VL::ROW;
        wt += part * 32;
        forget(ka);
        forget(va);
#pragma unroll
        for (int s = 0; s < 2 / PARTS; ++s) {
            const u2 v0 = tr4(vt + VL::go(va, 32 * s, 0)), v1 = tr4(vt + VL::go(va, 32 * s, 0, true));
            const uint32_t raw[4] = {v0[0], v0[1], v1[0], v1[1]};
            const f4 w0 = *reinterpret_cast<const f4*>(wt + 32 * s + 8 * g), w1 = *reinterpret_cast<const f4*>(wt + 32 * s + 8 * g + 4);
            const float w[8] = {w0[0], w0[1], w0[2], w0[3], w1[0], w1[1], w1[2], w1[3]};
            u4 p[3];
#pragma unroll
            for (int h = 0; h < DA / 64; ++h) {              // four accumulators' reads at a time
                u4 a[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int c = 64 * h + 16 * u;
                    const u2 a0 = tr4(kt + KL::go(ka, 32 * s, c)), a1 = tr4(kt + KL::go(ka, 32 * s, c, true));
                    a[u] = u4{a0[0], a0[1], a1[0], a1[1]};
                }
                if (h == 0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = __uint_as_float(raw[e] << 16) * w[2 * e];
                        float y = __uint_as_float(raw[e] & 0xffff0000u) * w[2 * e + 1];
#pragma unroll
                        for (int q = 0; q < 3; ++q) {
                            const uint32_t hx = __float_as_uint(x) & 0xffff0000u, hy = __float_as_uint(y) & 0xffff0000u;
                            p[q][e] = __builtin_amdgcn_perm(hy, hx, 0x07060302u);   // (hx >> 16) | hy
                            x -= __uint_as_float(hx);
                            y -= __uint_as_float(hy);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);           // the reads are under way before the first product
#pragma unroll
                for (int q = 0; q < 3; ++q)
#pragma unroll
                    for (int u = 0; u < 4; ++u) S[4 * h + u] = Frag<T>::mma(a[u], p[q], S[4 * h + u]);
            }
        }
    } else {
#pragma unroll
        for (int s = 0; s < 4 / PARTS; ++s) {
            const int t0 = 32 * part + 16 * s + 4 * g;
            const f4 w = *reinterpret_cast<const f4*>(wt + t0);
            u4 b;
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(vt[VL::at(t0 + e, 16 * wave + m)] * w[e]);
#pragma unroll
            for (int h = 0; h < DA / 64; ++h) {
                u4 a[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[u][e] = __float_as_uint(kt[KL::at(t0 + e, 64 * h + 16 * u + m)]);
#pragma unroll
                for (int u = 0; u < 4; ++u) S[4 * h + u] = Frag<T>::mma(a[u], b, S[4 * h + u]);
            }
        }
    }
}

// Weights of the state update of a chunk of n tokens, token by token in the 64 lanes of a wave:
// s_up lambda^{n - shift - j}; the rows behind the tokens hold zeros, and so do their weights.
__device__ __forceinline__ void fill_weights(float* wt, float l2, int n, int shift, float s_up, int lane) {
    wt[lane] = lane < n ? s_up * power(l2, n - shift - lane) : 0.0f;
}

template <typename T>
__device__ __forceinline__ const T* rows_of(const void* p, const LaArgs& A, const Seg& g, int64_t pos, int64_t ts, int head_off) {
    const int64_t t = A.reversed ? (int64_t)g.first + g.len - 1 - pos : (int64_t)g.first + pos;
    return (const T*)p + t * ts + head_off;
}

__device__ __forceinline__ int64_t state_at(const LaArgs& A, int at, int h, int tile, int da) {
    return (((int64_t)at * A.H + h) * A.nv + tile) * (da * kV);
}

// What a workgroup does.  Those that read the same rows (column tiles, heads that share keys) have
// numbers eight apart: workgroups go to the eight dies in turn, and such a group meets in one L2.
struct Unit { int seg, h, tile; };
__device__ __forceinline__ Unit unit_of(const LaArgs& A) {
    const int inner = A.share * A.nv, b = blockIdx.x;
    const int outer = b / (8 * inner) * 8 + b % 8, i = b / 8 % inner;
    const int groups = A.H / A.share;
    Unit u;
    u.tile = i % A.nv;
    u.h = outer % groups * A.share + i / A.nv;
    u.seg = A.seg0 + outer / groups;
    return u;
}
inline unsigned grid_of(const LaArgs& A) {
    const int64_t outer = (int64_t)(A.nseg - A.seg0) * (A.H / A.share);
    return (unsigned)((outer + 7) / 8 * 8 * A.share * A.nv);
}
// Segments whose grid_of a launch may have.
inline int64_t segments_of_launch(const LaArgs& A) {
    return (max_workgroups(kWalkThreads) - 7 * A.share * A.nv) / ((int64_t)A.H * A.nv);
}

// ------------------------------------------------------------------ plan ----
// The segments of more packed sequences than a workgroup should look through for itself, and those of
// more than kFewSegments segments (at most n_long of them, then -1).
__global__ void __launch_bounds__(64) k_la_plan(LaArgs A, Seg* plan, int2* seqs, int* longs, int n_long) {
    const int lane = threadIdx.x;
    int found = 0;
    Lane64 l;
    l.reach = l.segs = l.states = 0;
    for (int s0 = 0; s0 < A.n_seq; s0 += 64) {
        l.read(A, s0, lane);
        const int s = s0 + lane;
        const uint64_t many = __ballot(l.count > kFewSegments);
        const int place_of = found + __popcll(many & ((1ull << lane) - 1));
        if (l.count > kFewSegments && place_of < n_long) longs[place_of] = s;
        found += __popcll(many);
        if (s >= A.n_seq) continue;
        seqs[s] = make_int2(l.state, l.count);
        for (int i = 0; i < l.count; ++i) {
            Seg g{s, l.first, l.len, 0, 0, i, l.count, l.state + i};
            place(g);
            if (l.at + i < A.nseg) plan[l.at + i] = g;
        }
    }
    for (int i = l.segs + lane; i < A.nseg; i += 64) plan[i].seq = -1;
    for (int i = found + lane; i < n_long; i += 64) longs[i] = -1;
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

// Accumulator i of a wave's lane in a state's place in the workspace.
template <int DA>
__device__ __forceinline__ f4* state_piece(const LaArgs& A, int at, int h, int tile, int wave, int i, int lane) {
    return reinterpret_cast<f4*>(A.states + state_at(A, at, h, tile, DA)) + (wave * (DA / 16) + i) * 64 + lane;
}

// ---------------------------------------------------------- segment state ----
// Eight waves: a wave holds 16 value columns of the state and half of the tokens of each chunk, so
// that the weighted values' splitting, which costs more than the products, is shared out; the two
// halves are added up at the end.  Weights reach to the segment's end, so nothing is rescaled on the way.
// Bound by its reads.  16384 packed tokens of nine sequences, 16 heads of 128 x 64, bf16: 30.5 us for 96 MB
// (3.1 TB/s, matrix unit 11 % busy); 8190 tokens of 16 heads of 64 x 64 in fp32: 17.7 us for 72 MB (4.0 TB/s, 26 %).
template <typename T, int DA, bool VEC>
__global__ void __launch_bounds__(kWalkThreads) k_la_state(LaArgs A) {
    constexpr int NA = DA / 16, TILES = kC * (Tiled<T, DA>::ROW + Tiled<T, kV>::ROW) * (int)sizeof(T), SUMS = NA * 4 * 64 * 16;
    __shared__ __attribute__((aligned(16))) char mem[TILES > SUMS ? TILES : SUMS];
    __shared__ __attribute__((aligned(16))) float wt[2][kC];
    T* kt = reinterpret_cast<T*>(mem);
    T* vt = kt + kC * Tiled<T, DA>::ROW;
    const Unit u = unit_of(A);
    if (u.seg >= A.nseg) return;
    const Seg g = segment(A, u.seg);
    if (g.seq < 0 || is_last(g)) return;         // a last segment's end state is the final state: the walk makes it
    const int lane = threadIdx.x & 63, wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wave8 & 3, part = wave8 >> 2;
    const float l2 = log2_decay(A, u.h);
    const int64_t bs = A.reversed ? -A.b_ts : A.b_ts, cs = A.reversed ? -A.c_ts : A.c_ts;
    const T* kp = rows_of<T>(A.b, A, g, g.p0, A.b_ts, (u.h / A.b_rep) * A.Da);
    const T* vp = rows_of<T>(A.c, A, g, g.p0, A.c_ts, (u.h / A.c_rep) * A.Dv + u.tile * kV);
    const int vw = A.Dv - u.tile * kV;
    Tile<T, DA, VEC, kWalkThreads> k;
    Tile<T, kV, VEC, kWalkThreads> v;
    auto load = [&](int c0) {
        const int n = min(kC, g.n - c0);
        k.load(window(kp + c0 * bs, A.b_ts, A.reversed, n, A.Da), A.Da, threadIdx.x);
        v.load(window(vp + c0 * cs, A.c_ts, A.reversed, n, vw), vw, threadIdx.x);
    };
    load(0);
    f4 S[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) S[i] = f4{0, 0, 0, 0};
    if (g.idx == 0 && part == 0) {
        const float f = power(l2, g.n);
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const f4 h = load_h0(A, g.seq, u.h, u.tile, wave, i, lane);
            *state_piece<DA>(A, g.state + g.count - 1, u.h, u.tile, wave, i, lane) = h;
            S[i] = h * f;
        }
    }
    for (int c0 = 0; c0 < g.n; c0 += kC) {       // whole chunks: only a last segment has a ragged one
        float* w = wt[c0 / kC & 1];
        if (wave8 == 4) fill_weights(w, l2, g.n - c0, A.shift, A.s_up, lane);
        lds_barrier();
        k.store(kt, threadIdx.x);
        v.store(vt, threadIdx.x);
        lds_barrier();
        if (c0 + kC < g.n) load(c0 + kC);
        update_state<T, DA, 2>(S, kt, vt, w, wave, lane, part);
    }
    lds_barrier();
    f4* sums = reinterpret_cast<f4*>(mem) + wave * NA * 64 + lane;
    if (part) {
#pragma unroll
        for (int i = 0; i < NA; ++i) sums[i * 64] = S[i];
    }
    lds_barrier();
    if (!part) {
#pragma unroll
        for (int i = 0; i < NA; ++i) *state_piece<DA>(A, g.state, u.h, u.tile, wave, i, lane) = S[i] + sums[i * 64];
    }
}

// ---------------------------------------------------------------- carry ----
// In place over a sequence's places: the state that enters each of its segments.  A workgroup
// takes 1024 values (256 lanes of four) of one (long sequence, head, tile).  There are at most
// T / (kFewSegments target + 1) long sequences, so the launch does not grow with the short ones (64k tokens in
// 2000 sequences, 16 heads: the call 892 us where it did, 780 so; 721 now).  They are never more than 128: 2^23 workgroups
// with the most heads and columns.  Bound by latency: 5.4 us for 16.9 MB, 5.0 us where it finds none.
template <int DA>
__global__ void __launch_bounds__(256) k_la_carry(LaArgs A, const int* longs) {
    constexpr int PER = DA * kV / 1024;
    int b = blockIdx.x;
    const int part = b % PER;
    b /= PER;
    const int tile = b % A.nv;
    b /= A.nv;
    const int h = b % A.H;
    int which = b / A.H, seq = which;
    if (A.plan) {
        seq = longs[which];
    } else if (A.cu) {
        const int lane = threadIdx.x & 63, s = min(lane, A.n_seq - 1);
        const int64_t len = (int64_t)min(max(A.cu[s + 1], 0), A.T) - min(max(A.cu[s], 0), A.T);
        uint64_t many = __ballot(lane < A.n_seq && len > (int64_t)kFewSegments * A.target);
        for (; which > 0; --which) many &= many - 1;
        seq = __ffsll((unsigned long long)many) - 1;             // -1: fewer are long
    }
    if (seq < 0) return;
    int first, n, len;
    sequence(A, seq, first, n, len);
    if (n <= kFewSegments) return;
    const float f = power(log2_decay(A, h), segment_tokens(len, n));
    f4* p = reinterpret_cast<f4*>(A.states + state_at(A, first, h, tile, DA)) + part * 256 + threadIdx.x;
    const int64_t step = state_at(A, 1, 0, 0, DA) / 4;
    f4 run = p[0];
    p[0] = p[(n - 1) * step];                    // h0
    constexpr int B = 8;                         // states read ahead of the first one's use
    for (int i = 1; i < n; i += B) {
        f4 own[B];
#pragma unroll
        for (int j = 0; j < B; ++j) own[j] = i + j + 1 < n ? p[(i + j) * step] : f4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (i + j >= n) break;
            p[(i + j) * step] = run;
            run = run * f + own[j];
        }
    }
}

// ----------------------------------------------------------------- walk ----
// N rows of 16x16 products with the NK fragments of `q`: y = sum_s fetch(x, s) q[s], handed to use(x, y).  With PIECES = 2
// the other operand comes in two pieces, fetch(x, 2 s) and fetch(x, 2 s + 1).
// bf16 reads two operands ahead of the ones it multiplies; fp32 four at a time, whose 16
// instructions cover the next read themselves.
// fp32, bound by its products, leaves out the rows from `end` on (scores of later tokens): use gets zeros.
template <typename T, int N, int PIECES, int NK, typename Fetch, typename Use>
__device__ __forceinline__ void products(const u4 (&q)[NK], int end, Fetch fetch, Use use) {
    constexpr int GS = sizeof(T) == 2 ? 2 : 4, NG = NK * PIECES / GS, NB = sizeof(T) == 2 ? 2 : 1;
    u4 fr[NB][GS];
    auto read = [&](int z) {
#pragma unroll
        for (int s = 0; s < GS; ++s) fr[z % NB][s] = fetch(z / NG, z % NG * GS + s);
    };
    if (NB == 2) read(0);
#pragma unroll
    for (int x = 0; x < N; ++x) {
        f4 y = {0, 0, 0, 0};
        if (NB == 1 && x >= end) {
            use(x, y);
            continue;
        }
#pragma unroll
        for (int z = x * NG; z < (x + 1) * NG; ++z) {
            if (NB == 1) read(z);
            else if (z + 1 < N * NG) read(z + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < GS; ++s) y = Frag<T>::mma(fr[z % NB][s], q[(z % NG * GS + s) / PIECES], y);
        }
        use(x, y);
    }
}

// Value column of row 4 g of accumulator x: such that a lane's accumulators join to the 16 bytes it
// stores at a time, and the four lanes of a token store 64 bytes side by side.
template <typename TO>
__device__ __forceinline__ constexpr int column(int x, int g) {
    return sizeof(TO) == 2 ? 32 * (x >> 1) + 8 * g + 4 * (x & 1) : 16 * x + 4 * g;
}

// fp32 values as two bf16 pieces, the second what the first leaves: 16 of the 24 bits.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
template <typename T> constexpr int kPieces = sizeof(T) == 2 ? 2 : 1;

// Masked, decayed scores P^T (rows j, column i = 16 wave + m) of TOKENS tokens: what a lane holds of them is the operand
// of the product with the values as it stands, tokens in the same order on both sides.
template <typename T, int TOKENS>
struct Scores {
    u4 p[TOKENS / 16];                       // bf16: two pieces for every 32 tokens; fp32: 16 tokens each
};
// s_in lambda^{i - j} with j = 16 t + 4 gr + r: on the diagonal block (t = wave) as it is, in front of it
// through the power of the next block's distance, between 1 and 31, times lambda^{16 (wave - 1 - t)}.
// The powers are the same for all four waves and lie in LDS, two f4 a lane, diagonal and near: in eight
// registers they cost the walk for keys' and values' gradients its last ones (80 us from LDS, 103 so).
struct Decay {
    const f4* lds;
    float far[4];                            // uniform
    __device__ __forceinline__ Decay(f4* table, float l2, float s_in, int wave, int lane) : lds(table + lane) {
        const int m = lane & 15, gr = lane >> 4;
        f4 w;
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = s_in * power(l2, wave == 0 ? max(m - 4 * gr - r, 0) : m - 4 * gr - r + 16);
        if (wave < 2) table[wave * 64 + lane] = w;       // read behind the first barrier
#pragma unroll
        for (int t = 0; t < 4; ++t) far[t] = power(l2, 16 * max(wave - 1 - t, 0));
    }
    __device__ __forceinline__ f4 weights(int t, int wave) const { return lds[t == wave ? 0 : 64]; }
    // t: the block of 16 tokens in the chunk, x: in P
    template <typename T, int TOKENS>
    __device__ __forceinline__ void apply(Scores<T, TOKENS>& P, int x, int t, f4 y, int wave, int m, int gr) const {
        const f4 w = weights(t, wave);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            y[r] = t > wave || (t == wave && 4 * gr + r > m) ? 0.0f : y[r] * (t == wave ? w[r] : w[r] * far[t]);
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t hi, lo;
                split_bf16(y[2 * k], y[2 * k + 1], hi, lo);
                P.p[x & ~1][2 * (x & 1) + k] = hi;
                P.p[x | 1][2 * (x & 1) + k] = lo;
            }
        } else {
            P.p[x] = __builtin_bit_cast(u4, y);
        }
    }
};

// A fragment of the V tile, tokens from t on along the lane's elements, for accumulator x.
template <typename T, typename TO, int W>
__device__ __forceinline__ u4 value_fragment(const T* vt, int va, int x, int t, int m, int gr) {
    using VL = Tiled<T, W>;
    if constexpr (sizeof(T) == 2) {
        const u2 v0 = tr4(vt + VL::go(va, t, column<TO>(x, 0)));
        const u2 v1 = tr4(vt + VL::go(va, t + 16, column<TO>(x, 0)));
        return u4{v0[0], v0[1], v1[0], v1[1]};
    } else {
        u4 a;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = __float_as_uint(vt[VL::at(t + 4 * gr + e, column<TO>(x, m >> 2) + (m & 3))]);
        return a;
    }
}

// o[x] += V^T P^T for NT accumulators and the scores' tokens, from t0 on; V a tile of W columns.  The matrix product multiplies
// the zero scores of later tokens with whatever those hold: where the chunk has infinities or NaN among its values
// (`odd`), it is made once for each of the 16 tokens, later ones cleared from the tile's fragments.
template <typename T, typename TO, int W, int TOKENS, int NT>
__device__ __forceinline__ void add_values(f4 (&o)[NT], const Scores<T, TOKENS>& P, const T* vt, int t0, bool odd, int wave, int m, int gr) {
    using VL = Tiled<T, W>;
    constexpr int STEP = sizeof(T) == 2 ? 32 : 16;       // tokens of a fragment
    if (__builtin_expect(odd, false)) {
        int va = sizeof(T) == 2 ? VL::at(4 * gr + (m >> 2), column<TO>(0, m & 3)) : 0;
        forget(va);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            f4 own = o[x];
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                f4 y = o[x];
#pragma unroll
                for (int s = 0; s < TOKENS / STEP; ++s) {
                    u4 a = value_fragment<T, TO, W>(vt, va, x, t0 + STEP * s, m, gr);
                    const int left = 16 * wave + i - t0 - STEP * s - 4 * gr;      // the fragment's tokens up to the i-th
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (sizeof(T) == 2)
                            a[e] &= (left >= 16 * (e >> 1) + 2 * (e & 1) ? 0xffffu : 0u) | (left > 16 * (e >> 1) + 2 * (e & 1) ? 0xffff0000u : 0u);
                        else
                            a[e] = left >= e ? a[e] : 0u;
                    }
#pragma unroll
                    for (int k = 0; k < kPieces<T>; ++k) y = Frag<T>::mma(a, P.p[kPieces<T> * s + k], y);
                }
                if (m == i) own = y;
            }
            o[x] = own;
        }
        return;
    }
    if constexpr (sizeof(T) == 2) {
        int va = VL::at(4 * gr + (m >> 2), column<TO>(0, m & 3));
        forget(va);
#pragma unroll
        for (int h = 0; h < NT; h += 4) {
            u4 a[TOKENS / 32][4];
#pragma unroll
            for (int s = 0; s < TOKENS / 32; ++s)
#pragma unroll
                for (int x = 0; x < 4; ++x) a[s][x] = value_fragment<T, TO, W>(vt, va, h + x, t0 + 32 * s, m, gr);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < TOKENS / 16; ++s)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[h + x] = Frag<T>::mma(a[s / 2][x], P.p[s], o[h + x]);
        }
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t > wave) break;
#pragma unroll
            for (int h = 0; h < NT; h += 4) {
                u4 a[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) a[x] = value_fragment<T, TO, W>(vt, 0, h + x, 16 * t, m, gr);
#pragma unroll
                for (int x = 0; x < 4; ++x) o[h + x] = Frag<T>::mma(a[x], P.p[t], o[h + x]);
            }
        }
    }
}

// o += the chunk's own part for this wave's 16 tokens: the scores of `kt`, a tile of KW columns, with the fragments q, times the
// values in `vt`, a tile of W columns.  TOKENS: of the chunk at a time, none that are all later ones.  All 64 wait less (seven
// short prompts 17.7 us, 32 at a time 18.5); 32 take half the registers, which k_la_dkdv does not have.
template <typename T, typename TO, int KW, int W, int TOKENS, int NK, int NT>
__device__ __forceinline__ void add_chunk(f4 (&o)[NT], const u4 (&q)[NK], const Decay& dec, const T* kt, const T* vt, bool odd, int wave,
                                          int m, int gr) {
    using KL = Tiled<T, KW>;
    constexpr int N = TOKENS / 16;
    int ka = KL::at(m, Frag<T>::VE * gr);
    forget(ka);
#pragma unroll
    for (int c = 0; c < kC / TOKENS; ++c) {
        if (N * c > wave) break;
        Scores<T, TOKENS> P;
        products<T, N, 1>(
            q, 1 + wave, [&](int x, int s) { return fragment_at(kt + KL::go(ka, TOKENS * c + 16 * x, Frag<T>::K * s)); },
            [&](int x, f4 y) { dec.apply(P, x, N * c + x, y, wave, m, gr); });
        add_values<T, TO, W>(o, P, vt, TOKENS * c, odd, wave, m, gr);
    }
}

// The tokens' rows of `width` columns from their lanes' accumulators: token i of n lies at base + i step.
// LINES (16-bit rows): the lanes of two neighbouring tokens swap halves of 64 columns, so that eight
// lanes store a whole 128-byte line; packed prompt 86.5 -> 84 us.  The walk for keys' and values' gradients,
// short of registers, stores pieces of 64 bytes instead (80 us; with lines 90).
template <typename TO, bool VEC, bool LINES, int NT>
__device__ __forceinline__ void store_rows(TO* base, int64_t step, int i, int n, const f4 (&o)[NT], int width, int gr) {
    if constexpr (VEC && sizeof(TO) == 2) {
        const bool odd = LINES && (i & 1);
#pragma unroll
        for (int e = 0; e < NT / 2; e += 2) {
            u4 x[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                x[k] = u4{pack_bf16(o[2 * e + 2 * k][0], o[2 * e + 2 * k][1]), pack_bf16(o[2 * e + 2 * k][2], o[2 * e + 2 * k][3]),
                          pack_bf16(o[2 * e + 2 * k + 1][0], o[2 * e + 2 * k + 1][1]),
                          pack_bf16(o[2 * e + 2 * k + 1][2], o[2 * e + 2 * k + 1][3])};
            if constexpr (LINES) {
                u4 a, b;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t send = odd ? x[0][k] : x[1][k];
                    const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)send, 0xb1, 0xf, 0xf, true);   // lane ^ 1
                    a[k] = odd ? got : x[0][k];
                    b[k] = odd ? x[1][k] : got;
                }
                const int col = column<TO>(2 * e + (odd ? 2 : 0), gr), t = i & ~1;
                if (col < width) {
                    if (t < n) *reinterpret_cast<u4*>(base + t * step + col) = a;
                    if (t + 1 < n) *reinterpret_cast<u4*>(base + (t + 1) * step + col) = b;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (i < n && column<TO>(2 * e + 2 * k, gr) < width)
                        *reinterpret_cast<u4*>(base + i * step + column<TO>(2 * e + 2 * k, gr)) = x[k];
            }
        }
    } else if (i < n) {
        TO* row = base + i * step;
        if constexpr (sizeof(TO) == 4) {
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const int col = column<TO>(x, gr);
                if constexpr (VEC) {
                    if (col < width) *reinterpret_cast<f4*>(row + col) = o[x];
                } else if (col + 4 <= width) {
                    __builtin_memcpy(row + col, &o[x], 16);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (col + r < width) row[col + r] = o[x][r];
                }
            }
        } else {
#pragma unroll
            for (int x = 0; x < NT; x += 2) {
                const int col = column<TO>(x, gr);
                const u4 t = {pack_bf16(o[x][0], o[x][1]), pack_bf16(o[x][2], o[x][3]), pack_bf16(o[x + 1][0], o[x + 1][1]),
                              pack_bf16(o[x + 1][2], o[x + 1][3])};
                if (col + 8 <= width) {
                    __builtin_memcpy(row + col, &t, 16);
                } else {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        if (col + r < width) row[col + r] = (TO)(t[r / 2] >> (16 * (r % 2)));
                }
            }
        }
    }
}

// The state's waves of a walk: they hold the state, 16 value columns each, put its copy and the
// chunks' K and V tiles to LDS, and bring it to the next chunk.
template <typename T, int DA, bool VEC>
__device__ __forceinline__ void carry_state(const LaArgs& A, const Seg& g, const Unit& un, float l2, T* kt, T* vt, T* st, float* wt,
                                            int* odd, int wave, int lane) {
    using SL = Tiled<T, DA>;
    int thread = threadIdx.x & 255;
    const int64_t bs = A.reversed ? -A.b_ts : A.b_ts, cs = A.reversed ? -A.c_ts : A.c_ts;
    const T* kp = rows_of<T>(A.b, A, g, g.p0, A.b_ts, (un.h / A.b_rep) * A.Da);
    const T* vp = rows_of<T>(A.c, A, g, g.p0, A.c_ts, (un.h / A.c_rep) * A.Dv + un.tile * kV);
    const int vw = A.Dv - un.tile * kV;
    const int64_t hrow = is_last(g) && A.h_out ? state_row(A, g.seq) : -1;
    Tile<T, DA, VEC, 256> k;
    Tile<T, kV, VEC, 256> v;
    auto load = [&](int c0) {
        const int n = min(kC, g.n - c0);
        k.load(window(kp + c0 * bs, A.b_ts, A.reversed, n, A.Da), A.Da, thread);
        v.load(window(vp + c0 * cs, A.c_ts, A.reversed, n, vw), vw, thread);
    };
    load(0);
    f4 S[DA / 16];
    if (g.count == 1) {
#pragma unroll
        for (int i = 0; i < DA / 16; ++i) S[i] = load_h0(A, g.seq, un.h, un.tile, wave, i, lane);
    } else {
        const int base = g.state - g.idx;
        const bool few = g.count <= kFewSegments;
        const int from = !few ? g.state : g.idx ? base : base + g.count - 1;
#pragma unroll
        for (int i = 0; i < DA / 16; ++i) S[i] = *state_piece<DA>(A, from, un.h, un.tile, wave, i, lane);
        const float each = power(l2, g.p0 / max(g.idx, 1));
        for (int j = 1; few && j < g.idx; ++j) {
#pragma unroll
            for (int i = 0; i < DA / 16; ++i) S[i] = S[i] * each + *state_piece<DA>(A, base + j, un.h, un.tile, wave, i, lane);
        }
    }
    float f = power(l2, kC);
    for (int c0 = 0; c0 < g.n; c0 += kC) {
        forget_lane<T, DA>(thread);
        const int lane = thread & 63, sw = SL::at_state(16 * wave + (lane & 15), 4 * (lane >> 4));
        const int n = min(kC, g.n - c0);
        const bool more = c0 + kC < g.n;
        k.store(kt, thread);
        v.store(vt, thread);
        const int have = (__ballot(v.odd_values()) ? 1 : 0) | (__ballot(k.odd_values()) ? 2 : 0);
        if (lane == 0) odd[wave] = have;
        if (c0 == 0 || n < kC) {
            if (wave == 0) fill_weights(wt, l2, n, A.shift, A.s_up, lane);
            f = power(l2, n);
        }
#pragma unroll
        for (int i = 0; i < DA / 16; ++i) {      // the copy that this chunk's products read
            T* p = st + SL::go_state(sw, 0, 16 * i, false);
            if constexpr (sizeof(T) == 2) {
                u2 hi, lo;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t a, b;
                    split_bf16(S[i][2 * k], S[i][2 * k + 1], a, b);
                    hi[k] = a;
                    lo[k] = b;
                }
                *reinterpret_cast<u2*>(p) = hi;
                *reinterpret_cast<u2*>(p + kV * SL::ROW) = lo;
            } else {
                *reinterpret_cast<f4*>(p) = S[i];
            }
        }
        lds_barrier();
        if (more) load(c0 + kC);
        if (more || hrow >= 0) {
#pragma unroll
            for (int i = 0; i < DA / 16; ++i) S[i] *= f;
            update_state<T, DA>(S, kt, vt, wt, wave, lane);
        }
        lds_barrier();
    }
    if (hrow >= 0) {
        int late = lane;                         // keeps these addresses out of the walk's registers
        forget(late);
        float* p = A.h_out + (hrow * A.H + un.h) * (int64_t)A.Da * A.Dv;
        const int col = un.tile * kV + 16 * wave + (late & 15);
#pragma unroll
        for (int i = 0; i < DA / 16; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * (late >> 4) + r;
                if (col < A.Dv && row < A.Da) p[A.transposed ? (int64_t)col * A.Da + row : (int64_t)row * A.Dv + col] = S[i][r];
            }
    }
}

// Which 16 tokens of the chunk an output wave takes (or which 16 columns a state's wave holds).  In
// fp32 later tokens cost more products, and a wave's SIMD goes by its number: every other round of
// 256 workgroups counts backwards, so that two workgroups on a compute unit even out.
template <typename T>
__device__ __forceinline__ int block_of(int wave8) {
    const bool back = sizeof(T) == 4 && wave8 < 4 && (blockIdx.x >> 8 & 1);
    return back ? 3 - wave8 : wave8 & 3;
}

// Eight waves on one chunk: waves 0 - 3 make the outputs of 16 tokens each, waves 4 - 7
// bring the state to the next chunk at the same time.  Both read the chunk's K and V tiles; the
// state entering the chunk reaches the output waves as an LDS copy.  The state's waves load the
// next chunk's tiles into registers while this one is computed (the output waves the next
// queries, which only they read) and put them to LDS between two barriers.
// TO: type of the output (fp32 where several heads' gradients are still to be added up).
// bf16 is bound by its traffic: the packed prompt above 54 us for 222 MB, 4.1 TB/s, and the backward's run for dq (4 x 4096
// tokens, do and v to dq) 55 us for 210 MB, 3.8 TB/s, the matrix unit 21 - 24 % busy, LDS 26 - 32 %.  fp32, 49 us for 143 MB with
// the matrix unit 38 % busy, waits for both in turn.  Two workgroups of eight waves fit a compute unit: 128
// registers a wave.
template <typename T, typename TO, int DA, bool VEC>
__global__ void __launch_bounds__(kWalkThreads, sizeof(T) * DA > 256 ? 2 : 4) k_la_out(LaArgs A) {
    using KL = Tiled<T, DA>;
    constexpr int NK = DA / Frag<T>::K, P = kPieces<T>;
    __shared__ __attribute__((aligned(16))) T kt[kC * Tiled<T, DA>::ROW];
    __shared__ __attribute__((aligned(16))) T vt[kC * Tiled<T, kV>::ROW];
    __shared__ __attribute__((aligned(16))) T st[kPieces<T> * kV * KL::ROW];      // the state's copy [piece][value column][row]
    __shared__ __attribute__((aligned(16))) float wt[kC];
    __shared__ __attribute__((aligned(16))) f4 powers[128];
    __shared__ int odd[4];                       // infinities or NaN in the chunk: in the V tile 1, in the K tile 2
    const Unit un = unit_of(A);
    if (un.seg >= A.nseg) return;
    const Seg g = segment(A, un.seg);
    if (g.seq < 0) return;
    const int lane = threadIdx.x & 63, m = lane & 15, gr = lane >> 4;
    const int wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = block_of<T>(wave8);
    const float l2 = log2_decay(A, un.h);
    // Every wave meets the same barriers: two a chunk.
    if (wave8 >= 4) {
        carry_state<T, DA, VEC>(A, g, un, l2, kt, vt, st, wt, odd, wave, lane);
        return;
    }
    const int64_t as = A.reversed ? -A.a_ts : A.a_ts, os = A.reversed ? -A.o_ts : A.o_ts;
    const T* ap = rows_of<T>(A.a, A, g, g.p0, A.a_ts, (un.h / A.a_rep) * A.Da);
    TO* op = const_cast<TO*>(rows_of<TO>(A.o, A, g, g.p0, A.o_ts, un.h * A.Dv + un.tile * kV));
    const int qi = 16 * wave + m;                // this lane's query position in the chunk
    const float at_q = A.s_carry * power(l2, qi + A.shift);
    const Decay dec(powers, l2, A.s_in, wave, lane);
    u4 q[NK], qn[NK];
    auto load_q = [&](int c0) {
        const Window w = window(ap + c0 * as, A.a_ts, A.reversed, min(kC, g.n - c0), A.Da);
#pragma unroll
        for (int s = 0; s < NK; ++s) qn[s] = load_row<T, VEC>(w, qi, Frag<T>::K * s + Frag<T>::VE * gr, A.Da);
    };
    load_q(0);
    for (int c0 = 0; c0 < g.n; c0 += kC) {
#pragma unroll
        for (int s = 0; s < NK; ++s) q[s] = qn[s];
        lds_barrier();
        if (c0 + kC < g.n) load_q(c0 + kC);

        // the carried part O^T = S^T Q^T (four accumulators of value columns), then the chunk's own
        f4 o[4];
        int sa = KL::at_state(column<TO>(0, m >> 2) + (m & 3), Frag<T>::VE * gr);
        forget(sa);
        products<T, 4, kPieces<T>>(
            q, 4,
            [&](int x, int s) {
                return fragment_at(st + s % P * (kV * KL::ROW) + KL::go_state(sa, column<TO>(x, 0), Frag<T>::K * (s / P), x & 1));
            },
            [&](int x, f4 y) { o[x] = y * at_q; });      // lambda^{i + shift} of the lane's token
        const int has = odd[0] | odd[1] | odd[2] | odd[3];
        add_chunk<T, TO, DA, kV, kC>(o, q, dec, kt, vt, has & 1, wave, m, gr);
        store_rows<TO, VEC, true>(op + c0 * os, os, qi, g.n - c0, o, A.Dv - un.tile * kV, gr);
        lds_barrier();
    }
}

// The gradients of keys and values in one reversed walk, for values of one column tile.  In the roles of
// the walk: keys q, values do (A.b, A.c), queries k (A.a) give dv (A.o),
//     dv_j = scale sum_{i>=j} lambda^{i-j} (k_j . q_i) do_i + lambda^{..} k_j^T R,
// and on the same tiles and state, with queries v (X.v),
//     dk_j = scale sum_{i>=j} lambda^{i-j} (v_j . do_i) q_i + lambda^{..} R v_j   (X.dk).
// R's copy lies with its rows (key width) side by side: the first product reads it as it lies, the second
// transposed.  Bound by its traffic: 16384 tokens, 16 heads of 128 x 64, bf16: 86 us for 352 MB, 4.1 TB/s (matrix unit 20 % busy,
// LDS 36 %); before the operands came in two pieces 81 us, and the call
// with two runs instead 231 us, so 188.
struct SecondArgs {
    const void* v;
    void* dk;
    int64_t v_ts, dk_ts;
    int v_rep;
};
template <typename T, typename TO, int DA, bool VEC>
__global__ void __launch_bounds__(kWalkThreads, sizeof(T) == 4 ? 2 : 4) k_la_dkdv(LaArgs A, SecondArgs X) {
    using KL = Tiled<T, DA>;
    using VL = Tiled<T, kV>;
    constexpr int NK = DA / Frag<T>::K, NV = kV / Frag<T>::K, NA = DA / 16, P = kPieces<T>, TOK = sizeof(T) == 2 ? 32 : kC;
    __shared__ __attribute__((aligned(16))) T kt[kC * Tiled<T, DA>::ROW];
    __shared__ __attribute__((aligned(16))) T vt[kC * Tiled<T, kV>::ROW];
    __shared__ __attribute__((aligned(16))) T st[kPieces<T> * kV * KL::ROW];
    __shared__ __attribute__((aligned(16))) float wt[kC];
    __shared__ __attribute__((aligned(16))) f4 powers[128];
    __shared__ int odd[4];                       // infinities or NaN in the chunk: in the V tile 1, in the K tile 2
    const Unit un = unit_of(A);
    if (un.seg >= A.nseg) return;
    const Seg g = segment(A, un.seg);
    if (g.seq < 0) return;
    const int lane = threadIdx.x & 63;
    const int wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = block_of<T>(wave8);
    const float l2 = log2_decay(A, un.h);
    if (wave8 >= 4) {
        carry_state<T, DA, VEC>(A, g, un, l2, kt, vt, st, wt, odd, wave, lane);
        return;
    }
    const T* ap = rows_of<T>(A.a, A, g, g.p0, A.a_ts, (un.h / A.a_rep) * A.Da);
    const T* vp = rows_of<T>(X.v, A, g, g.p0, X.v_ts, (un.h / X.v_rep) * A.Dv);
    TO* dv = const_cast<TO*>(rows_of<TO>(A.o, A, g, g.p0, A.o_ts, un.h * A.Dv));
    TO* dk = const_cast<TO*>(rows_of<TO>(X.dk, A, g, g.p0, X.dk_ts, un.h * A.Da));
    const float at_q = A.s_carry * power(l2, 16 * wave + (lane & 15) + A.shift);
    const Decay dec(powers, l2, A.s_in, wave, lane);
    u4 q[NK], qn[NK], v[NV], vn[NV];
    int me = lane;
    auto load = [&](int c0) {
        const int n = min(kC, g.n - c0), i = 16 * wave + (me & 15), e = Frag<T>::VE * (me >> 4);
        const Window wq = window(ap - c0 * A.a_ts, A.a_ts, true, n, A.Da), wv = window(vp - c0 * X.v_ts, X.v_ts, true, n, A.Dv);
#pragma unroll
        for (int s = 0; s < NK; ++s) qn[s] = load_row<T, VEC>(wq, i, Frag<T>::K * s + e, A.Da);
#pragma unroll
        for (int s = 0; s < NV; ++s) vn[s] = load_row<T, VEC>(wv, i, Frag<T>::K * s + e, A.Dv);
    };
    load(0);
    for (int c0 = 0; c0 < g.n; c0 += kC) {
#pragma unroll
        for (int s = 0; s < NK; ++s) q[s] = qn[s];
#pragma unroll
        for (int s = 0; s < NV; ++s) v[s] = vn[s];
        lds_barrier();
        forget_lane<T, DA>(me);
        const int m = me & 15, gr = me >> 4, qi = 16 * wave + m;
        if (c0 + kC < g.n) load(c0 + kC);
        const int has = odd[0] | odd[1] | odd[2] | odd[3];
        {
            f4 o[4];
            int sa = KL::at_state(column<TO>(0, m >> 2) + (m & 3), Frag<T>::VE * gr);
            forget(sa);
            products<T, 4, kPieces<T>>(
                q, 4,
                [&](int x, int s) {
                    return fragment_at(st + s % P * (kV * KL::ROW) + KL::go_state(sa, column<TO>(x, 0), Frag<T>::K * (s / P), x & 1));
                },
                [&](int x, f4 y) { o[x] = y * at_q; });
            add_chunk<T, TO, DA, kV, TOK>(o, q, dec, kt, vt, has & 1, wave, m, gr);
            store_rows<TO, VEC, false>(dv - c0 * A.o_ts, -A.o_ts, qi, g.n - c0, o, A.Dv, gr);
        }
        {
            f4 o[NA];
            int sa = KL::at_state(8 * gr + (m >> 2), column<TO>(0, m & 3));
            forget(sa);
            products<T, NA, kPieces<T>>(
                v, NA,
                [&](int x, int sp) {
                    const int s = sp / P;
                    const T* copy = st + sp % P * (kV * KL::ROW);
                    if constexpr (sizeof(T) == 2) {      // rows of R: key columns of the copy, eight value columns a lane
                        const u2 a0 = tr4(copy + KL::go_state(sa, 32 * s, column<TO>(x, 0), false));
                        const u2 a1 = tr4(copy + KL::go_state(sa, 32 * s + 4, column<TO>(x, 0), true));
                        return u4{a0[0], a0[1], a1[0], a1[1]};
                    } else {
                        u4 a;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[e] = __float_as_uint(copy[KL::at_state(16 * s + 4 * gr + e, column<TO>(x, m >> 2) + (m & 3))]);
                        return a;
                    }
                },
                [&](int x, f4 y) { o[x] = y * at_q; });
            add_chunk<T, TO, kV, DA, TOK>(o, v, dec, vt, kt, has & 2, wave, m, gr);
            store_rows<TO, VEC, false>(dk - c0 * X.dk_ts, -X.dk_ts, qi, g.n - c0, o, A.Da, gr);
        }
        lds_barrier();
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
    int64_t row0, n_slots, q_ts, k_ts, v_ts;      // row0: first row of the launch
    int H, rep, Dk, Dv, cols, tiles;     // value columns of a workgroup, workgroups of a row's head
    float scale;
    bool stream;                         // states past the caches
};

// A workgroup owns CW = 4 LN value columns of one (row, head): LN lanes side by side hold
// four columns each, the 256 / LN rows of lanes share out the state's rows, and their parts
// of o are added up in LDS.  All its state reads are under way before the first is used.
// Bound by the states' bytes: 256 rows, 16 heads of 128 x 64: 48 us for 272 MB, 5.6 TB/s.  One row: 4.4 us, the
// latency of a load, a sum through LDS and a store.
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
    const int64_t row = A.row0 + b / A.H;
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
                if constexpr (VEC) put(reinterpret_cast<f4*>(p), f4{s[i][0], s[i][1], s[i][2], s[i][3]}, A.stream);
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

constexpr int kOneSegment = 1024;   // tokens in all up to which every sequence is one segment

// Longest segment: as many segments as it takes to put about two workgroups on each compute unit (all
// that fit at a time; packed sequences end in half a segment on average), no shorter than 256 tokens: a
// segment's state makes four trips through memory.  Up to 1024 tokens in all, one segment a sequence.
// Packed prompt and backward (above) with one workgroup a compute unit 115 and 212 us, with two 85 and 188, with
// four and segments from 128 tokens 99 and 212; seven prompts of 1021 tokens in all 15 us, cut 19.5.  The last rule goes by the sum of
// tokens and costs a long sequence that comes alone: one prompt of 1000 tokens, 16 heads, 44 us, of 1088, cut in five, 24.
int plan_target(int64_t n_seq, int64_t T, int64_t H, int64_t Dv, bool packed) {
    if (T <= kOneSegment) return kOneSegment;
    const int64_t units = H * ((Dv + kV - 1) / kV);
    int64_t want = (2 * (int64_t)device_cu_count() + units - 1) / units;
    if (packed) want = std::max(want - n_seq / 2, (want + 1) / 2);
    int64_t len = (T + want - 1) / want;
    len = (len + kC - 1) / kC * kC;
    if (len < 256) len = 256;
    if (len > 1 << 20) len = 1 << 20;
    return (int)len;
}

struct Plan {
    int target, nseg, per_seq;
    bool single;        // packed, kOneSegment tokens at most: a workgroup's sequence is its number
    bool table;         // more other packed sequences than kLookThrough
    size_t states, seqs_at, longs_at, table_bytes;
    int da, n_long;
};

Plan make_plan(int64_t n_seq, int64_t T, int64_t H, int64_t Da, int64_t Dv, bool packed) {
    Plan p;
    p.target = plan_target(n_seq, T, H, Dv, packed);
    p.da = Da <= 64 ? 64 : 128;
    const int64_t L = T / n_seq;
    const bool several = packed ? T > p.target : L > p.target;
    p.single = packed && T <= kOneSegment;
    p.table = packed && !p.single && n_seq > kLookThrough;
    p.per_seq = packed ? 0 : several ? (int)((L + p.target - 1) / p.target) : 1;
    const int64_t nseg = !packed ? n_seq * p.per_seq : several ? T / p.target + n_seq : n_seq;
    p.nseg = (int)std::min<int64_t>(nseg, 0x7fffffff);
    const int64_t nst = packed ? std::min(nseg, 2 * T / p.target) : nseg;
    p.states = several ? (size_t)nst * H * ((Dv + kV - 1) / kV) * p.da * kV * 4 : 0;
    p.seqs_at = up256((size_t)nseg * sizeof(Seg));
    p.n_long = packed ? (int)std::min(n_seq, T / ((int64_t)kFewSegments * p.target + 1)) : p.per_seq > kFewSegments ? (int)n_seq : 0;
    p.longs_at = p.seqs_at + up256((size_t)n_seq * 8);
    p.table_bytes = p.table ? p.longs_at + up256((size_t)p.n_long * 4) : 0;
    return p;
}

bool sizes_ok(int64_t n_seq, int64_t T, int64_t H, int64_t G, int64_t Dk, int64_t Dv) {
    if (n_seq < 0 || T < 0 || H < 1 || G < 1 || H % G || H > 4096 || Dk < 1 || Dk > kMaxDim || Dv < 1 || Dv > kMaxDim) return false;
    if (n_seq > 1 << 20 || T >= (int64_t)1 << 31) return false;
    return true;
}

// A chunk's rows are addressed in 31 bits: 64 strides of four bytes.
bool strides_ok(int64_t stride, int64_t row) { return stride >= row && stride < 1 << 22; }

template <typename T, typename TO, int DA, bool VEC>
mb_status run_passes(const LaArgs& A, const SecondArgs* X, const Plan& p, hipStream_t s) {
    const auto launch = [&](auto kern, const auto&... more) -> mb_status {
        mb_status st = MB_OK;
        const int64_t per = segments_of_launch(A);
        for (int64_t at = 0; at < p.nseg && st == MB_OK; at += per) {
            LaArgs B = A;
            B.seg0 = (int)at;
            B.nseg = (int)std::min<int64_t>(at + per, p.nseg);
            hipLaunchKernelGGL(kern, dim3(grid_of(B)), dim3(kWalkThreads), 0, s, B, more...);
            st = check_launch();
        }
        return st;
    };
    if (p.states) {
        mb_status st = launch(k_la_state<T, DA, VEC>);
        if (st != MB_OK) return st;
        if (p.n_long) {
            const dim3 blocks((unsigned)((int64_t)p.n_long * A.H * A.nv * (DA * kV / 1024)));
            const int* longs = p.table ? (const int*)((const char*)A.plan + p.longs_at) : nullptr;
            hipLaunchKernelGGL(k_la_carry<DA>, blocks, dim3(256), 0, s, A, longs);
            if ((st = check_launch()) != MB_OK) return st;
        }
    }
    return X ? launch(k_la_dkdv<T, TO, DA, VEC>, *X) : launch(k_la_out<T, TO, DA, VEC>);
}

template <typename T, typename TO>
mb_status run_typed(const LaArgs& A, const SecondArgs* X, const Plan& p, hipStream_t s) {
    constexpr int VE = Frag<T>::VE, VO = 16 / sizeof(TO);
    bool vec = A.Da % VE == 0 && A.Dv % VE == 0 && A.Dv % VO == 0 && A.a_ts % VE == 0 && A.b_ts % VE == 0 && A.c_ts % VE == 0 &&
               al16(A.a) && al16(A.b) && al16(A.c) && al16(A.o);
    if (X) vec = vec && X->v_ts % VE == 0 && A.Da % VO == 0 && al16(X->v) && al16(X->dk);
    if (p.da == 64) return vec ? run_passes<T, TO, 64, true>(A, X, p, s) : run_passes<T, TO, 64, false>(A, X, p, s);
    return vec ? run_passes<T, TO, 128, true>(A, X, p, s) : run_passes<T, TO, 128, false>(A, X, p, s);
}

// Fills in what the plan says.
void use_plan(LaArgs& A, const Plan& p, char* ws) {
    A.nv = (A.Dv + kV - 1) / kV;
    A.target = p.target;
    A.nseg = p.nseg;
    A.per_seq = p.per_seq;
    A.single = p.single;
    A.plan = p.table ? (const Seg*)ws : nullptr;
    A.seqs = p.table ? (const int2*)(ws + p.seqs_at) : nullptr;
    A.states = p.states ? (float*)(ws + p.table_bytes) : nullptr;
}

// One run of the chunked form (with X: of both gradients); `out_f32` where heads' gradients are added up afterwards.
mb_status run(const LaArgs& A, const SecondArgs* X, const Plan& p, mb_dtype dtype, bool out_f32, hipStream_t s) {
    if (dtype == MB_F32) return run_typed<float, float>(A, X, p, s);
    return out_f32 ? run_typed<bf16, float>(A, X, p, s) : run_typed<bf16, bf16>(A, X, p, s);
}

mb_status launch_plan(LaArgs A, const Plan& p, char* ws, hipStream_t s) {
    if (!p.table) return MB_OK;
    A.plan = nullptr;
    hipLaunchKernelGGL(k_la_plan, dim3(1), dim3(64), 0, s, A, (Seg*)ws, (int2*)(ws + p.seqs_at), (int*)(ws + p.longs_at), p.n_long);
    return check_launch();
}

// The backward: one run for dq, and for dk and dv one walk over both where one of them is at most a
// column tile wide (that one takes the values' role), two runs otherwise.
struct BwdPlan {
    Plan q, k, v;          // k, v: both runs, or v the common one
    bool both, swapped;    // swapped: keys have the values' role
    size_t states, fold[2], total;
};

BwdPlan bwd_plan(int64_t n_seq, int64_t T, int64_t H, int64_t G, int64_t Dk, int64_t Dv, bool packed) {
    BwdPlan b;
    b.both = Dv <= kV || Dk <= kV;
    b.swapped = b.both && Dv > kV;
    b.q = make_plan(n_seq, T, H, Dv, Dk, packed);
    b.k = b.q;
    b.v = b.swapped ? b.q : make_plan(n_seq, T, H, Dk, Dv, packed);
    b.states = up256(std::max(b.q.table_bytes + b.q.states, b.v.table_bytes + b.v.states));
    const auto rows = [&](int64_t D) { return G < H ? up256((size_t)T * H * D * 4) : 0; };
    b.fold[0] = b.both ? rows(Dk) : rows(std::max(Dk, Dv));       // dk, or both one after the other
    b.fold[1] = b.both ? rows(Dv) : 0;
    b.total = b.states + b.fold[0] + b.fold[1];
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
    if (n_slots > 0x7fffffff) return MB_ERR_SHAPE;
    if (!strides_ok(q_stride, H * Dk) || !strides_ok(k_stride, G * Dk) || !strides_ok(v_stride, G * Dv)) return MB_ERR_SHAPE;
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
    A.n_seq = (int)n_seq; A.T = (int)T; A.L = (int)(T / n_seq);
    A.share = rep;
    A.cu = cu_seqlens;
    A.h0 = h0; A.has_h0 = has_h0; A.slots = slots; A.n_slots = n_slots;
    A.h_out = h_out;
    use_plan(A, p, (char*)ws);
    mb_status st = launch_plan(A, p, (char*)ws, stream);
    return st != MB_OK ? st : run(A, nullptr, p, dtype, false, stream);
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
    if (!strides_ok(q_stride, H * Dk) || !strides_ok(k_stride, G * Dk) || !strides_ok(v_stride, G * Dv)) return MB_ERR_SHAPE;
    if (!cu_seqlens && (n_seq ? T % n_seq : T) != 0) return MB_ERR_SHAPE;
    if (T == 0 && n_seq == 0) return MB_OK;
    if (!log_decay || (T > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv))) return MB_ERR_NULL;
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)q % es || (uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)d_o % es || (uintptr_t)dq % es ||
        (uintptr_t)dk % es || (uintptr_t)dv % es || ((uintptr_t)log_decay & 3) || ((uintptr_t)cu_seqlens & 3) ||
        ((uintptr_t)h0 & 3) || ((uintptr_t)dh_out & 3) || ((uintptr_t)dh0 & 3))
        return MB_ERR_ALIGN;
    const BwdPlan bp = n_seq ? bwd_plan(n_seq, T, H, G, Dk, Dv, cu_seqlens != nullptr) : BwdPlan{};
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
    float* fold_k = (float*)(w + bp.states);
    float* fold_v = bp.both ? (float*)(w + bp.states + bp.fold[0]) : fold_k;
    LaArgs A{};
    A.H = (int)H;
    A.log_decay = log_decay;
    A.n_seq = (int)n_seq; A.T = (int)T; A.L = n_seq ? (int)(T / n_seq) : 0;
    A.share = rep;
    A.cu = cu_seqlens;
    mb_status st;
    auto add_up = [&](const float* in, void* out, int64_t D) -> mb_status {
        const int64_t n = T * G * D;
        if (rep == 1 || n == 0) return MB_OK;
        const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 8192);
        if (dtype == MB_F32) hipLaunchKernelGGL(k_la_fold<float>, dim3(blocks), dim3(256), 0, stream, in, (float*)out, n, (int)G, rep, (int)D);
        else hipLaunchKernelGGL(k_la_fold<bf16>, dim3(blocks), dim3(256), 0, stream, in, (bf16*)out, n, (int)G, rep, (int)D);
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
    if (n_seq) use_plan(Q, bp.q, w);
    if (n_seq && ((st = launch_plan(Q, bp.q, w, stream)) != MB_OK || (st = run(Q, nullptr, bp.q, dtype, false, stream)) != MB_OK)) return st;
    // dk: queries v, keys do, values q, reversed; the state is R^T and holds the scale.
    LaArgs K = A;
    K.a = v; K.b = d_o; K.c = q; K.o = rep > 1 ? (void*)fold_k : dk;
    K.a_ts = v_stride; K.b_ts = H * Dv; K.c_ts = q_stride; K.o_ts = H * Dk;
    K.a_rep = rep; K.b_rep = K.c_rep = 1;
    K.Da = (int)Dv; K.Dv = (int)Dk;
    K.s_in = K.s_up = scale; K.s_carry = 1.0f;
    K.shift = 0; K.reversed = 1;
    K.h0 = dh_out; K.transposed = 1;
    // dv: queries k, keys q, values do, reversed; the state is R.  The end of the state is the gradient of h0.
    LaArgs V = K;
    V.a = k; V.b = q; V.c = d_o; V.o = rep > 1 ? (void*)fold_v : dv;
    V.a_ts = k_stride; V.b_ts = q_stride; V.c_ts = H * Dv; V.o_ts = H * Dv;
    V.Da = (int)Dk; V.Dv = (int)Dv;
    V.transposed = 0;
    if (!n_seq) {
        // no sequence: the gradients of all tokens are zero, below
    } else if (bp.both) {
        LaArgs& B = bp.swapped ? K : V;
        const LaArgs& o = bp.swapped ? V : K;
        const SecondArgs X{o.a, o.o, o.a_ts, o.o_ts, o.a_rep};
        B.h_out = dh0;
        use_plan(B, bp.v, w);
        if ((st = launch_plan(B, bp.v, w, stream)) != MB_OK || (st = run(B, &X, bp.v, dtype, rep > 1, stream)) != MB_OK ||
            (st = add_up(fold_k, dk, Dk)) != MB_OK || (st = add_up(fold_v, dv, Dv)) != MB_OK)
            return st;
    } else {
        use_plan(K, bp.k, w);
        if ((st = run(K, nullptr, bp.k, dtype, rep > 1, stream)) != MB_OK || (st = add_up(fold_k, dk, Dk)) != MB_OK) return st;
        V.h_out = dh0;
        use_plan(V, bp.v, w);
        if ((st = launch_plan(V, bp.v, w, stream)) != MB_OK || (st = run(V, nullptr, bp.v, dtype, rep > 1, stream)) != MB_OK ||
            (st = add_up(fold_v, dv, Dv)) != MB_OK)
            return st;
    }
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
    if (!strides_ok(q_stride, H * Dk) || !strides_ok(k_stride, G * Dk) || !strides_ok(v_stride, G * Dv)) return MB_ERR_SHAPE;
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
    StepArgs A{q, k, v, log_decay, slots, h_in, h_out, o, 0, n_slots, q_stride, k_stride, v_stride,
               (int)H, (int)(H / G), (int)Dk, (int)Dv, 0, 0, scale, (size_t)n * H * Dk * Dv * 8 > kStreamBytes};
    // Few rows: narrow column tiles, so that the one token's states are read by more compute
    // units (one row of 16 heads: 4.4 us, with wide tiles 5.3); many rows: a tile as wide as a row of the
    // state (256 rows: 46.6 us, with narrow tiles 79.5).
    const bool few = n * H < 2 * device_cu_count();
    const int ln = few ? 4 : 16, cpl = vec ? 4 : 1;
    A.cols = ln * cpl;
    A.tiles = (int)((Dv + A.cols - 1) / A.cols);
    const auto go = [&](auto kern) -> mb_status {
        const int64_t per = max_workgroups(256) / (H * A.tiles);     // rows of a launch
        mb_status st = MB_OK;
        for (; A.row0 < n && st == MB_OK; A.row0 += per) {
            hipLaunchKernelGGL(kern, dim3((unsigned)(std::min(per, n - A.row0) * H * A.tiles)), dim3(256), 0, stream, A);
            st = check_launch();
        }
        return st;
    };
    if (dtype == MB_F32) {
        if (vec) return few ? go(k_la_step<float, 4, true>) : go(k_la_step<float, 16, true>);
        return few ? go(k_la_step<float, 4, false>) : go(k_la_step<float, 16, false>);
    }
    if (vec) return few ? go(k_la_step<bf16, 4, true>) : go(k_la_step<bf16, 16, true>);
    return few ? go(k_la_step<bf16, 4, false>) : go(k_la_step<bf16, 16, false>);
}
