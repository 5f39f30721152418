// gatedscan.hip -- gated linear recurrence with a decay per channel and token, its single-token step and its backward.
//
//     s = sigma(a_gate + a_bias), la = -decay s, a = e^la, beta = sqrt(1 - a^2)
//     b = beta sigma(x_gate + x_bias) x,  h_t = a_t h_{t-1} + b_t,  y = h
//     backward: G_t = dy_t + a_{t+1} G_{t+1}, and every gradient a product of G_t and what the token's gates give
//
// A span of tokens acts on the state that enters it as h -> e^S h + U, S the sum of its la, and two spans one behind the other as
// (S1 + S2, e^S2 U1 + U2).  The tokens of all sequences, one after another, are cut into tiles of 128 (backward: 64)
// tokens by 64 channels.  A workgroup reads its tile once, keeps a and b in registers, makes the tile's (S, U), hands it
// to the tiles behind it, takes the state that enters from those in front, and walks its tokens a second time in registers:
// one pass over memory, where cutting the sequence into a pass for end states and one for outputs reads everything twice.
//
// Handing on.  Workgroups take their tile from a counter, so that every tile in front of a taken one has been taken by a workgroup that
// runs; a wait for a tile in front therefore ends.  A tile publishes (S, U) for each channel in one 64-bit store, which
// readers poll until it is no longer the pattern that the first launch left there.  16 tiles make a group, whose last
// tile also publishes the state behind it (and with few columns the group's (S, U)).  The state that enters a tile is composed of the state
// behind the group before and the (S, U) of the group's tiles in front, always in this order: results do not depend on who came first.
// Tiles in front of the one in which the first token's sequence starts are not looked at.
//
// What bounds it: bytes (12 of x and gates and 4 of y a token and channel in fp32, half of it in bf16, once each), and beside them the
// gates' transcendentals and the waits for states, which four workgroups a compute unit hide in part.  Here and below: times of the kernel
// alone.  16384 packed tokens of 1536 bf16 channels, columns of one projection: 58 to 59 us for 201 MB, 3.4 TB/s (when it took 57, the
// loads and stores alone took 39, the gates 5 to 8, counters 3, waits for tiles in front 6 to 10; a pass for end states and one for
// outputs read 151 MB twice); one sequence of contiguous tensors 53.  65536 tokens of 768: 101 to 104 us, 403 MB.  The backward of 8 x 2048 by
// 1536: 109 us for 352 MB, 3.2 TB/s.  Few channels leave most of the card idle: 131072 tokens of 64 channels 37 us for 67 MB, their
// backward 64 for 117.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "mb_internal.h"

namespace mb {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

constexpr int kEvery = 64;                  // tokens between the rows of states
constexpr int kCols = 64;                   // channels of a tile
constexpr int kTile = 128, kTileBack = 64;  // its tokens, forward and backward
constexpr int kPer = 16, kPerBack = 8;      // tokens of a thread
constexpr int kGroup = 16;                  // tiles of a group, groups of a group of groups
constexpr int kDeep = 6;                    // columns up to which a group's last tile looks further (DEEP)
template <bool DEEP> constexpr int kLook = DEEP ? 2 * kGroup : kGroup;       // words that a tile looks at
constexpr int kCounter = 32;                // words between the counters of two columns
constexpr uint64_t kNone = ~0ull;           // not published yet
// Polls of one wait before it is given up: some seconds.  What was waited for counts as NaN then, in outputs and end states, and the
// call has returned MB_OK long before.  A workspace that something else writes to at the same time brings it about, and so would a
// workgroup of an earlier tile that is held up for as long (by a debugger, or where several processes share the card).
constexpr int kPolls = 1 << 22;

// What the tiles of one direction hand on to each other, in the workspace.
struct Chain {
    uint64_t* agg;       // (tiles, columns): (S, U) of a tile
    uint64_t* gagg;      // (groups, columns): (S, U) of a group
    uint32_t* incl;      // (groups, columns): the state behind a group
    int* first;          // (tiles + 1): the last offset of cu at or before the tile's first token
    uint32_t* ticket;
};

struct GsArgs {
    const void *x, *a, *g;
    int64_t x_ts, a_ts, g_ts;
    const float *decay, *a_bias, *x_bias;
    const int32_t* cu;
    const float* h0;
    const uint8_t* has_h0;
    const int32_t* slots;
    int64_t n_slots;
    void* y;
    float *h_out, *states;
    const void* dy;
    const float *dh_out, *kept;
    void *dx, *da, *dg;
    float *dh0, *part;
    int n_seq, T, L, D;
    int tiles, cols;     // tiles along the tokens, columns of tiles
    Chain ch;
};

// ---------------------------------------------------------------- gates ----
// Logarithms are held in base 2: x2 = la log2(e).
struct Gate {
    float x2, a, less, beta;     // less = 1 - a^2
};

// e^la - 1 next to zero, from x2 = la log2(e): the series of 2^x - 1, off by x^6 / 5040 of itself at |la| = 1/4, 2^-24.3.
// Further away 2^x - 1 loses two bits at most.
__device__ __forceinline__ float less_one(float x2, float a) {
    float p = fmaf(x2, 1.5403530394e-4f, 1.3333558146e-3f);
    p = fmaf(x2, p, 9.6181291076e-3f);
    p = fmaf(x2, p, 5.5504108665e-2f);
    p = fmaf(x2, p, 2.4022650696e-1f);
    p = fmaf(x2, p, 6.9314718056e-1f);
    return x2 > -0.36f ? p * x2 : a - 1.0f;
}

// s: sigma of the gate; nd: -decay log2(e).
__device__ __forceinline__ Gate gate(float s, float nd) {
    Gate r;
    r.x2 = nd * s;
    r.a = exp2_fast(r.x2);
    const float e = less_one(r.x2, r.a);
    r.less = -e * (2.0f + e);
    r.beta = __builtin_amdgcn_sqrtf(r.less);
    return r;
}

// e^-(v + bias), nb = -bias log2(e)
__device__ __forceinline__ float exp_minus(float v, float nb) { return exp2_fast(fmaf(v, -kLog2e, nb)); }
__device__ __forceinline__ float sigma(float v, float nb) { return __builtin_amdgcn_rcpf(1.0f + exp_minus(v, nb)); }

// sigma and 1 - sigma, both with all their digits.  The bound keeps e^-v finite (and NaN as it is).
__device__ __forceinline__ void sigma2(float v, float nb, float& s, float& not_s) {
    const float e = __builtin_elementwise_minimum(exp_minus(v, nb), 0x1p120f);
    s = __builtin_amdgcn_rcpf(1.0f + e);
    not_s = e * s;
}

// --------------------------------------------------------------- memory ----
// A thread's two channels: beside each other where both can be read at a time (PAIR: they start on a border of two elements everywhere),
// otherwise half a tile apart, so that a row's threads read neighbouring elements with each of two reads.  16384 tokens of 1001 bf16
// channels, forward and backward: channels beside each other, read one by one, 63 and 129 us, half a tile apart 49 and 121 (pairs from odd
// addresses 64 forward, where half a tile apart then took 52).
// PAIR: 0 half a tile apart, 1 pairs, 2 pairs whose tiles' rows are whole lines of memory, 128 bytes.  Those are read past the caches; lines
// that two tiles share are not.  16384 tokens of 1536 bf16 channels (whole lines): forward 53 us past the caches and 55.5 through
// them, backward 107 and 112; of 1000 (shared): 48.5 and 46.5, backward 87 both ways; 8192 of 1530 fp32 channels (shared): 50.5 and 52.5,
// 86 and 91, the one kind that reading past the caches would serve better.
template <int PAIR> constexpr int kNext = PAIR ? 1 : kCols / 2;
template <int PAIR> __device__ __forceinline__ int first_channel() { return (threadIdx.x & 31) * (PAIR ? 2 : 1); }
template <int PAIR> __device__ __forceinline__ int channels_of(int D, int c) { return (c < D) + (c + kNext<PAIR> < D); }

// Two channels as they come from memory.
template <typename T> struct Raw;
template <> struct Raw<bf16> {
    typedef uint32_t type;
    static __device__ __forceinline__ type open() { return 0x7f807f80u; }
};
template <> struct Raw<float> {
    typedef f2 type;
    static __device__ __forceinline__ type open() { return f2{__builtin_inff(), __builtin_inff()}; }
};

__device__ __forceinline__ float half_of(uint32_t v, int i) { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
__device__ __forceinline__ float half_of(f2 v, int i) { return v[i]; }

// `n` rows of a tile as a buffer: what lies outside reads zero.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const void* p, int64_t t0, int64_t ts, int n, int D) {
    // The same in all lanes, and known to be: a descriptor in vector registers costs a loop for every access.
    n = __builtin_amdgcn_readfirstlane(n);
    int row0 = __builtin_amdgcn_readfirstlane((int)t0);
    asm("" : "+s"(n), "+s"(row0));
    const uint32_t bytes = n > 0 ? (uint32_t)(n - 1) * (uint32_t)ts * sizeof(T) + (uint32_t)D * sizeof(T) : 0;
    return __builtin_amdgcn_make_buffer_rsrc((void*)((const T*)p + (int64_t)row0 * ts), 0, (int)bytes, 0x00027000);
}

// `row`: the same in all lanes, a scalar operand (a sum in a vector register for each row would be held over the whole walk); the
// buffer's range holds for the sum.  PAIR: two channels start on a border of two elements.
template <typename T, int PAIR>
__device__ __forceinline__ typename Raw<T>::type load2(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t row) {
    constexpr int kAux = PAIR == 2 ? 2 : 0;          // non-temporal
    if constexpr (sizeof(T) == 2) {
        if constexpr (PAIR) return __builtin_amdgcn_raw_buffer_load_b32(r, off, row, kAux);
        const uint32_t lo = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, row, 0);
        const uint32_t hi = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off + 2 * kNext<PAIR>, row, 0);
        return lo | hi << 16;
    } else {
        if constexpr (PAIR) return __builtin_bit_cast(f2, __builtin_amdgcn_raw_buffer_load_b64(r, off, row, kAux));
        f2 v;
        v[0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, row, 0));
        v[1] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off + 4 * kNext<PAIR>, row, 0));
        return v;
    }
}

// Where two channels of a thread are stored: channels that are not there lie outside every buffer.
struct Place2 {
    uint32_t lo, hi;
};
constexpr uint32_t kNowhere = 0x80000000u;

template <typename T, int PAIR>
__device__ __forceinline__ Place2 place2(uint32_t off, int live) {
    return Place2{live > 0 ? off : kNowhere, live > 1 ? off + (uint32_t)sizeof(T) * kNext<PAIR> : kNowhere};
}

// Rounds to nearest even.
template <typename T, int PAIR>
__device__ __forceinline__ void store2(__amdgpu_buffer_rsrc_t r, Place2 at, uint32_t row, float lo, float hi) {
    if constexpr (sizeof(T) == 2) {
        const f2 v = {lo, hi};
        const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
        if constexpr (PAIR) {
            __builtin_amdgcn_raw_buffer_store_b32(w, r, at.lo, row, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b16((short)(w & 0xffffu), r, at.lo, row, 0);
            __builtin_amdgcn_raw_buffer_store_b16((short)(w >> 16), r, at.hi, row, 0);
        }
    } else {
        if constexpr (PAIR) {
            typedef uint32_t u2 __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(u2{__float_as_uint(lo), __float_as_uint(hi)}, r, at.lo, row, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(lo), r, at.lo, row, 0);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(hi), r, at.hi, row, 0);
        }
    }
}

// A barrier for what waves share through LDS: loads and stores to memory stay under way.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);          // lgkmcnt(0), no other counter
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ------------------------------------------------------------ sequences ----
__device__ __forceinline__ int offset_at(const GsArgs& A, int i) { return min(max(A.cu[i], 0), A.T); }

// Tokens of sequence s.
__device__ __forceinline__ void range_of(const GsArgs& A, int s, int& b, int& e) {
    if (A.cu) {
        b = offset_at(A, s);
        e = offset_at(A, s + 1);
    } else {
        b = s * A.L;
        e = b + A.L;
    }
}

// Row of h0 and h_out of a sequence, or -1 where it has none.
__device__ __forceinline__ int row_of(const GsArgs& A, int s) {
    if (!A.slots) return s;
    const int r = A.slots[s];
    return r >= 0 && r < A.n_slots ? r : -1;
}

// A tile's place, the same in all threads.
struct Place {
    int t0, n;           // first token, tokens
    int sa, sb;          // sequences that may begin or end in it
    int src;             // tile in which the first (backward: last) token's sequence begins (ends); its own: nothing enters
    int lo, hi;          // its tokens that belong to a sequence
    bool plain;          // all its tokens belong to one sequence that neither begins nor ends in it
};

template <int TT, bool BACK>
__device__ __forceinline__ Place place(const GsArgs& A, int j) {
    Place p;
    p.t0 = j * TT;
    p.n = min(A.T - p.t0, TT);
    p.lo = 0;
    p.hi = p.n;
    p.src = j;
    const int end = p.t0 + p.n;
    if (A.cu) {
        int f0 = -1, f1 = A.n_seq;
        if (A.tiles > 1) {
            f0 = A.ch.first[j];
            f1 = min(A.ch.first[j + 1], A.n_seq);
        }
        p.sa = j == 0 ? 0 : max(f0, 0);
        p.sb = min(f1, A.n_seq - 1);
        p.plain = f0 == f1 && f0 >= 0 && f0 < A.n_seq && offset_at(A, f0) < p.t0 && p.n == TT;
        if (!p.plain) {
            p.lo = max(offset_at(A, 0) - p.t0, 0);
            p.hi = min(offset_at(A, A.n_seq) - p.t0, p.n);
        }
        if constexpr (BACK) {
            // the sequence of the last token: f1, but where it begins right behind the tile
            if (j + 1 < A.tiles && f1 >= 0) {
                int s = f1;
                if (offset_at(A, f1) >= end) s = -1;      // another one begins there: the last token ends its own
                if (s >= 0 && s < A.n_seq) p.src = max((offset_at(A, s + 1) - 1) / TT, j);
            }
        } else if (f0 >= 0 && f0 < A.n_seq) {
            p.src = min(offset_at(A, f0) / TT, j);
        }
    } else if (A.L == 0) {
        p.sa = 0;
        p.sb = A.n_seq - 1;
        p.plain = false;
    } else {
        p.sa = p.t0 / A.L;
        p.sb = (end - 1) / A.L;
        p.plain = p.sa == p.sb && p.sa * A.L < p.t0 && (p.sb + 1) * (int64_t)A.L > end && p.n == TT;
        p.src = BACK ? (int)(((p.sb + 1) * (int64_t)A.L - 1) / TT) : p.sa * A.L / TT;
    }
    return p;
}

// Where sequences begin and end in a tile: a bit for each of a group's tokens, and the rows (-1: none) of the sequences that begin and end.
template <int TT, int NG>
struct Events {
    uint32_t begins[NG], ends[NG];
    int begin[TT], end[TT];
};

// Fills them in, all threads together, a sequence each, and settles the sequences of no tokens: their `from` rows, or zeros, go to `to`, four
// rows of the column's 64 channels at a time in a wave (offsets padded to a thousand sequences and more are all in one tile).  BACK: rows
// are the sequences' numbers, and behind the last sequence one of no row begins, which keeps that one's state from the tokens there.
template <int TT, int NG, bool BACK>
__device__ __forceinline__ void find_events(const GsArgs& A, const Place& p, Events<TT, NG>& ev, int col, const float* from, float* to) {
    constexpr int K = TT / NG;
    const int lane = threadIdx.x & 63;
    if (threadIdx.x < NG) ev.begins[threadIdx.x] = ev.ends[threadIdx.x] = 0;
    lds_barrier();
    if (BACK && threadIdx.x == 0 && p.hi > 0 && p.hi < TT) {
        ev.begin[p.hi] = -1;
        atomicOr(&ev.begins[p.hi / K], 1u << p.hi % K);
    }
    for (int s0 = p.sa; s0 <= p.sb; s0 += NG * 32) {
        const int s = s0 + (int)threadIdx.x;
        int row = -1;
        bool has = false, copy = false;
        if (s <= p.sb) {
            int b, e;
            range_of(A, s, b, e);
            row = BACK ? s : row_of(A, s);
            has = BACK || (row >= 0 && A.h0 && (!A.has_h0 || A.has_h0[s]));
            copy = b >= e && to && row >= 0 && !(has && from == to);
            if (b < e) {
                b -= p.t0;
                e -= p.t0 + 1;
                if (b >= 0 && b < p.n) {
                    ev.begin[b] = has ? row : -1;
                    atomicOr(&ev.begins[b / K], 1u << b % K);
                }
                if (e >= 0 && e < p.n) {
                    ev.end[e] = row;
                    atomicOr(&ev.ends[e / K], 1u << e % K);
                }
            }
        }
        const uint64_t rows = __ballot(copy);
        const int with = (has && from) ? row : ~row;       // below zero: zeros
        for (int i = 0; i < 64; i += 4) {
            if ((rows >> i & 0xf) == 0) continue;
            const int src = i + (lane >> 4), r = __shfl(with, src), c = col * kCols + (lane & 15);
            if (!(rows >> src & 1)) continue;
            const int64_t at = (int64_t)(r < 0 ? ~r : r) * A.D + c;
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = r >= 0 && c + 16 * k < A.D ? from[at + 16 * k] : 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + 16 * k < A.D) to[at + 16 * k] = v[k];
        }
    }
    lds_barrier();
}

// -------------------------------------------------------------- handing on ----
__device__ __forceinline__ uint64_t peek(const uint64_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint32_t peek(const uint32_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// One NaN for all: none looks like kNone.
__device__ __forceinline__ uint32_t plain_bits(float v) { return v == v ? __float_as_uint(v) : 0x7fc00000u; }

__device__ __forceinline__ uint64_t word_of(float S, float U) { return (uint64_t)plain_bits(S) | (uint64_t)plain_bits(U) << 32; }

// Row `i` of a table of words, at channel c.
__device__ __forceinline__ void publish(const GsArgs& A, uint64_t* table, int i, int c, uint64_t w) {
    __hip_atomic_store(table + (int64_t)i * A.cols * kCols + c, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void publish_state(const GsArgs& A, int i, int c, float h) {
    __hip_atomic_store(A.ch.incl + (int64_t)i * A.cols * kCols + c, plain_bits(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The words that tile j of the chain (tiles counted in walking order, its sequence from tile `src` on) looks at.  Rows 0 to 14: the tiles
// of its group in front of it, from `tile` on.  Row 15: the state behind the group before.  States are so handed on from group to group, one
// after the other, 1.4 us each, which with few columns takes longer than memory.  DEEP: a group's last tile (`last`) does not wait for that
// state.  Its rows 16 to 30 are the groups of its group of groups in front of its own, from `group` on, row 31 the state behind the group of
// groups before.  One sequence, bf16, group by group and DEEP, us:
//     131072 tokens of    64 channels 122 and 37, 128 118 and 48, 256 126 and 79, 384 134 and 107, 512 170 and 160, 640 161 and 168
//     backward                        222 and 64,     225 and 98,     247 and 173,    264 and 249,    320 and 345,    355 and 399
//     16384 tokens of     64 channels 21.5 and 13.9, 384 27.5 and 22.2, 512 28.8 and 24.9;  backward 37 and 19, 48 and 45, 47 and 50
//     2048 tokens of      64 channels 10.5 and 11.4, 384 10.6 and 11.4;                     backward 12.8 and 14.6, 14 and 15
// 32 sequences of 2048 tokens of 64 channels 20 and 21, of 384 57 and 58, backward 39 and 41, 122 and 131.  One border (kDeep) serves both
// directions and every length: the forward would gain up to 512 channels, and short sequences lose a little by it.
template <bool DEEP>
struct Look {
    int j, src, tile, group;
    bool last, far;              // far: the sequence comes from another group
    __device__ __forceinline__ Look(int j_, int src_) : j(j_), src(src_) {
        tile = max(src, j / kGroup * kGroup);
        group = max(src / kGroup, j / (kGroup * kGroup) * kGroup);
        last = DEEP && j % kGroup == kGroup - 1;
        far = src < j / kGroup * kGroup;
    }
    __device__ __forceinline__ bool state() const { return src < j / (kGroup * kGroup) * (kGroup * kGroup); }
};

// All waves fetch the rows of tiles (HIGH: of groups), and wait for those that are not published yet.
template <int NW, bool HIGH, bool DEEP>
__device__ __forceinline__ void fetch_look(const GsArgs& A, const Look<DEEP>& q, int col, uint64_t (*look)[kCols]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t row = (int64_t)A.cols * kCols;
    const uint64_t* words = (HIGH ? A.ch.gagg + q.group * row : A.ch.agg + q.tile * row) + col * kCols;
    const int n_words = HIGH ? q.j / kGroup - q.group : q.j - q.tile, before = HIGH ? q.j / (kGroup * kGroup) * kGroup : q.j / kGroup;
    const uint32_t* incl = A.ch.incl + (before - 1) * row + col * kCols;
    const bool state = HIGH ? q.state() : q.far && !q.last;
    if (HIGH) look += kGroup;
    int polls = 0;
    const auto read = [&](int i) -> uint64_t {
        if (i < kGroup - 1) return i < n_words ? peek(words + i * row + lane) : 0;
        const uint32_t v = state ? peek(incl + lane) : 0;
        return v == (uint32_t)kNone ? kNone : v;
    };
    // All reads are under way at a time; what came too early is read again, one word after the other.
    constexpr int N = kGroup / NW;
    uint64_t w[N];
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = read(wave + n * NW);
#pragma unroll
    for (int n = 0; n < N; ++n) look[wave + n * NW][lane] = w[n];
#pragma unroll 1
    for (int i = wave; i < kGroup; i += NW) {
        uint64_t v = look[i][lane];
        if (v != kNone) continue;
        while (v == kNone && ++polls < kPolls) {
            __builtin_amdgcn_s_sleep(1);
            v = read(i);
        }
        look[i][lane] = v;
    }
}

__device__ __forceinline__ float low(uint64_t w) { return __uint_as_float((uint32_t)w); }
__device__ __forceinline__ float high(uint64_t w) { return __uint_as_float((uint32_t)(w >> 32)); }

// (S, U) of the group that ends with tile j, whose own is `own`: from the first tile of the sequence that goes on behind it; `cut`: which
// begins in tile j.
template <bool DEEP>
__device__ __forceinline__ uint64_t compose_group(const Look<DEEP>& q, uint64_t own, bool cut, const uint64_t (*look)[kCols]) {
    const int lane = threadIdx.x & 63;
    float S = 0.0f, U = 0.0f;
#pragma unroll 4
    for (int i = 0; q.tile + i < q.j; ++i) {
        const uint64_t w = look[i][lane];
        S += low(w);
        U = q.src == q.tile + i ? high(w) : fmaf(exp2_fast(low(w)), U, high(w));
    }
    return cut || q.src == q.j ? own : word_of(S + low(own), fmaf(exp2_fast(low(own)), U, high(own)));
}

// The state that enters tile j.
template <bool DEEP>
__device__ __forceinline__ float compose(const Look<DEEP>& q, const uint64_t (*look)[kCols]) {
    const int lane = threadIdx.x & 63;
    float h = 0.0f;
    if (q.far && !q.last) h = low(look[kGroup - 1][lane]);
    if constexpr (DEEP) {
        if (q.far && q.last) {
            if (q.state()) h = low(look[kLook<DEEP> - 1][lane]);
#pragma unroll 4
            for (int i = 0; q.group + i < q.j / kGroup; ++i) {
                const uint64_t w = look[kGroup + i][lane];
                h = q.src / kGroup == q.group + i ? high(w) : fmaf(exp2_fast(low(w)), h, high(w));
            }
        }
    }
#pragma unroll 4
    for (int i = 0; q.tile + i < q.j; ++i) {
        const uint64_t w = look[i][lane];
        h = q.src == q.tile + i ? high(w) : fmaf(exp2_fast(low(w)), h, high(w));
    }
    return h;
}

// Fetches what tile j looks at; all threads together.  A group's last tile hands the group's (S, U) on before it waits for other groups'; its
// own, `own`, is with the first 64 threads.
template <int NW, bool DEEP>
__device__ __forceinline__ void look_back(const GsArgs& A, const Look<DEEP>& q, int col, uint64_t own, bool cut, uint64_t (*look)[kCols]) {
    if (q.src < q.j) fetch_look<NW, false>(A, q, col, look);
    if constexpr (DEEP) {
        if (q.last) {
            lds_barrier();
            if (threadIdx.x < kCols) publish(A, A.ch.gagg, q.j / kGroup, col * kCols + threadIdx.x, compose_group(q, own, cut, look));
            if (q.far) fetch_look<NW, true>(A, q, col, look);
        }
    }
    lds_barrier();
}

__host__ __device__ __forceinline__ int64_t groups_of(int64_t tiles) { return (tiles + kGroup - 1) / kGroup; }

// Clears what the chains hand on and finds every tile's place among the offsets.  A launch of its own, 5 us behind another kernel's large
// writes (2.5 behind small ones): nothing of a chain may be taken before all of it is clear.
struct Setup {
    Chain ch[2];
    int tiles[2], tokens[2];     // 0 tiles: no chain
    const int32_t* cu;
    int n_seq, T, columns;
};

__global__ void __launch_bounds__(256) k_gs_setup(Setup S) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (S.tiles[k] < 2) continue;
        const int64_t words = (int64_t)S.tiles[k] * S.columns, groups = groups_of(S.tiles[k]) * S.columns;
        for (int64_t i = i0; i < words; i += step) S.ch[k].agg[i] = kNone;
        for (int64_t i = i0; i < groups; i += step) {
            S.ch[k].gagg[i] = kNone;
            S.ch[k].incl[i] = (uint32_t)kNone;
        }
        for (int64_t i = i0; i < S.columns / kCols; i += step) S.ch[k].ticket[i * kCounter] = 0;
        if (S.cu && S.n_seq < 64) {
            // one look at all offsets, a lane each
            const int lane = threadIdx.x & 63;
            const int own = lane <= S.n_seq ? min(max(S.cu[lane], 0), S.T) : 0x7fffffff;
            for (int64_t i = i0 >> 6; i <= S.tiles[k]; i += step >> 6) {
                const int n = __popcll(__ballot(own <= i * S.tokens[k]));
                if (lane == 0) S.ch[k].first[i] = n - 1;
            }
        } else if (S.cu)
            for (int64_t i = i0; i <= S.tiles[k]; i += step) {
                const int64_t t = i * S.tokens[k];
                int lo = 0, hi = S.n_seq + 1;              // offsets at or before t
                while (lo < hi) {
                    const int m = (lo + hi) >> 1;
                    if (min(max(S.cu[m], 0), S.T) <= t) lo = m + 1;
                    else hi = m;
                }
                S.ch[k].first[i] = lo - 1;
            }
    }
}

// A workgroup has a column by its number, and takes the column's tiles, in walking order, from a counter: the least unfinished one is
// then always in work.  One counter for all columns is slower: their adds come one after the other at one address, 12 us of the 73
// that 16384 tokens of 1536 bf16 channels took with it; with a counter each, 128 bytes apart, 3 to 5.
// Workgroups go to the eight dies in turn: a die, or two or four together where eight does not divide the columns, has columns that lie
// beside each other, whose rows share lines where they are not aligned and pages of memory everywhere.  Against column b % cols, 16384
// tokens of 1536 bf16 channels in 8 sequences: forward 52.6 and 51.1 us, backward 107 and 104; 16380 tokens of 1001 fp32 channels 71.1
// and 70.0, backward 139 and 128.
__device__ __forceinline__ int column_of(const GsArgs& A) {
    const uint32_t b = blockIdx.x, cols = A.cols, shift = cols & 1 ? 0 : cols & 2 ? 1 : cols & 4 ? 2 : 3, per = cols >> shift;
    return (int)((b & ((1u << shift) - 1)) * per + (b >> shift) % per);
}

// The bound holds it in range where something else writes to the workspace at the same time.
__device__ __forceinline__ int take(const GsArgs& A, int col) {
    if (A.tiles == 1) return 0;
    const uint32_t j = __hip_atomic_fetch_add(A.ch.ticket + col * kCounter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return (int)min(j, (uint32_t)A.tiles - 1);
}

// -decay log2(e) and the biases times -log2(e) of two channels; those behind the last are zero.
template <int PAIR>
struct Params {
    float nd[2], nab[2], nxb[2];
    __device__ __forceinline__ void load(const GsArgs& A, int c, int live) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = i < live;
            const int at = c + i * kNext<PAIR>;
            nd[i] = in ? -A.decay[at] * kLog2e : 0.0f;
            nab[i] = in && A.a_bias ? -A.a_bias[at] * kLog2e : 0.0f;
            nxb[i] = in && A.x_bias ? -A.x_bias[at] * kLog2e : 0.0f;
        }
    }
};

// A thread's K tokens of several tensors, token by token: work on the first ones begins while the others are on their way.
template <typename T>
struct Source {
    __amdgpu_buffer_rsrc_t rows;
    uint32_t off, step;
    __device__ __forceinline__ Source(const void* p, int64_t t0, int64_t ts, int n, int D, int first, int c) {
        rows = rows_at<T>(p, t0, ts, n, D);
        step = (uint32_t)ts * sizeof(T);
        off = first * step + c * sizeof(T);
    }
    template <int PAIR>
    __device__ __forceinline__ typename Raw<T>::type get(int k) const {
        return load2<T, PAIR>(rows, off, k * step);
    }
};

// -------------------------------------------------------------- forward ----
// A thread holds K tokens of two channels; 32 threads side by side make a group's rows of 64 channels, NG groups the tile.
// OUT: outputs and end states are written; otherwise the states for the backward alone.
// Four workgroups a compute unit; three where fp32 channels come in pairs, whose registers would not hold it all otherwise (16384 tokens of
// 2048 channels 113 us with four and 24 bytes of scratch, 106 with three; 8192 of 1536 48.8 and 44.7).
template <typename T, int PAIR, int K, bool OUT, bool DEEP>
__global__ void __launch_bounds__(kTile / K * 32, sizeof(T) == 4 && PAIR ? 3 : 4) k_gs_forward(GsArgs A) {
    constexpr int NG = kTile / K, NX = kNext<PAIR>;
    __shared__ f2 comp[NG][kCols];
    __shared__ float entry[NG][kCols];
    __shared__ uint64_t look[kLook<DEEP>][kCols];
    __shared__ Events<kTile, NG> ev;
    __shared__ int taken;
    const int c2 = first_channel<PAIR>(), grp = threadIdx.x >> 5;
    typename Raw<T>::type rx[K], ra[K], rg[K];
    Params<PAIR> par;
    const int col = column_of(A);
    if (threadIdx.x == 0) taken = take(A, col);
    __syncthreads();
    const int j = __builtin_amdgcn_readfirstlane(taken);
    {
        const int c = col * kCols + c2, live = channels_of<PAIR>(A.D, c);          // channels of this thread
        {
            const int t0 = j * kTile, n = min(A.T - t0, kTile);
            par.load(A, c, live);
            const Source<T> sa(A.a, t0, A.a_ts, n, A.D, grp * K, c), sx(A.x, t0, A.x_ts, n, A.D, grp * K, c);
            const Source<T> sg(A.g, t0, A.g_ts, A.g ? n : 0, A.D, grp * K, c);
            if (A.g) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    ra[k] = sa.template get<PAIR>(k);
                    rg[k] = sg.template get<PAIR>(k);
                    rx[k] = sx.template get<PAIR>(k);
                }
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    ra[k] = sa.template get<PAIR>(k);
                    rg[k] = Raw<T>::open();           // infinity: a gate of exactly one
                    rx[k] = sx.template get<PAIR>(k);
                }
            }
        }
        const Place p = place<kTile, false>(A, j);
        uint32_t begins = 0, ends = 0;         // of this thread's tokens: first and last ones of a sequence
        if (!p.plain) {
            find_events<kTile, NG, false>(A, p, ev, col, A.h0, OUT ? A.h_out : nullptr);
            begins = ev.begins[grp];
            ends = ev.ends[grp];
        }
        float a[K][2], b[K][2], S[2] = {0.0f, 0.0f}, U[2] = {0.0f, 0.0f};        // (S, U) of this thread's tokens
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const Gate q = gate(sigma(half_of(ra[k], i), par.nab[i]), par.nd[i]);
                const float x = half_of(rx[k], i);
                a[k][i] = q.a;
                b[k][i] = q.beta * sigma(half_of(rg[k], i), par.nxb[i]) * x;
                S[i] += q.x2;
            }
        // A first token's b takes in what its h0 gives, and its a is marked by -1: nothing of the token before.  This is the only read
        // of h0: a row that is updated in place may be written by the thread that holds its last token.
        for (uint32_t m = begins; m; m &= m - 1) {
            const int at = __builtin_ctz(m), row = ev.begin[grp * K + at];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float h0 = row >= 0 && i < live ? A.h0[(int64_t)row * A.D + c + i * NX] : 0.0f;
                if (at == 0 && A.states && i < live && grp * K % kEvery == 0) A.states[(int64_t)((p.t0 + grp * K) / kEvery) * A.D + c + i * NX] = h0;
                float av = 0.0f, bv = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    av = k == at ? a[k][i] : av;
                    bv = k == at ? b[k][i] : bv;
                }
                bv = fmaf(av, h0, bv);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    b[k][i] = k == at ? bv : b[k][i];
                    a[k][i] = k == at ? -1.0f : a[k][i];
                }
            }
        }
        if (p.plain) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) U[i] = fmaf(a[k][i], U[i], b[k][i]);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) U[i] = a[k][i] < 0.0f ? b[k][i] : fmaf(a[k][i], U[i], b[k][i]);
            if (begins) S[0] = S[1] = 1.0f;      // a logarithm above zero marks what is cut off from the state that enters
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) comp[grp][c2 + i * NX] = f2{S[i], U[i]};
        lds_barrier();
        const Look<DEEP> q(j, p.src);
        if (A.tiles > 1) {
            uint64_t own = 0;
            bool cut = false;
            if (threadIdx.x < kCols) {
                float St = 0.0f, Ut = 0.0f;
#pragma unroll 4
                for (int i = 0; i < NG; ++i) {
                    const f2 v = comp[i][threadIdx.x];
                    const bool off = v[0] > 0.0f;
                    cut = cut || off;
                    St += off ? 0.0f : v[0];
                    Ut = off ? v[1] : fmaf(exp2_fast(v[0]), Ut, v[1]);
                }
                own = word_of(St, Ut);
                publish(A, A.ch.agg, j, col * kCols + threadIdx.x, own);
            }
            look_back<NG / 2>(A, q, col, own, cut, look);
        }
        if (threadIdx.x < kCols) {
            float h = p.src < j ? compose(q, look) : 0.0f;
#pragma unroll 4
            for (int i = 0; i < NG; ++i) {
                const f2 v = comp[i][threadIdx.x];
                entry[i][threadIdx.x] = h;
                h = v[0] > 0.0f ? v[1] : fmaf(exp2_fast(v[0]), h, v[1]);
            }
            if (A.tiles > 1 && j % kGroup == kGroup - 1) publish_state(A, j / kGroup, col * kCols + threadIdx.x, h);
        }
        lds_barrier();
        // made here: behind the branch below it would come to lie in vector registers
        const __amdgpu_buffer_rsrc_t by = rows_at<T>(A.y, p.t0, A.D, p.n, A.D);
        float h[2] = {entry[grp][c2], entry[grp][c2 + NX]};
        if (A.states && grp * K % kEvery == 0 && grp * K < p.n && !(begins & 1)) {
            float* s = A.states + (int64_t)((p.t0 + grp * K) / kEvery) * A.D + c;
            if (live > 0) s[0] = h[0];
            if (live > 1) s[NX] = h[1];
        }
        if constexpr (OUT) {
            const uint32_t sy = (uint32_t)A.D * sizeof(T);
            const Place2 oy = place2<T, PAIR>(grp * K * sy + c * sizeof(T), live);
            if (p.plain) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) h[i] = fmaf(a[k][i], h[i], b[k][i]);
                    store2<T, PAIR>(by, oy, k * sy, h[0], h[1]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        h[i] = a[k][i] < 0.0f ? b[k][i] : fmaf(a[k][i], h[i], b[k][i]);
                        b[k][i] = h[i];                 // for the end states
                    }
                    const bool in = grp * K + k >= p.lo && grp * K + k < p.hi;
                    store2<T, PAIR>(by, in ? oy : Place2{kNowhere, kNowhere}, k * sy, h[0], h[1]);
                }
                for (uint32_t m = ends; m; m &= m - 1) {
                    const int at = __builtin_ctz(m), row = ev.end[grp * K + at];
                    if (row < 0 || !A.h_out) continue;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v = 0.0f;
#pragma unroll
                        for (int k = 0; k < K; ++k) v = k == at ? b[k][i] : v;
                        if (i < live) A.h_out[(int64_t)row * A.D + c + i * NX] = v;
                    }
                }
            }
        }
    }
}

// ------------------------------------------------------------- backward ----
// Tiles from the last to the first.  A tile needs the state that enters it, which the forward kept for every 64th token, and
// the gradient that comes back out of the tiles behind, handed on like the states forward.  The tokens are walked three times in
// registers: forward and back for what the tile hands on, forward for h_{t-1}, back for G and the gradients.  64 tokens, eight a thread: what
// is held of every token (two outputs' factors, a, s, the inputs) makes 160 registers, three workgroups a compute unit; four
// tokens a thread (92 registers, 512 threads) take 121 us where this takes 102 to 110 (8 x 2048 by 1536, bf16).
template <typename T, int PAIR, int K, bool DEEP>
__global__ void __launch_bounds__(kTileBack / K * 32, 3) k_gs_backward(GsArgs A) {
    constexpr int NG = kTileBack / K, NT = NG * 32, NX = kNext<PAIR>;
    __shared__ f4 comp[NG][kCols];          // of every group: (S, U) forward, (S, V) backward
    __shared__ f2 entry[NG][kCols];         // the state in front of it, the gradient from behind it
    __shared__ uint64_t look[kLook<DEEP>][kCols];
    __shared__ Events<kTileBack, NG> ev;
    __shared__ int taken;
    static_assert(kTileBack == kEvery, "a tile starts from a kept state");
    const int c2 = first_channel<PAIR>(), grp = threadIdx.x >> 5;
    typename Raw<T>::type rx[K], ra[K], rg[K], rd[K];
    Params<PAIR> par;
    const int col = column_of(A);
    if (threadIdx.x == 0) taken = take(A, col);
    __syncthreads();
    const int jr = __builtin_amdgcn_readfirstlane(taken), j = A.tiles - 1 - jr;
    const int c = col * kCols + c2, live = channels_of<PAIR>(A.D, c);
    {
        const int t0 = j * kTileBack, n = min(A.T - t0, kTileBack);
        par.load(A, c, live);
        const Source<T> sa(A.a, t0, A.a_ts, n, A.D, grp * K, c), sx(A.x, t0, A.x_ts, n, A.D, grp * K, c);
        const Source<T> sg(A.g, t0, A.g_ts, A.g ? n : 0, A.D, grp * K, c), sd(A.dy, t0, A.D, n, A.D, grp * K, c);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            ra[k] = sa.template get<PAIR>(k);
            rg[k] = A.g ? sg.template get<PAIR>(k) : Raw<T>::open();
            rx[k] = sx.template get<PAIR>(k);
        }
#pragma unroll
        for (int k = K - 1; k >= 0; --k) rd[k] = sd.template get<PAIR>(k);
    }
    const Place p = place<kTileBack, true>(A, j);
    uint32_t begins = 0, ends = 0;
    if (!p.plain) {
        find_events<kTileBack, NG, true>(A, p, ev, col, A.dh_out, A.dh0);
        begins = ev.begins[grp];
        ends = ev.ends[grp];
        // Tokens of no sequence count as zeros, whatever they hold; no gradient comes to them and no state that is not finite (the
        // walks are cut where a sequence begins, and behind the last one), so that they add nothing to the sums.
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool in = grp * K + k >= p.lo && grp * K + k < p.hi;
            ra[k] = in ? ra[k] : typename Raw<T>::type{};
            rx[k] = in ? rx[k] : typename Raw<T>::type{};
            rg[k] = in ? rg[k] : typename Raw<T>::type{};
            rd[k] = in ? rd[k] : typename Raw<T>::type{};
        }
    }
    // A row's values in place of what comes from the neighbouring token.  Not before its turn: rows of many tokens would be held.
    const auto set = [&](float (&v)[2], const float* q, int row) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = q && row >= 0 && i < live ? q[(int64_t)row * A.D + c + i * NX] : 0.0f;
    };

    // of every token: a, beta i, a^2 b / (1 - a^2) and then dla / G, the smaller of s and 1 - s (1 - s negated), b (1 - i)
    float a[K][2], bi[K][2], r[K][2], sm[K][2], bn[K][2];
    float S[2] = {0.0f, 0.0f}, U[2] = {0.0f, 0.0f}, V[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float s, not_s, ig, not_i;
            sigma2(half_of(ra[k], i), par.nab[i], s, not_s);
            const Gate q = gate(s, par.nd[i]);
            sigma2(half_of(rg[k], i), par.nxb[i], ig, not_i);
            a[k][i] = q.a;
            bi[k][i] = q.beta * ig;
            const float b = bi[k][i] * half_of(rx[k], i);
            bn[k][i] = b * not_i;
            sm[k][i] = s > not_s ? -not_s : s;
            const float root = q.a * q.a * b * __builtin_amdgcn_rcpf(q.less);
            r[k][i] = q.less < 0x1p-120f ? 0.0f : root;
            // made here and held, rather than their factors, of which there are more
            asm volatile("" : "+v"(sm[k][i]), "+v"(r[k][i]), "+v"(bn[k][i]));
            S[i] += q.x2;
        }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!p.plain && (begins >> k & 1)) set(U, A.h0, ev.begin[grp * K + k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) U[i] = fmaf(a[k][i], U[i], bi[k][i] * half_of(rx[k], i));
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        if (!p.plain && (ends >> k & 1)) set(V, A.dh_out, ev.end[grp * K + k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) V[i] = a[k][i] * (half_of(rd[k], i) + V[i]);
        if (!p.plain && (begins >> k & 1)) V[0] = V[1] = 0.0f;
    }
    const bool cut = begins != 0, cut_back = (begins | ends) != 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) comp[grp][c2 + i * NX] = f4{cut ? 1.0f : S[i], U[i], cut_back ? 1.0f : S[i], V[i]};
    lds_barrier();
    const int src = A.tiles - 1 - p.src;
    const Look<DEEP> look_at(jr, src);
    if (A.tiles > 1) {
        uint64_t own = 0;
        bool cut_any = false;
        if (threadIdx.x < kCols) {
            float St = 0.0f, Vt = 0.0f;
#pragma unroll 4
            for (int i = NG - 1; i >= 0; --i) {
                const f4 q = comp[i][threadIdx.x];
                const bool off = q[2] > 0.0f;
                cut_any = cut_any || off;
                St += off ? 0.0f : q[2];
                Vt = off ? q[3] : fmaf(exp2_fast(q[2]), Vt, q[3]);
            }
            own = word_of(St, Vt);
            publish(A, A.ch.agg, jr, col * kCols + threadIdx.x, own);
        }
        look_back<NG / 2>(A, look_at, col, own, cut_any, look);
    }
    if (threadIdx.x < kCols) {
        float g = src < jr ? compose(look_at, look) : 0.0f;
#pragma unroll 4
        for (int i = NG - 1; i >= 0; --i) {
            const f4 q = comp[i][threadIdx.x];
            entry[i][threadIdx.x][1] = g;
            g = q[2] > 0.0f ? q[3] : fmaf(exp2_fast(q[2]), g, q[3]);
        }
        if (A.tiles > 1 && jr % kGroup == kGroup - 1) publish_state(A, jr / kGroup, col * kCols + threadIdx.x, g);
    } else if (threadIdx.x < 2 * kCols) {
        const int lane = threadIdx.x - kCols, at = col * kCols + lane;
        // no state is kept where the first token is in no sequence
        float h = at < A.D && p.lo == 0 && p.hi > 0 ? A.kept[(int64_t)j * A.D + at] : 0.0f;
#pragma unroll 4
        for (int i = 0; i < NG; ++i) {
            const f4 q = comp[i][lane];
            entry[i][lane][0] = h;
            h = q[0] > 0.0f ? q[1] : fmaf(exp2_fast(q[0]), h, q[1]);
        }
    }
    lds_barrier();
    float h[2], g[2], sum[3][2];
    float la_open[2];        // -decay; held finite: with infinite decay dla is zero, and so is what comes to the gate
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        la_open[i] = __builtin_elementwise_maximum(par.nd[i], -0x1.fffffep127f) * 0.69314718056f;
        h[i] = entry[grp][c2 + i * NX][0];
        g[i] = entry[grp][c2 + i * NX][1];
        sum[0][i] = sum[1][i] = sum[2][i] = 0.0f;
    }
    const __amdgpu_buffer_rsrc_t bdx = rows_at<T>(A.dx, p.t0, A.D, p.n, A.D), bda = rows_at<T>(A.da, p.t0, A.D, p.n, A.D);
    const __amdgpu_buffer_rsrc_t bdg = rows_at<T>(A.dg, p.t0, A.D, A.g ? p.n : 0, A.D);
    const uint32_t sd = (uint32_t)A.D * sizeof(T);
    const Place2 od = place2<T, PAIR>(grp * K * sd + c * sizeof(T), live);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!p.plain && (begins >> k & 1)) set(h, A.h0, ev.begin[grp * K + k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            r[k][i] = fmaf(a[k][i], h[i], -r[k][i]);
            h[i] = fmaf(a[k][i], h[i], bi[k][i] * half_of(rx[k], i));
        }
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        float dx[2], da[2], dg[2];
        if (!p.plain && (ends >> k & 1)) set(g, A.dh_out, ev.end[grp * K + k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float G = half_of(rd[k], i) + g[i], dla = G * r[k][i];
            g[i] = a[k][i] * G;
            dx[i] = G * bi[k][i];
            dg[i] = G * bn[k][i];
            const float m = sm[k][i];
            const bool open = (int)__float_as_uint(m) < 0;       // the sign, not the value: -0 is a gate so far open that 1 - s is zero
            const float s = open ? 1.0f + m : m, not_s = open ? -m : 1.0f - m;
            da[i] = dla * (la_open[i] * s * not_s);
            sum[0][i] = fmaf(-dla, s, sum[0][i]);
            sum[1][i] += da[i];
            sum[2][i] += dg[i];
        }
        store2<T, PAIR>(bdx, od, k * sd, dx[0], dx[1]);
        store2<T, PAIR>(bda, od, k * sd, da[0], da[1]);
        store2<T, PAIR>(bdg, od, k * sd, dg[0], dg[1]);
        if (!p.plain && (begins >> k & 1)) {
            const int row = ev.begin[grp * K + k];
            const int64_t at = (int64_t)row * A.D + c;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (A.dh0 && row >= 0 && i < live) A.dh0[at + i * NX] = g[i];
                g[i] = 0.0f;            // for tokens of no sequence in front of it
            }
        }
    }
    if (p.lo > 0 || p.hi < p.n) {          // their rows: zeros, also behind a state that is not finite
#pragma unroll 1
        for (int k = 0; k < K; ++k) {
            if (grp * K + k >= p.lo && grp * K + k < p.hi) continue;
            store2<T, PAIR>(bdx, od, k * sd, 0.0f, 0.0f);
            store2<T, PAIR>(bda, od, k * sd, 0.0f, 0.0f);
            store2<T, PAIR>(bdg, od, k * sd, 0.0f, 0.0f);
        }
    }
    if (!A.part) return;
    float (*red)[3][kCols] = reinterpret_cast<float (*)[3][kCols]>(&comp[0][0]);       // comp has been read
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) red[grp][q][c2 + i * NX] = sum[q][i];
    lds_barrier();
    for (int i = threadIdx.x; i < 3 * kCols; i += NT) {
        float v = 0.0f;
#pragma unroll
        for (int n = 0; n < NG; ++n) v += red[n][i / kCols][i % kCols];
        A.part[((int64_t)j * 3 + i / kCols) * A.cols * kCols + col * kCols + i % kCols] = v;
    }
}

// The sums over tokens of ddecay, da_bias and dx_bias from the tiles' shares, in a fixed order: a workgroup adds up 32 columns of one of
// them, its 32 groups of lanes dealing the tiles out.
__global__ void __launch_bounds__(1024) k_gs_sums(const float* __restrict__ part, int tiles, int cols, int D, float* d0, float* d1, float* d2) {
    __shared__ float red[32][33];
    const int which = blockIdx.y, lane = threadIdx.x & 31, grp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float* d = which == 0 ? d0 : which == 1 ? d1 : d2;
    if (!d) return;
    const int64_t row = (int64_t)cols * kCols;
    float s = 0.0f;
    for (int i = grp; i < tiles; i += 32 * 8) {
        float t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = i + 32 * k < tiles ? part[((int64_t)(i + 32 * k) * 3 + which) * row + c] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += t[k];
    }
    red[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < D) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += red[i][lane];
        d[c] = s;
    }
}

// ----------------------------------------------------------------- step ----
// Two channels of one sequence a thread, nothing shared.  One row of 1536 channels 3.0 us, the latency of the launch and two loads; 256
// rows in a pool 4.3 us for 6.3 MB, most of it in the caches.
template <typename T, int PAIR>
__global__ void __launch_bounds__(256) k_gs_step(GsArgs A, int64_t n0, int blocks) {
    const int64_t n = n0 + blockIdx.x / blocks;
    constexpr int NX = kNext<PAIR>;
    const int c = ((int)(blockIdx.x % blocks) * 8 + (threadIdx.x >> 5)) * kCols + first_channel<PAIR>(), live = channels_of<PAIR>(A.D, c);
    if (live == 0) return;
    const __amdgpu_buffer_rsrc_t bx = rows_at<T>(A.x, n, A.x_ts, 1, A.D), ba = rows_at<T>(A.a, n, A.a_ts, 1, A.D);
    const __amdgpu_buffer_rsrc_t bg = rows_at<T>(A.g, n, A.g_ts, A.g ? 1 : 0, A.D), by = rows_at<T>(A.y, n, A.D, 1, A.D);
    const auto rx = load2<T, PAIR>(bx, c * sizeof(T), 0), ra = load2<T, PAIR>(ba, c * sizeof(T), 0);
    const auto rg = A.g ? load2<T, PAIR>(bg, c * sizeof(T), 0) : Raw<T>::open();
    int64_t row = n;
    if (A.slots) {
        row = A.slots[n];
        if (row < 0 || row >= A.n_slots) row = -1;
    }
    float h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = c + i * NX;
        h[i] = 0.0f;
        if (i < live) {
            if (A.h0 && row >= 0) h[i] = A.h0[row * A.D + at];
            const Gate q = gate(sigma(half_of(ra, i), A.a_bias ? -A.a_bias[at] * kLog2e : 0.0f), -A.decay[at] * kLog2e);
            const float ig = sigma(half_of(rg, i), A.x_bias ? -A.x_bias[at] * kLog2e : 0.0f);
            h[i] = fmaf(q.a, h[i], q.beta * ig * half_of(rx, i));
            if (row >= 0) A.h_out[row * A.D + at] = h[i];
        }
    }
    store2<T, PAIR>(by, place2<T, PAIR>(c * sizeof(T), live), 0, h[0], h[1]);
}

// ------------------------------------------------------------------ host ----
bool sizes_ok(int64_t n_seq, int64_t T, int64_t D) {
    if (n_seq < 0 || T < 0 || D < 1 || D >= 1 << 22 || n_seq > 1 << 20 || T >= (int64_t)1 << 31) return false;
    return ((T + kTileBack - 1) / kTileBack) * ((D + kCols - 1) / kCols) < (int64_t)1 << 23;
}

bool stride_ok(int64_t s, int64_t D) { return s >= D && s < 1 << 22; }

size_t span_of(int64_t tokens, int64_t stride, int64_t row, size_t es) {
    return tokens > 0 ? ((size_t)(tokens - 1) * stride + row) * es : 0;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t tiles_of(int64_t T, int tokens) { return T > 0 ? (T + tokens - 1) / tokens : 1; }
int64_t columns_of(int64_t D) { return (D + kCols - 1) / kCols * kCols; }

// Where a chain's parts lie in the workspace from `at` on; returns the bytes it takes (none for one tile).
size_t lay_out(Chain* ch, char* at, int64_t tiles, int64_t columns) {
    if (tiles < 2) return 0;
    const size_t agg = up256((size_t)tiles * columns * 8), gagg = up256((size_t)groups_of(tiles) * columns * 8);
    const size_t incl = up256((size_t)groups_of(tiles) * columns * 4), first = up256((size_t)(tiles + 1) * 4);
    if (ch) {
        ch->agg = (uint64_t*)at;
        ch->gagg = (uint64_t*)(at + agg);
        ch->incl = (uint32_t*)(at + agg + gagg);
        ch->first = (int*)(at + agg + gagg + incl);
        ch->ticket = (uint32_t*)(at + agg + gagg + incl + first);
    }
    return agg + gagg + incl + first + up256((size_t)(columns / kCols) * kCounter * 4);
}

// The backward's workspace: both chains, the tiles' shares of the sums, the states where they are made again.
struct BackPlan {
    int64_t tiles, tiles_back, columns;
    size_t back_at, part_at, states_at, bytes;
};

BackPlan back_plan(int64_t T, int64_t D) {
    BackPlan b;
    b.tiles = tiles_of(T, kTile);
    b.tiles_back = tiles_of(T, kTileBack);
    b.columns = columns_of(D);
    b.back_at = lay_out(nullptr, nullptr, b.tiles, b.columns);
    b.part_at = b.back_at + lay_out(nullptr, nullptr, b.tiles_back, b.columns);
    b.states_at = b.part_at + up256((size_t)b.tiles_back * 3 * b.columns * 4);
    b.bytes = b.states_at + up256((size_t)((T + kEvery - 1) / kEvery) * D * 4);
    return b;
}

// Which of the kernels' PAIR holds for a call: `more` are the outputs, contiguous.
template <typename T>
int pairs_of(const GsArgs& A, std::initializer_list<const void*> more) {
    uintptr_t all = (uintptr_t)A.D * sizeof(T) | (uintptr_t)A.x_ts * sizeof(T) | (uintptr_t)A.a_ts * sizeof(T) | (uintptr_t)A.x | (uintptr_t)A.a | (uintptr_t)A.g;
    if (A.g) all |= (uintptr_t)A.g_ts * sizeof(T);
    for (const void* p : more) all |= (uintptr_t)p;
    return all % (2 * sizeof(T)) ? 0 : all % 128 ? 1 : 2;
}

mb_status launch_setup(const GsArgs& A, const Chain& fwd, int64_t tiles, const Chain& back, int64_t tiles_back, hipStream_t s) {
    Setup S{};
    S.ch[0] = fwd;
    S.ch[1] = back;
    S.tiles[0] = (int)tiles;
    S.tiles[1] = (int)tiles_back;
    S.tokens[0] = kTile;
    S.tokens[1] = kTileBack;
    S.cu = A.cu;
    S.n_seq = A.n_seq;
    S.T = A.T;
    S.columns = A.cols * kCols;
    const int64_t most = std::max(tiles, tiles_back);
    if (most < 2) return MB_OK;
    const int64_t words = most * S.columns;
    hipLaunchKernelGGL(k_gs_setup, dim3((unsigned)std::min<int64_t>((words + 1023) / 1024, 1024)), dim3(256), 0, s, S);
    return check_launch();
}

template <typename T, bool OUT, bool DEEP>
mb_status run_forward_as(const GsArgs& A, hipStream_t s) {
    constexpr int K = kPer;
    const dim3 grid((unsigned)(A.tiles * A.cols)), block(kTile / K * 32);
    switch (pairs_of<T>(A, {A.y})) {
        case 0: hipLaunchKernelGGL((k_gs_forward<T, 0, K, OUT, DEEP>), grid, block, 0, s, A); break;
        case 1: hipLaunchKernelGGL((k_gs_forward<T, 1, K, OUT, DEEP>), grid, block, 0, s, A); break;
        default: hipLaunchKernelGGL((k_gs_forward<T, 2, K, OUT, DEEP>), grid, block, 0, s, A);
    }
    return check_launch();
}

template <typename T, bool OUT>
mb_status run_forward(const GsArgs& A, hipStream_t s) {
    return A.cols <= kDeep ? run_forward_as<T, OUT, true>(A, s) : run_forward_as<T, OUT, false>(A, s);
}

template <typename T>
mb_status run_step(const GsArgs& A, int64_t n, hipStream_t s) {
    const int64_t blocks = (A.D + 511) / 512, most = max_workgroups(256) / blocks;       // rows of a launch
    const int pairs = pairs_of<T>(A, {A.y});
    for (int64_t at = 0; at < n; at += most) {
        const dim3 grid((unsigned)(std::min(most, n - at) * blocks));
        if (pairs) hipLaunchKernelGGL((k_gs_step<T, 1>), grid, dim3(256), 0, s, A, at, (int)blocks);
        else hipLaunchKernelGGL((k_gs_step<T, 0>), grid, dim3(256), 0, s, A, at, (int)blocks);
        const mb_status st = check_launch();
        if (st != MB_OK) return st;
    }
    return MB_OK;
}

template <typename T, bool DEEP>
mb_status run_backward_as(const GsArgs& A, hipStream_t s) {
    constexpr int K = kPerBack;
    const dim3 grid((unsigned)(A.tiles * A.cols)), block(kTileBack / K * 32);
    switch (pairs_of<T>(A, {A.dy, A.dx, A.da, A.dg})) {
        case 0: hipLaunchKernelGGL((k_gs_backward<T, 0, K, DEEP>), grid, block, 0, s, A); break;
        case 1: hipLaunchKernelGGL((k_gs_backward<T, 1, K, DEEP>), grid, block, 0, s, A); break;
        default: hipLaunchKernelGGL((k_gs_backward<T, 2, K, DEEP>), grid, block, 0, s, A);
    }
    return check_launch();
}

template <typename T>
mb_status run_backward(const GsArgs& A, hipStream_t s) {
    return A.cols <= kDeep ? run_backward_as<T, true>(A, s) : run_backward_as<T, false>(A, s);
}

// What every entry point takes: sizes, pointers and alignment of the inputs.
mb_status check_inputs(const GsArgs& A, int64_t T, mb_dtype dtype) {
    const size_t es = dtype_size(dtype);
    if (!A.decay || (T > 0 && (!A.x || !A.a || (!A.g && A.x_bias)))) return MB_ERR_NULL;
    if ((uintptr_t)A.x % es || (uintptr_t)A.a % es || (uintptr_t)A.g % es || ((uintptr_t)A.decay & 3) || ((uintptr_t)A.a_bias & 3) ||
        ((uintptr_t)A.x_bias & 3) || ((uintptr_t)A.cu & 3) || ((uintptr_t)A.slots & 3) || ((uintptr_t)A.h0 & 3))
        return MB_ERR_ALIGN;
    return MB_OK;
}

}  // namespace

size_t gated_scan_workspace(int64_t n_seq, int64_t T, int64_t D) {
    if (!sizes_ok(n_seq, T, D)) return 0;
    return lay_out(nullptr, nullptr, tiles_of(T, kTile), columns_of(D));
}

size_t gated_scan_bwd_workspace(int64_t n_seq, int64_t T, int64_t D) {
    if (!sizes_ok(n_seq, T, D)) return 0;
    return back_plan(T, D).bytes;
}

}  // namespace mb

using namespace mb;

extern "C" mb_status mb_gated_scan(const void* x, const void* a_gate, const void* x_gate, const float* decay, const float* a_bias,
                                   const float* x_bias, const int32_t* cu_seqlens, const float* h0, const uint8_t* has_h0,
                                   const int32_t* slots, void* y, float* h_out, float* states, int64_t n_seq, int64_t T, int64_t D,
                                   int64_t n_slots, int64_t x_stride, int64_t a_stride, int64_t g_stride, mb_dtype dtype, void* ws,
                                   size_t ws_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (!sizes_ok(n_seq, T, D) || !stride_ok(x_stride, D) || !stride_ok(a_stride, D) || (x_gate && !stride_ok(g_stride, D))) return MB_ERR_SHAPE;
    if (n_slots > 0x7fffffff || (slots ? n_slots < 1 : n_slots != 0)) return MB_ERR_SHAPE;
    if (n_seq == 0) return MB_OK;
    if (!cu_seqlens && T % n_seq) return MB_ERR_SHAPE;
    GsArgs A{};
    A.x = x; A.a = a_gate; A.g = x_gate;
    A.x_ts = x_stride; A.a_ts = a_stride; A.g_ts = g_stride;
    A.decay = decay; A.a_bias = a_bias; A.x_bias = x_bias;
    A.cu = cu_seqlens; A.h0 = h0; A.has_h0 = has_h0; A.slots = slots; A.n_slots = n_slots;
    A.y = y; A.h_out = h_out; A.states = states;
    A.n_seq = (int)n_seq; A.T = (int)T; A.L = (int)(T / n_seq); A.D = (int)D;
    mb_status st = check_inputs(A, T, dtype);
    if (st != MB_OK) return st;
    if (T > 0 && !y) return MB_ERR_NULL;
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)y % es || ((uintptr_t)h_out & 3) || ((uintptr_t)states & 3)) return MB_ERR_ALIGN;
    const size_t need = gated_scan_workspace(n_seq, T, D);
    if (need && (!ws || ws_bytes < need || ((uintptr_t)ws & 255))) return MB_ERR_WORKSPACE;
    const size_t nh = (size_t)(slots ? n_slots : n_seq) * D * 4, no = (size_t)T * D * es, ns = (size_t)((T + kEvery - 1) / kEvery) * D * 4;
    const Span ins[10] = {{x, span_of(T, x_stride, D, es)}, {a_gate, span_of(T, a_stride, D, es)}, {x_gate, span_of(T, g_stride, D, es)},
                          {decay, (size_t)D * 4}, {a_bias, (size_t)D * 4}, {x_bias, (size_t)D * 4},
                          {cu_seqlens, (size_t)(n_seq + 1) * 4}, {has_h0, (size_t)n_seq}, {slots, (size_t)n_seq * 4}, {h0, nh}};
    const Span outs[3] = {{y, no}, {h_out, nh}, {states, ns}};
    for (int i = 0; i < 3; ++i) {
        if (overlaps_any(outs[i].p, outs[i].bytes, ins, i == 1 && h_out == h0 ? 9 : 10)) return MB_ERR_ALIAS;
        if (overlaps_any(outs[i].p, outs[i].bytes, outs, i)) return MB_ERR_ALIAS;
    }
    if (need && (overlaps_any(ws, need, ins, 10) || overlaps_any(ws, need, outs, 3))) return MB_ERR_ALIAS;
    A.tiles = (int)tiles_of(T, kTile);
    A.cols = (int)(columns_of(D) / kCols);
    lay_out(&A.ch, (char*)ws, A.tiles, columns_of(D));
    if ((st = launch_setup(A, A.ch, A.tiles, Chain{}, 0, stream)) != MB_OK) return st;
    return dtype == MB_F32 ? run_forward<float, true>(A, stream) : run_forward<bf16, true>(A, stream);
}

extern "C" mb_status mb_gated_scan_step(const void* x, const void* a_gate, const void* x_gate, const float* decay, const float* a_bias,
                                        const float* x_bias, const int32_t* slots, const float* h_in, float* h_out, void* y, int64_t n,
                                        int64_t D, int64_t n_slots, int64_t x_stride, int64_t a_stride, int64_t g_stride, mb_dtype dtype,
                                        hipStream_t stream) {
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (n < 0 || n > 1 << 20 || D < 1 || D >= 1 << 22 || !stride_ok(x_stride, D) || !stride_ok(a_stride, D) || (x_gate && !stride_ok(g_stride, D)))
        return MB_ERR_SHAPE;
    if (n_slots > 0x7fffffff || (slots ? n_slots < 1 : n_slots != 0)) return MB_ERR_SHAPE;
    if (n == 0) return MB_OK;
    GsArgs A{};
    A.x = x; A.a = a_gate; A.g = x_gate;
    A.x_ts = x_stride; A.a_ts = a_stride; A.g_ts = g_stride;
    A.decay = decay; A.a_bias = a_bias; A.x_bias = x_bias;
    A.slots = slots; A.n_slots = n_slots; A.h0 = h_in; A.h_out = h_out; A.y = y;
    A.D = (int)D;
    mb_status st = check_inputs(A, n, dtype);
    if (st != MB_OK) return st;
    if (!y || !h_out) return MB_ERR_NULL;
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)y % es || ((uintptr_t)h_out & 3)) return MB_ERR_ALIGN;
    const size_t nh = (size_t)(slots ? n_slots : n) * D * 4, no = (size_t)n * D * es;
    const Span ins[8] = {{x, span_of(n, x_stride, D, es)}, {a_gate, span_of(n, a_stride, D, es)}, {x_gate, span_of(n, g_stride, D, es)},
                         {decay, (size_t)D * 4}, {a_bias, (size_t)D * 4}, {x_bias, (size_t)D * 4}, {slots, (size_t)n * 4}, {h_in, nh}};
    if (overlaps_any(y, no, ins, 8) || overlaps_any(h_out, nh, ins, h_out == h_in ? 7 : 8) || overlaps(y, no, h_out, nh)) return MB_ERR_ALIAS;
    return dtype == MB_F32 ? run_step<float>(A, n, stream) : run_step<bf16>(A, n, stream);
}

extern "C" mb_status mb_gated_scan_bwd(const void* x, const void* a_gate, const void* x_gate, const float* decay, const float* a_bias,
                                       const float* x_bias, const int32_t* cu_seqlens, const float* h0, const void* dy,
                                       const float* dh_out, const float* states, void* dx, void* da_gate, void* dx_gate, float* ddecay,
                                       float* da_bias, float* dx_bias, float* dh0, int64_t n_seq, int64_t T, int64_t D, int64_t x_stride,
                                       int64_t a_stride, int64_t g_stride, mb_dtype dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (!sizes_ok(n_seq, T, D) || !stride_ok(x_stride, D) || !stride_ok(a_stride, D) || (x_gate && !stride_ok(g_stride, D))) return MB_ERR_SHAPE;
    if (!cu_seqlens && (n_seq ? T % n_seq : T) != 0) return MB_ERR_SHAPE;
    GsArgs A{};
    A.x = x; A.a = a_gate; A.g = x_gate;
    A.x_ts = x_stride; A.a_ts = a_stride; A.g_ts = g_stride;
    A.decay = decay; A.a_bias = a_bias; A.x_bias = x_bias;
    A.cu = cu_seqlens; A.h0 = h0; A.dy = dy; A.dh_out = dh_out; A.kept = states;
    A.dx = dx; A.da = da_gate; A.dg = dx_gate; A.dh0 = dh0;
    A.n_seq = (int)n_seq; A.T = (int)T; A.L = n_seq ? (int)(T / n_seq) : 0; A.D = (int)D;
    mb_status st = check_inputs(A, T, dtype);
    if (st != MB_OK) return st;
    if (T > 0 && (!dy || !dx || !da_gate || (x_gate != nullptr) != (dx_gate != nullptr) || (!x_gate && dx_bias))) return MB_ERR_NULL;
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)dy % es || (uintptr_t)dx % es || (uintptr_t)da_gate % es || (uintptr_t)dx_gate % es || ((uintptr_t)dh_out & 3) ||
        ((uintptr_t)states & 3) || ((uintptr_t)ddecay & 3) || ((uintptr_t)da_bias & 3) || ((uintptr_t)dx_bias & 3) || ((uintptr_t)dh0 & 3))
        return MB_ERR_ALIGN;
    const size_t need = gated_scan_bwd_workspace(n_seq, T, D);
    if (need && (!ws || ws_bytes < need || ((uintptr_t)ws & 255))) return MB_ERR_WORKSPACE;
    const size_t nh = (size_t)n_seq * D * 4, no = (size_t)T * D * es, ns = (size_t)((T + kEvery - 1) / kEvery) * D * 4, nd = (size_t)D * 4;
    const Span ins[11] = {{x, span_of(T, x_stride, D, es)}, {a_gate, span_of(T, a_stride, D, es)}, {x_gate, span_of(T, g_stride, D, es)},
                          {decay, nd}, {a_bias, nd}, {x_bias, nd}, {cu_seqlens, (size_t)(n_seq + 1) * 4}, {h0, nh}, {dy, no}, {dh_out, nh}, {states, ns}};
    const Span outs[7] = {{dx, no}, {da_gate, no}, {dx_gate, no}, {ddecay, nd}, {da_bias, nd}, {dx_bias, nd}, {dh0, nh}};
    for (int i = 0; i < 7; ++i)
        if (overlaps_any(outs[i].p, outs[i].bytes, ins, 11) || overlaps_any(outs[i].p, outs[i].bytes, outs, i)) return MB_ERR_ALIAS;
    if (need && (overlaps_any(ws, need, ins, 11) || overlaps_any(ws, need, outs, 7))) return MB_ERR_ALIAS;
    const BackPlan bp = back_plan(T, D);
    char* base = (char*)ws;
    A.cols = (int)(bp.columns / kCols);
    Chain fwd{}, back{};
    if (!states) lay_out(&fwd, base, bp.tiles, bp.columns);
    lay_out(&back, base + bp.back_at, bp.tiles_back, bp.columns);
    if ((st = launch_setup(A, fwd, states ? 0 : bp.tiles, back, bp.tiles_back, stream)) != MB_OK) return st;
    if (!states) {
        GsArgs F = A;
        F.states = (float*)(base + bp.states_at);
        F.tiles = (int)bp.tiles;
        F.ch = fwd;
        if (T && (st = dtype == MB_F32 ? run_forward<float, false>(F, stream) : run_forward<bf16, false>(F, stream)) != MB_OK) return st;
        A.kept = F.states;
    }
    A.tiles = (int)bp.tiles_back;
    A.ch = back;
    A.part = ddecay || da_bias || dx_bias ? (float*)(base + bp.part_at) : nullptr;
    if ((st = dtype == MB_F32 ? run_backward<float>(A, stream) : run_backward<bf16>(A, stream)) != MB_OK) return st;
    if (!A.part) return MB_OK;
    hipLaunchKernelGGL(k_gs_sums, dim3((unsigned)A.cols * (kCols / 32), 3), dim3(1024), 0, stream, A.part, A.tiles, A.cols, A.D, ddecay, da_bias, dx_bias);
    return check_launch();
}
