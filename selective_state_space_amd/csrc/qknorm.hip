// qknorm.hip -- root-mean-square norm of every head of queries and keys with the rotation by their position, and its
// backward.
//
//     n = x / sqrt(mean x^2 + eps) * w;   pairs (u, v) of n turn by the angle position * freqs[j]
//     backward: e = the gradient turned back, xh = x rstd, g = e w:
//         dx = rstd (g - xh mean(g xh)),  dw = sum e xh
//
// Bound by HBM: a head's row is read once, kept in registers between the sum of squares and the turn, and written once.
// LPR lanes (the power of two that holds D / 8) share a row, eight columns each as four pairs: the pairs' members lie in
// one lane whichever way they are paired, two pieces of four neighbouring columns.  A workgroup takes some tokens with all
// their heads, and makes the tokens' sines and cosines once, in LDS, for all of them.  Times of the kernel alone: 16384 tokens of 16 and
// 16 heads of 128, bf16, 52 to 58 us for 268 MB, 4.6 to 5.2 TB/s, about the rate of a large copy (288 with the angles, reduced in fp64,
// made for every row); the backward with 16 and 4 heads 49 to 52 us for 252 MB, 4.8 to 5.1 TB/s, and 4.3 to 5.0 for the sum over
// workgroups.  One token 3.4 us.  4095 tokens of 6 and 2 heads of 80 in fp32, 32 columns turned, 9.8 us for 21 MB: 512 of them take
// 5.6, load, angle, sum and store one behind the other; the angles are 1.2 of the 9.8; the rest grows with the bytes (8190 tokens 14.4).
#include <algorithm>
#include <type_traits>

#include "mb_internal.h"

namespace mb {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

constexpr int kMaxD = 512;
constexpr int kTokens = 16;       // most tokens of a workgroup at a time
constexpr int kParts = 1024;      // most workgroups of the backward, each with its own share of dw
constexpr int kBatch = 4;         // rows of a lane under way at a time

struct QkArgs {
    const void* in[2];        // queries, keys
    void* out[2];
    const void* d[2];         // backward: their outputs' gradients
    const float* w[2];
    float* part;              // (workgroups, 2, D) shares of dw
    int64_t in_ts[2], out_ts[2];
    const float* freqs;
    const int32_t* positions;
    int64_t T, L;
    int64_t first;            // forward: the launch's first token
    int H[2], D, R, inter;
    int tokens, heads;        // of a workgroup at a time
    float eps;
};

// Sum (or maximum) over the LPR lanes of a row, the same in all of them.
template <int LPR, bool MAX = false>
__device__ __forceinline__ float row_all(float v) {
    const auto with = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#define MB_DPP(ctrl) with(v, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), ctrl, 0xf, 0xf, true)))
    v = MB_DPP(0xB1);                            // neighbour
    v = MB_DPP(0x4E);                            // neighbouring pair
    if constexpr (LPR > 4) v = MB_DPP(0x141);    // mirrored in eight lanes
    if constexpr (LPR > 8) v = MB_DPP(0x140);    // mirrored in sixteen
#undef MB_DPP
    if constexpr (LPR > 16) v = with(v, __shfl_xor(v, 16));
    if constexpr (LPR > 32) v = with(v, __shfl_xor(v, 32));
    return v;
}

// Four neighbouring columns as they lie in memory.
template <typename T> struct Four;
template <> struct Four<bf16> {
    typedef u2 type;
    static __device__ __forceinline__ float get(u2 v, int i) { return __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16); }
    static __device__ __forceinline__ u2 make(float a, float b, float c, float d) {
        const f2 x = {a, b}, y = {c, d};
        return u2{__builtin_bit_cast(uint32_t, __builtin_convertvector(x, b2)), __builtin_bit_cast(uint32_t, __builtin_convertvector(y, b2))};
    }
};
template <> struct Four<float> {
    typedef f4 type;
    static __device__ __forceinline__ float get(f4 v, int i) { return v[i]; }
    static __device__ __forceinline__ f4 make(float a, float b, float c, float d) { return f4{a, b, c, d}; }
};

// A lane's columns: member o of its pair i lies at at<VEC>(i, o), or nowhere (-1).  VEC: two pieces of four.
struct Columns {
    int first, second;       // the pieces
    int pair, R, D, inter;   // its first pair
    template <bool VEC>
    __device__ __forceinline__ int at(int i, int o) const {
        int d;
        if constexpr (VEC) {
            d = inter ? first + 2 * i + o : (o ? second : first) + i;
        } else {
            const int p = pair + i;
            d = 2 * p < R && !inter ? p + o * (R / 2) : 2 * p + o;
        }
        return d < D ? d : -1;
    }
    // VEC: all four or none
    template <bool VEC>
    __device__ __forceinline__ bool turns(int i) const { return 2 * (pair + (VEC ? 0 : i)) < R; }
};

__device__ __forceinline__ Columns columns(const QkArgs& A, int lane) {
    Columns c;
    c.pair = 4 * lane;
    c.R = A.R;
    c.D = A.D;
    c.inter = A.inter;
    const bool apart = !A.inter && 8 * lane < A.R;
    c.first = apart ? 4 * lane : 8 * lane;
    c.second = apart ? A.R / 2 + 4 * lane : 8 * lane + 4;
    return c;
}

// A weight's values for a lane's columns.
template <bool VEC>
__device__ __forceinline__ void load_weights(const float* w, const Columns& c, float (&u)[4], float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = c.at<VEC>(i, 0), e = c.at<VEC>(i, 1);
        u[i] = w && d >= 0 ? w[d] : 1.0f;
        v[i] = w && e >= 0 ? w[e] : 1.0f;
    }
}

// A lane's part of a row, before it is taken apart.
template <typename T, bool VEC> struct Part {
    typename Four<T>::type a, b;
    __device__ __forceinline__ void load(const T* p, const Columns& c) {
        if (c.first < c.D) {
            a = *reinterpret_cast<const typename Four<T>::type*>(p + c.first);
            b = *reinterpret_cast<const typename Four<T>::type*>(p + c.second);
        } else {
            a = b = typename Four<T>::type{};
        }
    }
    // pairs (u, v)
    __device__ __forceinline__ void get(float (&u)[4], float (&v)[4], const Columns& c) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[i] = c.inter ? Four<T>::get(i < 2 ? a : b, 2 * (i & 1)) : Four<T>::get(a, i);
            v[i] = c.inter ? Four<T>::get(i < 2 ? a : b, 2 * (i & 1) + 1) : Four<T>::get(b, i);
        }
    }
    static __device__ __forceinline__ void store(T* p, const float (&u)[4], const float (&v)[4], const Columns& c) {
        if (c.first >= c.D) return;
        typedef typename Four<T>::type F;
        const bool x = c.inter;
        *reinterpret_cast<F*>(p + c.first) = x ? Four<T>::make(u[0], v[0], u[1], v[1]) : Four<T>::make(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<F*>(p + c.second) = x ? Four<T>::make(u[2], v[2], u[3], v[3]) : Four<T>::make(v[0], v[1], v[2], v[3]);
    }
};
template <typename T> struct Part<T, false> {
    T e[4][2];
    __device__ __forceinline__ void load(const T* p, const Columns& c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int d = c.at<false>(i, o);
                e[i][o] = d >= 0 ? p[d] : (T)0;
            }
    }
    __device__ __forceinline__ void get(float (&u)[4], float (&v)[4], const Columns&) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[i] = to_f32(e[i][0]);
            v[i] = to_f32(e[i][1]);
        }
    }
    static __device__ __forceinline__ void store(T* p, const float (&u)[4], const float (&v)[4], const Columns& c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = c.at<false>(i, 0), e = c.at<false>(i, 1);
            if (d >= 0) store_out(p + d, u[i]);
            if (e >= 0) store_out(p + e, v[i]);
        }
    }
};

// 1 / sqrt(mean x^2 + eps) of a row of the sum of squares ss.  Where squares leave fp32's range, above or, with an eps that does not
// cover it, below (2^-100: those below the range are off by up to 2^-150 each), the row is multiplied by `up`, a power of two that brings
// the larger of its values and of sqrt(eps) to between 1 and 4, and summed once more; `up` is 1 otherwise.
template <int LPR>
__device__ __forceinline__ float inverse_rms(float ss, float (&u)[4], float (&v)[4], float inv_d, float eps, float& up) {
    up = 1.0f;
    if (__builtin_expect(ss > 3.0e38f || ss + eps < 0x1p-100f, false)) {
        float top = sqrtf(eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(u[i]), fabsf(v[i])));
        const uint32_t bits = __float_as_uint(row_all<LPR, true>(top));
        if (bits != 0 && bits < 0x7f800000u) {       // neither zeros alone nor infinities; NaN does not come here
            up = __uint_as_float((uint32_t)max(254 - (int)(bits >> 23), 1) << 23);
            ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] *= up;
                v[i] *= up;
                ss = fmaf(u[i], u[i], fmaf(v[i], v[i], ss));
            }
            ss = row_all<LPR>(ss);
            eps = eps * up * up;          // in this order: a square of up leaves fp32
        }
    }
    return __builtin_amdgcn_rsqf(fmaf(ss, inv_d, eps));
}

// Sines and cosines of `n` tokens from t0 on, LPR * 4 pairs each; pairs that do not turn are left out.  The angle in turns
// is reduced in 64 bits: at a position of 2^31 it is off by 2^-24 of a turn.
template <int LPR>
__device__ __forceinline__ void fill_turns(const QkArgs& A, int64_t t0, int n, f2* cs) {
    const int half = A.R / 2;
    for (int i = threadIdx.x; i < n * LPR * 4; i += 256) {
        const int t = i / (LPR * 4), p = i % (LPR * 4);
        if (p >= half || t0 + t >= A.T) continue;
        const int64_t pos = A.positions ? A.positions[t0 + t] : (t0 + t) % A.L;
        const double r = (double)pos * (double)A.freqs[p] * 0.15915494309189533577;
        float s, c;
        sincospif(2.0f * (float)(r - rint(r)), &s, &c);
        cs[i] = f2{c, s};
    }
}

// (u, v) turned by (cos, sin)
__device__ __forceinline__ void turn(float& u, float& v, float c, float s) {
    const float a = u;
    u = fmaf(-v, s, a * c);
    v = fmaf(v, c, a * s);
}

template <typename T, int LPR, bool VEC>
__global__ void __launch_bounds__(256) k_qk_forward(QkArgs A) {
    constexpr int RS = 256 / LPR;
    __shared__ f2 cs[kTokens * LPR * 4];
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const Columns c = columns(A, lane);
    const int64_t t0 = A.first + (int64_t)blockIdx.x * A.tokens;
    const int all = A.H[0] + A.H[1], h0 = blockIdx.y * A.heads, nh = min(A.heads, all - h0);
    const int rows = (int)min((int64_t)A.tokens, A.T - t0) * nh;
    const float inv_nh = 1.0f / (float)nh, inv_d = 1.0f / (float)A.D;
    const auto place = [&](int r, int& t, int& k, int& h) {
        t = (int)(((float)r + 0.5f) * inv_nh);       // at most 16 tokens and 8192 heads: off by less than 0.5 / nh
        h = h0 + r - t * nh;
        k = h >= A.H[0];
        h -= k ? A.H[0] : 0;
    };
    float wu[2][4], wv[2][4];
    Part<T, VEC> x[kBatch];
    const auto fetch = [&](int r0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + b * RS;
            if (r < rows) {
                int t, k, h;
                place(r, t, k, h);
                x[b].load((const T*)(k ? A.in[1] : A.in[0]) + (t0 + t) * (k ? A.in_ts[1] : A.in_ts[0]) + h * A.D, c);
            }
        }
    };
    fetch(slot);
    load_weights<VEC>(A.w[0], c, wu[0], wv[0]);
    load_weights<VEC>(A.w[1], c, wu[1], wv[1]);
    if (A.R) fill_turns<LPR>(A, t0, A.tokens, cs);
    __syncthreads();
    for (int r0 = slot; r0 < rows; r0 += kBatch * RS) {
        if (r0 != slot) fetch(r0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + b * RS;
            if (r >= rows) continue;
            int t, k, h;
            place(r, t, k, h);
            float u[4], v[4], ss = 0.0f, up;
            x[b].get(u, v, c);
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = fmaf(u[i], u[i], fmaf(v[i], v[i], ss));
            const float rs = inverse_rms<LPR>(row_all<LPR>(ss), u, v, inv_d, A.eps, up);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] *= rs * (k ? wu[1][i] : wu[0][i]);
                v[i] *= rs * (k ? wv[1][i] : wv[0][i]);
                if (c.turns<VEC>(i)) {
                    const f2 q = cs[t * LPR * 4 + c.pair + i];
                    turn(u[i], v[i], q[0], q[1]);
                }
            }
            Part<T, VEC>::store((T*)(k ? A.out[1] : A.out[0]) + (t0 + t) * (k ? A.out_ts[1] : A.out_ts[0]) + h * A.D, u, v, c);
        }
    }
}

// A workgroup walks over blocks of tokens; a lane keeps its columns' shares of both weights' gradients in registers, which are added up
// in LDS at the end.
template <typename T, int LPR, bool VEC>
__global__ void __launch_bounds__(256) k_qk_backward(QkArgs A) {
    constexpr int RS = 256 / LPR, B = 2;
    __shared__ f2 cs[kTokens * LPR * 4];
    __shared__ float red[RS][LPR * 8 + 1];
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const Columns c = columns(A, lane);
    float wu[2][4], wv[2][4], du[2][4], dv[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) du[k][i] = dv[k][i] = 0.0f;
        load_weights<VEC>(A.w[k], c, wu[k], wv[k]);
    }
    const float inv_d = 1.0f / (float)A.D;
    // The rows of n tokens from t0 on of queries or of keys: which of both is known where it is compiled.
    const auto rows_of = [&](auto which, int64_t t0, int n) {
        constexpr int k = decltype(which)::value;
        const int nh = A.H[k], rows = n * nh;
        const float inv_nh = 1.0f / (float)nh;
        const T* in = (const T*)A.in[k] + t0 * A.in_ts[k];
        const T* up = (const T*)A.d[k] + t0 * A.out_ts[k];
        T* out = (T*)A.out[k] + t0 * A.out_ts[k];
        for (int r0 = slot; r0 < rows; r0 += B * RS) {
            Part<T, VEC> x[B], d[B];
            int t[B], h[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int r = min(r0 + b * RS, rows - 1);           // rows behind the last are the last one again, and not written
                t[b] = (int)(((float)r + 0.5f) * inv_nh);
                h[b] = (r - t[b] * nh) * A.D;
                x[b].load(in + t[b] * A.in_ts[k] + h[b], c);
                d[b].load(up + t[b] * A.out_ts[k] + h[b], c);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const bool live = r0 + b * RS < rows;
                float u[4], v[4], eu[4], ev[4], ss = 0.0f, dot = 0.0f, scale_up;
                x[b].get(u, v, c);
                d[b].get(eu, ev, c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ss = fmaf(u[i], u[i], fmaf(v[i], v[i], ss));
                    if (c.turns<VEC>(i)) {
                        const f2 q = cs[t[b] * LPR * 4 + c.pair + i];
                        turn(eu[i], ev[i], q[0], -q[1]);
                    }
                }
                const float rs = inverse_rms<LPR>(row_all<LPR>(ss), u, v, inv_d, A.eps, scale_up);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] *= rs;
                    v[i] *= rs;
                    du[k][i] = live ? fmaf(eu[i], u[i], du[k][i]) : du[k][i];
                    dv[k][i] = live ? fmaf(ev[i], v[i], dv[k][i]) : dv[k][i];
                    eu[i] *= wu[k][i];
                    ev[i] *= wv[k][i];
                    dot = fmaf(eu[i], u[i], fmaf(ev[i], v[i], dot));
                }
                dot = row_all<LPR>(dot) * inv_d;
                const float scale = rs * scale_up;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    eu[i] = scale * fmaf(-u[i], dot, eu[i]);
                    ev[i] = scale * fmaf(-v[i], dot, ev[i]);
                }
                if (live) Part<T, VEC>::store(out + t[b] * A.out_ts[k] + h[b], eu, ev, c);
            }
        }
    };
    for (int64_t t0 = (int64_t)blockIdx.x * A.tokens; t0 < A.T; t0 += (int64_t)gridDim.x * A.tokens) {
        const int n = (int)min((int64_t)A.tokens, A.T - t0);
        __syncthreads();                          // the turns of the block before have been read
        if (A.R) fill_turns<LPR>(A, t0, A.tokens, cs);
        __syncthreads();
        rows_of(std::integral_constant<int, 0>{}, t0, n);
        if (A.H[1]) rows_of(std::integral_constant<int, 1>{}, t0, n);
    }
    if (!A.part) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int d = c.at<VEC>(i, o);
                if (d >= 0) red[slot][d] = o ? dv[k][i] : du[k][i];
            }
        __syncthreads();
        for (int d = threadIdx.x; d < A.D; d += 256) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < RS; ++i) s += red[i][d];
            A.part[((int64_t)blockIdx.x * 2 + k) * A.D + d] = s;
        }
    }
}

// dw from the workgroups' shares, in a fixed order: 32 columns a workgroup, its 32 groups of lanes dealing the shares out.
__global__ void __launch_bounds__(1024) k_qk_sum(const float* __restrict__ part, int n, int D, float* dq, float* dk) {
    __shared__ float red[32][33];
    float* dw = blockIdx.y ? dk : dq;
    if (!dw) return;
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (d < D)
        for (int i = grp; i < n; i += 32 * 8) {
            float t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = i + 32 * k < n ? part[((int64_t)(i + 32 * k) * 2 + blockIdx.y) * D + d] : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += t[k];
        }
    red[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && d < D) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += red[i][lane];
        dw[d] = s;
    }
}

// ------------------------------------------------------------------ host ----
bool sizes_ok(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R) {
    return T >= 0 && T <= (int64_t)1 << 30 && Hq >= 1 && Hq <= 4096 && Hk >= 0 && Hk <= 4096 && D >= 1 && D <= kMaxD && R >= 0 && R <= D && R % 2 == 0;
}

bool stride_ok(int64_t s, int64_t row) { return s >= row && s < 1 << 22; }

size_t span_of(int64_t tokens, int64_t stride, int64_t row, size_t es) {
    return tokens > 0 ? ((size_t)(tokens - 1) * stride + row) * es : 0;
}

// T rows of `row` elements, `stride` apart.
struct Rows {
    const void* p;
    int64_t stride, row;
};

// Whether two tensors of tokens share memory.  Columns of one buffer lie in each other's span and do not: with one
// stride it is the rows' places within it that count.
bool rows_overlap(const Rows& a, const Rows& b, int64_t T, size_t es) {
    if (!overlaps(a.p, span_of(T, a.stride, a.row, es), b.p, span_of(T, b.stride, b.row, es))) return false;
    if (T == 1 || a.stride != b.stride) return true;
    const int64_t s = a.stride * (int64_t)es;
    int64_t off = ((intptr_t)b.p - (intptr_t)a.p) % s;
    if (off < 0) off += s;
    return off < a.row * (int64_t)es || off + b.row * (int64_t)es > s;
}

// Lanes of a row: the power of two that holds its width, four at least.
int lanes_of(int64_t D) {
    int l = 4;
    while (l * 8 < D) l *= 2;
    return l;
}

// Tokens that a workgroup takes at a time: eight rows or more for every place that it has, no more than leaves two workgroups a
// compute unit.  A power of two: heads mostly come in numbers that then fill the batches (16384 tokens of 16 and 4 heads of 128, bf16, with
// 7 tokens 45.6 us, 8 39.6, 10 44.4 and 16 42.0; the backward 54.0, 51.0, 54.4 and 52.0).
int tokens_of(int64_t T, int64_t heads, int64_t D) {
    const int64_t places = 256 / lanes_of(D), want = 2 * (int64_t)device_cu_count();
    int64_t n = 1;
    while (n < kTokens && n * heads < 8 * places) n *= 2;
    while (n > 1 && (T + n - 1) / n < want) n /= 2;
    return (int)n;
}

// Pieces of four columns may be read as they are.
bool pieces_ok(const QkArgs& A, size_t es) {
    bool ok = A.D % 8 == 0 && A.R % 8 == 0;
    for (int i = 0; i < 2; ++i)
        ok = ok && A.in_ts[i] % 4 == 0 && A.out_ts[i] % 4 == 0 && (uintptr_t)A.in[i] % (4 * es) == 0 && (uintptr_t)A.out[i] % (4 * es) == 0 &&
             (uintptr_t)A.d[i] % (4 * es) == 0;
    return ok;
}

template <typename T, bool VEC>
void launch_forward(const QkArgs& A, dim3 grid, hipStream_t s) {
    switch (lanes_of(A.D)) {
        case 4: hipLaunchKernelGGL((k_qk_forward<T, 4, VEC>), grid, dim3(256), 0, s, A); break;
        case 8: hipLaunchKernelGGL((k_qk_forward<T, 8, VEC>), grid, dim3(256), 0, s, A); break;
        case 16: hipLaunchKernelGGL((k_qk_forward<T, 16, VEC>), grid, dim3(256), 0, s, A); break;
        case 32: hipLaunchKernelGGL((k_qk_forward<T, 32, VEC>), grid, dim3(256), 0, s, A); break;
        default: hipLaunchKernelGGL((k_qk_forward<T, 64, VEC>), grid, dim3(256), 0, s, A);
    }
}

template <typename T, bool VEC>
void launch_backward(const QkArgs& A, dim3 grid, hipStream_t s) {
    switch (lanes_of(A.D)) {
        case 4: hipLaunchKernelGGL((k_qk_backward<T, 4, VEC>), grid, dim3(256), 0, s, A); break;
        case 8: hipLaunchKernelGGL((k_qk_backward<T, 8, VEC>), grid, dim3(256), 0, s, A); break;
        case 16: hipLaunchKernelGGL((k_qk_backward<T, 16, VEC>), grid, dim3(256), 0, s, A); break;
        case 32: hipLaunchKernelGGL((k_qk_backward<T, 32, VEC>), grid, dim3(256), 0, s, A); break;
        default: hipLaunchKernelGGL((k_qk_backward<T, 64, VEC>), grid, dim3(256), 0, s, A);
    }
}

// Workgroups of the backward.
int64_t parts_of(int64_t T, int64_t heads, int64_t D) {
    const int64_t n = tokens_of(T, heads, D);
    return std::min<int64_t>((T + n - 1) / n, kParts);
}

}  // namespace

size_t qk_norm_rope_bwd_workspace(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
    if (!sizes_ok(T, Hq, Hk, D, 0) || T == 0) return 0;
    return (size_t)parts_of(T, Hq + Hk, D) * D * 4 * 2;
}

}  // namespace mb

using namespace mb;

extern "C" mb_status mb_qk_norm_rope(const void* q, const void* k, const float* q_weight, const float* k_weight, const float* freqs,
                                     const int32_t* positions, void* q_out, void* k_out, int64_t T, int64_t L, int64_t Hq, int64_t Hk,
                                     int64_t D, int64_t R, int64_t q_stride, int64_t k_stride, int64_t q_out_stride,
                                     int64_t k_out_stride, int interleaved, float eps, mb_dtype dtype, hipStream_t stream) {
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (!sizes_ok(T, Hq, Hk, D, R) || !stride_ok(q_stride, Hq * D) || !stride_ok(q_out_stride, Hq * D)) return MB_ERR_SHAPE;
    if (Hk && (!stride_ok(k_stride, Hk * D) || !stride_ok(k_out_stride, Hk * D))) return MB_ERR_SHAPE;
    if ((!positions && L < 1) || !(eps >= 0.0f) || eps > 3.0e38f) return MB_ERR_SHAPE;
    if (T == 0) return MB_OK;
    if (!q || !q_out || (Hk && (!k || !k_out)) || (R && !freqs)) return MB_ERR_NULL;
    if (!Hk) {
        k = k_out = nullptr;
        k_weight = nullptr;
    }
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)q % es || (uintptr_t)k % es || (uintptr_t)q_out % es || (uintptr_t)k_out % es || ((uintptr_t)q_weight & 3) ||
        ((uintptr_t)k_weight & 3) || ((uintptr_t)freqs & 3) || ((uintptr_t)positions & 3))
        return MB_ERR_ALIGN;
    const Span in[4] = {{q_weight, (size_t)D * 4}, {k_weight, (size_t)D * 4}, {freqs, (size_t)R * 2}, {positions, (size_t)T * 4}};
    const Rows x[2] = {{q, q_stride, Hq * D}, {k, k_stride, Hk * D}}, y[2] = {{q_out, q_out_stride, Hq * D}, {k_out, k_out_stride, Hk * D}};
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 2; ++j)
            if (!(i == j && y[i].p == x[j].p && (T == 1 || y[i].stride == x[j].stride)) && rows_overlap(y[i], x[j], T, es)) return MB_ERR_ALIAS;
        if (overlaps_any(y[i].p, span_of(T, y[i].stride, y[i].row, es), in, 4)) return MB_ERR_ALIAS;
    }
    if (rows_overlap(y[0], y[1], T, es)) return MB_ERR_ALIAS;
    QkArgs A{};
    A.in[0] = q; A.in[1] = k; A.out[0] = q_out; A.out[1] = k_out;
    A.w[0] = q_weight; A.w[1] = k_weight;
    A.in_ts[0] = q_stride; A.in_ts[1] = k_stride; A.out_ts[0] = q_out_stride; A.out_ts[1] = k_out_stride;
    A.freqs = freqs; A.positions = positions;
    A.T = T; A.L = L < 1 ? 1 : L; A.H[0] = (int)Hq; A.H[1] = (int)Hk; A.D = (int)D; A.R = (int)R; A.inter = interleaved; A.eps = eps;
    // Few tokens: their heads are dealt out to several workgroups.
    A.tokens = tokens_of(T, Hq + Hk, D);
    int64_t parts = 1;
    const int64_t blocks = (T + A.tokens - 1) / A.tokens, places = 256 / lanes_of(D);
    while (blocks * parts < 2 * device_cu_count() && (Hq + Hk + parts - 1) / parts > places) parts *= 2;
    A.heads = (int)((Hq + Hk + parts - 1) / parts);
    const int64_t groups = (Hq + Hk + A.heads - 1) / A.heads, most = max_workgroups(256) / groups;        // blocks of a launch
    const bool vec = pieces_ok(A, es);
    for (int64_t at = 0; at < blocks; at += most) {
        A.first = at * A.tokens;
        const dim3 grid((unsigned)std::min(most, blocks - at), (unsigned)groups);
        if (dtype == MB_F32) vec ? launch_forward<float, true>(A, grid, stream) : launch_forward<float, false>(A, grid, stream);
        else vec ? launch_forward<bf16, true>(A, grid, stream) : launch_forward<bf16, false>(A, grid, stream);
        const mb_status st = check_launch();
        if (st != MB_OK) return st;
    }
    return MB_OK;
}

extern "C" mb_status mb_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, const float* q_weight,
                                         const float* k_weight, const float* freqs, const int32_t* positions, void* dq, void* dk,
                                         float* dq_weight, float* dk_weight, int64_t T, int64_t L, int64_t Hq, int64_t Hk, int64_t D,
                                         int64_t R, int64_t q_stride, int64_t k_stride, int interleaved, float eps, mb_dtype dtype,
                                         void* ws, size_t ws_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (!sizes_ok(T, Hq, Hk, D, R) || !stride_ok(q_stride, Hq * D) || (Hk && !stride_ok(k_stride, Hk * D))) return MB_ERR_SHAPE;
    if ((!positions && L < 1) || !(eps >= 0.0f) || eps > 3.0e38f) return MB_ERR_SHAPE;
    if (T && (!dq_out || !q || !dq || (Hk && (!dk_out || !k || !dk)) || (R && !freqs))) return MB_ERR_NULL;
    if (!Hk) {
        k = dk_out = dk = nullptr;
        k_weight = nullptr;
        dk_weight = nullptr;
    }
    const size_t es = dtype_size(dtype);
    if ((uintptr_t)q % es || (uintptr_t)k % es || (uintptr_t)dq_out % es || (uintptr_t)dk_out % es || (uintptr_t)dq % es || (uintptr_t)dk % es ||
        ((uintptr_t)q_weight & 3) || ((uintptr_t)k_weight & 3) || ((uintptr_t)freqs & 3) || ((uintptr_t)positions & 3) ||
        ((uintptr_t)dq_weight & 3) || ((uintptr_t)dk_weight & 3))
        return MB_ERR_ALIGN;
    const size_t need = dq_weight || dk_weight ? qk_norm_rope_bwd_workspace(T, Hq, Hk, D) : 0;
    if (need && (!ws || ws_bytes < need || ((uintptr_t)ws & 255))) return MB_ERR_WORKSPACE;
    const size_t nq = (size_t)T * Hq * D * es, nk = (size_t)T * Hk * D * es, nd = (size_t)D * 4;
    const Span ins[8] = {{dq_out, nq}, {dk_out, nk}, {q, span_of(T, q_stride, Hq * D, es)}, {k, span_of(T, k_stride, Hk * D, es)},
                         {q_weight, nd}, {k_weight, nd}, {freqs, (size_t)R * 2}, {positions, (size_t)T * 4}};
    const Span outs[4] = {{dq, nq}, {dk, nk}, {dq_weight, nd}, {dk_weight, nd}};
    for (int i = 0; i < 4; ++i)
        if (overlaps_any(outs[i].p, outs[i].bytes, ins, 8) || overlaps_any(outs[i].p, outs[i].bytes, outs, i)) return MB_ERR_ALIAS;
    if (need && (overlaps_any(ws, need, ins, 8) || overlaps_any(ws, need, outs, 4))) return MB_ERR_ALIAS;
    QkArgs A{};
    A.in[0] = q; A.in[1] = k; A.out[0] = dq; A.out[1] = dk; A.d[0] = dq_out; A.d[1] = dk_out;
    A.w[0] = q_weight; A.w[1] = k_weight;
    A.in_ts[0] = q_stride; A.in_ts[1] = k_stride; A.out_ts[0] = Hq * D; A.out_ts[1] = Hk * D;
    A.freqs = freqs; A.positions = positions;
    A.T = T; A.L = L < 1 ? 1 : L; A.H[0] = (int)Hq; A.H[1] = (int)Hk; A.D = (int)D; A.R = (int)R; A.inter = interleaved; A.eps = eps;
    mb_status st;
    const int64_t parts = T ? parts_of(T, Hq + Hk, D) : 0;
    A.part = need ? (float*)ws : nullptr;
    if (T) {
        A.tokens = tokens_of(T, Hq + Hk, D);
        const dim3 grid((unsigned)parts);
        const bool vec = pieces_ok(A, es);
        if (dtype == MB_F32) vec ? launch_backward<float, true>(A, grid, stream) : launch_backward<float, false>(A, grid, stream);
        else vec ? launch_backward<bf16, true>(A, grid, stream) : launch_backward<bf16, false>(A, grid, stream);
        if ((st = check_launch()) != MB_OK) return st;
    }
    if (!dq_weight && !dk_weight) return MB_OK;
    hipLaunchKernelGGL(k_qk_sum, dim3((unsigned)((D + 31) / 32), 2), dim3(1024), 0, stream, (const float*)A.part, (int)parts, (int)D, dq_weight,
                       dk_weight);
    return check_launch();
}
