// gatedscan.hip -- gated linear recurrence with a decay per channel and token, its single-token step and its backward.
//
//     s = sigma(a_gate + a_bias), la = -decay s, a = e^la, beta = sqrt(1 - a^2)
//     b = beta sigma(x_gate + x_bias) x,  h_t = a_t h_{t-1} + b_t,  y = h
//
// A lane walks one channel of one sequence.
#include "mb_internal.h"

namespace mb {
namespace {

constexpr int kEvery = 64;       // tokens between the rows of states

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
    const float* dh_out;
    void *dx, *da, *dg;
    float* dh0;
    float *before, *part;
    int n_seq, T, L, D;
};

struct Gate {
    float s, la, a, b1, beta, i;     // b1 = 1 - a^2
};

template <typename T>
__device__ __forceinline__ Gate gate(const GsArgs& A, int64_t t, int c) {
    Gate r;
    const float va = to_f32(((const T*)A.a)[t * A.a_ts + c]) + (A.a_bias ? A.a_bias[c] : 0.0f);
    r.s = 1.0f / (1.0f + expf(-va));
    r.la = -A.decay[c] * r.s;
    const float e = expm1f(r.la);
    r.a = expf(r.la);                 // 1 + e has lost the digits of a small a
    r.b1 = -e * (2.0f + e);
    r.beta = sqrtf(r.b1);
    r.i = 1.0f;
    if (A.g) r.i = 1.0f / (1.0f + expf(-(to_f32(((const T*)A.g)[t * A.g_ts + c]) + (A.x_bias ? A.x_bias[c] : 0.0f))));
    return r;
}

__device__ __forceinline__ void range(const GsArgs& A, int s, int& b, int& e) {
    if (A.cu) {
        b = min(max(A.cu[s], 0), A.T);
        e = min(max(A.cu[s + 1], 0), A.T);
    } else {
        b = s * A.L;
        e = b + A.L;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_gs_walk(GsArgs A) {
    const int c = blockIdx.x * 256 + threadIdx.x, s = blockIdx.y;
    if (c >= A.D) return;
    int b, e;
    range(A, s, b, e);
    int64_t row = s;
    if (A.slots) {
        row = A.slots[s];
        if (row < 0 || row >= A.n_slots) row = -1;
    }
    float h = A.h0 && row >= 0 && (!A.has_h0 || A.has_h0[s]) ? A.h0[row * A.D + c] : 0.0f;
    for (int t = b; t < e; ++t) {
        const Gate r = gate<T>(A, t, c);
        if (A.states && t % kEvery == 0) A.states[(int64_t)(t / kEvery) * A.D + c] = h;
        h = fmaf(r.a, h, r.beta * r.i * to_f32(((const T*)A.x)[t * A.x_ts + c]));
        store_out((T*)A.y + (int64_t)t * A.D + c, h);
    }
    if (A.h_out && row >= 0) A.h_out[row * A.D + c] = h;
}

template <typename T>
__global__ void __launch_bounds__(256) k_gs_back(GsArgs A) {
    const int c = blockIdx.x * 256 + threadIdx.x, s = blockIdx.y;
    if (c >= A.D) return;
    int b, e;
    range(A, s, b, e);
    float h = A.h0 ? A.h0[(int64_t)s * A.D + c] : 0.0f;
    for (int t = b; t < e; ++t) {
        const Gate r = gate<T>(A, t, c);
        A.before[(int64_t)t * A.D + c] = h;
        h = fmaf(r.a, h, r.beta * r.i * to_f32(((const T*)A.x)[t * A.x_ts + c]));
    }
    float G = A.dh_out ? A.dh_out[(int64_t)s * A.D + c] : 0.0f;
    float sd = 0.0f, sa = 0.0f, sx = 0.0f;
    for (int t = e - 1; t >= b; --t) {
        const Gate r = gate<T>(A, t, c);
        const int64_t at = (int64_t)t * A.D + c;
        const float x = to_f32(((const T*)A.x)[t * A.x_ts + c]);
        G += to_f32(((const T*)A.dy)[at]);
        const float bb = r.beta * r.i * x, root = r.b1 < 0x1p-120f ? 0.0f : bb / r.b1;
        const float dla = G * (r.a * A.before[at] - r.a * r.a * root);
        const float va = to_f32(((const T*)A.a)[t * A.a_ts + c]) + (A.a_bias ? A.a_bias[c] : 0.0f);
        const float da = dla * r.la / (1.0f + expf(va));
        store_out((T*)A.dx + at, G * r.beta * r.i);
        store_out((T*)A.da + at, da);
        sd -= dla * r.s;
        sa += da;
        if (A.g) {
            const float vg = to_f32(((const T*)A.g)[t * A.g_ts + c]) + (A.x_bias ? A.x_bias[c] : 0.0f);
            const float dg = G * bb / (1.0f + expf(vg));
            store_out((T*)A.dg + at, dg);
            sx += dg;
        }
        G *= r.a;
    }
    if (A.dh0) A.dh0[(int64_t)s * A.D + c] = G;
    float* p = A.part + (int64_t)s * 3 * A.D + c;
    p[0] = sd;
    p[A.D] = sa;
    p[2 * (int64_t)A.D] = sx;
}

template <typename T>
__global__ void __launch_bounds__(256) k_gs_clear(GsArgs A) {
    const int64_t t = blockIdx.x;
    const int b = A.n_seq ? min(max(A.cu[0], 0), A.T) : A.T, e = min(max(A.cu[A.n_seq], 0), A.T);
    if (t >= b && t < e) return;
    for (int c = threadIdx.x; c < A.D; c += 256) {
        const int64_t at = t * A.D + c;
        store_out((T*)A.dx + at, 0.0f);
        store_out((T*)A.da + at, 0.0f);
        if (A.g) store_out((T*)A.dg + at, 0.0f);
    }
}

__global__ void __launch_bounds__(256) k_gs_sums(const float* part, int n, int D, float* d0, float* d1, float* d2) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= D) return;
    float s[3] = {0.0f, 0.0f, 0.0f};
    for (int i = 0; i < n; ++i)
        for (int k = 0; k < 3; ++k) s[k] += part[((int64_t)i * 3 + k) * D + c];
    if (d0) d0[c] = s[0];
    if (d1) d1[c] = s[1];
    if (d2) d2[c] = s[2];
}

template <typename T>
__global__ void __launch_bounds__(256) k_gs_step(GsArgs A, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n * A.D) return;
    const int64_t r = i / A.D;
    const int c = (int)(i - r * A.D);
    int64_t row = r;
    if (A.slots) {
        row = A.slots[r];
        if (row < 0 || row >= A.n_slots) row = -1;
    }
    const Gate q = gate<T>(A, r, c);
    const float h0 = A.h0 && row >= 0 ? A.h0[row * A.D + c] : 0.0f;
    const float h = fmaf(q.a, h0, q.beta * q.i * to_f32(((const T*)A.x)[r * A.x_ts + c]));
    store_out((T*)A.y + i, h);
    if (row >= 0) A.h_out[row * A.D + c] = h;
}

// ------------------------------------------------------------------ host ----
constexpr int kTile = 128, kCols = 64;      // tokens and channels of a tile

bool sizes_ok(int64_t n_seq, int64_t T, int64_t D) {
    if (n_seq < 0 || T < 0 || D < 1 || D >= 1 << 22 || n_seq > 1 << 20 || T >= (int64_t)1 << 31) return false;
    return ((T + kTile - 1) / kTile) * ((D + kCols - 1) / kCols) < (int64_t)1 << 24;
}

bool stride_ok(int64_t s, int64_t D) { return s >= D && s < 1 << 22; }

size_t span_of(int64_t tokens, int64_t stride, int64_t row, size_t es) {
    return tokens > 0 ? ((size_t)(tokens - 1) * stride + row) * es : 0;
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
    return 0;
}

size_t gated_scan_bwd_workspace(int64_t n_seq, int64_t T, int64_t D) {
    if (!sizes_ok(n_seq, T, D)) return 0;
    return (size_t)T * D * 4 + (size_t)n_seq * 3 * D * 4;
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
    const dim3 grid((unsigned)((D + 255) / 256), (unsigned)n_seq);
    if (dtype == MB_F32) hipLaunchKernelGGL(k_gs_walk<float>, grid, dim3(256), 0, stream, A);
    else hipLaunchKernelGGL(k_gs_walk<bf16>, grid, dim3(256), 0, stream, A);
    return check_launch();
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
    const dim3 grid((unsigned)((n * D + 255) / 256));
    if (dtype == MB_F32) hipLaunchKernelGGL(k_gs_step<float>, grid, dim3(256), 0, stream, A, n);
    else hipLaunchKernelGGL(k_gs_step<bf16>, grid, dim3(256), 0, stream, A, n);
    return check_launch();
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
    A.cu = cu_seqlens; A.h0 = h0; A.dy = dy; A.dh_out = dh_out; A.states = const_cast<float*>(states);
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
    A.before = (float*)ws;
    A.part = A.before + T * D;
    const unsigned cols = (unsigned)((D + 255) / 256);
    if (n_seq) {
        const dim3 grid(cols, (unsigned)n_seq);
        if (dtype == MB_F32) hipLaunchKernelGGL(k_gs_back<float>, grid, dim3(256), 0, stream, A);
        else hipLaunchKernelGGL(k_gs_back<bf16>, grid, dim3(256), 0, stream, A);
        if ((st = check_launch()) != MB_OK) return st;
    }
    if (cu_seqlens && T) {
        if (dtype == MB_F32) hipLaunchKernelGGL(k_gs_clear<float>, dim3((unsigned)T), dim3(256), 0, stream, A);
        else hipLaunchKernelGGL(k_gs_clear<bf16>, dim3((unsigned)T), dim3(256), 0, stream, A);
        if ((st = check_launch()) != MB_OK) return st;
    }
    hipLaunchKernelGGL(k_gs_sums, dim3(cols), dim3(256), 0, stream, A.part, A.n_seq, A.D, ddecay, da_bias, dx_bias);
    return check_launch();
}
