// qknorm.hip -- root-mean-square norm of every head of queries and keys with the rotation by their position, and its
// backward.
//
//     n = x / sqrt(mean x^2 + eps) * w;   pairs (u, v) of n turn by the angle position * freqs[j]
//     backward: e = the gradient turned back, xh = x rstd, g = e w:
//         dx = rstd (g - xh mean(g xh)),  dw = sum e xh
//
// A wave takes one head of one token at a time.
#include "mb_internal.h"

namespace mb {
namespace {

constexpr int kMaxD = 512, kE = kMaxD / 64;
constexpr int kParts = 256;       // workgroups of the backward, each with its own share of dw

struct QkArgs {
    const void* in[2];        // queries, keys
    void* out[2];
    const void* d[2];         // backward: their outputs' gradients
    const float* w[2];
    float* part[2];
    int64_t in_ts[2], out_ts[2];
    const float* freqs;
    const int32_t* positions;
    int64_t T, L;
    int H[2], D, R, inter;
    float eps;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Columns of element i of lane: pairs' members beside each other in a lane.  -1: none.
__device__ __forceinline__ int column(const QkArgs& A, int lane, int i) {
    const int p = (i / 2) * 64 + lane, o = i & 1;
    if (2 * p < A.R) return A.inter ? 2 * p + o : p + o * (A.R / 2);
    return 2 * p + o < A.D ? 2 * p + o : -1;
}

__device__ __forceinline__ void turn(const QkArgs& A, int64_t pos, int lane, int i, float& c, float& s) {
    const int p = i * 64 + lane;
    c = 1.0f;
    s = 0.0f;
    if (2 * p < A.R) {
        const double r = (double)pos * (double)A.freqs[p] * 0.15915494309189533577;
        sincospif(2.0f * (float)(r - rint(r)), &s, &c);
    }
}

template <typename T, bool BACK>
__global__ void __launch_bounds__(256) k_qk(QkArgs A) {
    __shared__ float red[4][2][kMaxD];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int heads = A.H[0] + A.H[1];
    float dw[2][kE];
    for (int i = 0; i < kE; ++i) dw[0][i] = dw[1][i] = 0.0f;
    for (int64_t r = (int64_t)blockIdx.x * 4 + wave; r < A.T * heads; r += (int64_t)gridDim.x * 4) {
        const int64_t t = r / heads;
        const int hh = (int)(r - t * heads), k = hh >= A.H[0], h = hh - (k ? A.H[0] : 0);
        const int64_t pos = A.positions ? A.positions[t] : t % A.L;
        const T* x = (const T*)A.in[k] + t * A.in_ts[k] + (int64_t)h * A.D;
        float v[kE], top = 0.0f, ss = 0.0f;
        for (int i = 0; i < kE; ++i) {
            const int d = column(A, lane, i);
            v[i] = d >= 0 ? to_f32(x[d]) : 0.0f;
            ss = fmaf(v[i], v[i], ss);
            top = fmaxf(top, fabsf(v[i]));
        }
        ss = wave_sum(ss);
        float rs = 1.0f / sqrtf(ss / (float)A.D + A.eps);
        if (ss > 3.0e38f || ss + A.eps < 0x1p-100f) {
            for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
            top = fmaxf(top, sqrtf(A.eps));
            if (top > 0.0f && top < 3.4e38f) {
                const float f = exp2f(-(float)ilogbf(top));
                ss = 0.0f;
                for (int i = 0; i < kE; ++i) ss = fmaf(v[i] * f, v[i] * f, ss);
                rs = f / sqrtf(wave_sum(ss) / (float)A.D + A.eps * f * f);
            }
        }
        float w[kE], c[kE / 2], s[kE / 2];
        for (int i = 0; i < kE; ++i) {
            const int d = column(A, lane, i);
            w[i] = A.w[k] && d >= 0 ? A.w[k][d] : 1.0f;
        }
        for (int i = 0; i < kE / 2; ++i) turn(A, pos, lane, i, c[i], s[i]);
        const int64_t at = t * A.out_ts[k] + (int64_t)h * A.D;
        if (!BACK) {
            for (int i = 0; i < kE; i += 2) {
                const float a = v[i] * rs * w[i], b = v[i + 1] * rs * w[i + 1];
                const int d0 = column(A, lane, i), d1 = column(A, lane, i + 1);
                if (d0 >= 0) store_out((T*)A.out[k] + at + d0, 2 * ((i / 2) * 64 + lane) < A.R ? a * c[i / 2] - b * s[i / 2] : a);
                if (d1 >= 0) store_out((T*)A.out[k] + at + d1, 2 * ((i / 2) * 64 + lane) < A.R ? a * s[i / 2] + b * c[i / 2] : b);
            }
        } else {
            float dot = 0.0f, g[kE];
            for (int i = 0; i < kE; i += 2) {
                const int d0 = column(A, lane, i), d1 = column(A, lane, i + 1);
                const float a = d0 >= 0 ? to_f32(((const T*)A.d[k])[at + d0]) : 0.0f, b = d1 >= 0 ? to_f32(((const T*)A.d[k])[at + d1]) : 0.0f;
                g[i] = a * c[i / 2] + b * s[i / 2];
                g[i + 1] = b * c[i / 2] - a * s[i / 2];
            }
            for (int i = 0; i < kE; ++i) {
                v[i] *= rs;
                dw[k][i] += g[i] * v[i];
                g[i] *= w[i];
                dot = fmaf(g[i], v[i], dot);
            }
            dot = wave_sum(dot) / (float)A.D;
            for (int i = 0; i < kE; ++i) {
                const int d = column(A, lane, i);
                if (d >= 0) store_out((T*)A.out[k] + at + d, rs * (g[i] - v[i] * dot));
            }
        }
    }
    if (BACK) {
        for (int k = 0; k < 2; ++k)
            for (int i = 0; i < kE; ++i) {
                const int d = column(A, lane, i);
                if (d >= 0) red[wave][k][d] = dw[k][i];
            }
        __syncthreads();
        for (int k = 0; k < 2; ++k)
            for (int d = threadIdx.x; d < A.D; d += 256)
                if (A.part[k]) A.part[k][(int64_t)blockIdx.x * A.D + d] = red[0][k][d] + red[1][k][d] + red[2][k][d] + red[3][k][d];
    }
}

__global__ void __launch_bounds__(256) k_qk_sum(const float* part, int n, int D, float* dw) {
    const int d = blockIdx.x * 256 + threadIdx.x;
    if (d >= D) return;
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s += part[(int64_t)i * D + d];
    dw[d] = s;
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

}  // namespace

size_t qk_norm_rope_bwd_workspace(int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
    if (!sizes_ok(T, Hq, Hk, D, 0) || T == 0) return 0;
    return (size_t)kParts * D * 4 * 2;
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
    const int64_t rows = T * (Hq + Hk);
    const dim3 grid((unsigned)(rows < 4 * 65536 ? (rows + 3) / 4 : 65536));
    if (dtype == MB_F32) hipLaunchKernelGGL((k_qk<float, false>), grid, dim3(256), 0, stream, A);
    else hipLaunchKernelGGL((k_qk<bf16, false>), grid, dim3(256), 0, stream, A);
    return check_launch();
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
    A.part[0] = dq_weight ? (float*)ws : nullptr;
    A.part[1] = dk_weight ? (float*)ws + (size_t)kParts * D : nullptr;
    mb_status st;
    if (T) {
        if (dtype == MB_F32) hipLaunchKernelGGL((k_qk<float, true>), dim3(kParts), dim3(256), 0, stream, A);
        else hipLaunchKernelGGL((k_qk<bf16, true>), dim3(kParts), dim3(256), 0, stream, A);
        if ((st = check_launch()) != MB_OK) return st;
    }
    float* dw[2] = {dq_weight, dk_weight};
    for (int i = 0; i < 2; ++i)
        if (dw[i]) {
            hipLaunchKernelGGL(k_qk_sum, dim3((unsigned)((D + 255) / 256)), dim3(256), 0, stream, A.part[i], T ? kParts : 0, (int)D, dw[i]);
            if ((st = check_launch()) != MB_OK) return st;
        }
    return MB_OK;
}
