// rmsnorm.hip -- root-mean-square norm with the residual's addition, its 8-bit
// output form, and its backward.
//
//     r = x + residual,  rstd = 1 / sqrt(mean_d r_d^2 + eps),  y_d = r_d rstd w_d
//     8 bits: q_d = e4m3(y_d / s), s = max(amax over the group's |y|, 2^-96) / 448
//     backward: g = dy w, xh = r rstd:
//         dr = dr_in + rstd (g - xh mean_d(g xh)),  dw_d = sum_rows dy_d xh_d
//
// All three are bound by HBM: a row is read once, kept in registers between the
// sum of squares and the scaling, and written once.  A row belongs to one wave
// (D <= 1024, some to 2048), a workgroup of 256 (D <= 8192) or of 1024 threads (D <= 16384);
// a thread holds E of its elements as E / VEC vectors, lanes side by side.
// Rows that no vector is aligned to are read and written in vectors all the same, which the memory
// takes at any element's address; only a row's last vector goes element by element.
// Measured: 16384 rows of 2048 bf16 with residual to 8 bits 46.9 us for 237 MB, 5.0 TB/s; 4097 rows of 1001 fp32, none of
// them aligned, 12.7 us for 66 MB, 5.2 TB/s (one element at a time 17.6), 16384 of 1001 bf16 30 us (72);
// four rows 3.4 us, the latency of one load, one sum and one store.  Short rows leave most lanes of their wave idle: 2^20
// rows of 64 bf16 with residual 429 us for 537 MB.
#include "mb_internal.h"

namespace mb {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxMin = 0x1p-96f;     // keeps 1 / scale and y / scale in range for a group of zeros
constexpr int64_t kMaxD = 16384;

// VEC neighbouring elements of a row, `left` of which (and at least one) are in it: those behind read as zero
// and are not written.  AL: pointers and widths are multiples of the vector and a vector lies in the row
// as a whole; otherwise it may start at any element, and the row's last one may be cut short.
template <int VEC, bool AL>
__device__ __forceinline__ void load_vec(const float* p, float* v, int left) {
    if (AL || left >= VEC) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            f4 t;
            if constexpr (AL) t = reinterpret_cast<const f4*>(p)[i];
            else __builtin_memcpy(&t, p + 4 * i, 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * i + k] = t[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = k < left ? p[k] : 0.0f;
    }
}

template <int VEC, bool AL>
__device__ __forceinline__ void load_vec(const bf16* p, float* v, int left) {
    static_assert(VEC == 8, "bf16 vectors hold eight elements");
    if (AL || left >= VEC) {
        u4 t;
        if constexpr (AL) t = *reinterpret_cast<const u4*>(p);
        else __builtin_memcpy(&t, p, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(t[i] << 16);
            v[2 * i + 1] = __uint_as_float(t[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = k < left ? to_f32(p[k]) : 0.0f;
    }
}

template <int VEC, bool AL>
__device__ __forceinline__ void store_vec(float* p, const float* v, int left, bool stream) {
    if (AL || left >= VEC) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const f4 t = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            if constexpr (AL) put(reinterpret_cast<f4*>(p) + i, t, stream);
            else __builtin_memcpy(p + 4 * i, &t, 16);
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (k < left) p[k] = v[k];
    }
}

template <int VEC, bool AL>
__device__ __forceinline__ void store_vec(bf16* p, const float* v, int left, bool stream) {
    if (AL || left >= VEC) {
        u4 t;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t[i] = (uint32_t)f32_to_bf16(v[2 * i]) | ((uint32_t)f32_to_bf16(v[2 * i + 1]) << 16);
        if constexpr (AL) put(reinterpret_cast<u4*>(p), t, stream);
        else __builtin_memcpy(p, &t, 16);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (k < left) p[k] = f32_to_bf16(v[k]);
    }
}

// Sum over the TPR threads of a row, the same value in all of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (TPR > 64) {
        __syncthreads();                       // the previous use of lds is over
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += lds[i];
    }
    return v;
}

// Maximum over the row of absolute values given as bits: NaN's bits are the largest, so NaN wins.
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* lds) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    if constexpr (TPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v = max(v, lds[i]);
    }
    return v;
}

// Scale of a group from its amax bits (NaN stays NaN).
__device__ __forceinline__ float group_scale(uint32_t amax) {
    float a = __uint_as_float(amax);
    a = a < kAmaxMin ? kAmaxMin : a;
    return a / kE4m3Max;
}

// Sum of squares of a row whose squares as they are leave fp32's range, above or, with an eps that does not
// cover it, below: of its values times a power of two (v is left so) that brings the larger of them and of
// sqrt(eps) to between 1 and 4.  Returns it; 1 where there is nothing to scale by: infinities, NaN, zeros alone.
template <int E, int TPR>
__device__ __forceinline__ float rescale(float (&v)[E], float& ss, float eps, float* lds) {
    uint32_t top = __float_as_uint(sqrtf(eps));
#pragma unroll
    for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = row_max<TPR>(top, (uint32_t*)lds);
    if (top == 0 || top >= 0x7f800000u) return 1.0f;
    const float f = __uint_as_float((uint32_t)max(254 - (int)(top >> 23), 1) << 23);
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        v[i] *= f;
        t = fmaf(v[i], v[i], t);
    }
    ss = row_sum<TPR>(t, lds);
    return f;
}

// v / scale: the reciprocal's product with one residual correction is the
// correctly rounded quotient but for rare cases, so values on a border of two
// e4m3 steps fall as they do for the division.  An infinite scale (its group
// then holds infinities) takes the product alone: the residual would be NaN.
__device__ __forceinline__ float over(float v, float scale, float inv) {
    float q = v * inv;
    float c = fmaf(fmaf(-q, scale, v), inv, q);
    return __builtin_isinf(scale) ? q : c;
}

struct NormArgs {
    const void* x;
    const void* res;
    const float* w;
    void* y;
    float* scales;
    void* r_out;
    float* rstd;
    int64_t row0, rows, x_stride;        // row0: first row of the launch
    int D, group, ngroups;
    float eps;
    bool stream;
};

// MODE 0: y in the type of x.  MODE 1: e4m3 with scales.
template <typename TX, typename TR, int VEC, bool AL, int E, int TPR, int MODE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_rms_norm(NormArgs a) {
    constexpr int NT = TPR < 256 ? 256 : TPR;
    constexpr int ROWS = NT / TPR;
    constexpr int NV = E / VEC;
    __shared__ float red[16];
    const int lane = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const int64_t row = a.row0 + (int64_t)blockIdx.x * ROWS + slot;
    const bool live = row < a.rows;
    const TX* x = (const TX*)a.x + row * a.x_stride;
    const TR* res = (const TR*)a.res + row * a.D;

    float v[E];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int d = (c * TPR + lane) * VEC;
        if (live && d < a.D) {
            load_vec<VEC, AL>(x + d, v + c * VEC, a.D - d);
            if (a.res) {
                float t[VEC];
                load_vec<VEC, AL>(res + d, t, a.D - d);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[c * VEC + k] += t[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[c * VEC + k] = 0.0f;
        }
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int d = (c * TPR + lane) * VEC;
        if (a.r_out && live && d < a.D) store_vec<VEC, AL>((TR*)a.r_out + row * a.D + d, v + c * VEC, a.D - d, a.stream);
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss = fmaf(v[c * VEC + k], v[c * VEC + k], ss);
    }
    ss = row_sum<TPR>(ss, red);
    float rstd = 1.0f / sqrtf(ss / (float)a.D + a.eps), rstd_out = rstd;
    // A row's threads agree.  2^-100: squares below fp32's range are off by up to 2^-150 each.
    if (__builtin_expect(ss > 3.0e38f || ss + a.eps < 0x1p-100f, false)) {
        const float f = rescale<E, TPR>(v, ss, a.eps, red);
        rstd = 1.0f / sqrtf(ss / (float)a.D + a.eps * f * f);      // of the values times f
        rstd_out = rstd * f;
    }
    if (a.rstd && live && lane == 0) a.rstd[row] = rstd_out;

#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int d = (c * TPR + lane) * VEC;
        float w[VEC];
        if (a.w && d < a.D) {
            load_vec<VEC, AL>(a.w + d, w, a.D - d);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) w[k] = 1.0f;
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[c * VEC + k] = v[c * VEC + k] * rstd * w[k];
        if constexpr (MODE == 0) {
            if (live && d < a.D) store_vec<VEC, AL>((TX*)a.y + row * a.D + d, v + c * VEC, a.D - d, a.stream);
        }
    }
    if constexpr (MODE == 1) {
        float* scales = a.scales + row * a.ngroups;
        uint8_t* q = (uint8_t*)a.y + row * a.D;
        uint32_t m[NV];
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            m[c] = 0;
#pragma unroll
            for (int k = 0; k < VEC; ++k) m[c] = max(m[c], __float_as_uint(v[c * VEC + k]) & 0x7fffffffu);
        }
        if (a.group == 0) {
            uint32_t t = 0;
#pragma unroll
            for (int c = 0; c < NV; ++c) t = max(t, m[c]);
            t = row_max<TPR>(t, (uint32_t*)red);
#pragma unroll
            for (int c = 0; c < NV; ++c) m[c] = t;
            if (live && lane == 0) scales[0] = group_scale(t);
        } else {
            const int lanes = a.group / VEC;       // a power of two, at most 32
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                for (int o = 1; o < lanes; o <<= 1) m[c] = max(m[c], (uint32_t)__shfl_xor((int)m[c], o));
                const int d = (c * TPR + lane) * VEC;
                if (live && d < a.D && (lane & (lanes - 1)) == 0) scales[d / a.group] = group_scale(m[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int d = (c * TPR + lane) * VEC;
            const float s = group_scale(m[c]), inv = 1.0f / s;
            if (live && d < a.D) {
                float t[VEC];
#pragma unroll
                for (int k = 0; k < VEC; ++k) t[k] = over(v[c * VEC + k], s, inv);
                uint32_t o[VEC / 4];
#pragma unroll
                for (int k = 0; k < VEC / 4; ++k) {
                    int p = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * k], t[4 * k + 1], 0, false);
                    o[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[4 * k + 2], t[4 * k + 3], p, true);
                }
                if constexpr (AL) {
                    if constexpr (VEC == 8) put(reinterpret_cast<u2*>(q + d), u2{o[0], o[1]}, a.stream);
                    else put(reinterpret_cast<uint32_t*>(q + d), o[0], a.stream);
                } else if (a.D - d >= VEC) {
                    __builtin_memcpy(q + d, o, VEC);
                } else {
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        if (k < a.D - d) q[d + k] = (uint8_t)(o[k / 4] >> (8 * (k % 4)));
                }
            }
        }
    }
}

struct NormBwdArgs {
    const void* dy;
    const void* r;
    const float* rstd;
    const float* w;
    const void* dr_in;
    void* dx;
    void* dr;
    float* part;        // (gridDim.x, D) partial sums of dw, or dw itself when the grid is one workgroup
    int64_t rows;
    int D;
};

// A workgroup walks rows; every thread keeps its columns' share of dw in registers
// and the rows' slots are added up in LDS at the end.  16384 rows of 1536, bf16 with fp32 residual: 76 us for
// 403 MB, 5.3 TB/s, and 4.7 us for the sum over workgroups.
template <typename TX, typename TR, int VEC, bool AL, int E, int TPR>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_rms_norm_bwd(NormBwdArgs a) {
    constexpr int NT = TPR < 256 ? 256 : TPR;
    constexpr int ROWS = NT / TPR;
    constexpr int NV = E / VEC;
    __shared__ float red[16];
    __shared__ float dwl[ROWS > 1 ? (ROWS - 1) * TPR * E : 1];
    const int lane = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    float dw[E], w[E];
#pragma unroll
    for (int i = 0; i < E; ++i) { dw[i] = 0.0f; w[i] = 1.0f; }
    if (a.w) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int d = (c * TPR + lane) * VEC;
            if (d < a.D) load_vec<VEC, AL>(a.w + d, w + c * VEC, a.D - d);
        }
    }
    const float inv_d = 1.0f / (float)a.D;
    for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.rows; base += (int64_t)gridDim.x * ROWS) {
        const int64_t row = base + slot;
        const bool live = row < a.rows;
        float dy[E], xh[E], in[E];
        const float rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int d = (c * TPR + lane) * VEC;
            if (live && d < a.D) {
                load_vec<VEC, AL>((const TX*)a.dy + row * a.D + d, dy + c * VEC, a.D - d);
                load_vec<VEC, AL>((const TR*)a.r + row * a.D + d, xh + c * VEC, a.D - d);
                if (a.dr_in) {
                    load_vec<VEC, AL>((const TR*)a.dr_in + row * a.D + d, in + c * VEC, a.D - d);
                } else {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) in[c * VEC + k] = 0.0f;
                }
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k) dy[c * VEC + k] = xh[c * VEC + k] = in[c * VEC + k] = 0.0f;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            xh[i] *= rstd;
            dw[i] = fmaf(dy[i], xh[i], dw[i]);
            dy[i] *= w[i];
            dot = fmaf(dy[i], xh[i], dot);
        }
        dot = row_sum<TPR>(dot, red) * inv_d;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int d = (c * TPR + lane) * VEC;
            if (live && d < a.D) {
                float o[VEC];
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    o[k] = fmaf(rstd, fmaf(-xh[c * VEC + k], dot, dy[c * VEC + k]), in[c * VEC + k]);
                if (a.dr) store_vec<VEC, AL>((TR*)a.dr + row * a.D + d, o, a.D - d, false);
                if (a.dx) store_vec<VEC, AL>((TX*)a.dx + row * a.D + d, o, a.D - d, false);
            }
        }
    }
    if (!a.part) return;
    if constexpr (ROWS > 1) {
        if (slot > 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) dwl[((slot - 1) * E + i) * TPR + lane] = dw[i];
        }
        __syncthreads();
        if (slot > 0) return;
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int s = 0; s < ROWS - 1; ++s) dw[i] += dwl[(s * E + i) * TPR + lane];
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int d = (c * TPR + lane) * VEC;
        if (d < a.D) store_vec<VEC, AL>(a.part + (int64_t)blockIdx.x * a.D + d, dw + c * VEC, a.D - d, false);
    }
}

// dw = the sum of the workgroups' partial rows: 32 columns a workgroup, the rows dealt to its
// VEC * 8 groups of lanes, eight reads of each under way at a time.
template <int VEC>
__global__ void __launch_bounds__(256) k_dw_sum(const float* __restrict__ part, float* __restrict__ dw, int n, int D) {
    constexpr int LN = 32 / VEC, SUB = 256 / LN;
    __shared__ float red[SUB][33];
    const int ln = threadIdx.x % LN, sub = threadIdx.x / LN;
    const int d = blockIdx.x * 32 + ln * VEC;
    float s[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[k] = 0.0f;
    if (d < D)
        for (int i = sub; i < n; i += 8 * SUB) {
            float t[8][VEC];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (i + j * SUB < n) {
                    if constexpr (VEC == 1) t[j][0] = part[(int64_t)(i + j * SUB) * D + d];
                    else load_vec<VEC, true>(part + (int64_t)(i + j * SUB) * D + d, t[j], VEC);
                } else {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) t[j][k] = 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int k = 0; k < VEC; ++k) s[k] += t[j][k];
        }
#pragma unroll
    for (int k = 0; k < VEC; ++k) red[sub][ln * VEC + k] = s[k];
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + (int)threadIdx.x < D) {
        float x = 0.0f;
#pragma unroll 8
        for (int i = 0; i < SUB; ++i) x += red[i][threadIdx.x];
        dw[blockIdx.x * 32 + threadIdx.x] = x;
    }
}

inline bool vec_ok(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename TX, typename TR, int MODE, int VEC, bool AL>
mb_status launch_norm(NormArgs a, hipStream_t s) {
    const int per = a.D;
    mb_status st = MB_OK;
    auto go = [&](auto kern, int nt, int rows) {
        const int64_t most = max_workgroups(nt) * rows;              // rows of a launch
        for (; a.row0 < a.rows && st == MB_OK; a.row0 += most) {
            const int64_t n = a.rows - a.row0 < most ? a.rows - a.row0 : most;
            hipLaunchKernelGGL(kern, dim3((unsigned)((n + rows - 1) / rows)), dim3(nt), 0, s, a);
            st = check_launch();
        }
    };
    // A whole row in one wave needs no barrier; of 32 values a thread it reads at lower rate than a
    // workgroup of 8 a thread does, as long as that leaves few threads idle.  16384 rows, wave and workgroup:
    // bf16 of 2048 columns 50.4 and 47.9 us (to 8 bits 51.0 and 47.4), of 1536 to 8 bits 41.0 and 44.3;
    // fp32 of 1280 65 and 58.4.
    constexpr bool F32 = sizeof(TX) == 4;
    if (per <= 64 * 8) go(k_rms_norm<TX, TR, VEC, AL, 8, 64, MODE>, 256, 4);
    else if (per <= 64 * 16) go(k_rms_norm<TX, TR, VEC, AL, 16, 64, MODE>, 256, 4);
    else if (per > (F32 ? 1024 : 1792) && per <= 256 * 8) go(k_rms_norm<TX, TR, VEC, AL, 8, 256, MODE>, 256, 1);
    else if (per <= 64 * 32) go(k_rms_norm<TX, TR, VEC, AL, 32, 64, MODE>, 256, 4);
    else if (per <= 256 * 16) go(k_rms_norm<TX, TR, VEC, AL, 16, 256, MODE>, 256, 1);
    else if (per <= 256 * 32) go(k_rms_norm<TX, TR, VEC, AL, 32, 256, MODE>, 256, 1);
    else go(k_rms_norm<TX, TR, VEC, AL, 16, 1024, MODE>, 1024, 1);
    return st;
}

template <int MODE>
mb_status norm(const void* x, const void* res, const float* w, void* y, float* scales, void* r_out, float* rstd,
               int64_t rows, int64_t D, int64_t x_stride, int64_t group, float eps, mb_dtype dtype, mb_dtype rdtype,
               hipStream_t stream) {
    if (!dtype_ok(dtype) || !dtype_ok(rdtype) || (rdtype == MB_BF16 && dtype == MB_F32)) return MB_ERR_DTYPE;
    if (rows < 0 || D < 1 || D > kMaxD || x_stride < D || !(eps >= 0.0f) || eps > 3.0e38f) return MB_ERR_SHAPE;
    if (rows > (int64_t)1 << 30 || x_stride > 0x7fffffff) return MB_ERR_SHAPE;
    if (MODE == 1 && group != 0 && group != 32 && group != 64 && group != 128) return MB_ERR_SHAPE;
    if (rows == 0) return MB_OK;
    if (!x || !y || (MODE == 1 && !scales)) return MB_ERR_NULL;
    const size_t ex = dtype_size(dtype), er = dtype_size(rdtype);
    const int64_t ng = group ? (D + group - 1) / group : 1;
    const size_t n = (size_t)rows * D;
    const size_t nx = ((size_t)(rows - 1) * x_stride + D) * ex;
    if (((uintptr_t)x % ex) || ((uintptr_t)res % er) || ((uintptr_t)r_out % er) || (MODE == 0 && (uintptr_t)y % ex) ||
        ((uintptr_t)w & 3) || ((uintptr_t)scales & 3) || ((uintptr_t)rstd & 3))
        return MB_ERR_ALIGN;
    const Span ins[3] = {{x, nx}, {res, n * er}, {w, (size_t)D * 4}};
    Span outs[4] = {{y, n * (MODE == 1 ? 1 : ex)}, {r_out, n * er}, {rstd, (size_t)rows * 4}, {scales, (size_t)rows * ng * 4}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j) {
            if (i == 1 && j == 1 && r_out == res) continue;      // the residual stream is updated in place
            if (overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return MB_ERR_ALIAS;
        }
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return MB_ERR_ALIAS;
    }
    NormArgs a{x, res, w, y, scales, r_out, rstd, 0, rows, x_stride, (int)D, (int)group, (int)ng, eps,
               nx + outs[0].bytes + (res ? n * er : 0) + (r_out ? n * er : 0) > kStreamBytes};
    const int V = dtype == MB_BF16 ? 8 : 4;
    const bool vec = D % V == 0 && x_stride % V == 0 && vec_ok(x) && vec_ok(res) && vec_ok(w) && vec_ok(y) && vec_ok(r_out);
    if (dtype == MB_F32)
        return vec ? launch_norm<float, float, MODE, 4, true>(a, stream) : launch_norm<float, float, MODE, 4, false>(a, stream);
    if (rdtype == MB_F32)
        return vec ? launch_norm<bf16, float, MODE, 8, true>(a, stream) : launch_norm<bf16, float, MODE, 8, false>(a, stream);
    return vec ? launch_norm<bf16, bf16, MODE, 8, true>(a, stream) : launch_norm<bf16, bf16, MODE, 8, false>(a, stream);
}

// Workgroups of the backward: enough to fill the device twice, so that the partial
// rows of dw stay few (the call above: once 79.4, twice 79.6, four times 81.5 us).
int bwd_grid(int64_t rows, int64_t D) {
    const int64_t per = D <= 2048 ? 4 : 1;
    const int64_t want = (rows + per - 1) / per, cap = 2 * (int64_t)device_cu_count();
    return (int)(want < cap ? want : cap);
}

template <typename TX, typename TR, int VEC, bool AL>
void launch_bwd(const NormBwdArgs& a, int grid, hipStream_t s) {
    auto go = [&](auto kern, int nt) { hipLaunchKernelGGL(kern, dim3(grid), dim3(nt), 0, s, a); };
    if (a.D <= 64 * 8) go(k_rms_norm_bwd<TX, TR, VEC, AL, 8, 64>, 256);
    else if (a.D <= 64 * 16) go(k_rms_norm_bwd<TX, TR, VEC, AL, 16, 64>, 256);
    else if (a.D <= 64 * 32) go(k_rms_norm_bwd<TX, TR, VEC, AL, 32, 64>, 256);
    else if (a.D <= 256 * 16) go(k_rms_norm_bwd<TX, TR, VEC, AL, 16, 256>, 256);
    else if (a.D <= 256 * 32) go(k_rms_norm_bwd<TX, TR, VEC, AL, 32, 256>, 256);
    else go(k_rms_norm_bwd<TX, TR, VEC, AL, 16, 1024>, 1024);
}

}  // namespace

size_t rms_norm_bwd_workspace(int64_t rows, int64_t D) {
    if (rows < 1 || D < 1 || D > kMaxD || rows > (int64_t)1 << 30) return 0;
    const int g = bwd_grid(rows, D);
    return g == 1 ? 0 : ((size_t)g * D * 4 + 255) / 256 * 256;
}

}  // namespace mb

extern "C" mb_status mb_rms_norm(const void* x, const void* residual, const float* weight, void* y, void* residual_out,
                                 float* rstd, int64_t rows, int64_t D, int64_t x_stride, float eps, mb_dtype dtype,
                                 mb_dtype residual_dtype, hipStream_t stream) {
    return mb::norm<0>(x, residual, weight, y, nullptr, residual_out, rstd, rows, D, x_stride, 0, eps, dtype,
                       residual_dtype, stream);
}

extern "C" mb_status mb_rms_norm_fp8(const void* x, const void* residual, const float* weight, void* y, float* scales,
                                     void* residual_out, float* rstd, int64_t rows, int64_t D, int64_t x_stride,
                                     int64_t group, float eps, mb_dtype dtype, mb_dtype residual_dtype,
                                     hipStream_t stream) {
    return mb::norm<1>(x, residual, weight, y, scales, residual_out, rstd, rows, D, x_stride, group, eps, dtype,
                       residual_dtype, stream);
}

extern "C" mb_status mb_rms_norm_bwd(const void* dy, const void* r, const float* rstd, const float* weight,
                                     const void* dr_in, void* dx, void* dr, float* dweight, int64_t rows, int64_t D,
                                     mb_dtype dtype, mb_dtype residual_dtype, void* ws, size_t ws_bytes,
                                     hipStream_t stream) {
    using namespace mb;
    if (!dtype_ok(dtype) || !dtype_ok(residual_dtype) || (residual_dtype == MB_BF16 && dtype == MB_F32)) return MB_ERR_DTYPE;
    if (rows < 0 || D < 1 || D > kMaxD || rows > (int64_t)1 << 30) return MB_ERR_SHAPE;
    if (rows == 0) return dweight ? copy_state(nullptr, dweight, D, stream) : MB_OK;
    if (!dy || !r || !rstd || (!dx && !dr && !dweight)) return MB_ERR_NULL;
    const size_t ex = dtype_size(dtype), er = dtype_size(residual_dtype), n = (size_t)rows * D;
    if (((uintptr_t)dy % ex) || ((uintptr_t)dx % ex) || ((uintptr_t)r % er) || ((uintptr_t)dr_in % er) ||
        ((uintptr_t)dr % er) || ((uintptr_t)rstd & 3) || ((uintptr_t)weight & 3) || ((uintptr_t)dweight & 3))
        return MB_ERR_ALIGN;
    const size_t need = dweight ? rms_norm_bwd_workspace(rows, D) : 0;
    if (need && (!ws || ws_bytes < need || ((uintptr_t)ws & 255))) return MB_ERR_WORKSPACE;
    const Span ins[5] = {{dy, n * ex}, {r, n * er}, {rstd, (size_t)rows * 4}, {weight, (size_t)D * 4}, {dr_in, n * er}};
    const Span outs[4] = {{dx, n * ex}, {dr, n * er}, {dweight, (size_t)D * 4}, {need ? ws : nullptr, need}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j) {
            if (i == 1 && j == 4 && dr == dr_in) continue;      // the stream's gradient is updated in place
            if (overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return MB_ERR_ALIAS;
        }
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return MB_ERR_ALIAS;
    }
    const int grid = bwd_grid(rows, D);
    float* part = !dweight ? nullptr : need ? (float*)ws : dweight;
    NormBwdArgs a{dy, r, rstd, weight, dr_in, dx, dr, part, rows, (int)D};
    const int V = dtype == MB_BF16 ? 8 : 4;
    const bool vec = D % V == 0 && vec_ok(dy) && vec_ok(r) && vec_ok(weight) && vec_ok(dr_in) && vec_ok(dx) && vec_ok(dr) &&
                     vec_ok(part);
    if (dtype == MB_F32)
        vec ? launch_bwd<float, float, 4, true>(a, grid, stream) : launch_bwd<float, float, 4, false>(a, grid, stream);
    else if (residual_dtype == MB_F32)
        vec ? launch_bwd<bf16, float, 8, true>(a, grid, stream) : launch_bwd<bf16, float, 8, false>(a, grid, stream);
    else
        vec ? launch_bwd<bf16, bf16, 8, true>(a, grid, stream) : launch_bwd<bf16, bf16, 8, false>(a, grid, stream);
    mb_status st = check_launch();
    if (st != MB_OK || !need) return st;
    const dim3 cols((unsigned)((D + 31) / 32));
    if (D % 4 == 0) hipLaunchKernelGGL(k_dw_sum<4>, cols, dim3(256), 0, stream, (const float*)ws, dweight, grid, (int)D);
    else hipLaunchKernelGGL(k_dw_sum<1>, cols, dim3(256), 0, stream, (const float*)ws, dweight, grid, (int)D);
    return check_launch();
}
