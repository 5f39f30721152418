// gradclip.hip -- the global 2-norm of many gradient tensors, and their clipping.
//
//     norm = sqrt(sum over all tensors and elements of g^2)
//     out  = g * min(1, max_norm / (norm + eps))
//
// Bound by HBM: the gradients are read once for the norm and once more, with a
// write, for the scaling.  Each square is summed in fp64: no fp32 gradient's
// square overflows or vanishes there, and the two extra fp64 operations an element
// cost less than its load.  129 M bf16 gradients of 24 layers, which the last-level cache cannot hold: norm 47 us
// for 258 MB (5.5 TB/s), scaling 89 us for 517 MB (5.8 TB/s); pieces of twice the size, or half or twice as many
// workgroups, change neither by 2 %.  A workgroup's sum goes to its own place in the
// workspace and every reader adds these in the same order: results do not depend on
// the order in which workgroups run.
//
// The tensors' addresses travel as kernel arguments, so a captured graph holds them
// itself: up to kPer of them with the two passes' own launches, more through a table in the
// workspace that launches of kPer each write first.
#include <algorithm>
#include <memory>
#include <new>

#include "mb_internal.h"

namespace mb {
namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kPer = 120;             // tensors whose table entries fit one launch's arguments
constexpr int kMaxTensors = 1 << 16;
constexpr int64_t kPiece = 16384;     // bytes a workgroup takes at a time: four 16-byte vectors a thread
constexpr int kGrid = 2048;           // partial sums at most

struct Entry {
    const void* g;
    void* o;
    int64_t n;
    int64_t first;      // pieces of the tensors before this one
};

struct Batch {
    Entry e[kPer];
};
struct InWorkspace {
    const Entry* e;
};

__global__ void k_table(Batch b, Entry* table, int at, int n) {
    // each entry is four words of eight bytes
    const int64_t* src = (const int64_t*)b.e;
    int64_t* dst = (int64_t*)(table + at);
    for (int i = threadIdx.x; i < n * 4; i += blockDim.x) dst[i] = src[i];
}

// A workgroup's run of pieces, and the tensor that its first belongs to: the last whose first
// piece is not behind it, found by all lanes of a wave together, 64 tensors a step.
struct Run {
    int64_t p, end;
    int at;
};
template <typename Table>
__device__ __forceinline__ Run run_of(const Table& t, int n, int64_t pieces, int64_t block) {
    Run r;
    r.p = pieces * block / gridDim.x;
    r.end = pieces * (block + 1) / gridDim.x;
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64, i = lo + lane * step;
        const int c = __popcll(__ballot(i < hi && t.e[i].first <= r.p));
        lo += (c - 1) * step;
        hi = min(lo + step, hi);
    }
    r.at = lo;
    return r;
}

// Calls f(entry, first element, elements) for each piece of a run.
template <typename T, typename Table, typename F>
__device__ __forceinline__ void for_pieces(const Table& t, int n, const Run& r, F f) {
    int at = r.at;
    Entry e = t.e[at];
    int64_t next = at + 1 < n ? t.e[at + 1].first : INT64_MAX;
    for (int64_t p = r.p; p < r.end; ++p) {
        if (p >= next) {                  // a tensor has at least one piece
            e = t.e[++at];
            next = at + 1 < n ? t.e[at + 1].first : INT64_MAX;
        }
        constexpr int64_t M = kPiece / sizeof(T);
        const int64_t first = (p - e.first) * M, left = e.n - first;
        f(e, first, (int)(left < M ? left : M));
    }
}

__device__ __forceinline__ double sum_block(double v, double* lds) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0] + lds[1] + lds[2] + lds[3];
    return v;
}

// Sixteen bytes at any element's address, which the memory takes in one access: gradients are often
// views at odd offsets of one buffer (the norm and scaling of 129 M bf16 values from an odd address on: one
// element at a time 329 us, so 136; 266 tensors each at an odd address 147 - 158 us, aligned 145 - 148).
typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
__device__ __forceinline__ u4 load16(const T* p) {
    u4 t;
    __builtin_memcpy(&t, p, 16);
    return t;
}
template <typename T>
__device__ __forceinline__ void put16(T* p, u4 t, bool stream) {
    if (stream) {
        asm volatile("");     // keeps the two kinds of store apart
        __builtin_nontemporal_store(t, reinterpret_cast<any4*>(p));
        asm volatile("");
    } else {
        __builtin_memcpy(p, &t, 16);
    }
}

template <typename T>
__device__ __forceinline__ double sum_piece(const T* g, int n) {
    double s0 = 0.0, s1 = 0.0;
    constexpr int V = 16 / sizeof(T);
    const int nv = n / V;
    const auto add = [&](u4 t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) {
                const double a = (double)__uint_as_float(t[j]);
                (j & 1 ? s1 : s0) += a * a;
            } else {
                // the square of a bf16 value is exact in fp32 but may leave its range
                const double a = (double)__uint_as_float(t[j] << 16), b = (double)__uint_as_float(t[j] & 0xffff0000u);
                s0 += a * a;
                s1 += b * b;
            }
        }
    };
    constexpr int B = 4;              // reads under way
    int k = threadIdx.x;
    for (; k + (B - 1) * 256 < nv; k += B * 256) {
        u4 t[B];
#pragma unroll
        for (int j = 0; j < B; ++j) t[j] = load16(g + (k + j * 256) * V);
#pragma unroll
        for (int j = 0; j < B; ++j) add(t[j]);
    }
    for (; k < nv; k += 256) add(load16(g + k * V));
    for (k = nv * V + threadIdx.x; k < n; k += 256) {
        const double a = (double)to_f32(g[k]);
        s0 += a * a;
    }
    return s0 + s1;
}

template <typename T, typename Table>
__global__ void __launch_bounds__(256, 8) k_norm_parts(Table t, int n, int64_t pieces, double* __restrict__ part) {
    __shared__ double lds[4];
    double s = 0.0;
    for_pieces<T>(t, n, run_of(t, n, pieces, blockIdx.x), [&](const Entry& e, int64_t at, int m) { s += sum_piece((const T*)e.g + at, m); });
    s = sum_block(s, lds);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* g, T* o, int n, float f, bool stream) {
    constexpr int V = 16 / sizeof(T);
    const int nv = n / V;
    const auto scaled = [&](u4 t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) {
                t[j] = __float_as_uint(__uint_as_float(t[j]) * f);
            } else {
                const float a = __uint_as_float(t[j] << 16) * f, b = __uint_as_float(t[j] & 0xffff0000u) * f;
                t[j] = (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
            }
        }
        return t;
    };
    constexpr int B = 4;              // reads under way
    int k = threadIdx.x;
    for (; k + (B - 1) * 256 < nv; k += B * 256) {
        u4 t[B];
#pragma unroll
        for (int j = 0; j < B; ++j) t[j] = load16(g + (k + j * 256) * V);
#pragma unroll
        for (int j = 0; j < B; ++j) put16(o + (k + j * 256) * V, scaled(t[j]), stream);
    }
    for (; k < nv; k += 256) put16(o + k * V, scaled(load16(g + k * V)), false);
    for (k = nv * V + threadIdx.x; k < n; k += 256) store_out(o + k, to_f32(g[k]) * f);
}

// The pieces in the opposite order: what the first pass read last may still lie in the last-level cache.
template <typename T, typename Table>
__global__ void __launch_bounds__(256) k_clip(Table t, int n, int64_t pieces, const double* __restrict__ part, int parts,
                                              float* __restrict__ norm_out, float max_norm, float eps, bool stream) {
    __shared__ double lds[4];
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 256) s += part[i];
    const Run r = run_of(t, n, pieces, gridDim.x - 1 - blockIdx.x);
    const float norm = (float)sqrt(sum_block(s, lds));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    const float c = max_norm / (norm + eps);
    const float f = c > 1.0f || __builtin_isinf(max_norm) ? 1.0f : c;      // NaN stays
    for_pieces<T>(t, n, r, [&](const Entry& e, int64_t at, int m) {
        if (f == 1.0f && e.g == e.o) return;          // in place and nothing to scale
        scale_piece((const T*)e.g + at, (T*)e.o + at, m, f, stream);
    });
}

template <typename T, typename Table>
mb_status passes(const Table& t, int n, int64_t pieces, double* part, float* norm, float max_norm, float eps, hipStream_t s) {
    const bool stream = pieces * 2 * kPiece > (int64_t)kStreamBytes;
    const int grid = (int)(pieces < kGrid ? pieces : kGrid);
    hipLaunchKernelGGL((k_norm_parts<T, Table>), dim3(grid), dim3(256), 0, s, t, n, pieces, part);
    mb_status st = check_launch();
    if (st != MB_OK) return st;
    hipLaunchKernelGGL((k_clip<T, Table>), dim3(grid), dim3(256), 0, s, t, n, pieces, part, grid, norm, max_norm, eps, stream);
    return check_launch();
}

// Whether a tensor that is written overlaps any other one.  Tensors that are only read may.
struct Range {
    uintptr_t b, e;
    bool written;
};
bool any_overlap(Range* r, int64_t n) {
    const auto before = [](const Range& x, const Range& y) { return x.b < y.b; };
    if (!std::is_sorted(r, r + n, before)) std::sort(r, r + n, before);
    uintptr_t all = 0, out = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (r[i].b < (r[i].written ? all : out)) return true;
        all = std::max(all, r[i].e);
        if (r[i].written) out = std::max(out, r[i].e);
    }
    return false;
}

size_t table_bytes(int64_t n) { return ((size_t)n * sizeof(Entry) + 255) / 256 * 256; }

}  // namespace

size_t grad_clip_workspace(int64_t n) {
    if (n < 1 || n > kMaxTensors) return 0;
    return table_bytes(n) + kGrid * sizeof(double);
}

}  // namespace mb

extern "C" mb_status mb_grad_norm_clip(const void* const* grads, void* const* outs, const int64_t* sizes, int64_t n,
                                       float max_norm, float eps, float* norm, mb_dtype dtype, void* ws,
                                       size_t ws_bytes, hipStream_t stream) {
    using namespace mb;
    if (!dtype_ok(dtype)) return MB_ERR_DTYPE;
    if (n < 0 || n > kMaxTensors || !(max_norm >= 0.0f) || !(eps >= 0.0f) || eps > 3.0e38f) return MB_ERR_SHAPE;
    if (!norm || (n > 0 && (!grads || !sizes))) return MB_ERR_NULL;
    const size_t es = dtype_size(dtype);
    const int64_t piece = kPiece / (int64_t)es;
    if ((uintptr_t)norm & 3) return MB_ERR_ALIGN;
    const size_t need = grad_clip_workspace(n);
    if (n > 0 && (!ws || ws_bytes < need || ((uintptr_t)ws & 255))) return MB_ERR_WORKSPACE;
    constexpr int64_t kOnStack = 512;
    Range few[kOnStack];
    std::unique_ptr<Range[]> many(2 * n > kOnStack ? new (std::nothrow) Range[2 * n] : nullptr);
    Range* const ranges = 2 * n > kOnStack ? many.get() : few;
    if (!ranges) return MB_ERR_WORKSPACE;
    int64_t total = 0, spans = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (sizes[i] < 0 || sizes[i] > ((int64_t)1 << 40)) return MB_ERR_SHAPE;
        if (sizes[i] == 0) continue;
        const void* o = outs ? outs[i] : grads[i];
        if (!grads[i] || !o) return MB_ERR_NULL;
        if ((uintptr_t)grads[i] % es || (uintptr_t)o % es) return MB_ERR_ALIGN;
        const size_t b = (size_t)sizes[i] * es;
        if ((o != grads[i] && overlaps(o, b, grads[i], b)) || overlaps(o, b, norm, 4) || overlaps(grads[i], b, norm, 4) ||
            overlaps(ws, need, o, b) || overlaps(ws, need, grads[i], b))
            return MB_ERR_ALIAS;
        ranges[spans++] = {(uintptr_t)o, (uintptr_t)o + b, true};
        if (o != grads[i]) ranges[spans++] = {(uintptr_t)grads[i], (uintptr_t)grads[i] + b, false};
        total += (sizes[i] + piece - 1) / piece;
    }
    if ((n > 0 && overlaps(ws, need, norm, 4)) || any_overlap(ranges, spans)) return MB_ERR_ALIAS;
    if (total == 0) return copy_state(nullptr, norm, 1, stream);
    Entry* table = (Entry*)ws;
    double* part = (double*)((char*)ws + table_bytes(n));
    int64_t filled = 0;
    for (int64_t i = 0; i < n; ++i) filled += sizes[i] != 0;
    int used = 0, at = 0;
    int64_t pieces = 0;
    Batch b;
    for (int64_t i = 0; i < n; ++i) {
        if (sizes[i] == 0) continue;
        b.e[used++] = Entry{grads[i], outs ? outs[i] : const_cast<void*>(grads[i]), sizes[i], pieces};
        pieces += (sizes[i] + piece - 1) / piece;
        if (filled > kPer && (used == kPer || at + used == filled)) {
            hipLaunchKernelGGL(k_table, dim3(1), dim3(256), 0, stream, b, table, at, used);
            mb_status st = check_launch();
            if (st != MB_OK) return st;
            at += used;
            used = 0;
        }
    }
    if (filled > kPer) {
        const InWorkspace t{table};
        return dtype == MB_F32 ? passes<float>(t, at, pieces, part, norm, max_norm, eps, stream)
                               : passes<bf16>(t, at, pieces, part, norm, max_norm, eps, stream);
    }
    return dtype == MB_F32 ? passes<float>(b, used, pieces, part, norm, max_norm, eps, stream)
                           : passes<bf16>(b, used, pieces, part, norm, max_norm, eps, stream);
}
