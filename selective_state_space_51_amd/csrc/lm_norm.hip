// libselscan_lm - residual addition with root-mean-square norm, forward (with an 8-bit output) and gradients
// (add_rms_norm_fwd, add_rms_norm_bwd of include/selscan_lm.h).  MI355X (gfx950).
//
// Both directions read each row once and keep it in registers between the row's reductions: TPR
// threads share a row, each with 8 NV of its elements, the fewest threads that hold it in 32 registers each or fewer (a
// wave up to 1,024 elements, so that no barrier is needed; four waves up to 8,192; 16 beyond).
//
// HBM bound where there are many rows: 16,384 x 2,048, bf16 with an fp32 residual, takes 72 us forward (5.6 TB/s of what it
// reads and writes; with an int8 output 69 us, with e4m3 68, 5.4 TB/s) and 110 + 5 us backward (4.9 TB/s).  With few it is the launch and one trip to memory: 5 x 2,048 with an
// int8 output 2.8 us in a graph.
#include "lm_common.h"

#include <float.h>

namespace {

struct NormParams {
    const void *x, *residual;  // backward: dy, s
    const float *weight;
    void *y, *residual_out;    // backward: dx, dresidual
    const void *dres;          // backward: gradient of residual_out
    const void *add;           // backward: x, where the sum is formed anew; row stride x_stride
    float *scale, *rstd;       // backward: rstd is read
    float *partial;            // backward: [slots][width] sums of dweight
    int64_t rows, x_stride;
    int width, kind, slots;
    int64_t rows_per;          // backward: consecutive rows of a slot
    float eps, inv_width;      // (inv_width: backward; inv_width64: forward)
    double inv_width64;
};

// element e of piece v of a thread: 8 adjacent ones (rows that move as 16-byte vectors), or elements TPR
// apart, so that the lanes of a wave read adjacent elements of a row of any alignment
template <int TPR, bool VEC>
__device__ __forceinline__ int col_of(int v, int e, int tr) {
    return VEC ? (v * TPR + tr) * 8 + e : (v * 8 + e) * TPR + tr;
}

template <typename T, int TPR, bool VEC, bool NT = false>
__device__ __forceinline__ void load_piece(const T *row, int v, int tr, int width, float (&out)[8]) {
    if constexpr (VEC) {
        const int c = col_of<TPR, VEC>(v, 0, tr);
        const Raw8<T> r = c < width ? NT ? load_stream8<NT>(row + c) : load_raw8(row + c, 8, true) : Raw8<T>{};
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = raw_f32(r, e);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = col_of<TPR, VEC>(v, e, tr);
            out[e] = c < width ? Io<T>::f32(row[c]) : 0.f;
        }
    }
}

template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void store_piece(T *row, int v, int tr, int width, const float (&val)[8]) {
    if constexpr (VEC) {
        const int c = col_of<TPR, VEC>(v, 0, tr);
        if (c < width) store8(row + c, 8, true, val);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = col_of<TPR, VEC>(v, e, tr);
            if (c < width) row[c] = Io<T>::to(val[e]);
        }
    }
}

// the sum (or maximum) over the TPR threads of a row; sh: one value per wave of the workgroup, two buffers
// used in turn (buf), so that one barrier per reduction is enough
template <int TPR, bool MAX, typename V>
__device__ __forceinline__ V row_reduce(V v, V *sh, int buf) {
    if constexpr (MAX) v = wave_max(v);
    else v = wave_sum(v);
    if constexpr (TPR > 64) {
        constexpr int NW = TPR / 64;
        V *s = sh + buf * NW;
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        lds_barrier();
        v = s[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) {
            if constexpr (MAX) v = fmaxf(v, s[i]);
            else v += s[i];
        }
    }
    return v;
}

template <int KIND>
__device__ __forceinline__ uint2 pack8(const float (&q)[8]) {
    uint32_t w[2] = {0, 0};
    if constexpr (KIND == SELSCAN_LM_OUT_INT8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = (int)__builtin_amdgcn_fmed3f(rintf(q[e]), -127.f, 127.f);
            w[e >> 2] |= (uint32_t)(i & 255) << (8 * (e & 3));
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
            w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], w[h], true);
        }
    }
    return make_uint2(w[0], w[1]);
}

// Forward.  The squares are added in 64 bits, which hides behind the row's loads: rstd is then the rounded exact one whatever
// the split over threads, and a value between two steps of an 8-bit output does not move with the width's thread count.
template <typename T, typename R, int TPR, int NV, bool VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd(NormParams p) {
    constexpr int BLOCK = TPR < 256 ? 256 : TPR;
    __shared__ double sums[BLOCK / 64];
    __shared__ float sh[BLOCK / 64];
    const int tr = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * (BLOCK / TPR) + threadIdx.x / TPR;
    if (row >= p.rows) return;  // with more than one row per workgroup, rows do not share barriers
    const T *x = (const T *)p.x + row * p.x_stride;
    const R *res = p.residual ? (const R *)p.residual + row * p.width : nullptr;
    float s[NV][8];
    double ss = 0.;
#pragma unroll
    for (int v = 0; v < NV; ++v) load_piece<T, TPR, VEC>(x, v, tr, p.width, s[v]);
    if (res) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float r[8];
            load_piece<R, TPR, VEC>(res, v, tr, p.width, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[v][e] += r[e];
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fma((double)s[v][e], (double)s[v][e], ss);
    if (p.residual_out) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            store_piece<R, TPR, VEC>((R *)p.residual_out + row * p.width, v, tr, p.width, s[v]);
    }
    const double mean64 = row_reduce<TPR, false>(ss, sums, 0) * p.inv_width64;
    const float mean = (float)mean64, under = mean + p.eps;
    float rstd = 1.f / sqrtf(under);
    // a row of values past 1.8e19, or below 1e-19 with an eps of 0: its mean square is no normal number of fp32, its root is
    if (!(under >= FLT_MIN && under < INFINITY)) rstd = (float)(1. / sqrt(mean64 + (double)p.eps));
    if (p.rstd && tr == 0) p.rstd[row] = rstd;
    // the largest magnitude as a whole number, in whose order a NaN is the largest (fmaxf would drop it)
    uint32_t most = 0;
    // (a row of zeros with an eps of 0 has an infinite rstd; its 8-bit output is zeros all the same)
    const float by = p.kind != SELSCAN_LM_OUT_IO && mean64 == 0. ? 0.f : rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float w[8];
        load_piece<float, TPR, VEC>(p.weight, v, tr, p.width, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[v][e] = s[v][e] * by * w[e];
            const uint32_t u = __float_as_uint(s[v][e]) & 0x7FFFFFFFu;
            most = u > most ? u : most;
        }
    }
    if (p.kind == SELSCAN_LM_OUT_IO) {
#pragma unroll
        for (int v = 0; v < NV; ++v) store_piece<T, TPR, VEC>((T *)p.y + row * p.width, v, tr, p.width, s[v]);
        return;
    }
    const float amax = row_reduce<TPR, true>(most > 0x7F800000u ? INFINITY : __uint_as_float(most), sh, 0);
    const float top = p.kind == SELSCAN_LM_OUT_INT8 ? 127.f : 448.f;
    // a row that holds an infinity or a NaN (or whose mean square overflows) is marked by its scale
    const bool bad = !(mean < INFINITY) || amax == INFINITY, zero = bad || amax < 1e-32f;
    const float inv = zero ? 0.f : top * (1.f / amax);
    if (tr == 0) p.scale[row] = bad ? NAN : zero ? 0.f : amax * (1.f / top);
    uint8_t *y = (uint8_t *)p.y + row * p.width;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = zero ? 0.f : s[v][e] * inv;
        const uint2 w = p.kind == SELSCAN_LM_OUT_INT8 ? pack8<SELSCAN_LM_OUT_INT8>(q) : pack8<SELSCAN_LM_OUT_FP8>(q);
        if constexpr (VEC) {
            const int c = col_of<TPR, VEC>(v, 0, tr);
            if (c < p.width) *(uint2 *)(y + c) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = col_of<TPR, VEC>(v, e, tr);
                if (c < p.width) y[c] = (uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
            }
        }
    }
}

// Gradients: a slot (the threads of a row) walks rows_per consecutive rows with the weight and its sums of
// dweight in registers, and leaves the sums in its row of `partial`; norm_dw adds those in order.
//
// NT: dy, s and dresidual_out are read without a place in the caches.
template <typename T, typename R, int TPR, int NV, bool VEC, bool NT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd(NormParams p) {
    constexpr int BLOCK = TPR < 256 ? 256 : TPR;
    __shared__ float sh[2 * (BLOCK / 64)];
    const int tr = threadIdx.x % TPR;
    const int64_t slot = (int64_t)blockIdx.x * (BLOCK / TPR) + threadIdx.x / TPR;
    if (slot >= p.slots) return;
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load_piece<float, TPR, VEC>(p.weight, v, tr, p.width, w[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = 0.f;
    }
    const int64_t r0 = slot * p.rows_per, r1 = r0 + p.rows_per < p.rows ? r0 + p.rows_per : p.rows;
    int buf = 0;
    for (int64_t row = r0; row < r1; ++row, buf ^= 1) {
        const int64_t at = row * p.width;
        float g[NV][8], xh[NV][8], dot = 0.f;
        const float rstd = p.rstd[row];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            load_piece<T, TPR, VEC, NT>((const T *)p.x + at, v, tr, p.width, g[v]);
            load_piece<R, TPR, VEC, NT>((const R *)p.residual + at, v, tr, p.width, xh[v]);
        }
        if (p.add) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float a[8];
                load_piece<T, TPR, VEC>((const T *)p.add + row * p.x_stride, v, tr, p.width, a);
#pragma unroll
                for (int e = 0; e < 8; ++e) xh[v][e] += a[e];
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[v][e] *= rstd;
                dw[v][e] = fmaf(g[v][e], xh[v][e], dw[v][e]);
                g[v][e] *= w[v][e];
                dot = fmaf(g[v][e], xh[v][e], dot);
            }
        dot = row_reduce<TPR, false>(dot, sh, buf) * p.inv_width;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (p.dres) load_piece<R, TPR, VEC, NT>((const R *)p.dres + at, v, tr, p.width, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = fmaf(rstd, fmaf(-xh[v][e], dot, g[v][e]), d[e]);
            if (p.y) store_piece<T, TPR, VEC>((T *)p.y + at, v, tr, p.width, d);
            if (p.residual_out) store_piece<R, TPR, VEC>((R *)p.residual_out + at, v, tr, p.width, d);
        }
    }
    if (p.partial) {
#pragma unroll
        for (int v = 0; v < NV; ++v) store_piece<float, TPR, VEC>(p.partial + slot * p.width, v, tr, p.width, dw[v]);
    }
}

// dweight: 32 columns per workgroup, 32 threads each summing every 32nd slot, then those in order
__global__ __launch_bounds__(1024) void norm_dw(NormParams p) {
    __shared__ float sh[32][33];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    float a = 0.f;
    if (col < p.width) {
#pragma unroll 8
        for (int s = g; s < p.slots; s += 32) a += p.partial[(int64_t)s * p.width + col];
    }
    sh[g][c] = a;
    __syncthreads();
    if (g == 0 && col < p.width) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += sh[i][c];
        ((float *)p.y)[col] = a;
    }
}

constexpr int kMaxWidth = 32768;

// threads per row and 8-element pieces per thread of a width
struct Shape {
    int tpr, nv;
};
Shape shape_of(int64_t width) {
    if (width <= 512) return {64, 1};
    if (width <= 1024) return {64, 2};
    if (width <= 2048) return {256, 1};
    if (width <= 4096) return {256, 2};
    if (width <= 8192) return {256, 4};
    if (width <= 16384) return {1024, 2};
    return {1024, 4};
}

// slots of the backward: enough rows in flight to fill the chip, few enough that their sums of
// dweight (4 bytes per slot and column) stay a few per cent of what the rows move
int64_t bwd_slots(int64_t rows, int64_t width) {
    const Shape s = shape_of(width);
    const int64_t most = s.tpr == 64 ? 2048 : s.tpr == 256 ? 1024 : 512;
    return rows < most ? rows : most;
}

// Gradients of a 16-bit residual stream read dy, the residual and its gradient without a place in the caches once they and x
// pass this many bytes (forward and gradients, us, with a place and without: 4,096 x 2,048, 67 MB, 32 and 34; 6,000, 98 MB, 46.5
// and 46; 8,192, 134 MB, 58 and 56.5; 12,000 88 and 80; 16,384 120 and 109; 20,000 x 1,024 82 and 75).  With an fp32 stream it
// is 1 or 2 % either way, and none does it.
constexpr int64_t kReadsPast = INT64_C(112) << 20;

template <typename T, typename R, bool BWD, bool VEC>
int launch_norm(const NormParams &p, void *stream) {
    const Shape s = shape_of(p.width);
    const int64_t units = BWD ? p.slots : p.rows;
    const int block = s.tpr < 256 ? 256 : s.tpr, per = block / s.tpr;
    const int64_t blocks = (units + per - 1) / per;
    if (!grid_fits(blocks, block)) return SELSCAN_E_UNSUPPORTED;
    const dim3 grid((unsigned)blocks), bl(block);
    const bool past = BWD && p.rows * p.width * 8 >= kReadsPast;
#define GO(TPR, NV)                                                                        \
    if (s.tpr == TPR && s.nv == NV) {                                                      \
        if constexpr (BWD) {                                                               \
            if constexpr (VEC && sizeof(R) == 2) {                                         \
                if (past) return enqueue(norm_bwd<T, R, TPR, NV, true, true>, grid, bl, p, stream); \
            }                                                                              \
            return enqueue(norm_bwd<T, R, TPR, NV, VEC, false>, grid, bl, p, stream);      \
        } else return enqueue(norm_fwd<T, R, TPR, NV, VEC>, grid, bl, p, stream);            \
    }
    GO(64, 1) GO(64, 2) GO(256, 1) GO(256, 2) GO(256, 4) GO(1024, 2) GO(1024, 4)
#undef GO
    return SELSCAN_E_UNSUPPORTED;
}

template <bool BWD>
int launch_types(const NormParams &p, int io, int res, bool vec, void *stream) {
    if (io == SELSCAN_F32) return vec ? launch_norm<float, float, BWD, true>(p, stream) : launch_norm<float, float, BWD, false>(p, stream);
    if (res == SELSCAN_F32)
        return vec ? launch_norm<uint16_t, float, BWD, true>(p, stream) : launch_norm<uint16_t, float, BWD, false>(p, stream);
    return vec ? launch_norm<uint16_t, uint16_t, BWD, true>(p, stream) : launch_norm<uint16_t, uint16_t, BWD, false>(p, stream);
}

int norm_sizes(int64_t rows, int64_t width, int io, int res) {
    if (rows < 0 || width < 0) return SELSCAN_E_SHAPE;
    if (!io_known(io) || (res != SELSCAN_F32 && res != io)) return SELSCAN_E_UNSUPPORTED;
    if (width > kMaxWidth) return SELSCAN_E_UNSUPPORTED;
    if (mul_size(rows, width) < 0) return SELSCAN_E_SHAPE;
    return SELSCAN_OK;
}

}  // namespace

extern "C" {

int add_rms_norm_fwd(const void *x, int64_t x_stride, const void *residual, const float *weight, float eps,
                     int out_kind, void *y, void *residual_out, float *scale, float *rstd, int64_t rows, int64_t width,
                     int io_dtype, int residual_dtype, void *stream) {
    int rc = norm_sizes(rows, width, io_dtype, residual_dtype);
    if (rc != SELSCAN_OK) return rc;
    if (out_kind < SELSCAN_LM_OUT_IO || out_kind > SELSCAN_LM_OUT_FP8 || !(eps >= 0.f) || !(eps < INFINITY))
        return SELSCAN_E_UNSUPPORTED;
    if (rows == 0 || width == 0) return SELSCAN_OK;
    if (x_stride < width || mul_size(rows, x_stride) < 0) return SELSCAN_E_SHAPE;
    const bool q8 = out_kind != SELSCAN_LM_OUT_IO;
    if (!x || !weight || !y || (q8 && !scale)) return SELSCAN_E_NULL;
    const size_t s = io_bytes(io_dtype), r = io_bytes(residual_dtype), o = q8 ? 1 : s;
    if (!span_aligned(x, s) || !span_aligned(residual, r) || !span_aligned(residual_out, r) || !span_aligned(y, o) ||
        !span_aligned(weight, 4) || !span_aligned(scale, 4) || !span_aligned(rstd, 4))
        return SELSCAN_E_ALIGN;
    const size_t n = (size_t)rows * width;
    // residual_out may be residual itself
    const Span in[] = {{x, strided_bytes(rows, width, x_stride, s)},
                       {weight, (size_t)width * 4},
                       {residual != residual_out ? residual : nullptr, n * r}};
    const Span out[] = {{y, n * o}, {residual_out, n * r}, {q8 ? scale : nullptr, (size_t)rows * 4}, {rstd, (size_t)rows * 4}};
    if (any_alias(in, 3, out, 4)) return SELSCAN_E_ALIAS;
    NormParams p{};
    p.x = x, p.residual = residual, p.weight = weight, p.y = y, p.residual_out = residual_out;
    p.scale = scale, p.rstd = rstd, p.rows = rows, p.x_stride = x_stride;
    p.width = (int)width, p.kind = out_kind, p.eps = eps, p.inv_width64 = 1. / (double)width;
    const bool vec = width % 8 == 0 && x_stride * s % 16 == 0 && span_aligned(x, 16) && span_aligned(residual, 16) &&
                     span_aligned(residual_out, 16) && span_aligned(y, q8 ? 8 : 16) && span_aligned(weight, 16);
    return launch_types<false>(p, io_dtype, residual_dtype, vec, stream);
}

size_t add_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t width) {
    if (rows <= 0 || width <= 0 || width > kMaxWidth) return 0;
    return (size_t)bwd_slots(rows, width) * (size_t)width * sizeof(float);
}

int add_rms_norm_bwd(const void *dy, const void *s, const void *x, int64_t x_stride, const float *weight,
                     const float *rstd, const void *dresidual_out, void *dx, void *dresidual, float *dweight,
                     int64_t rows, int64_t width, int io_dtype, int residual_dtype, void *workspace,
                     size_t workspace_bytes, void *stream) {
    int rc = norm_sizes(rows, width, io_dtype, residual_dtype);
    if (rc != SELSCAN_OK) return rc;
    if (width == 0 || (rows == 0 && !dweight)) return SELSCAN_OK;
    if (x && (x_stride < width || mul_size(rows, x_stride) < 0)) return SELSCAN_E_SHAPE;
    if (rows > 0 && (!dy || !s || !weight || !rstd)) return SELSCAN_E_NULL;
    const size_t b = io_bytes(io_dtype), r = io_bytes(residual_dtype);
    const size_t need = dweight ? add_rms_norm_bwd_workspace_bytes(rows, width) : 0;
    if (!span_aligned(dy, b) || !span_aligned(x, b) || !span_aligned(dx, b) || !span_aligned(s, r) ||
        !span_aligned(dresidual_out, r) ||
        !span_aligned(dresidual, r) || !span_aligned(weight, 4) || !span_aligned(rstd, 4) || !span_aligned(dweight, 4) ||
        (need && !span_aligned(workspace, 16)))
        return SELSCAN_E_ALIGN;
    if (need && (!workspace || workspace_bytes < need)) return SELSCAN_E_WORKSPACE;
    const size_t n = (size_t)rows * width;
    const Span in[] = {{dy, n * b}, {s, n * r}, {weight, (size_t)width * 4}, {rstd, (size_t)rows * 4}, {dresidual_out, n * r},
                       {x, strided_bytes(rows, width, x_stride, b)}};
    const Span out[] = {{dx, n * b}, {dresidual, n * r}, {dweight, (size_t)width * 4}, {need ? workspace : nullptr, need}};
    if (any_alias(in, 6, out, 4)) return SELSCAN_E_ALIAS;
    NormParams p{};
    p.x = dy, p.residual = s, p.weight = weight, p.y = dx, p.residual_out = dresidual, p.dres = dresidual_out;
    p.add = x, p.x_stride = x_stride;
    p.rstd = (float *)rstd, p.rows = rows, p.width = (int)width, p.inv_width = 1.f / (float)width;
    p.partial = dweight ? (float *)workspace : nullptr;
    p.slots = (int)bwd_slots(rows, width);
    if (rows > 0) {
        // consecutive rows per slot; rounding up can leave fewer slots with rows than were asked for
        p.rows_per = (rows + p.slots - 1) / p.slots;
        p.slots = (int)((rows + p.rows_per - 1) / p.rows_per);
        const bool vec = width % 8 == 0 && span_aligned(dy, 16) && span_aligned(s, 16) && span_aligned(weight, 16) &&
                         span_aligned(dresidual_out, 16) && span_aligned(dx, 16) && span_aligned(dresidual, 16) &&
                         (!x || (span_aligned(x, 16) && x_stride * b % 16 == 0));
        rc = launch_types<true>(p, io_dtype, residual_dtype, vec, stream);
        if (rc != SELSCAN_OK || !dweight) return rc;
    }
    p.y = dweight;
    return enqueue(norm_dw, dim3((unsigned)((width + 31) / 32)), dim3(1024), p, stream);
}

}  // extern "C"
