// lm_common.h - what the sources of libselscan_lm share beyond selscan_common.h: host-side argument
// checks and launches, unaligned vector reads, reductions across a wave and a workgroup.
#pragma once

#include "selscan_common.h"
#include "selscan_lm.h"

namespace {

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------

inline bool io_known(int dtype) { return dtype == SELSCAN_F32 || dtype == SELSCAN_BF16; }
inline size_t io_bytes(int dtype) { return dtype == SELSCAN_BF16 ? 2 : 4; }

// bytes from the first to the last element of `rows` rows of `width` elements, `stride` apart
inline size_t strided_bytes(int64_t rows, int64_t width, int64_t stride, size_t elem) {
    return rows <= 0 || width <= 0 ? 0 : ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * elem;
}

inline bool span_aligned(const void *p, size_t a) { return !p || aligned(p, a); }

// a * b for non-negative sizes, or -1 where it passes 2^62 (then no array of that size exists)
inline int64_t mul_size(int64_t a, int64_t b) {
    if (a == 0 || b == 0) return 0;
    return a > (INT64_C(1) << 62) / b ? -1 : a * b;
}

// A dispatch counts its threads along an axis in 32 bits: whether that many workgroups of that many threads are a launch
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

// every output against every input and every other output
inline bool any_alias(const Span *in, int nin, const Span *out, int nout) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlap(out[i], in[j])) return true;
        for (int j = i + 1; j < nout; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

template <class P>
int enqueue(void (*kernel)(P), dim3 grid, dim3 block, const P &p, void *stream, unsigned lds = 0) {
    P copy = p;
    void *args[] = {&copy};
    const hipError_t e = hipLaunchKernel((const void *)kernel, grid, block, args, lds, (hipStream_t)stream);
    if (e != hipSuccess) {
        record_hip_error(e);
        return SELSCAN_E_HIP;
    }
    return SELSCAN_OK;
}

// ------------------------------------------------------------------------------------
// device side
// ------------------------------------------------------------------------------------

// 4 floats from an address that is 4-byte aligned (one 16-byte load)
__device__ __forceinline__ float4 load_f4(const float *p) {
    struct __attribute__((packed, aligned(4))) U {
        float a, b, c, d;
    };
    const U u = *(const U *)p;
    return make_float4(u.a, u.b, u.c, u.d);
}

// 8 elements from any address aligned to the element
template <typename T>
__device__ __forceinline__ Raw8<T> load_any8(const T *p) {
    struct __attribute__((packed, aligned(sizeof(T)))) U {
        uint32_t w[sizeof(T) * 2];
    };
    const U u = *(const U *)p;
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) * 2; ++i) r.w[i] = u.w[i];
    return r;
}
// the same without a place in the caches (NT), for what no one reads again before the caches have seen that much else
template <bool NT, typename T>
__device__ __forceinline__ Raw8<T> load_stream8(const T *p) {
    if constexpr (!NT) return load_any8(p);
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const V v = __builtin_nontemporal_load((const V *)p + i);
        r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void store_any8(T *p, const float (&v)[8]) {
    struct __attribute__((packed, aligned(sizeof(T)))) U {
        uint32_t w[sizeof(T) * 2];
    };
    U u;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u.w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) u.w[i] = Io<T>::to2(v[2 * i], v[2 * i + 1]);
    }
    *(U *)p = u;
}

// Sum and maximum over the 64 lanes, the same in every lane.  DPP moves along rows of 16 and then across them
// (lane 63 ends with all), without LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float other, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(other), __float_as_int(v), CTRL, ROWS, 0xF, false));
}
template <class F>
__device__ __forceinline__ float wave_reduce(float v, float identity, F f) {
    v = f(v, dpp_or<0x111, 0xF>(identity, v));  // row_shr 1, 2, 4, 8
    v = f(v, dpp_or<0x112, 0xF>(identity, v));
    v = f(v, dpp_or<0x114, 0xF>(identity, v));
    v = f(v, dpp_or<0x118, 0xF>(identity, v));
    v = f(v, dpp_or<0x142, 0xA>(identity, v));  // row_bcast 15 into rows 1 and 3, 31 into rows 2 and 3
    v = f(v, dpp_or<0x143, 0xC>(identity, v));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
    return wave_reduce(v, 0.f, [](float a, float b) { return a + b; });
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double v) {
    const int64_t b = __double_as_longlong(v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, ROWS, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xF, false);
    return __longlong_as_double((int64_t)hi << 32 | (uint32_t)lo);
}
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp_or_zero<0x111, 0xF>(v);
    v += dpp_or_zero<0x112, 0xF>(v);
    v += dpp_or_zero<0x114, 0xF>(v);
    v += dpp_or_zero<0x118, 0xF>(v);
    v += dpp_or_zero<0x142, 0xA>(v);
    v += dpp_or_zero<0x143, 0xC>(v);
    const int64_t b = __double_as_longlong(v);
    const int lo = __builtin_amdgcn_readlane((int)b, 63), hi = __builtin_amdgcn_readlane((int)(b >> 32), 63);
    return __longlong_as_double((int64_t)hi << 32 | (uint32_t)lo);
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace
