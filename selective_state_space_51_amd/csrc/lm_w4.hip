// libselscan_lm - a few rows times a 4-bit weight matrix with group scales (w4_matvec of
// include/selscan_lm.h).  MI355X (gfx950).
//
// y[r][j] = sum over groups of  scale * (sum_k q x - zero * sum_k x).  The inner sums run on the matrix
// cores (16 rows of x by 16 rows of the matrix by 32 k), with the 4-bit values as bf16 numbers 16 + q: a
// nibble put into the top of the mantissa of 16.0 is that number exactly, one shift and one and-or for two
// weights.  The 16 leaves with the zero point, both times sum_k x, which one more product with ones gives
// in the same register layout.  (128 + q would save nothing and cost 8 times the cancellation.)
//
// HBM bound: each weight is read once per 32 rows.
#include "lm_common.h"

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct W4Params {
    const void *x;
    const uint8_t *q, *zeros;
    const uint16_t *scales;
    const float *bias;
    void *y;
    int64_t x_stride, n;
    int rows, k, groups, units, upw;  // units of 128 k; upw: units per wave
};

struct Frag {
    uint32_t w[4];
};
__device__ __forceinline__ bf16x8 frag(const Frag &f) { return __builtin_bit_cast(bf16x8, f); }

// 8 nibbles as 16 + q, in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ Frag dequant(uint32_t d) {
    constexpr uint32_t mask = 0x00780078u, one = 0x41804180u;  // 16.0 twice
    return {{((d << 3) & mask) | one, ((d >> 1) & mask) | one, ((d >> 5) & mask) | one, ((d >> 9) & mask) | one}};
}

// 8 values of x as NS bf16 fragments in that order whose sum is x: x itself for bf16; for fp32 its upper,
// middle and lower 8 bits
template <typename T>
struct Split {
    static constexpr int NS = sizeof(T) == 2 ? 1 : 3;
    Frag f[NS];
};
template <typename T>
__device__ __forceinline__ Split<T> split_x(const Raw8<T> &r) {
    Split<T> s;
    if constexpr (sizeof(T) == 2) {
        s.f[0].w[0] = __builtin_amdgcn_perm(r.w[2], r.w[0], 0x05040100u);
        s.f[0].w[1] = __builtin_amdgcn_perm(r.w[2], r.w[0], 0x07060302u);
        s.f[0].w[2] = __builtin_amdgcn_perm(r.w[3], r.w[1], 0x05040100u);
        s.f[0].w[3] = __builtin_amdgcn_perm(r.w[3], r.w[1], 0x07060302u);
    } else {
        uint32_t p[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = __uint_as_float(r.w[e]);
            p[0][e] = r.w[e];
            const float m = v - __uint_as_float(r.w[e] & 0xFFFF0000u);
            p[1][e] = __float_as_uint(m);
            p[2][e] = __float_as_uint(m - __uint_as_float(p[1][e] & 0xFFFF0000u));
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int h = 0; h < 4; ++h) s.f[i].w[h] = __builtin_amdgcn_perm(p[i][h + 4], p[i][h], 0x07060302u);
    }
    return s;
}

// 16-byte pieces (lane group g, word d) -> (d, g): lane group g holds 32 consecutive k of its row, and
// product j then finds k = 32 j + 8 g in word j of lane group g, so that a product's 32 k are consecutive
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
    typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
    u32x2 a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    u32x2 b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    u32x2 c = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
    u32x2 d = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
    w[0] = c.x, w[1] = c.y, w[2] = d.x, w[3] = d.y;
}

// One workgroup: 16 RT rows of the matrix for 16 TM rows of x; its waves share out k, upw units of 128 each,
// and add their sums in LDS.  Lane (i, g): row i of each 16 and k piece g.  GM: products per group (group / 32).
template <typename T, int GM, int RT, int TM>
__global__ __launch_bounds__(512) void w4_kernel(W4Params p) {
    extern __shared__ float red[];
    constexpr int NS = Split<T>::NS, NG = 4 / GM;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * (16 * RT);
    const int tok0 = blockIdx.y * (16 * TM);
    const T *x[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        // rows past the last repeat it: their products fall into columns that are not stored
        const int r = tok0 + 16 * t + i < p.rows ? tok0 + 16 * t + i : p.rows - 1;
        x[t] = (const T *)p.x + r * p.x_stride;
    }
    int64_t wr[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t row = row0 + 16 * r + i;
        wr[r] = row < p.n ? row : p.n - 1;
    }
    f32x4 acc[RT][TM];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TM; ++t) acc[r][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const Frag ones = {{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}};
    const f32x4 nil = {0.f, 0.f, 0.f, 0.f};

    struct Unit {
        uint32_t w[RT][4];
        float s[RT][NG], z[RT][NG];
    };
    auto load_unit = [&](int u, Unit &d) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int kb = u * 128 + 32 * g;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (kb < p.k) v = *(const uint4 *)(p.q + wr[r] * (p.k >> 1) + (kb >> 1));
            d.w[r][0] = v.x, d.w[r][1] = v.y, d.w[r][2] = v.z, d.w[r][3] = v.w;
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                int gi = u * NG + a;
                gi = gi < p.groups ? gi : p.groups - 1;
                d.s[r][a] = Io<uint16_t>::f32(p.scales[wr[r] * p.groups + gi]);
                d.z[r][a] = p.zeros ? (float)(p.zeros[wr[r] * p.groups + gi] & 15) : 8.f;
            }
        }
    };
    const int u0 = wave * p.upw, u1 = u0 + p.upw < p.units ? u0 + p.upw : p.units;
    Unit cur;
    if (u0 < u1) load_unit(u0, cur);
    for (int u = u0; u < u1; ++u) {
        Raw8<T> xr[4][TM];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                xr[j][t] = Raw8<T>{};
                if (u * 128 + 32 * j < p.k) xr[j][t] = load_any8(x[t] + u * 128 + 32 * j + 8 * g);
            }
        Unit next;
        if (u + 1 < u1) load_unit(u + 1, next);
#pragma unroll
        for (int r = 0; r < RT; ++r) transpose4(cur.w[r]);
        f32x4 part[RT][TM], xs[TM];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Split<T> sx[TM];
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                sx[t] = split_x<T>(xr[j][t]);
#pragma unroll
                for (int e = 0; e < NS; ++e)
                    xs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(sx[t].f[e]), frag(ones),
                                                                   j % GM == 0 && e == 0 ? nil : xs[t], 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const Frag w = dequant(cur.w[r][j]);
#pragma unroll
                for (int t = 0; t < TM; ++t)
#pragma unroll
                    for (int e = 0; e < NS; ++e)
                        part[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(sx[t].f[e]), frag(w),
                                                                            j % GM == 0 && e == 0 ? nil : part[r][t], 0, 0, 0);
            }
            if (j % GM == GM - 1) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float s = cur.s[r][j / GM], z = -16.f - cur.z[r][j / GM];
#pragma unroll
                    for (int t = 0; t < TM; ++t)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[r][t][c] = fmaf(s, fmaf(z, xs[t][c], part[r][t][c]), acc[r][t][c]);
                }
            }
        }
        cur = next;
    }
    // the waves' sums, in order; element c of lane (i, g): row i of the matrix, row 4 g + c of x
    const int nw = blockDim.x >> 6;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) red[((wave * RT + r) * TM + t) * 256 + c * 64 + lane] = acc[r][t][c];
    __syncthreads();
    for (int o = tid; o < RT * TM * 256; o += blockDim.x) {
        const int l = o & 63, c = (o >> 6) & 3, t = (o >> 8) % TM, r = (o >> 8) / TM;
        const int tok = tok0 + 16 * t + 4 * (l >> 4) + c;
        const int64_t row = row0 + 16 * r + (l & 15);
        if (tok >= p.rows || row >= p.n) continue;
        float v = 0.f;
        for (int w = 0; w < nw; ++w) v += red[w * RT * TM * 256 + o];
        if (p.bias) v += p.bias[row];
        ((T *)p.y)[tok * p.n + row] = Io<T>::to(v);
    }
}

template <typename T, int GM, int RT>
int launch_w4(const W4Params &p, int tm, int waves, void *stream) {
    const dim3 grid((unsigned)((p.n + 16 * RT - 1) / (16 * RT)), (unsigned)((p.rows + 16 * tm - 1) / (16 * tm)));
    const unsigned lds = waves * RT * tm * 1024;
    return tm == 1 ? enqueue(w4_kernel<T, GM, RT, 1>, grid, dim3(64 * waves), p, stream, lds)
                   : enqueue(w4_kernel<T, GM, RT, 2>, grid, dim3(64 * waves), p, stream, lds);
}

template <typename T, int GM>
int launch_rt(const W4Params &p, int tm, void *stream) {
    // rows of the matrix per wave: x is fetched once for them, so 64 (fp32 x, whose three fragments take
    // more registers: 32) where that still leaves three workgroups per compute unit, else 16
    constexpr int RT = sizeof(T) == 2 ? 4 : 2;
    const int64_t tiles = (p.n + 15) / 16;
    const bool big = tiles >= RT * 768;
    W4Params c = p;
    // waves over k: four, or eight where there are few workgroups; at most one per unit
    int waves = (big ? tiles / RT : tiles) >= 512 ? 4 : 8;
    if (waves > p.units) waves = p.units;
    c.upw = (p.units + waves - 1) / waves;
    return big ? launch_w4<T, GM, RT>(c, tm, waves, stream) : launch_w4<T, GM, 1>(c, tm, waves, stream);
}

template <typename T>
int launch_group(const W4Params &p, int64_t group, int tm, void *stream) {
    if (group == 32) return launch_rt<T, 1>(p, tm, stream);
    if (group == 64) return launch_rt<T, 2>(p, tm, stream);
    return launch_rt<T, 4>(p, tm, stream);
}

}  // namespace

extern "C" {

int w4_matvec(const void *x, int64_t x_stride, const void *qweight, const void *scales, const void *zeros,
              const float *bias, void *y, int64_t rows, int64_t n, int64_t k, int64_t group, int io_dtype,
              void *stream) {
    if (rows < 0 || n < 0 || k < 0) return SELSCAN_E_SHAPE;
    if (!io_known(io_dtype) || (group != 32 && group != 64 && group != 128)) return SELSCAN_E_UNSUPPORTED;
    if (k % group) return SELSCAN_E_SHAPE;
    if (rows == 0 || n == 0) return SELSCAN_OK;
    if (k == 0 || x_stride < k || mul_size(rows, x_stride) < 0 || mul_size(rows, n) < 0 || mul_size(n, k) < 0) return SELSCAN_E_SHAPE;
    // sizes that the launch grid and 32-bit indexes within a row hold
    if (k > (1 << 30) || rows > 32 * INT64_C(65535) || n > 16 * (int64_t)INT32_MAX) return SELSCAN_E_UNSUPPORTED;
    if (!x || !qweight || !scales || !y) return SELSCAN_E_NULL;
    const size_t s = io_bytes(io_dtype);
    if (!span_aligned(x, s) || !span_aligned(y, s) || !span_aligned(qweight, 16) || !span_aligned(scales, 2) ||
        !span_aligned(bias, 4))
        return SELSCAN_E_ALIGN;
    const size_t ng = (size_t)n * (size_t)(k / group);
    const Span in[] = {{x, strided_bytes(rows, k, x_stride, s)},
                       {qweight, (size_t)n * k / 2},
                       {scales, ng * 2},
                       {zeros, ng},
                       {bias, (size_t)n * 4}};
    const Span out[] = {{y, (size_t)rows * n * s}};
    if (any_alias(in, 5, out, 1)) return SELSCAN_E_ALIAS;
    W4Params p{};
    p.x = x, p.q = (const uint8_t *)qweight, p.zeros = (const uint8_t *)zeros, p.scales = (const uint16_t *)scales;
    p.bias = bias, p.y = y, p.x_stride = x_stride, p.n = n, p.rows = (int)rows, p.k = (int)k;
    p.groups = (int)(k / group), p.units = (int)((k + 127) / 128);
    const int tm = rows <= 16 ? 1 : 2;
    return io_dtype == SELSCAN_BF16 ? launch_group<uint16_t>(p, group, tm, stream) : launch_group<float>(p, group, tm, stream);
}

}  // extern "C"
