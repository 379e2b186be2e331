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
#ifndef RTV
#define RTV 4
#endif

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
    int rows, k, groups, upw;  // upw: units of 128 k per wave
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

// N values of consecutive groups, from any address aligned to one
template <typename V, int N>
struct __attribute__((packed, aligned(sizeof(V)))) Group {
    V v[N];
};
// 16 bytes of x from any address aligned to 2
struct __attribute__((packed, aligned(2))) Raw16 {
    uint32_t w[4];
};

// The LDS of one wave, staged anew for every unit of 128 k.  Pieces of 16 bytes of a row are stored at their number
// xor a function of the row, so that the 16 rows of a product's operand lie in different banks.
template <typename T, int RT, int TM, int NG>
struct Stage {
    static constexpr int XP = 8 * (int)sizeof(T);  // 16-byte pieces of a row of x
    static constexpr int XL = TM * XP / 4;         // loads of 64 pieces
    uint4 x[16 * TM * XP];
    uint4 w[16 * RT * 4];
    uint32_t sz[16 * RT * 4 * NG];  // scale (bf16) above, zero point below; 4 units' groups of a row together
    __device__ static int xat(int row, int piece) { return row * XP + (piece ^ (row & 15)); }
    __device__ static int wat(int row, int piece) { return row * 4 + (piece ^ ((row >> 2) & 3)); }
};

// One workgroup: 16 RT rows of the matrix for 16 TM rows of x; its waves share out k, upw units of 128 each,
// and add their sums in LDS.  GM: products per group (group / 32).
//
// The matrix products want each lane to hold another row; loads in that form touch a cache line per lane, and the
// address unit, at one line a clock, bounds the kernel (47 us for 24 x 2,048 x 50,280, of which 512 cycles a unit were
// that).  So every load takes whole pieces of rows, 4 (matrix) or 16 (x) lanes to a row, goes through the
// wave's own LDS, and comes back in operand form without bank conflicts; scales and zero points come for 4
// units at a time, one row to 4 / RT lanes.
template <typename T, int GM, int RT, int TM>
__global__ __launch_bounds__(512) void w4_kernel(W4Params p) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    constexpr int NS = Split<T>::NS, NG = 4 / GM;
    using S = Stage<T, RT, TM, NG>;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, i = lane & 15, g = lane >> 4;
    S &st = ((S *)lds)[wave];
    const int64_t row0 = (int64_t)blockIdx.x * (16 * RT);
    const int64_t tok0 = (int64_t)blockIdx.y * (16 * TM);
    // Addresses: a base that is the same for the wave and advances with k, and a 32-bit offset per lane.  Rows of x
    // or of the matrix past the last repeat it: their products fall where nothing is stored.
    const int rows_left = (int)(p.rows - tok0) - 1;
    const int n_left = (int)(p.n - row0 < 16 * RT ? p.n - row0 : 16 * RT) - 1;
    auto clamp = [](int r, int most) { return (uint32_t)(r < most ? r : most); };
    // load l of x: pieces 64 l + lane; of the matrix: rows 16 l .. 16 l + 15, 4 lanes each
    uint32_t xo[S::XL], wo[RT];
#pragma unroll
    for (int l = 0; l < S::XL; ++l)
        xo[l] = clamp((64 * l + lane) / S::XP, rows_left) * (uint32_t)p.x_stride + (lane % S::XP) * (16 / sizeof(T));
#pragma unroll
    for (int l = 0; l < RT; ++l) wo[l] = clamp(16 * l + (lane >> 2), n_left) * (uint32_t)(p.k >> 1) + 16 * (lane & 3);
    const T *xb = (const T *)p.x + tok0 * p.x_stride;
    const uint8_t *wb = p.q + row0 * (p.k >> 1);
    // scales and zero points of 4 units: NG RT adjacent ones of row lane / (4 / RT)
    constexpr int NP = NG * RT, LP = 4 / RT;
    const uint32_t so = clamp(lane / LP, n_left) * (uint32_t)p.groups + (lane % LP) * NP;
    const int sg = (lane % LP) * NP;  // its first group among the 4 NG
    const uint16_t *sb = p.scales + row0 * p.groups;
    const bool zeros = p.zeros != nullptr;
    const uint8_t *zb = zeros ? p.zeros + row0 * p.groups : (const uint8_t *)sb;  // (read and not used without zeros)

    f32x4 acc[RT][TM];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TM; ++t) acc[r][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const Frag ones = {{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}};
    const f32x4 nil = {0.f, 0.f, 0.f, 0.f};

    uint4 xv[S::XL], wv[RT];
    Group<uint16_t, NP> sv;
    Group<uint8_t, NP> zv;
    auto load_unit = [&](int u) {
        const T *xu = xb + (int64_t)u * 128;
        const uint8_t *wu = wb + (int64_t)u * 64;
#pragma unroll
        for (int l = 0; l < S::XL; ++l) {
            const Raw16 r = *(const Raw16 *)(xu + xo[l]);
            xv[l] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        }
#pragma unroll
        for (int l = 0; l < RT; ++l) wv[l] = *(const uint4 *)(wu + wo[l]);
    };
    // of units u .. u + 3; where the row ends before them, its last group again
    auto load_scales = [&](int u) {
        const int g0 = u * NG;
        if (g0 + 4 * NG <= p.groups) {
            sv = *(const Group<uint16_t, NP> *)(sb + g0 + so);
            zv = *(const Group<uint8_t, NP> *)(zb + g0 + so);
        } else {
#pragma unroll
            for (int a = 0; a < NP; ++a) {
                const int over = g0 + sg + a - (p.groups - 1);
                sv.v[a] = sb[g0 + so + a - (over > 0 ? over : 0)];
                zv.v[a] = zb[g0 + so + a - (over > 0 ? over : 0)];
            }
        }
    };
    auto store_unit = [&]() {
#pragma unroll
        for (int l = 0; l < S::XL; ++l) st.x[S::xat((64 * l + lane) / S::XP, lane % S::XP)] = xv[l];
#pragma unroll
        for (int l = 0; l < RT; ++l) st.w[S::wat(16 * l + (lane >> 2), lane & 3)] = wv[l];
    };
    auto store_scales = [&]() {
#pragma unroll
        for (int a = 0; a < NP; ++a) st.sz[lane * NP + a] = (uint32_t)sv.v[a] << 16 | (zeros ? zv.v[a] & 15 : 8);
    };
    // q: the unit's number among the 4 whose scales are staged
    auto compute = [&](int q) {
        f32x4 part[RT][TM], xs[TM];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Split<T> sx[TM];
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                Raw8<T> r;
#pragma unroll
                for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
                    const uint4 v = st.x[S::xat(16 * t + i, (4 * j + g) * ((int)sizeof(T) / 2) + h)];
                    r.w[4 * h] = v.x, r.w[4 * h + 1] = v.y, r.w[4 * h + 2] = v.z, r.w[4 * h + 3] = v.w;
                }
                sx[t] = split_x<T>(r);
#pragma unroll
                for (int e = 0; e < NS; ++e)
                    xs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(sx[t].f[e]), frag(ones),
                                                                   j % GM == 0 && e == 0 ? nil : xs[t], 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const Frag w = dequant(((const uint32_t *)&st.w[S::wat(16 * r + i, j)])[g]);
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
                    const uint32_t v = st.sz[(16 * r + i) * 4 * NG + q * NG + j / GM];
                    const float s = __uint_as_float(v & 0xFFFF0000u), z = -16.f - (float)(v & 255);
#pragma unroll
                    for (int t = 0; t < TM; ++t)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[r][t][c] = fmaf(s, fmaf(z, xs[t][c], part[r][t][c]), acc[r][t][c]);
                }
            }
        }
    };
    // this wave's whole units, the next one (and the next four's scales) in flight during each
    const int whole = p.k >> 7;
    const int u0 = wave * p.upw, u1 = u0 + p.upw < whole ? u0 + p.upw : whole;
    if (u0 < u1) {
        load_scales(u0);
        load_unit(u0);
    }
    for (int u = u0; u < u1; ++u) {
        const int q = (u - u0) & 3;
        if (q == 0) {
            store_scales();
            load_scales(u + 4 < u1 ? u + 4 : u);
        }
        store_unit();
        load_unit(u + 1 < u1 ? u + 1 : u);
        compute(q);
    }
    // what k leaves past the whole units: pieces that exist, the others with x and q of zero
    if ((p.k & 127) && wave == (int)(blockDim.x >> 6) - 1) {
        load_scales(whole);
        const int left = p.k - whole * 128;
#pragma unroll
        for (int l = 0; l < S::XL; ++l) {
            Raw16 r{};
            if ((lane % S::XP) * (int)(16 / sizeof(T)) < left) r = *(const Raw16 *)(xb + (int64_t)whole * 128 + xo[l]);
            xv[l] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        }
#pragma unroll
        for (int l = 0; l < RT; ++l) {
            wv[l] = make_uint4(0, 0, 0, 0);
            if (32 * (lane & 3) < left) wv[l] = *(const uint4 *)(wb + (int64_t)whole * 64 + wo[l]);
        }
        store_scales();
        store_unit();
        compute(0);
    }
    // the waves' sums, in order; element c of lane (i, g): row i of the matrix, row 4 g + c of x
    const int nw = blockDim.x >> 6;
    float *red = (float *)lds;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) red[((wave * RT + r) * TM + t) * 256 + c * 64 + lane] = acc[r][t][c];
    __syncthreads();
    for (int o = tid; o < RT * TM * 256; o += blockDim.x) {
        const int l = o & 63, c = (o >> 6) & 3, t = (o >> 8) % TM, r = (o >> 8) / TM;
        const int64_t tok = tok0 + 16 * t + 4 * (l >> 4) + c;
        const int64_t row = row0 + 16 * r + (l & 15);
        if (tok >= p.rows || row >= p.n) continue;
        float v = 0.f;
        for (int w = 0; w < nw; ++w) v += red[w * RT * TM * 256 + o];
        if (p.bias) v += p.bias[row];
        ((T *)p.y)[tok * p.n + row] = Io<T>::to(v);
    }
}

template <typename T, int GM, int RT, int TM>
int launch_w4(const W4Params &p, int waves, void *stream) {
    using S = Stage<T, RT, TM, 4 / GM>;
    const dim3 grid((unsigned)((p.n + 16 * RT - 1) / (16 * RT)), (unsigned)((p.rows + 16 * TM - 1) / (16 * TM)));
    const int sums = RT * TM * 1024, per = (int)sizeof(S) > sums ? (int)sizeof(S) : sums;
    while (waves > 1 && waves * per > 65536) waves >>= 1;  // (64 KB: what a launch gets without asking for more)
    W4Params c = p;
    const int units = p.k >> 7 > 0 ? p.k >> 7 : 1;
    if (waves > units) waves = units;
    c.upw = (units + waves - 1) / waves;
    return enqueue(w4_kernel<T, GM, RT, TM>, grid, dim3(64 * waves), c, stream, (unsigned)(waves * per));
}

template <typename T, int GM>
int launch_rt(const W4Params &p, int tm, void *stream) {
    // rows of the matrix per wave: x is staged once for them, so 64 (fp32 x, whose three fragments take
    // more registers: 32) where that still leaves three workgroups per compute unit, else 16
    constexpr int RT = sizeof(T) == 2 ? RTV : 2;
    const int64_t tiles = (p.n + 15) / 16;
    const bool big = tiles >= RT * 768;
    // waves over k: four, or eight where there are few workgroups
    const int waves = (big ? tiles / RT : tiles) >= 512 ? 4 : 8;
    if (big) return tm == 1 ? launch_w4<T, GM, RT, 1>(p, waves, stream) : launch_w4<T, GM, RT, 2>(p, waves, stream);
    return tm == 1 ? launch_w4<T, GM, 1, 1>(p, waves, stream) : launch_w4<T, GM, 1, 2>(p, waves, stream);
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
    if (k > (1 << 24) || x_stride > (1 << 26) || rows > 32 * INT64_C(65535) || n > 16 * (int64_t)INT32_MAX) return SELSCAN_E_UNSUPPORTED;
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
    p.groups = (int)(k / group);
    const int tm = rows <= 16 ? 1 : 2;
    return io_dtype == SELSCAN_BF16 ? launch_group<uint16_t>(p, group, tm, stream) : launch_group<float>(p, group, tm, stream);
}

}  // extern "C"
