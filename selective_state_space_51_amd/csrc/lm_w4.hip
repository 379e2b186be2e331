// libselscan_lm - a few rows times a 4-bit weight matrix with group scales (w4_matvec of
// include/selscan_lm.h).  MI355X (gfx950).
//
// y[r][j] = sum over groups of  scale * (sum_k q x - zero * sum_k x).  The inner sums run on the matrix
// cores (16 rows of x by 16 rows of the matrix by 32 k), with the 4-bit values as bf16 numbers 16 + q: a
// nibble put into the top of the mantissa of 16.0 is that number exactly, one shift and one and-or for two
// weights.  The 16 leaves together with the zero point, by a second product with the constant -(16 + zero).
// (128 + q would save nothing and cost 8 times the cancellation.)
//
// Each weight is read once per 32 rows of x.  One row (n 50,280, k 2,048, groups of 64): 18 us, of which 14 are the matrix at
// the rate that reads alone reach (4.05 TB/s).  24 rows: 25 us; two tiles of x double the matrix products and the reads of x
// from LDS, and each compute unit's fourth workgroup (3.07 on average) adds 5 us to its first three.
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
    int rows, k, groups, upw;  // upw: units of 128 k per wave
};

struct Frag {
    uint32_t w[4];
};
__device__ __forceinline__ bf16x8 frag(const Frag &f) { return __builtin_bit_cast(bf16x8, f); }

// 16.0 twice, in a vector register: and-or is one instruction if only one of its operands is scalar
__device__ __forceinline__ uint32_t two_16s() {
    uint32_t v = 0x41804180u;
    asm("" : "+v"(v));
    return v;
}
// 8 nibbles as 16 + q, in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ Frag dequant(uint32_t d, uint32_t base) {
    constexpr uint32_t mask = 0x00780078u;
    return {{((d << 3) & mask) | base, ((d >> 1) & mask) | base, ((d >> 5) & mask) | base, ((d >> 9) & mask) | base}};
}

// The operand of -(16 + zero), exact in bf16, eight times, for each zero point: a 16-byte read in place of forming it.
__device__ __forceinline__ void fill_zero_table(uint4 *zt, int lane) {
    if (lane >= 16) return;
    const uint32_t z = 0xC180u | (uint32_t)lane << 3, v = z << 16 | z;
    zt[lane] = make_uint4(v, v, v, v);
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

template <int V>
struct IntC {
    static constexpr int value = V;
};

// N values of consecutive groups, from any address aligned to one
template <typename V, int N>
struct __attribute__((packed, aligned(sizeof(V)))) Group {
    V v[N];
};
// 16 bytes of x from any address aligned to 2
struct __attribute__((packed, aligned(2))) Raw16 {
    uint32_t w[4];
};

// Every load takes whole pieces of rows: the matrix products want each lane to hold another row, but loads in that form
// touch a cache line per lane, and the address unit, at a line a clock, then bounds the kernel (47 us for 24 x 2,048 x
// 50,280).  The pieces go through LDS and come back in operand form.  A piece of 16 bytes is stored at its number
// xor a function of its row, so that the 16 rows of an operand lie in different banks.
//
// Loads ahead are never under a condition (past the end they read what is there again), so that the wait for one does
// not become a wait for all.

// the matrix: 16 rows x 4 pieces of a unit
__device__ __forceinline__ int w_at(int row, int piece) { return row * 4 + (piece ^ (row >> 2)); }

// what a wave needs of 16 rows of the matrix
template <int GM>
struct MatrixRows {
    static constexpr int NG = 4 / GM;  // groups of a unit
    const uint8_t *wb, *zb;
    const uint16_t *sb;
    uint32_t wo, so;  // offsets: 4 lanes to a row
    int groups, lane;
    bool zeros;
    Group<uint16_t, NG> sv;
    Group<uint8_t, NG> zv;

    __device__ __forceinline__ MatrixRows(const W4Params &p, int64_t row0, int lane_) : lane(lane_) {
        // rows past the last repeat it: their products are not stored
        const int64_t rowc = row0 < p.n ? row0 : p.n - 1;
        const int most = (int)(p.n - rowc < 16 ? p.n - rowc : 16) - 1;
        const uint32_t r = (lane >> 2) < most ? lane >> 2 : most;
        groups = p.groups;
        zeros = p.zeros != nullptr;
        wb = p.q + rowc * (p.k >> 1);
        sb = p.scales + rowc * p.groups;
        zb = zeros ? p.zeros + rowc * p.groups : (const uint8_t *)sb;  // (read and not used without zeros)
        wo = r * (uint32_t)(p.k >> 1) + 16 * (lane & 3);
        so = r * (uint32_t)p.groups;
    }
    __device__ __forceinline__ uint4 load(int u) const { return *(const uint4 *)(wb + (int64_t)u * 64 + wo); }
    // scales and zero points of units u .. u + 3, one unit to a lane (of a unit past the last: some that exist)
    __device__ __forceinline__ void load_scales(int u) {
        int at = (u + (lane & 3)) * NG;
        at = at + NG <= groups ? at : groups - NG;
        sv = *(const Group<uint16_t, NG> *)(sb + so + at);
        zv = *(const Group<uint8_t, NG> *)(zb + so + at);
    }
    // of unit u alone, which may end early
    __device__ __forceinline__ void load_scales_of_last(int u) {
#pragma unroll
        for (int a = 0; a < NG; ++a) {
            const int at = u * NG + a < groups ? u * NG + a : groups - 1;
            sv.v[a] = sb[so + at];
            zv.v[a] = zb[so + at];
        }
    }
    // [4 units][NG][16 rows]: scale (bf16) above, the zero point's byte offset in its table below
    __device__ __forceinline__ void store_scales(uint32_t *sz) const {
#pragma unroll
        for (int a = 0; a < NG; ++a)
            sz[((lane & 3) * NG + a) * 16 + (lane >> 2)] = (uint32_t)sv.v[a] << 16 | (zeros ? zv.v[a] & 15 : 8) << 4;
    }
};

// acc += the products of one unit: x as fragments from `fx(t, e, j)`, the matrix from w, scales from sz.  The 16 and the
// zero point leave by a second product, of x with -(16 + zero) for every k of the group.
template <int GM, int TM, int NS, class F>
__device__ __forceinline__ void unit_products(F fx, const uint4 *w, const uint32_t *sz, const uint4 *zt, uint32_t base, int q, int i,
                                              int g, f32x4 (&acc)[TM]) {
    constexpr int NG = 4 / GM;
    const f32x4 nil = {0.f, 0.f, 0.f, 0.f};
    f32x4 part[TM];
    float s;
    Frag zf;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j % GM == 0) {
            const uint32_t v = sz[(q * NG + j / GM) * 16 + i];
            s = __uint_as_float(v & 0xFFFF0000u);
            const uint4 z = *(const uint4 *)((const char *)zt + (v & 0xFFFFu));
            zf = {{z.x, z.y, z.z, z.w}};
        }
        const Frag wf = dequant(((const uint32_t *)&w[w_at(i, j)])[g], base);
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int e = 0; e < NS; ++e) {
                const bf16x8 x = frag(fx(t, e, j));
                part[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, frag(wf), j % GM == 0 && e == 0 ? nil : part[t], 0, 0, 0);
                part[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, frag(zf), part[t], 0, 0, 0);
            }
        if (j % GM == GM - 1) {
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[t][c] = fmaf(s, part[t][c], acc[t][c]);
        }
    }
}

// One output by its definition in 64 bits, for those that the matrix cores leave infinite or NaN.  An infinite x or one
// above 1e37 does that where the definition has a number or an infinity: (16 + q) x and -(16 + zero) x overflow before they
// cancel.  Neither goes away in what is added after it, so the end is where to look; a row without such x never comes here (24 x 2,048 x 50,280
// with one infinite row 215 us, without 23.5).  The arguments are read afresh, so that they take nothing of the other path's.
template <typename T, int GM>
__device__ __forceinline__ float output_in_64_bits(int64_t tok, int64_t row) {
    const auto &p = fresh_args<W4Params>();
    const T *x = (const T *)p.x + tok * p.x_stride;
    const uint8_t *q = p.q + row * (p.k >> 1);
    double sum = 0.;
#pragma unroll 1
    for (int g = 0; g < p.groups && sum == sum; ++g) {
        const double scale = Io<uint16_t>::f32(p.scales[row * p.groups + g]);
        const int zero = p.zeros ? p.zeros[row * p.groups + g] & 15 : 8;
#pragma unroll 1
        for (int i = 0; i < 16 * GM; ++i) {
            const int b = q[g * 16 * GM + i];
            const T *at = x + 2 * (g * 16 * GM + i);
            sum = fma((double)((b & 15) - zero) * scale, (double)Io<T>::f32(at[0]), sum);
            sum = fma((double)((b >> 4) - zero) * scale, (double)Io<T>::f32(at[1]), sum);
        }
    }
    return (float)(p.bias ? sum + p.bias[row] : sum);
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// Many rows of the matrix: the four waves of a workgroup take 16 rows each and the whole of k together, so that x is
// staged, split and reordered once for all of them, and no sums are left to join.  x has two buffers: one barrier
// per unit.  The matrix is loaded two units ahead, x one.
template <typename T, int GM, int TM>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) void w4_rows(W4Params p) {
    constexpr int NS = Split<T>::NS, NG = 4 / GM;
    __shared__ uint4 xl[2][NS][16 * TM * 16];  // bf16 pieces of 8 k, 16 a row
    __shared__ uint4 wl[4][64];
    __shared__ uint32_t szl[4][64 * NG];
    __shared__ uint4 zt[16];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 64 + wave * 16, tok0 = (int64_t)blockIdx.y * (16 * TM);
    MatrixRows<GM> m(p, row0, lane);
    const uint32_t base = two_16s();
    fill_zero_table(zt, tid);  // (the first unit's barrier comes before it is read)
    // x: this thread brings piece tid & 15 (8 k) of row tid / 16, and of row 16 + tid / 16 where TM = 2
    const int most = (int)(p.rows - tok0) - 1;
    uint32_t xo[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const int r = 16 * t + (tid >> 4);
        xo[t] = (uint32_t)(r < most ? r : most) * (uint32_t)p.x_stride + 8 * (tid & 15);
    }
    const T *xb = (const T *)p.x + tok0 * p.x_stride;
    f32x4 acc[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    Raw8<T> xv[TM];
    auto load_x = [&](int u) {
#pragma unroll
        for (int t = 0; t < TM; ++t) xv[t] = load_any8(xb + (int64_t)u * 128 + xo[t]);
    };
    const int whole = p.k >> 7;
    // unit u, q = u % 4; more: loads ahead
    auto step = [&](int u, uint4 &wv, auto qc, auto more) {
        constexpr int q = decltype(qc)::value, buf = q & 1;
        if (q == 0 || !decltype(more)::value) {
            m.store_scales(szl[wave]);
            if constexpr (decltype(more)::value) m.load_scales(u + 4);
        }
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const Split<T> sx = split_x<T>(xv[t]);
#pragma unroll
            for (int e = 0; e < NS; ++e)
                xl[buf][e][(16 * t + (tid >> 4)) * 16 + ((tid & 15) ^ (tid >> 4))] =
                    make_uint4(sx.f[e].w[0], sx.f[e].w[1], sx.f[e].w[2], sx.f[e].w[3]);
        }
        wl[wave][w_at(lane >> 2, lane & 3)] = wv;
        lds_barrier();
        if constexpr (decltype(more)::value) {
            load_x(u + 1 < whole ? u + 1 : u);
            wv = m.load(u + 2 < whole ? u + 2 : u);
        }
        auto fx = [&](int t, int e, int j) {
            const uint4 v = xl[buf][e][(16 * t + i) * 16 + ((4 * j + g) ^ i)];
            return Frag{{v.x, v.y, v.z, v.w}};
        };
        unit_products<GM, TM, NS>(fx, wl[wave], szl[wave], zt, base, q, i, g, acc);
    };
    uint4 wa, wc;  // the matrix: units of even and of odd number
    if (whole > 0) {
        m.load_scales(0);
        load_x(0);
        wa = m.load(0);
        wc = m.load(whole > 1 ? 1 : 0);
        for (int u = 0; u < whole; u += 4) {
            step(u, wa, IntC<0>{}, BoolC<true>{});
            if (u + 1 >= whole) break;
            step(u + 1, wc, IntC<1>{}, BoolC<true>{});
            if (u + 2 >= whole) break;
            step(u + 2, wa, IntC<2>{}, BoolC<true>{});
            if (u + 3 >= whole) break;
            step(u + 3, wc, IntC<3>{}, BoolC<true>{});
        }
    }
    // what k leaves past the whole units: pieces that exist, the others with x and q of zero
    const int left = p.k - whole * 128;
    if (left) {
        m.load_scales_of_last(whole);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            xv[t] = Raw8<T>{};
            if (8 * (tid & 15) < left) xv[t] = load_any8(xb + (int64_t)whole * 128 + xo[t]);
        }
        wa = make_uint4(0, 0, 0, 0);
        if (32 * (lane & 3) < left) wa = m.load(whole);
        lds_barrier();  // (the buffer of q = 0 may still be read)
        step(whole, wa, IntC<0>{}, BoolC<false>{});
    }
    const int64_t row = row0 + i;
    if (row >= p.n) return;
    const float b = p.bias ? p.bias[row] : 0.f;
    uint32_t again = 0;  // outputs 4 t + c
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int64_t tok = tok0 + 16 * t + 4 * g + c;
            if (tok < p.rows) {
                ((T *)p.y)[tok * p.n + row] = Io<T>::to(acc[t][c] + b);
                if (!finite(acc[t][c])) again |= 1u << (4 * t + c);
            }
        }
#pragma unroll 1
    for (; again; again &= again - 1) {
        const int o = __builtin_ctz(again);
        const int64_t tok = tok0 + 16 * (o >> 2) + 4 * g + (o & 3);
        ((T *)p.y)[tok * p.n + row] = Io<T>::to(output_in_64_bits<T, GM>(tok, row));
    }
}

// Few rows of the matrix: a workgroup takes 16 of them and its waves share out k, upw units each, and add their sums in
// LDS.  A wave stages its own units of x and waits for no other until the end.
template <typename T, int TM, int NG>
struct WaveLds {
    static constexpr int XP = 8 * (int)sizeof(T);  // 16-byte pieces of a row of x
    static constexpr int XL = TM * XP / 4;         // loads of 64 pieces
    uint4 x[16 * TM * XP];
    uint4 w[64];
    uint4 zt[16];
    uint32_t sz[64 * NG];
};

template <typename T, int GM, int TM>
__global__ __launch_bounds__(512) void w4_split(W4Params p) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    constexpr int NS = Split<T>::NS, NG = 4 / GM, H = (int)sizeof(T) / 2;
    using S = WaveLds<T, TM, NG>;
    constexpr int XP = S::XP, XL = S::XL;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, i = lane & 15, g = lane >> 4;
    S &st = ((S *)lds)[wave];
    const int64_t row0 = (int64_t)blockIdx.x * 16, tok0 = (int64_t)blockIdx.y * (16 * TM);
    MatrixRows<GM> m(p, row0, lane);
    const uint32_t base = two_16s();
    fill_zero_table(st.zt, lane);
    const int most = (int)(p.rows - tok0) - 1;
    uint32_t xo[XL];
#pragma unroll
    for (int l = 0; l < XL; ++l) {
        const int r = (64 * l + lane) / XP;
        xo[l] = (uint32_t)(r < most ? r : most) * (uint32_t)p.x_stride + (lane % XP) * (16 / sizeof(T));
    }
    const T *xb = (const T *)p.x + tok0 * p.x_stride;
    f32x4 acc[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    uint4 xv[XL], wv[4];  // the matrix: four units ahead
    auto load_piece = [&](int u, int l) {
        const Raw16 r = *(const Raw16 *)(xb + (int64_t)u * 128 + xo[l]);
        return make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    };
    auto load_x = [&](int u) {
#pragma unroll
        for (int l = 0; l < XL; ++l) xv[l] = load_piece(u, l);
    };
    auto store_unit = [&](const uint4 &w) {
#pragma unroll
        for (int l = 0; l < XL; ++l) {
            const int r = (64 * l + lane) / XP;
            st.x[r * XP + ((lane % XP) ^ (r & 15))] = xv[l];
        }
        st.w[w_at(lane >> 2, lane & 3)] = w;
    };
    auto compute = [&](int q) {
        Split<T> sx[TM][4];
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                Raw8<T> r;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const uint4 v = st.x[(16 * t + i) * XP + (((4 * j + g) * H + h) ^ i)];
                    r.w[4 * h] = v.x, r.w[4 * h + 1] = v.y, r.w[4 * h + 2] = v.z, r.w[4 * h + 3] = v.w;
                }
                sx[t][j] = split_x<T>(r);
            }
        unit_products<GM, TM, NS>([&](int t, int e, int j) { return sx[t][j].f[e]; }, st.w, st.sz, st.zt, base, q, i, g, acc);
    };
    const int whole = p.k >> 7;
    const int u0 = wave * p.upw, u1 = u0 + p.upw < whole ? u0 + p.upw : whole;
    if (u0 < u1) {
#pragma unroll
        for (int h = 0; h < 4; ++h) wv[h] = m.load(u0 + h < u1 ? u0 + h : u0);
        m.load_scales(u0);
        load_x(u0);
        auto step = [&](int u, auto qc) {
            constexpr int q = decltype(qc)::value;
            if constexpr (q == 0) {
                m.store_scales(st.sz);
                m.load_scales(u + 4);
            }
            store_unit(wv[q]);
            load_x(u + 1 < u1 ? u + 1 : u);
            wv[q] = m.load(u + 4 < u1 ? u + 4 : u);
            compute(q);
        };
        for (int u = u0; u < u1; u += 4) {
            step(u, IntC<0>{});
            if (u + 1 >= u1) break;
            step(u + 1, IntC<1>{});
            if (u + 2 >= u1) break;
            step(u + 2, IntC<2>{});
            if (u + 3 >= u1) break;
            step(u + 3, IntC<3>{});
        }
    }
    const int left = p.k - whole * 128;
    if (left && wave == (int)(blockDim.x >> 6) - 1) {
        m.load_scales_of_last(whole);
#pragma unroll
        for (int l = 0; l < XL; ++l) {
            xv[l] = make_uint4(0, 0, 0, 0);
            if ((lane % XP) * (int)(16 / sizeof(T)) < left) xv[l] = load_piece(whole, l);
        }
        wv[0] = make_uint4(0, 0, 0, 0);
        if (32 * (lane & 3) < left) wv[0] = m.load(whole);
        m.store_scales(st.sz);
        store_unit(wv[0]);
        compute(0);
    }
    // the waves' sums, in order; element c of lane (i, g): row i of the matrix, row 4 g + c of x
    const int nw = blockDim.x >> 6;
    float *red = (float *)lds;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) red[(wave * TM + t) * 256 + c * 64 + lane] = acc[t][c];
    __syncthreads();
    for (int o = tid; o < TM * 256; o += blockDim.x) {
        const int l = o & 63, c = (o >> 6) & 3, t = o >> 8;
        const int64_t tok = tok0 + 16 * t + 4 * (l >> 4) + c, row = row0 + (l & 15);
        if (tok >= p.rows || row >= p.n) continue;
        float v = 0.f;
        for (int w = 0; w < nw; ++w) v += red[w * TM * 256 + o];
        if (__builtin_expect(!finite(v), 0)) v = output_in_64_bits<T, GM>(tok, row);
        else if (p.bias) v += p.bias[row];
        ((T *)p.y)[tok * p.n + row] = Io<T>::to(v);
    }
}

template <typename T, int GM, int TM>
int launch_w4(const W4Params &p, void *stream) {
    const int64_t tiles = (p.n + 15) / 16, blocks_y = (p.rows + 16 * TM - 1) / (16 * TM);
    // shared x where that leaves two workgroups per compute unit, of fp32 x one: its stages let fewer waves share out k.
    // Measured at 1 and 32 rows, us, with it and without, k 2,048: n 16,384 bf16 11.2 and 13.8, 8.6 and 14.4; n 50,280 bf16
    // 16.9 and 23.3, 21.1 and 37.4; n 8,192 fp32 14.2 and 22.8, 9.0 and 21.7; n 16,384 fp32 14.5 and 23.4, 15.8 and 26.1; n 24,576
    // fp32 17.5 and 28.1, 22.3 and 43.7.  k 8,192: n 20,000 bf16 43.5 and 51.5, 26.8 and 46.0, fp32 59.6 and 97, 57.6 and 121.
    if (tiles >= 4 * 256 * (sizeof(T) == 2 ? 2 : 1))
        return enqueue(w4_rows<T, GM, TM>, dim3((unsigned)((tiles + 3) / 4), (unsigned)blocks_y), dim3(256), p, stream);
    // waves over k: four, or eight where there are few workgroups (n 8,192, k 2,048, one row: 5.6 us with four, 6.3 with
    // eight; n 16,384: 8.2 and 10.8); at most one per unit
    const int units = p.k >> 7 > 0 ? p.k >> 7 : 1, per = (int)sizeof(WaveLds<T, TM, 4 / GM>);
    static_assert(sizeof(WaveLds<T, TM, 4 / GM>) >= TM * 1024, "the sums reuse the stages");
    int waves = tiles >= 512 ? 4 : 8;
    while (waves * per > 65536) waves >>= 1;  // (64 KB: what a launch gets without asking for more)
    if (waves > units) waves = units;
    W4Params c = p;
    c.upw = (units + waves - 1) / waves;
    return enqueue(w4_split<T, GM, TM>, dim3((unsigned)tiles, (unsigned)blocks_y), dim3(64 * waves), c, stream,
                   (unsigned)(waves * per));
}

template <typename T, int GM>
int launch_rt(const W4Params &p, int tm, void *stream) {
    return tm == 1 ? launch_w4<T, GM, 1>(p, stream) : launch_w4<T, GM, 2>(p, stream);
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
    if (k > (1 << 24) || x_stride > (1 << 26) || rows > 32 * INT64_C(65535) || !grid_fits((n + 63) / 64, 256)) return SELSCAN_E_UNSUPPORTED;
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
