// libselscan_lm - linear attention with a decay for each head, on packed prompts and on single tokens, with states in a
// cache (linear_attn_packed_fwd, linear_attn_step of include/selscan_lm.h).  MI355X (gfx950).
#include "lm_packed.h"

namespace {

constexpr int kMaxKeys = 256, kMaxValues = 1024;

struct LaParams {
    const void *q, *k, *v;
    const float *decay;
    float *state;
    void *out;
    Seqs s;
    int64_t q_stride, k_stride, v_stride, decay_stride;
    int heads, share, dk, dv, vblocks;  // share: heads of a group
    float scale;
};

// A log decay as it is used: one of -infinity, or below any whose exponential is not 0 in fp32, is a number of which a
// chunk's worth can be added and subtracted again.
__device__ __forceinline__ float finite_decay(float g) { return g < -16384.f ? -16384.f : g; }

// Packed prompts, token by token: 64 columns of a head's state in a workgroup, a quarter of their rows in each thread.
template <typename T>
__global__ __launch_bounds__(256) void la_tokens(LaParams p) {
    __shared__ float kq[2][kMaxKeys];
    __shared__ float part[4][64];
    const int col = threadIdx.x & 63, quarter = threadIdx.x >> 6;
    const int vb = blockIdx.x % p.vblocks, hs = blockIdx.x / p.vblocks, h = hs % p.heads;
    const Segment g = whole_sequence(p.s, hs / p.heads);
    const int c = vb * 64 + col, rows = (p.dk + 3) / 4;
    const bool live = c < p.dv;
    float *cache = p.state && g.slot >= 0 ? p.state + ((int64_t)g.slot * p.heads + h) * p.dk * p.dv : nullptr;
    float S[kMaxKeys / 4];
#pragma unroll
    for (int i = 0; i < kMaxKeys / 4; ++i) {
        const int d = quarter * rows + i;
        S[i] = cache && g.carry && live && i < rows && d < p.dk ? cache[(int64_t)d * p.dv + c] : 0.f;
    }
    for (int t = 0; t < g.len; ++t) {
        const int64_t row = g.t0 + t;
        for (int d = threadIdx.x; d < kMaxKeys; d += 256) {
            const int64_t at = (int64_t)(h / p.share) * p.dk + d;
            kq[0][d] = d < p.dk ? Io<T>::f32(((const T *)p.k)[row * p.k_stride + at]) : 0.f;
            kq[1][d] = d < p.dk ? Io<T>::f32(((const T *)p.q)[row * p.q_stride + at]) : 0.f;
        }
        __syncthreads();
        const float e = __builtin_amdgcn_exp2f(finite_decay(p.decay[row * p.decay_stride + h]) * kLog2e);
        const float x = live ? Io<T>::f32(((const T *)p.v)[row * p.v_stride + (int64_t)h * p.dv + c]) : 0.f;
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxKeys / 4; ++i) {
            const int d = quarter * rows + i;
            if (i < rows && d < p.dk) {
                S[i] = fmaf(e, S[i], kq[0][d] * x);
                o = fmaf(kq[1][d], S[i], o);
            }
        }
        part[quarter][col] = o;
        __syncthreads();
        if (quarter == 0 && live)
            ((T *)p.out)[(row * p.heads + h) * p.dv + c] =
                Io<T>::to(p.scale * (part[0][col] + part[1][col] + part[2][col] + part[3][col]));
    }
    if (!cache || !live) return;
#pragma unroll
    for (int i = 0; i < kMaxKeys / 4; ++i) {
        const int d = quarter * rows + i;
        if (i < rows && d < p.dk) cache[(int64_t)d * p.dv + c] = S[i];
    }
}

// One token per sequence: 4 x CG columns of a head's state in a workgroup, CG lanes side by side in a row of it, ND rows in
// each thread, all of them in flight at once.
template <typename T, int CG, int ND, bool VEC>
__global__ __launch_bounds__(256) void la_step(LaParams p) {
    __shared__ float4 part[4][CG];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cg = lane % CG;
    const int vb = blockIdx.x % p.vblocks, hs = blockIdx.x / p.vblocks, h = hs % p.heads;
    const int row = hs / p.heads;
    const int64_t slot = slot_of(p.s, row);
    const int c = (vb * CG + cg) * 4, nc = p.dv - c < 4 ? p.dv - c : 4;
    const int d0 = (threadIdx.x / CG) * ND;
    float *cache = p.state + ((slot < 0 ? 0 : slot) * p.heads + h) * p.dk * p.dv + c;
    const T *q = (const T *)p.q + row * p.q_stride + (int64_t)(h / p.share) * p.dk;
    const T *k = (const T *)p.k + row * p.k_stride + (int64_t)(h / p.share) * p.dk;
    const T *v = (const T *)p.v + row * p.v_stride + (int64_t)h * p.dv + c;
    float S[ND][4], kv[ND], qv[ND], x[4];
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        const bool on = d0 + i < p.dk && slot >= 0;
        const float *at = cache + (int64_t)(d0 + i) * p.dv;
        if constexpr (VEC) {
            const float4 w = on && nc > 0 ? *(const float4 *)at : make_float4(0.f, 0.f, 0.f, 0.f);
            S[i][0] = w.x, S[i][1] = w.y, S[i][2] = w.z, S[i][3] = w.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = on && j < nc ? at[j] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        kv[i] = d0 + i < p.dk ? Io<T>::f32(k[d0 + i]) : 0.f;
        qv[i] = d0 + i < p.dk ? Io<T>::f32(q[d0 + i]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = j < nc ? Io<T>::f32(v[j]) : 0.f;
    const float e = __builtin_amdgcn_exp2f(finite_decay(p.decay[row * p.decay_stride + h]) * kLog2e);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ND; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            S[i][j] = fmaf(e, S[i][j], kv[i] * x[j]);
            o[j] = fmaf(qv[i], S[i][j], o[j]);
        }
        if (d0 + i < p.dk && slot >= 0) {
            float *at = cache + (int64_t)(d0 + i) * p.dv;
            if constexpr (VEC) {
                if (nc > 0) *(float4 *)at = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < nc) at[j] = S[i][j];
            }
        }
    }
#pragma unroll
    for (int m = CG; m < 64; m *= 2)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], m);
    if (lane < CG) part[wave][cg] = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (threadIdx.x >= CG) return;
    T *out = (T *)p.out + ((int64_t)row * p.heads + h) * p.dv + c;
    const float4 a = part[0][cg], b = part[1][cg], e2 = part[2][cg], f = part[3][cg];
    const float s[4] = {a.x + b.x + e2.x + f.x, a.y + b.y + e2.y + f.y, a.z + b.z + e2.z + f.z, a.w + b.w + e2.w + f.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < nc) out[j] = Io<T>::to(p.scale * s[j]);
}

constexpr int64_t kMaxStride = INT64_C(1) << 26;

struct LaArgs {
    const void *q;
    int64_t q_stride;
    const void *k;
    int64_t k_stride;
    const void *v;
    int64_t v_stride;
    const float *decay;
    int64_t decay_stride;
    float scale;
    const int32_t *cu, *slots;
    const uint8_t *carry;
    float *state;
    void *out;
    int64_t rows, nseq, nslots, heads, groups, dk, dv;
    int dtype;
    void *ws;
    size_t ws_need, ws_bytes;
    bool packed;
};

int la_check(const LaArgs &a, bool *nothing) {
    *nothing = false;
    if (a.rows < 0 || a.nseq < 0 || a.nslots < 0 || a.heads < 0 || a.groups < 0 || a.dk < 0 || a.dv < 0) return SELSCAN_E_SHAPE;
    if (!io_known(a.dtype) || !(a.scale - a.scale == 0.f)) return SELSCAN_E_UNSUPPORTED;
    if (a.rows > kMaxTokens || a.nseq > INT32_MAX / 2) return SELSCAN_E_UNSUPPORTED;
    if (a.heads == 0 || a.dv == 0 || a.nseq == 0) {
        *nothing = true;
        return a.nseq == 0 && a.rows > 0 && a.heads > 0 && a.dv > 0 ? SELSCAN_E_SHAPE : SELSCAN_OK;
    }
    if (a.groups == 0 || a.dk == 0 || a.heads % a.groups) return SELSCAN_E_SHAPE;
    if (a.dk > kMaxKeys || a.dv > kMaxValues || a.heads > kMaxStride) return SELSCAN_E_UNSUPPORTED;
    const int64_t qk = a.groups * a.dk, vw = a.heads * a.dv;
    if (a.q_stride < qk || a.k_stride < qk || a.v_stride < vw || (a.decay_stride != 0 && a.decay_stride < a.heads)) return SELSCAN_E_SHAPE;
    if (a.q_stride > kMaxStride || a.k_stride > kMaxStride || a.v_stride > kMaxStride || a.decay_stride > kMaxStride)
        return SELSCAN_E_UNSUPPORTED;
    if (a.state && !a.slots && a.nslots < a.nseq) return SELSCAN_E_SHAPE;
    const int64_t entry = vw * a.dk;  // below 2^26 * 2^8
    if (mul_size(a.nslots, entry) < 0) return SELSCAN_E_SHAPE;
    if ((a.rows > 0 && (!a.q || !a.k || !a.v || !a.decay || !a.out)) || (a.packed && !a.cu) || (!a.packed && !a.state)) return SELSCAN_E_NULL;
    const size_t s = io_bytes(a.dtype);
    const void *io[] = {a.q, a.k, a.v, a.out};
    for (const void *x : io)
        if (!span_aligned(x, s)) return SELSCAN_E_ALIGN;
    if (!span_aligned(a.decay, 4) || !span_aligned(a.cu, 4) || !span_aligned(a.slots, 4) || !span_aligned(a.state, 16) ||
        (a.ws_need && !span_aligned(a.ws, 16)))
        return SELSCAN_E_ALIGN;
    if (a.ws_need && (!a.ws || a.ws_bytes < a.ws_need)) return SELSCAN_E_WORKSPACE;
    const Span in[] = {{a.q, strided_bytes(a.rows, qk, a.q_stride, s)},
                       {a.k, strided_bytes(a.rows, qk, a.k_stride, s)},
                       {a.v, strided_bytes(a.rows, vw, a.v_stride, s)},
                       {a.decay, strided_bytes(a.rows, a.heads, a.decay_stride, 4)},
                       {a.cu, (size_t)(a.nseq + 1) * 4},
                       {a.slots, (size_t)a.nseq * 4},
                       {a.carry, (size_t)a.nseq}};
    const Span out[] = {{a.out, (size_t)a.rows * vw * s}, {a.state, (size_t)a.nslots * entry * 4}, {a.ws_need ? a.ws : nullptr, a.ws_need}};
    return any_alias(in, 7, out, 3) ? SELSCAN_E_ALIAS : SELSCAN_OK;
}

LaParams la_params(const LaArgs &a, int columns) {
    LaParams p{};
    p.q = a.q, p.k = a.k, p.v = a.v, p.decay = a.decay, p.state = a.state, p.out = a.out;
    p.s = {a.cu, a.slots, a.carry, a.nslots, (int)a.rows, (int)a.nseq};
    p.q_stride = a.q_stride, p.k_stride = a.k_stride, p.v_stride = a.v_stride, p.decay_stride = a.decay_stride;
    p.heads = (int)a.heads, p.share = (int)(a.heads / a.groups), p.dk = (int)a.dk, p.dv = (int)a.dv;
    p.vblocks = (int)((a.dv + columns - 1) / columns), p.scale = a.scale;
    return p;
}

template <typename T, int CG, int ND>
int launch_step(const LaParams &p, int64_t blocks, bool vec, void *stream) {
    return enqueue(vec ? la_step<T, CG, ND, true> : la_step<T, CG, ND, false>, dim3((unsigned)blocks), dim3(256), p, stream);
}

}  // namespace

extern "C" {

size_t linear_attn_packed_workspace_bytes(int64_t tokens, int64_t nseq, int64_t max_seqlen, int64_t heads, int64_t dk,
                                          int64_t dv) {
    return 0;
}

int linear_attn_packed_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                           int64_t v_stride, const float *log_decay, int64_t decay_stride, float scale,
                           const int32_t *cu_seqlens, const int32_t *slots, const uint8_t *carry, float *state, void *out,
                           int64_t tokens, int64_t nseq, int64_t nslots, int64_t max_seqlen, int64_t heads, int64_t groups,
                           int64_t dk, int64_t dv, int io_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (max_seqlen < 0) return SELSCAN_E_SHAPE;
    const size_t need = linear_attn_packed_workspace_bytes(tokens, nseq, max_seqlen, heads, dk, dv);
    const LaArgs a{q, q_stride, k, k_stride, v, v_stride, log_decay, decay_stride, scale, cu_seqlens, slots, carry, state, out,
                   tokens, nseq, nslots, heads, groups, dk, dv, io_dtype, workspace, need, workspace_bytes, true};
    bool nothing;
    const int rc = la_check(a, &nothing);
    if (rc != SELSCAN_OK || nothing) return rc;
    const LaParams p = la_params(a, 64);
    const int64_t per = heads * p.vblocks;
    if (mul_size(nseq, per) < 0 || !grid_fits(nseq * per, 256)) return SELSCAN_E_UNSUPPORTED;
    return enqueue(io_dtype == SELSCAN_BF16 ? la_tokens<uint16_t> : la_tokens<float>, dim3((unsigned)(nseq * per)), dim3(256), p, stream);
}

int linear_attn_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                     const float *log_decay, int64_t decay_stride, float scale, const int32_t *slots, float *state,
                     void *out, int64_t rows, int64_t nslots, int64_t heads, int64_t groups, int64_t dk, int64_t dv,
                     int io_dtype, void *stream) {
    const LaArgs a{q,    q_stride, k,      k_stride, v,      v_stride, log_decay, decay_stride, scale, nullptr, slots, nullptr,
                   state, out,      rows,   rows,     nslots, heads,    groups,    dk,           dv,    io_dtype, nullptr, 0,
                   0,    false};
    bool nothing;
    const int rc = la_check(a, &nothing);
    if (rc != SELSCAN_OK || nothing) return rc;
    const int cg = dv > 32 ? 16 : dv > 16 ? 8 : 4;
    const LaParams p = la_params(a, 4 * cg);
    const int64_t per = heads * p.vblocks;
    if (mul_size(rows, per) < 0 || !grid_fits(rows * per, 256)) return SELSCAN_E_UNSUPPORTED;
    const int64_t blocks = rows * per;
    const bool vec = dv % 4 == 0;
    const int rowlanes = 256 / cg, nd = (int)((dk + rowlanes - 1) / rowlanes);
#define GO(CG, ND)                                                                                   \
    if (cg == CG && nd <= ND)                                                                        \
        return io_dtype == SELSCAN_BF16 ? launch_step<uint16_t, CG, ND>(p, blocks, vec, stream) : launch_step<float, CG, ND>(p, blocks, vec, stream);
    GO(16, 4) GO(16, 8) GO(16, 16) GO(8, 2) GO(8, 4) GO(8, 8) GO(4, 1) GO(4, 2) GO(4, 4)
#undef GO
    return SELSCAN_E_UNSUPPORTED;
}

}  // extern "C"
