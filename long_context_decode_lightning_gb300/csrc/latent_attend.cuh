// Attention over a latent cache, absorbed form: every query head's key is the
// whole entry and its value the entry's first 512 dims.
//   s_e = scale q.c_e,  out = sum p_e c_e[:512] / sum p_e,  p_e = exp(s_e - max)
// over the entries that a token sees, or those of a list it brings.
#pragma once
#include <cstdint>

#include "attend.cuh"
#include "common.cuh"
#include "latent.cuh"

namespace hsi {

struct LatentAttendParams {
    LatentView c;
    const void* q;
    int64_t qt, qh;  // token and head strides (elements)
    const int32_t* q_start;
    int64_t T;
    int max_q, max_kv, H;  // host bounds of new tokens and entries; query heads
    const int32_t* idx;    // [T][ld_idx], k entries a token, or null
    int64_t ld_idx;
    int k;
    float sl2;             // scale * log2(e)
    int causal;
    void* out;
    int64_t ot, oh;
    float* lse;            // [T][H] or null
};

constexpr int LS_HEADS = 8, LS_KEYS = 16, LS_THREADS = 128;

// Eight values of an entry in the cache's format as 16-bit numbers of type T; m is a multiple of 8.
template <int FMT>
__device__ __forceinline__ uint4 latent_load8(const uint8_t* e, int m, int dim) {
    uint32_t o[4];
    if constexpr (FMT == LF_FP8) {
        const int codes = dim - LT_TAIL;
        if (m >= codes) return __ldg(reinterpret_cast<const uint4*>(e + codes + 2 * (m - codes)));
        decode8_fp8(__ldg(reinterpret_cast<const uint2*>(e + m)), __ldg(e + codes + 2 * LT_TAIL + m / 64), o);
    } else if constexpr (FMT == LF_FP4) {
        decode8_bf16(__ldg(reinterpret_cast<const uint32_t*>(e + m / 2)), __ldg(e + 256 + m / 16), o);
    } else {
        return __ldg(reinterpret_cast<const uint4*>(e + 2 * m));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A block takes a token's eight heads and goes through its entries, 16 at a time: a thread
// per (entry, head) for the scores, four value dims of all heads a thread for the sums.
template <typename T, int FMT>
__global__ void __launch_bounds__(LS_THREADS) latent_attend_simple_kernel(const __grid_constant__ LatentAttendParams p) {
    __shared__ uint4 s_e[LS_KEYS][576 / 8], s_q[LS_HEADS][576 / 8];
    __shared__ float s_p[LS_HEADS][LS_KEYS];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    const int dim = p.c.dim, vecs = dim / 8, h0 = blockIdx.y * LS_HEADS;
    int32_t first, past;
    const int b = token_seq_warp(p.q_start, p.c.B, t, p.T, &first, &past);
    if (b < 0) return;
    const int len = latent_len(p.c, b, p.max_kv);
    const int seen = p.causal ? min(len, len - (past - (int)t) + 1) : len;
    const int n = p.idx ? p.k : max(seen, 0);
    for (int i = threadIdx.x; i < LS_HEADS * vecs; i += LS_THREADS) {
        const int h = h0 + i / vecs;
        s_q[i / vecs][i % vecs] = h < p.H ? __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + t * p.qt +
                                                                                 h * p.qh) + i % vecs)
                                          : make_uint4(0u, 0u, 0u, 0u);
    }
    const int me = threadIdx.x % LS_KEYS, mh = threadIdx.x / LS_KEYS;  // the score of this thread
    float m = -INFINITY, l = 0.f, acc[LS_HEADS][4] = {};
    for (int k0 = 0; k0 < n; k0 += LS_KEYS) {
        __syncthreads();
        for (int i = threadIdx.x; i < LS_KEYS * vecs; i += LS_THREADS) {
            const int j = k0 + i / vecs;
            int e = -1;
            if (j < n) e = p.idx ? __ldg(p.idx + t * p.ld_idx + j) : j;
            if (e >= seen) {
                raise_error(DEVERR_ARG);
                e = -1;
            }
            const uint8_t* at = e >= 0 ? latent_entry(p.c, b, e) : nullptr;
            s_e[i / vecs][i % vecs] = at ? latent_load8<FMT>(at, i % vecs * 8, dim) : make_uint4(0u, 0u, 0u, 0u);
        }
        __syncthreads();
        float s = 0.f;
        for (int v = 0; v < vecs; ++v) {
            const uint32_t *a = &s_e[me][v].x, *q = &s_q[mh][v].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = unpack2<T>(a[j]), y = unpack2<T>(q[j]);
                s += x.x * y.x + x.y * y.y;
            }
        }
        s *= p.sl2;
        const int j = k0 + me;
        if (j >= n || (p.idx && (uint32_t)__ldg(p.idx + t * p.ld_idx + j) >= (uint32_t)max(seen, 0))) s = -INFINITY;
        float top = s;
#pragma unroll
        for (int o = 1; o < LS_KEYS; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        top = fmaxf(top, m);
        const float f = m == -INFINITY ? 1.f : ex2(m - top), pe = s == -INFINITY ? 0.f : ex2(s - top);
        float sum = pe;
#pragma unroll
        for (int o = 1; o < LS_KEYS; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
        l = l * f + sum;
        m = top;
        s_p[mh][me] = pe;
        __shared__ float s_f[LS_HEADS];
        if (me == 0) s_f[mh] = f;
        __syncthreads();
#pragma unroll
        for (int h = 0; h < LS_HEADS; ++h)
#pragma unroll
            for (int d = 0; d < 4; ++d) acc[h][d] *= s_f[h];
        for (int e = 0; e < LS_KEYS; ++e) {
            const uint2 w = *(reinterpret_cast<const uint2*>(s_e[e]) + threadIdx.x);
            const float2 a = unpack2<T>(w.x), c = unpack2<T>(w.y);
#pragma unroll
            for (int h = 0; h < LS_HEADS; ++h) {
                const float pe2 = s_p[h][e];
                acc[h][0] += pe2 * a.x;
                acc[h][1] += pe2 * a.y;
                acc[h][2] += pe2 * c.x;
                acc[h][3] += pe2 * c.y;
            }
        }
    }
    __shared__ float s_l[LS_HEADS];
    if (me == 0) {
        s_l[mh] = l;
        if (p.lse && h0 + mh < p.H) p.lse[t * p.H + h0 + mh] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
    __syncthreads();
    for (int h = 0; h < LS_HEADS && h0 + h < p.H; ++h) {
        const float li = s_l[h], inv = li > 0.f || li != li ? 1.f / li : 0.f;
        *(reinterpret_cast<uint2*>(static_cast<T*>(p.out) + t * p.ot + (h0 + h) * p.oh) + threadIdx.x) =
            make_uint2(pack2<T>(acc[h][0] * inv, acc[h][1] * inv), pack2<T>(acc[h][2] * inv, acc[h][3] * inv));
    }
}

}  // namespace hsi
