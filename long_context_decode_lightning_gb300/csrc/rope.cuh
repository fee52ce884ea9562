// Rotary positions, alone and fused with the append to a paged cache.
//
// Pair i of R/2 turns by pos * step_i / 2^64 turns, step_i a 64-bit fraction of
// a turn per position: the product wraps in integer arithmetic exactly as the
// angle wraps, so a position of a million is as exact as position 1 (an fp32
// angle would be off by 0.06 rad there) and no table of cosines is read. The
// top of the wrapped phase becomes an fp32 number of half turns in [-1, 1) for
// sincospif; the rotation is fp32 and rounds once, at the store. The transpose
// (the gradient) turns by the negative angle.
//
// Bound: HBM, one read and one write of the tensor. A block takes a few whole
// tokens; its threads load their 16-byte vectors first, then share the
// tokens' sines and cosines through shared memory (one sincospif per pair and
// token for all heads) while the loads are in flight.
//
// Measured: 8192 tokens of 32 heads of 128 in fp32 41.3 us, 96% of the copy rate; 64
// tokens of 32 heads of 128 in bf16 2.5 us. Append of 6400 tokens of 32 query and 8
// KV heads of 64 in fp16 19.4 us (floor 12.1), of 64 tokens of 128-wide heads 4.3 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"
#include "paged.cuh"

namespace hsi {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_CS = 2048;    // (token, pair) cosines and sines a block holds
constexpr int ROPE_UNROLL = 4;   // work items a thread loads before it needs the cosines

struct RopeTurn {
    const unsigned long long* steps;  // [rot / 2] turns per position, in 2^-64
    const int32_t* pos;               // [tokens]
    int rot, off;                     // rotated dims [off, off + rot)
    int pairs;                        // 1: pairs (2i, 2i+1); 0: (i, i + rot/2)
    float gain, sign;                 // sign -1: the transpose
};

struct RopeParams {
    RopeTurn r;
    const void* x;
    void* y;
    int64_t xt, xh, yt, yh;  // token and head strides (elements)
    int64_t T;
    int H, D, tb;            // heads, dims, tokens per block
};

// cos and sin (times gain) of `pos` at one pair.
__device__ __forceinline__ float2 rope_turn(const RopeTurn& r, int pair, int32_t pos) {
    const unsigned long long phase = (unsigned long long)(long long)pos * __ldg(r.steps + pair);
    float s, c;
    sincospif(__ll2float_rn((long long)phase) * 0x1p-63f, &s, &c);
    return make_float2(c * r.gain, s * r.gain * r.sign);
}

template <typename T>
struct Vec16 {
    static constexpr int N = 16 / sizeof(T);
    union {
        uint4 raw;
        T v[N];
    };
    __device__ Vec16() {}
};

template <typename T>
__device__ __forceinline__ float to_f(T v) { return static_cast<float>(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v) { return static_cast<T>(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// One work vector of a head: the 16 bytes at element `m`, and for a rotated
// vector of the halves layout its partner at `m + rot/2`; `pair` is the first
// pair (-1: not rotated).
struct RopeSpan {
    int m, n, pair;
};
template <int V>
__device__ __forceinline__ RopeSpan rope_span(int w, int rot, int off, int pairs) {
    RopeSpan s{w * V, -1, -1};
    if (pairs) {
        if (s.m >= off && s.m < off + rot) s.pair = (s.m - off) / 2;
    } else if (s.m >= off && s.m < off + rot / 2) {
        s.pair = s.m - off;
        s.n = s.m + rot / 2;
    } else if (s.m >= off + rot / 2) {
        s.m += rot / 2;  // the partners are done with their first halves
    }
    return s;
}
// Work vectors of a head of D dims.
template <int V>
__host__ __device__ constexpr int rope_spans(int D, int rot, int pairs) {
    return pairs ? D / V : (D - rot / 2) / V;
}

// cs: the token's (cos, sin) pairs, 16-byte aligned where a vector's pairs start.
template <typename T>
__device__ __forceinline__ void rope_rotate(const RopeSpan& s, bool pairs, const float2* cs, Vec16<T>& a, Vec16<T>& b) {
    if (s.pair < 0) return;
    if constexpr (sizeof(T) == 4) {
        if (pairs) {
            const float4 c = *reinterpret_cast<const float4*>(cs + s.pair);
            const float u0 = a.v[0], v0 = a.v[1], u1 = a.v[2], v1 = a.v[3];
            a.v[0] = u0 * c.x - v0 * c.y;
            a.v[1] = u0 * c.y + v0 * c.x;
            a.v[2] = u1 * c.z - v1 * c.w;
            a.v[3] = u1 * c.w + v1 * c.z;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float4 c = *reinterpret_cast<const float4*>(cs + s.pair + i);
            const float u0 = a.v[i], u1 = a.v[i + 1], v0 = b.v[i], v1 = b.v[i + 1];
            a.v[i] = u0 * c.x - v0 * c.y;
            b.v[i] = u0 * c.y + v0 * c.x;
            a.v[i + 1] = u1 * c.z - v1 * c.w;
            b.v[i + 1] = u1 * c.w + v1 * c.z;
        }
    } else {  // 32-bit words of two values
        uint32_t* x = &a.raw.x;
        uint32_t* y = &b.raw.x;
        if (pairs) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float4 c = *reinterpret_cast<const float4*>(cs + s.pair + i);
                const float2 p = unpack2<T>(x[i]), q = unpack2<T>(x[i + 1]);
                x[i] = pack2<T>(p.x * c.x - p.y * c.y, p.x * c.y + p.y * c.x);
                x[i + 1] = pack2<T>(q.x * c.z - q.y * c.w, q.x * c.w + q.y * c.z);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 c = *reinterpret_cast<const float4*>(cs + s.pair + 2 * i);
                const float2 u = unpack2<T>(x[i]), v = unpack2<T>(y[i]);
                x[i] = pack2<T>(u.x * c.x - v.x * c.y, u.y * c.z - v.y * c.w);
                y[i] = pack2<T>(u.x * c.y + v.x * c.x, u.y * c.w + v.y * c.z);
            }
        }
    }
}

// Whole 16-byte vectors: D, rot, off and every stride and address allow them
// (the caller checked).
template <typename T>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(RopeParams p) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int V = Vec16<T>::N;
    __shared__ __align__(16) float2 cs[ROPE_CS];
    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.y);
    const int64_t t0 = (int64_t)blockIdx.x * p.tb;
    const int nt = (int)(p.T - t0 < p.tb ? p.T - t0 : p.tb);
    const int half = p.r.rot / 2;
    const int W = rope_spans<V>(p.D, p.r.rot, p.r.pairs);
    const int per = p.H * W, items = nt * per;
    const bool in_place = p.x == p.y;
    for (int i0 = 0; i0 < items; i0 += ROPE_THREADS * ROPE_UNROLL) {
        Vec16<T> a[ROPE_UNROLL], b[ROPE_UNROLL];
        RopeSpan sp[ROPE_UNROLL];
        int tk[ROPE_UNROLL], hd[ROPE_UNROLL];
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) {
            const int i = i0 + u * ROPE_THREADS + threadIdx.x;
            tk[u] = -1;
            if (i >= items) continue;
            const int t = i / per, r = i - t * per, h = r / W;
            sp[u] = rope_span<V>(r - h * W, p.r.rot, p.r.off, p.r.pairs);
            if (in_place && sp[u].pair < 0) continue;
            tk[u] = t;
            hd[u] = h;
            const T* row = x + (t0 + t) * p.xt + h * p.xh;
            a[u].raw = *reinterpret_cast<const uint4*>(row + sp[u].m);
            if (sp[u].n >= 0) b[u].raw = *reinterpret_cast<const uint4*>(row + sp[u].n);
        }
        if (i0 == 0) {
            for (int i = threadIdx.x; i < nt * half; i += ROPE_THREADS)
                cs[i] = rope_turn(p.r, i % half, __ldg(p.r.pos + t0 + i / half));
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) {
            if (tk[u] < 0) continue;
            rope_rotate<T>(sp[u], p.r.pairs, cs + tk[u] * half, a[u], b[u]);
            T* row = y + (t0 + tk[u]) * p.yt + hd[u] * p.yh;
            *reinterpret_cast<uint4*>(row + sp[u].m) = a[u].raw;
            if (sp[u].n >= 0) *reinterpret_cast<uint4*>(row + sp[u].n) = b[u].raw;
        }
    }
}

// Any dims, strides and addresses: one pair, or one dim that is not rotated, a thread,
// each with its own sine and cosine. 8192 tokens of 32 heads of 128 in bf16, rows off 16
// bytes: 106 us (the vector kernel on aligned rows 30).
template <typename T>
__global__ void __launch_bounds__(ROPE_THREADS) rope_scalar_kernel(RopeParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.y);
    const int half = p.r.rot / 2, W = p.D - half;
    const int64_t per = (int64_t)p.H * W, items = p.T * per;
    for (int64_t i = (int64_t)blockIdx.x * ROPE_THREADS + threadIdx.x; i < items; i += (int64_t)gridDim.x * ROPE_THREADS) {
        const int64_t t = i / per;
        const int r = (int)(i - t * per), h = r / W, w = r - h * W;
        const T* in = x + t * p.xt + h * p.xh;
        T* out = y + t * p.yt + h * p.yh;
        if (w < half) {
            const int m = p.r.off + (p.r.pairs ? 2 * w : w), n = p.r.pairs ? m + 1 : m + half;
            const float2 c = rope_turn(p.r, w, __ldg(p.r.pos + t));
            const float a = to_f(in[m]), b = to_f(in[n]);
            out[m] = from_f<T>(a * c.x - b * c.y);
            out[n] = from_f<T>(a * c.y + b * c.x);
        } else {
            const int d = w - half, m = d < p.r.off ? d : d + p.r.rot;
            out[m] = in[m];
        }
    }
}

// ------------------------------------------------ append to a paged cache --

struct PagedAppendParams {
    RopeTurn r;  // steps null: nothing is rotated
    PagedView kv;
    const int32_t* q_start;
    const void *q, *k, *v;  // q may be null
    void* q_out;
    int64_t qt, qh, ot, oh, kt, kh, vt, vh;
    int64_t T;
    int Hq, tb;  // query heads; tokens per block
};

// Blocks of up to sixteen new tokens: their query heads are rotated (when given),
// their key heads are rotated into their pages, their value heads copied there.
// One launch in place of four, each of which would be little but its ramp at
// one token per sequence. A thread keeps its vectors' places in a token and
// goes from token to token, so that what finding them costs (two divisions) is
// shared; the first vectors are loaded at once, and the tokens' places in the
// pages (three dependent lookups, a warp a token) and cosines come in the
// loads' shadow.
constexpr int APPEND_UNROLL = 4, APPEND_TOKENS = 16, APPEND_CTAS = 4;

template <typename T>
__global__ void __launch_bounds__(ROPE_THREADS, APPEND_CTAS) paged_append_kernel(PagedAppendParams p) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int V = Vec16<T>::N;
    __shared__ __align__(16) float2 cs[APPEND_TOKENS * 64];   // heads of at most 128 dims
    __shared__ int64_t s_row[APPEND_TOKENS];    // element offset of a token's place in the pages, or why it has none
    const int64_t t0 = (int64_t)blockIdx.x * p.tb;
    const int nt = (int)(p.T - t0 < p.tb ? p.T - t0 : p.tb);
    const int half = p.r.steps ? p.r.rot / 2 : 0;
    const int D = p.kv.D, Hkv = p.kv.H;
    const int W = half ? rope_spans<V>(D, p.r.rot, p.r.pairs) : D / V, Wv = D / V;
    const int nq = p.q ? p.Hq * W : 0, nk = Hkv * W, per = nq + nk + Hkv * Wv;
    bool first = true;
    for (int i0 = 0; i0 < per; i0 += ROPE_THREADS) {
        const int i = i0 + threadIdx.x;
        const int kind = i >= per ? -1 : i < nq ? 0 : i < nq + nk ? 1 : 2;  // q, k, v
        const int r = i - (kind == 1 ? nq : kind == 2 ? nq + nk : 0), wide = kind == 2 ? Wv : W, h = r / wide;
        const RopeSpan sp = half && kind < 2 ? rope_span<V>(r - h * wide, p.r.rot, p.r.off, p.r.pairs)
                                             : RopeSpan{(r - h * wide) * V, -1, -1};
        const int64_t in_step = kind == 0 ? p.qt : kind == 1 ? p.kt : p.vt;
        const T* in = kind == 0   ? static_cast<const T*>(p.q) + h * p.qh
                      : kind == 1 ? static_cast<const T*>(p.k) + h * p.kh
                                  : static_cast<const T*>(p.v) + h * p.vh;
        in += t0 * in_step + sp.m;
        T* out = kind == 0   ? static_cast<T*>(p.q_out) + t0 * p.ot + h * p.oh
                 : kind == 1 ? static_cast<T*>(p.kv.k) + h * p.kv.head_stride
                             : static_cast<T*>(p.kv.v) + h * p.kv.head_stride;
        out += sp.m;
        const int pair_step = sp.n - sp.m;  // to a half's partner
        for (int k0 = 0; k0 < nt; k0 += APPEND_UNROLL) {
            Vec16<T> a[APPEND_UNROLL], b[APPEND_UNROLL];
#pragma unroll
            for (int u = 0; u < APPEND_UNROLL; ++u) {
                if (kind < 0 || k0 + u >= nt) continue;
                a[u].raw = *reinterpret_cast<const uint4*>(in + (k0 + u) * in_step);
                if (sp.n >= 0) b[u].raw = *reinterpret_cast<const uint4*>(in + (k0 + u) * in_step + pair_step);
            }
            if (first) {
                for (int j = threadIdx.x >> 5; j < nt; j += ROPE_THREADS / 32) {
                    const int64_t row = paged_new_row_warp(p.kv, p.q_start, t0 + j, p.T);
                    if ((threadIdx.x & 31) == 0) s_row[j] = row;
                }
                for (int j = threadIdx.x; j < nt * half; j += ROPE_THREADS)
                    cs[j] = rope_turn(p.r, j % half, __ldg(p.r.pos + t0 + j / half));
                __syncthreads();
                first = false;
            }
#pragma unroll
            for (int u = 0; u < APPEND_UNROLL; ++u) {
                if (kind < 0 || k0 + u >= nt) continue;
                const int64_t row = s_row[k0 + u];
                if (row == PAGED_NO_TOKEN || (kind > 0 && row < 0)) continue;
                T* to = out + (kind == 0 ? (k0 + u) * p.ot : row);
                rope_rotate<T>(sp, p.r.pairs, cs + (k0 + u) * half, a[u], b[u]);
                *reinterpret_cast<uint4*>(to) = a[u].raw;
                if (sp.n >= 0) *reinterpret_cast<uint4*>(to + pair_step) = b[u].raw;
            }
        }
    }
}

}  // namespace hsi
