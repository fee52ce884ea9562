// The latent cache: one vector of 512 or 576 values a token that all query heads
// share (its first 512 are the value, all of it is the key), its formats, the
// append of new tokens and reading entries back.
//
// Formats of an entry of `dim` values:
//  16-bit  dim values.
//  FP8     E4M3 codes of the first dim - 64 values, the last 64 (where rotary
//          dims lie) in bf16, then a byte for each 64 codes, 127 + e: their values are
//          code * 2^e, e the smallest by which the largest of the 64 is at most 448. As
//          the scale is a power of two, decoded values are exact in bf16 (at the largest e
//          codes end at 240, as 256 * 2^120 is no bf16 number). Padded to 16 bytes:
//          dim + 80 in all.
//  FP4     the main KV's entry (mainkv.cuh): 512 values in 288 bytes.
//
// Append and read are bound by HBM where there is much to move, and by a chain of
// dependent loads (sequence, length, page) where there is little. Both give a warp whole
// rows with 8 values a lane and step, so that every access is 4, 8 or 16 bytes a lane
// side by side, and look places up a lane each.
//
// Measured: 75000 FP8 entries of 576 read back 24.9 us, 86% of the copy rate; 64 x 512
// listed ones 13.1 us (67%); 13300 tokens appended as FP8 with rotation 8 us, and read
// back 7.5 us; 64 tokens appended 3 us (6 a call).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"
#include "mainkv.cuh"
#include "paged.cuh"
#include "quantize.cuh"
#include "rope.cuh"

namespace hsi {

enum LatentFormat { LF_BF16 = 0, LF_FP16 = 1, LF_FP8 = 2, LF_FP4 = 3 };

constexpr int LT_VALUE = 512;      // dims of the value
constexpr int LT_TAIL = 64;        // values of an FP8 entry that stay in bf16
constexpr int LT_MIN_E = -118, LT_MAX_E = 120;  // scales' exponents

__host__ __device__ constexpr int latent_entry_bytes(int fmt, int dim) {
    return fmt == LF_FP8 ? dim + 80 : fmt == LF_FP4 ? KV_BYTES : 2 * dim;
}

struct LatentView {
    uint8_t* data;
    int64_t page_stride, token_stride;  // bytes
    int64_t n_pages;                    // without a table: entries
    const int32_t* table;               // [B][ld_table], or null: entry e of sequence b is entry off[b] + e
    int64_t ld_table;
    const int64_t* off;
    const int32_t* kv_len;
    int B, dim, page_shift;
    int capacity;                       // entries that a row of the table lists (without a table: of the cache)
};

// Entries of sequence b, clamped to what the cache can hold for it and to the host's bound.
__device__ __forceinline__ int32_t latent_len(const LatentView& c, int b, int32_t bound = INT32_MAX) {
    const int32_t n = __ldg(c.kv_len + b);
    int64_t most = min(c.capacity, bound);
    if (!c.table) {
        const int64_t at = __ldg(c.off + b);
        most = at < 0 || at > c.n_pages ? 0 : min(most, c.n_pages - at);
    }
    if (n < 0 || n > most) {
        raise_error(DEVERR_ARG);
        return n < 0 ? 0 : (int32_t)most;
    }
    return n;
}

// The entry's address; null (reported) where the table names no page. e is below the sequence's length.
__device__ __forceinline__ uint8_t* latent_entry(const LatentView& c, int b, int32_t e) {
    if (!c.table) return c.data + (__ldg(c.off + b) + e) * c.token_stride;
    const int32_t page = __ldg(c.table + b * c.ld_table + (e >> c.page_shift));
    if (page < 0 || page >= c.n_pages) {
        raise_error(DEVERR_ARG);
        return nullptr;
    }
    return c.data + page * c.page_stride + (int64_t)(e & ((1 << c.page_shift) - 1)) * c.token_stride;
}

// Four E4M3 codes as two pairs of bf16 numbers, 2^-120 of their values: the code's seven bits
// are moved to the bf16 fields, subnormal codes among them (0x7F is 480, not NaN).
__device__ __forceinline__ void e4m3x4_fields(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = __byte_perm(w, 0u, 0x1404), b = __byte_perm(w, 0u, 0x3424);
    lo = (a & 0x80008000u) | ((a & 0x7F007F00u) >> 4);
    hi = (b & 0x80008000u) | ((b & 0x7F007F00u) >> 4);
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&p);
}
// Eight codes times 2^e, e = scale byte - 127: one product by 2^(120 + e), and where e > 0 and that might be past
// bf16, a second one. All are exact.
__device__ __forceinline__ void decode8_fp8(uint2 codes, uint32_t scale, uint32_t (&o)[4]) {
    const uint32_t first = min(scale, 127u) + 120u, s = first << 7 | first << 23;
    e4m3x4_fields(codes.x, o[0], o[1]);
    e4m3x4_fields(codes.y, o[2], o[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = bf16x2_mul(o[i], s);
    if (scale > 127u) {
        const uint32_t more = scale << 7 | scale << 23;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = bf16x2_mul(o[i], more);
    }
}

// An E4M3 scale as a pair of bf16 numbers, and eight E2M1 codes (value 2 i in the low nibble of byte i) times it: the
// values' bytes are looked up by permutes, four codes each, as conversions run at a quarter of their rate. Exact.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t byte) {
    const uint32_t f = (byte & 0x7Fu) << 4 | (byte & 0x80u) << 8;
    return bf16x2_mul(f | f << 16, 0x7B807B80u);  // 2^120
}
__device__ __forceinline__ void decode8_fp4(uint32_t codes, uint32_t scale, uint32_t (&o)[4]) {
    const uint32_t even = codes << 4;  // signs at the bytes' tops: of the even values here, of the odd ones in codes
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t pick = codes >> 16 * h & 0x7777u;  // 0, .5, 1, 1.5, 2, 3, 4, 6 in bf16
        const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, pick), hi = __byte_perm(0x3F3F3F00u, 0x40404040u, pick);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = __byte_perm(lo, hi, i ? 0x7362 : 0x5140);
            const uint32_t sign = __byte_perm(even, codes, (2 * h + i) * 0x1111 + 0x4000);
            o[2 * h + i] = bf16x2_mul(v | (sign & 0x80008000u), scale);
        }
    }
}

// ------------------------------------------------------------------- append --

struct LatentAppendParams {
    LatentView c;
    RopeTurn r;        // steps null: no rotation
    const void* x;     // [T] rows of dim values, xt apart
    int64_t xt, T;
    const int32_t* q_start;
};

// The sequence of token t of `total`, by a whole warp: -1 where it lies outside every one, or (reported) where q_start
// descends around it or its sequence leaves the tokens. *first, *past: the sequence's tokens.
__device__ __forceinline__ int token_seq_warp(const int32_t* q_start, int B, int64_t t, int64_t total, int32_t* first,
                                              int32_t* past) {
    int b = 0, last = 0;
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < B; i += 32) {
        if (__ldg(q_start + i + 1) > t) continue;
        ++b;
        last = i + 1;
    }
    b = __reduce_add_sync(~0u, b);
    if (__reduce_max_sync(~0u, last) != b) {
        raise_error(DEVERR_ARG);
        return -1;
    }
    if (b >= B) return -1;
    *first = __ldg(q_start + b);
    *past = __ldg(q_start + b + 1);
    if (t < *first) return -1;
    if (*first < 0 || *past > total) {
        raise_error(DEVERR_ARG);
        return -1;
    }
    return b;
}

// The same for N tokens at once, lane j < N's being its t: one pass over q_start for all of them.
template <int N>
__device__ __forceinline__ int token_seqs_warp(const int32_t* q_start, int B, int64_t t, int64_t total, int32_t* first,
                                               int32_t* past) {
    const int lane = threadIdx.x & 31;
    int b = 0, last = 0;
    int64_t tj[N];
#pragma unroll
    for (int j = 0; j < N; ++j) tj[j] = __shfl_sync(~0u, (long long)t, j);
    for (int i0 = 0; i0 < B; i0 += 32) {
        const int64_t end = i0 + lane < B ? __ldg(q_start + i0 + lane + 1) : INT64_MAX;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t before = __ballot_sync(~0u, end <= tj[j]);
            if (lane != j || !before) continue;
            b += __popc(before);
            last = i0 + 32 - __clz(before);
        }
    }
    __syncwarp();
    if (lane >= N || b >= B) return -1;
    if (last != b) {
        raise_error(DEVERR_ARG);
        return -1;
    }
    *first = __ldg(q_start + b);
    *past = __ldg(q_start + b + 1);
    if (t < *first) return -1;
    if (*first < 0 || *past > total) {
        raise_error(DEVERR_ARG);
        return -1;
    }
    return b;
}
template <typename P>
__device__ __forceinline__ P* shfl_ptr(P* p, int lane) {
    return reinterpret_cast<P*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(p), lane));
}

constexpr int LT_WARPS = 8;

// Four E4M3 codes of LT_MAX_E, whose values are at most 256: that is past bf16 times 2^120, so that it becomes 240 (255 *
// 2^120, the largest bf16 number, is 15 in 255 off then, less than half a step's 2^-4).
__device__ __forceinline__ uint32_t e4m3x4_to_240(uint32_t w) {
    return w - ((w >> 3 & w >> 4 & w >> 5 & w >> 6) & 0x01010101u);
}

// A token's values, eight a lane and step, as the cache's format keeps them. Whole warp.
template <typename T, int FMT>
__device__ __forceinline__ void latent_keep(int dim, const uint4 (&raw)[3], uint8_t* dst) {
    const int lane = threadIdx.x & 31;
    if constexpr (FMT == LF_BF16 || FMT == LF_FP16) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (lane + 32 * i < dim / 8) *(reinterpret_cast<uint4*>(dst) + lane + 32 * i) = raw[i];
        return;
    }
    const int codes = FMT == LF_FP8 ? dim - LT_TAIL : dim;
    uint32_t scales[2] = {0u, 0u};  // FP8: the scale bytes of groups 0-3, 4-7
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int m = 8 * (lane + 32 * i);
        const uint32_t* w = &raw[i].x;
        float v[8], amax = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<T>(w[j]);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
        // a NaN is passed over by the maximum, so values are looked at one by one
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            finite = finite && isfinite(v[j]);
            amax = fmaxf(amax, fabsf(v[j]));
        }
        if constexpr (FMT == LF_FP8) {
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
            const uint32_t bits = __float_as_uint(amax);  // 448 = 1.75 * 2^8
            int ex = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
            ex = max(LT_MIN_E, min(LT_MAX_E, ex));
            const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
            if (m < codes) {
                uint32_t c[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    asm("{ .reg .b16 t; cvt.rn.satfinite.e4m3x2.f32 t, %1, %2; cvt.u32.u16 %0, t; }"
                        : "=r"(c[j])
                        : "f"(v[2 * j + 1] * inv), "f"(v[2 * j] * inv));
                uint2 w = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                if (ex == LT_MAX_E) w = make_uint2(e4m3x4_to_240(w.x), e4m3x4_to_240(w.y));
                *reinterpret_cast<uint2*>(dst + m) = w;
            } else if (m < dim) {
                *reinterpret_cast<uint4*>(dst + codes + 2 * (m - codes)) = raw[i];
            }
            if (i < 2) {
                const uint32_t byte = m < codes ? (uint32_t)(ex + 127) << (lane & 24) : 0u;
                scales[i] = __reduce_or_sync(~0u, (lane & 7) == 0 ? byte : 0u);
            }
        } else if (i < 2) {
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            const uint32_t sb = f32_to_e4m3_rn_sat(__fdiv_rn(amax, 6.0f));
            const float sc = e4m3_to_f32(sb);
            uint32_t c = 0u;
            if (sc != 0.0f) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __fdiv_rn(v[j], sc);
                c = f32x4_to_e2m1x4(v[0], v[1], v[2], v[3]) | f32x4_to_e2m1x4(v[4], v[5], v[6], v[7]) << 16;
            }
            *reinterpret_cast<uint32_t*>(dst + m / 2) = c;
            if ((lane & 1) == 0) dst[256 + m / 16] = (uint8_t)sb;
        }
    }
    if (!finite) raise_error(DEVERR_ARG);
    if (FMT == LF_FP8 && lane == 0)
        *reinterpret_cast<uint4*>(dst + codes + 2 * LT_TAIL) = make_uint4(scales[0], scales[1], 0u, 0u);
}

// Cosines and sines (times gain) of a position, a pair a lane and turn.
__device__ __forceinline__ void latent_turn(const RopeTurn& r, int32_t pos, float2* cs) {
    for (int i = threadIdx.x & 31; i < r.rot / 2; i += 32) cs[i] = rope_turn(r, i, pos);
    __syncwarp();
}

// Token t's rotated dims; rot is a multiple of 16, off of 8, so that eight values are rotated or not.
template <typename T>
__device__ __forceinline__ void latent_rotate(const LatentAppendParams& p, int64_t t, const float2* cs, uint4 (&raw)[3]) {
    const int lane = threadIdx.x & 31, half = p.r.rot / 2;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int m = 8 * (lane + 32 * i), d = m - p.r.off;
        if (m >= p.c.dim || d < 0 || d >= p.r.rot) continue;
        uint32_t* w = &raw[i].x;
        if (p.r.pairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 c = cs[d / 2 + j], v = unpack2<T>(w[j]);
                w[j] = pack2<T>(v.x * c.x - v.y * c.y, v.x * c.y + v.y * c.x);
            }
            continue;
        }
        const bool low = d < half;
        const T* x = static_cast<const T*>(p.x) + t * p.xt;
        const uint4 other = __ldg(reinterpret_cast<const uint4*>(x + (low ? m + half : m - half)));
        const uint32_t* o = &other.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int pair = (low ? d : d - half) + 2 * j;
            const float2 c0 = cs[pair], c1 = cs[pair + 1], v = unpack2<T>(w[j]), u = unpack2<T>(o[j]);
            // (u, v) -> (u cos - v sin, u sin + v cos): this lane holds u below half, v from there
            w[j] = low ? pack2<T>(v.x * c0.x - u.x * c0.y, v.y * c1.x - u.y * c1.y)
                       : pack2<T>(u.x * c0.y + v.x * c0.x, u.y * c1.y + v.y * c1.x);
        }
    }
}

constexpr int LT_PAIRS = 288;  // rotated pairs of a token, at most

// A warp per token, whose loads are in flight while its place is looked up (two or four tokens a warp: no faster). A
// rotated value is rounded to the tokens' type, then kept as the format keeps it, so that the entry is the unrotated
// append of hsi_rope's result; the cosines and sines are worked out once, a pair a lane.
template <typename T, int FMT>
__global__ void __launch_bounds__(32 * LT_WARPS) latent_append_kernel(const __grid_constant__ LatentAppendParams p) {
    __shared__ float2 s_cs[LT_WARPS][LT_PAIRS];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * LT_WARPS + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int lane = threadIdx.x & 31, dim = p.c.dim;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + t * p.xt);
    uint4 raw[3] = {};
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (lane + 32 * i < dim / 8) raw[i] = __ldg(x + lane + 32 * i);
    const int32_t pos = p.r.steps ? __ldg(p.r.pos + t) : 0;
    int32_t first, past;
    const int b = token_seqs_warp<1>(p.q_start, p.c.B, t, p.T, &first, &past);
    uint8_t* dst = nullptr;
    if (lane == 0 && b >= 0) {
        // by the length as it is: by one clamped to the row, the tokens would land on the entries before them
        const int32_t len = __ldg(p.c.kv_len + b);
        const int64_t e = (int64_t)len - (past - t);
        int64_t most = p.c.capacity;
        if (!p.c.table) {
            const int64_t at = __ldg(p.c.off + b);
            most = at < 0 || at > p.c.n_pages ? 0 : min(most, p.c.n_pages - at);
        }
        if (len > most || e < 0) raise_error(DEVERR_ARG);
        if (e >= 0 && e < most) dst = latent_entry(p.c, b, (int32_t)e);
    }
    __syncwarp();
    dst = shfl_ptr(dst, 0);
    if (!dst) return;
    if (p.r.steps) {
        float2* const cs = s_cs[threadIdx.x >> 5];
        latent_turn(p.r, pos, cs);
        latent_rotate<T>(p, t, cs, raw);
        __syncwarp();
    }
    latent_keep<T, FMT>(dim, raw, dst);
}

// --------------------------------------------------------------------- read --

struct LatentReadParams {
    LatentView c;
    const int32_t* start;  // [B + 1]: the rows (with lists: the tokens) of each sequence
    const int32_t* first;  // [B] the entry of a sequence's first row, or null (0); not with lists
    const int32_t* idx;    // [T][ld_idx], k entries a token, or null
    int64_t ld_idx;
    int32_t k;
    int64_t T, rows;       // tokens (without lists: rows), rows
    uint16_t* out;
    int64_t ot;            // elements between rows (with lists: between tokens, whose rows lie side by side)
};

constexpr int LT_RPW = 4;  // rows a warp reads at once

// A warp takes four rows side by side and has all their loads in flight.
template <int FMT>
__global__ void __launch_bounds__(32 * LT_WARPS) latent_read_kernel(const __grid_constant__ LatentReadParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t r0 = ((int64_t)blockIdx.x * LT_WARPS + (threadIdx.x >> 5)) * LT_RPW;
    if (r0 >= p.rows) return;
    const int lane = threadIdx.x & 31, dim = p.c.dim;
    // the rows' entries, a lane each
    const int64_t r = r0 + lane;
    const bool mine = lane < LT_RPW && r < p.rows;
    const int64_t t = p.idx ? r / p.k : r;
    int64_t e = mine && p.idx ? __ldg(p.idx + t * p.ld_idx + (r - t * p.k)) : 0;
    int32_t from, past;
    const int b = token_seqs_warp<LT_RPW>(p.start, p.c.B, mine ? t : INT64_MAX, p.T, &from, &past);
    const uint8_t* at = nullptr;
    if (mine && b >= 0) {
        if (!p.idx) e = t - from + (p.first ? __ldg(p.first + b) : 0);
        const int32_t len = latent_len(p.c, b);
        if (e >= 0 && e < len) at = latent_entry(p.c, b, (int32_t)e);
        else if (!p.idx || e >= 0) raise_error(DEVERR_ARG);
    }
    __syncwarp();
    const uint32_t known = __ballot_sync(~0u, mine && b >= 0);
    const uint8_t* src[LT_RPW];  // null: zeros
    bool live[LT_RPW];           // rows of some sequence
#pragma unroll
    for (int j = 0; j < LT_RPW; ++j) {
        src[j] = shfl_ptr(at, j);
        live[j] = known >> j & 1;
    }
    constexpr int N = FMT == LF_FP8 || FMT == LF_FP4 ? 2 : 3;
    uint4 v[LT_RPW][3] = {};
    uint32_t sc[LT_RPW][2] = {};
#pragma unroll
    for (int j = 0; j < LT_RPW; ++j) {
        if (!src[j]) continue;
        if constexpr (FMT == LF_FP8) {
            const int codes = dim - LT_TAIL;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int m = 8 * (lane + 32 * i);
                if (m >= codes) continue;
                const uint2 c = __ldcs(reinterpret_cast<const uint2*>(src[j] + m));
                v[j][i].x = c.x;
                v[j][i].y = c.y;
                sc[j][i] = __ldcs(src[j] + codes + 2 * LT_TAIL + m / 64);
            }
            if (lane < 8) v[j][2] = __ldcs(reinterpret_cast<const uint4*>(src[j] + codes) + lane);
        } else if constexpr (FMT == LF_FP4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[j][i].x = __ldcs(reinterpret_cast<const uint32_t*>(src[j]) + lane + 32 * i);
                sc[j][i] = __ldcs(src[j] + 256 + (lane + 32 * i) / 2);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (lane + 32 * i < dim / 8) v[j][i] = __ldcs(reinterpret_cast<const uint4*>(src[j]) + lane + 32 * i);
        }
    }
#pragma unroll
    for (int j = 0; j < LT_RPW; ++j) {
        if (!live[j]) continue;
        const int64_t rj = r0 + j, tj = __shfl_sync(~0u, (long long)t, j);
        uint16_t* row = p.idx ? p.out + tj * p.ot + (rj - tj * p.k) * dim : p.out + rj * p.ot;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int m = 8 * (lane + 32 * i);
            uint32_t o[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
            if constexpr (FMT == LF_FP8) decode8_fp8(make_uint2(v[j][i].x, v[j][i].y), sc[j][i], o);
            if constexpr (FMT == LF_FP4) decode8_fp4(v[j][i].x, e4m3_pair(sc[j][i]), o);
            if (m < (FMT == LF_FP8 ? dim - LT_TAIL : dim))
                __stcs(reinterpret_cast<uint4*>(row + m), make_uint4(o[0], o[1], o[2], o[3]));
        }
        if (FMT == LF_FP8 && lane < 8) __stcs(reinterpret_cast<uint4*>(row + dim - LT_TAIL) + lane, v[j][2]);
    }
}

}  // namespace hsi
