// The paged K/V cache as the kernels see it, and its TMA loads.
//
// Pages of 2^page_shift entries; entry e of sequence b is entry e mod page of
// page table[b][e / page]. A page id outside [0, n_pages) is reported through
// the sticky error word: a load then reads zeros (the TMA's fill for a
// coordinate past the tensor), a store is skipped.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"

namespace hsi {

template <typename T>
constexpr bool is_bf16 = false;
template <>
constexpr bool is_bf16<__nv_bfloat16> = true;

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

struct PagedView {
    void *k, *v;
    int64_t page_stride, token_stride, head_stride;  // elements
    int64_t n_pages;
    const int32_t* table;
    int64_t ld_table;  // distance of the table's rows
    const int32_t* kv_len;
    int B, H, D, page_shift;
    int capacity;      // entries that a row of the table lists
};

constexpr int64_t PAGED_NO_ENTRY = -1, PAGED_NO_TOKEN = -2;

// Entries of sequence b, clamped to what its table row can hold and to the host's bound.
__device__ __forceinline__ int32_t paged_len(const PagedView& kv, int b, int32_t bound = INT32_MAX) {
    const int32_t n = __ldg(kv.kv_len + b);
    const int32_t most = min(kv.capacity, bound);
    if (n < 0 || n > most) {
        raise_error(DEVERR_ARG);
        return n < 0 ? 0 : most;
    }
    return n;
}

// New tokens of sequence b: [*first, *first + returned); a descending q_start counts as none.
__device__ __forceinline__ int32_t paged_new(const int32_t* q_start, int b, int32_t most, int64_t total, int32_t* first) {
    const int32_t a = __ldg(q_start + b), e = __ldg(q_start + b + 1);
    *first = a;
    if (a < 0 || e < a || e > total || e - a > most) {
        raise_error(DEVERR_ARG);
        return 0;
    }
    return e - a;
}

// Element offset (head 0) of the place of new token t of `total`: entry kv_len -
// (new tokens of its sequence) + its index among them. PAGED_NO_TOKEN where t
// lies outside every sequence, PAGED_NO_ENTRY (reported) where it has no valid
// place. Whole warp; the sequence is the number of those that end at or before
// t, so that its lookup is one round of loads (for up to 32 sequences) and no
// chain. Those are the first ones, or q_start descends around t: reported then,
// as where the sequence leaves the tokens, and t belongs to none.
__device__ __forceinline__ int64_t paged_new_row_warp(const PagedView& kv, const int32_t* q_start, int64_t t,
                                                      int64_t total) {
    const int lane = threadIdx.x & 31;
    int b = 0, last = 0;
#pragma unroll 4
    for (int i = lane; i < kv.B; i += 32) {
        if (__ldg(q_start + i + 1) > t) continue;
        ++b;
        last = i + 1;
    }
    b = __reduce_add_sync(~0u, b);
    if (__reduce_max_sync(~0u, last) != b) {
        raise_error(DEVERR_ARG);
        return PAGED_NO_TOKEN;
    }
    if (b >= kv.B || t < __ldg(q_start + b)) return PAGED_NO_TOKEN;
    const int32_t a = __ldg(q_start + b), e1 = __ldg(q_start + b + 1);
    if (a < 0 || e1 > total) {
        raise_error(DEVERR_ARG);
        return PAGED_NO_TOKEN;
    }
    // (by the length as it is: by one clamped to the row, the tokens would land on the entries before them)
    const int32_t n = __ldg(kv.kv_len + b);
    const int64_t e = (int64_t)n - (e1 - t);
    if (n > kv.capacity) raise_error(DEVERR_ARG);
    if (e < 0 || e >= kv.capacity) {
        raise_error(DEVERR_ARG);
        return PAGED_NO_ENTRY;
    }
    const int32_t page = __ldg(kv.table + b * kv.ld_table + (e >> kv.page_shift));
    if (page < 0 || page >= kv.n_pages) {
        raise_error(DEVERR_ARG);
        return PAGED_NO_ENTRY;
    }
    return page * kv.page_stride + (e & ((1 << kv.page_shift) - 1)) * kv.token_stride;
}

// Page id of page `i` of sequence b; n_pages (past the tensor: zeros) where the table is wrong.
__device__ __forceinline__ int32_t paged_page(const PagedView& kv, int b, int64_t i) {
    const int32_t page = __ldg(kv.table + b * kv.ld_table + i);
    if (page < 0 || page >= kv.n_pages) {
        raise_error(DEVERR_ARG);
        return (int32_t)kv.n_pages;
    }
    return page;
}

// One box of a {dim, entry, head, page} tensor map into 128-byte-swizzled rows
// of 64 values. The dim coordinate is a multiple of 64: 16-byte aligned.
__device__ __forceinline__ void tma_page_box(void* dst, const CUtensorMap* map, int dim, int entry, int head, int page,
                                             uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(dim), "r"(entry), "r"(head), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

// One box of a {dim, head, token} tensor map of the query rows.
__device__ __forceinline__ void tma_rows_box(void* dst, const CUtensorMap* map, int dim, int head, int token,
                                             uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(dim), "r"(head), "r"(token), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace hsi
