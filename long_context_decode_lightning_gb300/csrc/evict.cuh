// Eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, KV head): of L entries keep the first `sink`, the last
// `recent` and the largest weights among the others, ties to the lowest index,
// `budget` in all; the kept indices come out ascending and the kept entries
// move, in that order, to places 0 .. budget - 1.
//
// evict_select_kernel: one cluster per row. Each CTA reads its slice of the
// weights once and keeps them in shared memory (past EV_CAP of them it reads the
// rest again each pass, and then acc_out must not be acc); three radix passes
// (11, 11, 10 bits from the top) find the key of the last kept entry, the
// histograms of the slices added up through distributed shared memory. A
// second walk over the slice counts, then writes, in index order. Bound: one
// 4-byte read per entry, and the latency of the passes.
//
// paged_compact_kernel: copies of 64-byte column slices, 64 entries at a time
// and eight such rounds in flight. In place (the same table), a CTA walks its
// slice from the front: the sources of places i >= c lie at c or behind, so
// nothing that is still to be read has been written when a round's reads
// precede its writes. To other pages the places are split over more CTAs.
// Bound: HBM, one read and one write of the kept entries.
#pragma once
#include <cstdint>

#include "common.cuh"
#include "paged.cuh"

namespace hsi {

constexpr int EV_THREADS = 1024;
constexpr int EV_CAP = 49152;     // keys a CTA holds in shared memory
constexpr int EV_MAX_CLUSTER = 8;
constexpr int EV_BINS = 2048;

struct EvictParams {
    const float* acc;   // [B][H][ld_acc]
    int64_t ld_acc;
    const int32_t* kv_len;
    int B, H;
    int64_t max_len;
    int budget, sink, recent;
    int32_t* keep;      // [B][H][ld_keep]
    int64_t ld_keep;
    float* acc_out;     // [B][H][ld_out] or null
    int64_t ld_out, n_out;
    int32_t* new_len;   // [B]
};

struct EvictSmem {
    uint32_t hist[EV_BINS];
    uint32_t warp_gt[EV_THREADS / 32], warp_eq[EV_THREADS / 32];
    uint32_t gt, eq;         // of this slice
    uint32_t digit, above;   // the pass's bin and the entries above it
    uint32_t scan[EV_THREADS / 32];
    float w[EV_CAP];         // the slice's weights
};

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 32-bit word of another CTA of the cluster, at the address it has in this one.
__device__ __forceinline__ uint32_t dsmem_load(const uint32_t* mine, uint32_t rank) {
    uint32_t addr, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__global__ void __launch_bounds__(EV_THREADS, 1) evict_select_kernel(EvictParams p, int csize) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    EvictSmem& s = *reinterpret_cast<EvictSmem*>(smem_raw);
    griddep_wait();
    griddep_launch_dependents();
    const int rank = csize > 1 ? (int)cluster_ctarank() : 0;
    const int row = blockIdx.x / csize, b = row / p.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t len = __ldg(p.kv_len + b);
    if (len < 0 || len > p.max_len) {
        if (tid == 0) raise_error(DEVERR_ARG);
        len = len < 0 ? 0 : p.max_len;
    }
    const float* acc = p.acc + row * p.ld_acc;
    int32_t* keep = p.keep + row * p.ld_keep;
    float* out = p.acc_out ? p.acc_out + row * p.ld_out : nullptr;
    const int n_keep = (int)(len < p.budget ? len : p.budget);
    if (rank == 0 && row % p.H == 0 && tid == 0) p.new_len[b] = n_keep;

    // this CTA's slice [lo, hi), in whole warps' turns of 32
    const int64_t per = ((len + csize - 1) / csize + 31) / 32 * 32;
    const int64_t lo = min(len, rank * per), hi = min(len, lo + per);
    const int n = (int)(hi - lo), held = n < EV_CAP ? n : EV_CAP;
    const int head = (int)min((int64_t)held, (int64_t)((16 - ((reinterpret_cast<uintptr_t>(acc + lo) & 15))) % 16 / 4));
    for (int i = tid; i < head; i += EV_THREADS) s.w[i] = acc[lo + i];
    for (int i = head + 4 * tid; i < held; i += 4 * EV_THREADS) {
        if (i + 4 <= held) {
            const float4 v = *reinterpret_cast<const float4*>(acc + lo + i);
            s.w[i] = v.x;
            s.w[i + 1] = v.y;
            s.w[i + 2] = v.z;
            s.w[i + 3] = v.w;
        } else {
            for (int j = i; j < held; ++j) s.w[j] = acc[lo + j];
        }
    }
    __syncthreads();
    auto weight_at = [&](int i) { return i < held ? s.w[i] : acc[lo + i]; };
    // protected entries rank above every weight: order_key of a number is below ~0u
    auto key_at = [&](int i) {
        const int64_t g = lo + i;
        return g < p.sink || g >= len - p.recent ? ~0u : order_key(weight_at(i));
    };

    // the key of the last kept entry and how many entries with that key are kept
    uint32_t thr = 0, need = 0;
    const bool all = n_keep >= len;
    if (!all) {
        uint32_t want = (uint32_t)n_keep;
        const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
        for (int pass = 0; pass < 3; ++pass) {
            const int nb = 1 << bits[pass];
            for (int i = tid; i < EV_BINS; i += EV_THREADS) s.hist[i] = 0;
            __syncthreads();
            const uint32_t mask = pass == 0 ? 0u : ~0u << (shifts[pass] + bits[pass]);
            for (int i = tid; i < n; i += EV_THREADS) {
                const uint32_t k = key_at(i);
                if ((k & mask) == (thr & mask)) atomicAdd(&s.hist[(k >> shifts[pass]) & (nb - 1)], 1u);
            }
            if (csize > 1) cluster_sync();
            else __syncthreads();
            // whole-row counts; thread t takes bins nb - 1 - 2t and the one below (from the top)
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int bin = nb - 1 - (2 * tid + j);
                if (bin < 0) continue;
                if (csize == 1) c[j] = s.hist[bin];
                else
                    for (int r = 0; r < csize; ++r) c[j] += dsmem_load(&s.hist[bin], r);
            }
            uint32_t incl = c[0] + c[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t up = __shfl_up_sync(~0u, incl, o);
                if (lane >= o) incl += up;
            }
            if (lane == 31) s.scan[warp] = incl;
            __syncthreads();
            if (warp == 0) {
                uint32_t v = s.scan[lane];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t up = __shfl_up_sync(~0u, v, o);
                    if (lane >= o) v += up;
                }
                s.scan[lane] = v;
            }
            __syncthreads();
            uint32_t above = incl - c[0] - c[1] + (warp ? s.scan[warp - 1] : 0u);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (above < want && above + c[j] >= want) {
                    s.digit = nb - 1 - (2 * tid + j);
                    s.above = above;
                }
                above += c[j];
            }
            if (csize > 1) cluster_sync();  // also: every slice's histogram has been read
            else __syncthreads();
            thr |= s.digit << shifts[pass];
            want -= s.above;
        }
        need = want;
    }

    // counts of this slice, by warp: each warp owns a run of whole turns of 32
    const int turns = (n + 31) / 32, wt = (turns + EV_THREADS / 32 - 1) / (EV_THREADS / 32);
    const int i0 = warp * wt * 32, i1 = min(n, i0 + wt * 32);
    uint32_t gt = 0, eq = 0;
    for (int i = i0; i < i1; i += 32) {
        const bool live = i + lane < n;
        const uint32_t k = live ? key_at(i + lane) : 0u;
        gt += __popc(__ballot_sync(~0u, live && (all || k > thr)));
        eq += __popc(__ballot_sync(~0u, live && !all && k == thr));
    }
    if (lane == 0) {
        s.warp_gt[warp] = gt;
        s.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t g = 0, e = 0;
        for (int i = 0; i < EV_THREADS / 32; ++i) {
            const uint32_t tg = s.warp_gt[i], te = s.warp_eq[i];
            s.warp_gt[i] = g;
            s.warp_eq[i] = e;
            g += tg;
            e += te;
        }
        s.gt = g;
        s.eq = e;
    }
    uint32_t g0 = 0, e0 = 0;
    if (csize > 1) {
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            g0 += dsmem_load(&s.gt, r);
            e0 += dsmem_load(&s.eq, r);
        }
        cluster_sync();  // nobody leaves while its counts are read; every weight has been read
    } else {
        __syncthreads();
    }
    g0 += s.warp_gt[warp];
    e0 += s.warp_eq[warp];
    for (int i = i0; i < i1; i += 32) {
        const bool live = i + lane < n;
        const uint32_t k = live ? key_at(i + lane) : 0u;
        const uint32_t bg = __ballot_sync(~0u, live && (all || k > thr));
        const uint32_t be = __ballot_sync(~0u, live && !all && k == thr);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t er = e0 + __popc(be & below), gr = g0 + __popc(bg & below);
        const bool is_g = bg >> lane & 1, is_e = (be >> lane & 1) && er < need;
        if (is_g || is_e) {
            const uint32_t at = gr + (er < need ? er : need);
            keep[at] = (int32_t)(lo + i + lane);
            if (out) out[at] = weight_at(i + lane);
        }
        g0 += __popc(bg);
        e0 += __popc(be);
    }
    // padding: -1 indices, zero weights
    const int64_t pad0 = n_keep + (int64_t)rank * EV_THREADS + tid, pads = (int64_t)csize * EV_THREADS;
    for (int64_t i = pad0; i < p.budget; i += pads) keep[i] = -1;
    if (out)
        for (int64_t i = pad0; i < p.n_out; i += pads) out[i] = 0.f;
}

struct CompactParams {
    PagedView kv;
    const int32_t* keep;     // [B][H][ld_keep]
    int64_t ld_keep;
    const int32_t* new_len;  // [B]
    int budget;
    const int32_t* dst;      // [B][ld_dst] pages of the places
    int64_t ld_dst;
};

constexpr int CP_THREADS = 256;
constexpr int CP_ROWS = CP_THREADS / 4;  // entries of a round: four threads copy 64 bytes of each
constexpr int CP_ROUNDS = 8;             // rounds in flight

__global__ void __launch_bounds__(CP_THREADS) paged_compact_kernel(CompactParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int slices = p.kv.D * 2 / 64;
    int id = blockIdx.x;
    const int slice = id % slices;
    id /= slices;
    const int kind = id & 1;
    id >>= 1;
    const int h = id % p.kv.H, b = id / p.kv.H;
    uint8_t* const base = static_cast<uint8_t*>(kind ? p.kv.v : p.kv.k) +
                          ((int64_t)h * p.kv.head_stride * 2 + slice * 64 + (threadIdx.x & 3) * 16);
    const int32_t* keep = p.keep + ((int64_t)b * p.kv.H + h) * p.ld_keep;
    int n = __ldg(p.new_len + b);
    const int32_t len = paged_len(p.kv, b);
    if (n < 0 || n > p.budget) {
        if (threadIdx.x == 0) raise_error(DEVERR_ARG);
        n = n < 0 ? 0 : p.budget;
    }
    const int mask = (1 << p.kv.page_shift) - 1;
    const int step = CP_ROWS * CP_ROUNDS;
    for (int i0 = blockIdx.y * step; i0 < n; i0 += gridDim.y * step) {
        uint4 v[CP_ROUNDS];
        uint8_t* to[CP_ROUNDS];
        int src[CP_ROUNDS];
#pragma unroll
        for (int u = 0; u < CP_ROUNDS; ++u) {
            const int i = i0 + u * CP_ROWS + (threadIdx.x >> 2);
            src[u] = i < n ? __ldg(keep + i) : -2;
        }
#pragma unroll
        for (int u = 0; u < CP_ROUNDS; ++u) {
            const int i = i0 + u * CP_ROWS + (threadIdx.x >> 2);
            to[u] = nullptr;
            if (src[u] == -2) continue;
            if (src[u] < 0 || src[u] >= len) {
                raise_error(DEVERR_ARG);
                continue;
            }
            const int32_t a = __ldg(p.kv.table + b * p.kv.ld_table + (src[u] >> p.kv.page_shift));
            const int32_t d = __ldg(p.dst + b * p.ld_dst + (i >> p.kv.page_shift));
            if (a < 0 || a >= p.kv.n_pages || d < 0 || d >= p.kv.n_pages) {
                raise_error(DEVERR_ARG);
                continue;
            }
            v[u] = *reinterpret_cast<const uint4*>(base + 2 * (a * p.kv.page_stride + (src[u] & mask) * p.kv.token_stride));
            to[u] = base + 2 * (d * p.kv.page_stride + (i & mask) * p.kv.token_stride);
        }
        __syncthreads();  // the rounds' reads precede their writes
#pragma unroll
        for (int u = 0; u < CP_ROUNDS; ++u)
            if (to[u]) *reinterpret_cast<uint4*>(to[u]) = v[u];
    }
}

}  // namespace hsi
