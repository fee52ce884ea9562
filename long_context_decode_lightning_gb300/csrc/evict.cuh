// Eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, KV head): of L entries keep the first `sink`, the last
// `recent` and the largest weights among the others, ties to the lowest index,
// `budget` in all; the kept indices come out ascending and the kept entries
// move, in that order, to places 0 .. budget - 1.
//
// evict_select_kernel: one cluster per row. Each CTA reads its slice of the
// weights once and keeps them in shared memory (past EV_CAP of them it reads the
// rest again each pass, and then acc_out must not be acc). Passes of 2048 bins
// over the keys' own range (a fixed first digit would drop all weights of like
// size into a few bins, whose atomics serialise) narrow down the key of the
// last kept entry; the histograms of the slices are added up through
// distributed shared memory. Two passes mostly do, three always. A
// last walk over the slice counts, then writes, in index order. Bound: one
// 4-byte read per entry, and the latency of the passes.
//
// paged_compact_kernel: copies of whole entries, eight 16-byte vectors of each
// thread in flight. In place (the same table), the places are walked from the
// front in turns: the sources of places i >= c lie at c or behind, so nothing
// that is still to be read has been written when a turn's reads precede its
// writes; the blocks of a turn are a cluster with a barrier between the two.
// To other pages every block goes its own way.
// Bound: HBM, one read and one write of the kept entries.
//
// Measured: 8 sequences of 16384 entries, 8 KV heads of 128, back to 8192: selection
// 17 to 19 us (load 8000 cycles, passes 4000 each, counting and writing 4000 each), copy
// to other pages 85 us (93% of the copy rate), in place 109 us. Selection in clusters, 8
// heads of one sequence: 131072 entries 39 us, 500000 (past the shared memory) 87.
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
    uint32_t scan[EV_THREADS / 32], scan2[EV_THREADS / 32];
    uint32_t low, high;            // of this slice: the range of the unprotected keys; later its two counts
    uint32_t digit, above, count;  // the pass's bin, the entries above it and in it
    alignas(16) float w[EV_CAP];   // the slice's weights
};

// The sum of v over the threads before this one. Whole block; scan: a word a warp.
__device__ __forceinline__ uint32_t block_before(uint32_t* scan, uint32_t v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    return incl - v + __reduce_add_sync(~0u, lane < warp ? scan[lane] : 0u);
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

    // this CTA's slice: entries [lo, lo + n)
    const int64_t per = (len + csize - 1) / csize;
    const int64_t lo = min(len, rank * per);
    const int n = (int)(min(len, lo + per) - lo), held = n < EV_CAP ? n : EV_CAP;
    acc += lo;
    // protected: i < p_lo or i >= p_hi; they rank above every weight (whose keys are held below ~0u, so that
    // even a NaN's, which has no place of its own, is counted like any other)
    const int p_lo = (int)max((int64_t)0, min((int64_t)n, p.sink - lo));
    const int p_hi = (int)max((int64_t)0, min((int64_t)n, len - p.recent - lo));
    auto weight_at = [&](int i) { return i < held ? s.w[i] : acc[i]; };
    auto rank_of = [&](float w) { return min(order_key(w), ~0u - 1u); };
    auto key_of = [&](int i, float w) { return i < p_lo || i >= p_hi ? ~0u : rank_of(w); };

    // the weights into shared memory, and the range of the unprotected keys
    uint32_t low = ~0u, high = 0u;
    auto seen = [&](int i, float w) {
        const uint32_t k = key_of(i, w);
        low = min(low, k);
        if (k != ~0u) high = max(high, k);
    };
    const int head = min(held, (int)((16 - (reinterpret_cast<uintptr_t>(acc) & 15)) % 16 / 4));
    if (tid < head) {
        s.w[tid] = acc[tid];
        seen(tid, s.w[tid]);
    }
    const int vecs = (held - head) / 4, tail = head + 4 * vecs;
#pragma unroll 4
    for (int v = tid; v < vecs; v += EV_THREADS) {
        const int i = head + 4 * v;
        const float4 f = *reinterpret_cast<const float4*>(acc + i);
        s.w[i] = f.x;
        s.w[i + 1] = f.y;
        s.w[i + 2] = f.z;
        s.w[i + 3] = f.w;
        seen(i, f.x);
        seen(i + 1, f.y);
        seen(i + 2, f.z);
        seen(i + 3, f.w);
    }
    if (tid < held - tail) {
        s.w[tail + tid] = acc[tail + tid];
        seen(tail + tid, s.w[tail + tid]);
    }
    for (int i = held + tid; i < n; i += EV_THREADS) seen(i, acc[i]);
    __syncthreads();

    // thr: entries of larger keys are kept, and the first `need` of its own
    uint32_t thr = 0, need = 0;
    const bool all = n_keep >= len;
    if (!all) {
        uint32_t want = (uint32_t)(n_keep - p.sink - p.recent);  // unprotected ones (len > budget: all protected fit)
        low = __reduce_min_sync(~0u, low);
        high = __reduce_max_sync(~0u, high);
        if (lane == 0) {
            s.scan[warp] = low;
            s.scan2[warp] = high;
        }
        __syncthreads();
        low = __reduce_min_sync(~0u, s.scan[lane]);
        high = __reduce_max_sync(~0u, s.scan2[lane]);
        if (csize > 1) {
            if (tid == 0) {
                s.low = low;
                s.high = high;
            }
            cluster_sync();
            if (lane < csize) {
                low = dsmem_load(&s.low, lane);
                high = dsmem_load(&s.high, lane);
            }
            low = __reduce_min_sync(~0u, low);
            high = __reduce_max_sync(~0u, high);
        }
        // passes over the range [base, base + width]: 2048 bins of 2^shift keys
        uint32_t base = low, width = high - low;
        thr = ~0u - 1u;  // where no unprotected entry is wanted: above every rank
        while (want > 0) {
            const int top = 32 - __clz(width), shift = top > 11 ? top - 11 : 0;
            for (int i = tid; i < EV_BINS; i += EV_THREADS) s.hist[i] = 0;
            __syncthreads();
            auto count = [&](float w) {  // of the unprotected [p_lo, p_hi)
                const uint32_t k = rank_of(w) - base;
                if (k <= width) atomicAdd(&s.hist[k >> shift], 1u);
            };
            // whole vectors between v_lo and v_hi, single entries before and behind
            const int last = min(p_hi, held), v_lo = min(last, (p_lo + 3) & ~3), v_hi = max(v_lo, last & ~3);
            if (tid < v_lo - p_lo) count(s.w[p_lo + tid]);
            if (tid < last - v_hi) count(s.w[v_hi + tid]);
#pragma unroll 2
            for (int i = v_lo + 4 * tid; i < v_hi; i += 4 * EV_THREADS) {
                const float4 v = *reinterpret_cast<const float4*>(&s.w[i]);
                count(v.x);
                count(v.y);
                count(v.z);
                count(v.w);
            }
            for (int i = max(held, p_lo) + tid; i < p_hi; i += EV_THREADS) count(acc[i]);
            if (csize > 1) cluster_sync();
            else __syncthreads();
            // whole-row counts; thread t takes bins 2047 - 2t and the one below (from the top)
            uint32_t c[2] = {0, 0};
            if (csize == 1) {
                c[0] = s.hist[EV_BINS - 1 - 2 * tid];
                c[1] = s.hist[EV_BINS - 2 - 2 * tid];
            } else {
                for (int r = 0; r < csize; ++r) {
                    c[0] += dsmem_load(&s.hist[EV_BINS - 1 - 2 * tid], r);
                    c[1] += dsmem_load(&s.hist[EV_BINS - 2 - 2 * tid], r);
                }
            }
            uint32_t above = block_before(s.scan, c[0] + c[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (above < want && above + c[j] >= want) {
                    s.digit = EV_BINS - 1 - (2 * tid + j);
                    s.above = above;
                    s.count = c[j];
                }
                above += c[j];
            }
            if (csize > 1) cluster_sync();  // also: every slice's histogram has been read
            else __syncthreads();
            base += s.digit << shift;
            width = (1u << shift) - 1u;
            want -= s.above;
            if (shift == 0) {  // one key
                thr = base;
                need = want;
                break;
            }
            if (s.count == want && base > 0) {  // the whole bin
                thr = base - 1u;
                break;
            }
        }
    }

    // turns of 32 entries, a run of them a warp: counted, then written side by side behind the
    // runs before (a run of entries a thread would store them apart: 16000 cycles against 4000)
    const int turns = (n + 31) / 32, run = (turns + EV_THREADS / 32 - 1) / (EV_THREADS / 32) * 32;
    const int i0 = min(n, warp * run), i1 = min(n, i0 + run);
    uint32_t gt = 0, eq = 0;
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
        const bool live = i + lane < i1;
        const uint32_t k = live ? key_of(i + lane, weight_at(i + lane)) : 0u;
        gt += __popc(__ballot_sync(~0u, live && (all || k > thr)));
        eq += __popc(__ballot_sync(~0u, live && !all && k == thr));
    }
    if (lane == 0) {
        s.scan[warp] = gt;
        s.scan2[warp] = eq;
    }
    __syncthreads();
    uint32_t g0 = __reduce_add_sync(~0u, lane < warp ? s.scan[lane] : 0u);
    uint32_t e0 = __reduce_add_sync(~0u, lane < warp ? s.scan2[lane] : 0u);
    if (csize > 1) {
        if (tid == EV_THREADS - 1) {
            s.low = g0 + gt;
            s.high = e0 + eq;
        }
        cluster_sync();
        uint32_t gr = lane < rank ? dsmem_load(&s.low, lane) : 0u, er = lane < rank ? dsmem_load(&s.high, lane) : 0u;
        g0 += __reduce_add_sync(~0u, gr);
        e0 += __reduce_add_sync(~0u, er);
        cluster_sync();  // nobody leaves while its counts are read; every weight has been read
    }
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 2
    for (int i = i0; i < i1; i += 32) {
        const bool live = i + lane < i1;
        const float w = live ? weight_at(i + lane) : 0.f;
        const uint32_t k = key_of(i + lane, w);
        const uint32_t bg = __ballot_sync(~0u, live && (all || k > thr));
        const uint32_t be = __ballot_sync(~0u, live && !all && k == thr);
        const uint32_t er = e0 + __popc(be & below);
        if ((bg >> lane & 1) || ((be >> lane & 1) && er < need)) {
            const uint32_t at = g0 + __popc(bg & below) + min(er, need);
            if (at < (uint32_t)n_keep) {  // (always, unless somebody writes the weights meanwhile)
                keep[at] = (int32_t)(lo + i + lane);
                if (out) out[at] = w;
            }
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
    int in_place;
};

constexpr int CP_THREADS = 256;

// Blocks of a (sequence, KV head, K or V): `csize` (in place, as a cluster) or
// gridDim.x / (2 B H) (to other pages) share its places, ROUNDS times the
// entries that 16-byte loads of CP_THREADS threads cover at a time: eight
// rounds in flight a thread, or two where that leaves SMs without blocks (512
// places of two sequences to other pages: 2.5 us against 4.2).
// AHEAD: the next turn's indices and pages are looked up before the barrier,
// which leaves one round trip between two barriers; for few blocks in place,
// where the SMs have the registers (one sequence of 131072 entries 199 us to 154; with
// every SM full it lost, 131 us against 109).
template <int ROUNDS, bool AHEAD>
__global__ void __launch_bounds__(CP_THREADS, AHEAD ? 2 : 4)
    paged_compact_kernel(CompactParams p, int split, int csize) {
    griddep_wait();
    griddep_launch_dependents();
    const int lanes = p.kv.D / 8, rows = CP_THREADS / lanes;  // threads of an entry, entries of a round
    const int part = blockIdx.x % split, id = blockIdx.x / split;
    const int kind = id & 1, h = (id >> 1) % p.kv.H, b = (id >> 1) / p.kv.H;
    const int row = threadIdx.x / lanes;
    uint8_t* const base = static_cast<uint8_t*>(kind ? p.kv.v : p.kv.k) +
                          ((int64_t)h * p.kv.head_stride * 2 + (threadIdx.x % lanes) * 16);
    const int32_t* keep = p.keep + ((int64_t)b * p.kv.H + h) * p.ld_keep;
    int n = __ldg(p.new_len + b);
    const int32_t len = paged_len(p.kv, b);
    if (n < 0 || n > p.budget) {
        if (threadIdx.x == 0) raise_error(DEVERR_ARG);
        n = n < 0 ? 0 : p.budget;
    }
    const int mask = (1 << p.kv.page_shift) - 1;
    const int step = rows * ROUNDS * split;
    if constexpr (AHEAD) {
        int src[ROUNDS], page[ROUNDS], to_page[ROUNDS];  // page < 0: nothing to copy
        auto look_up = [&](int i0) {
#pragma unroll
            for (int u = 0; u < ROUNDS; ++u) {
                const int i = i0 + (part * ROUNDS + u) * rows + row;
                src[u] = i < n ? __ldg(keep + i) : -2;
            }
#pragma unroll
            for (int u = 0; u < ROUNDS; ++u) {
                const int i = i0 + (part * ROUNDS + u) * rows + row;
                page[u] = -1;
                if (src[u] == -2) continue;
                if (src[u] < 0 || src[u] >= len) {
                    raise_error(DEVERR_ARG);
                    continue;
                }
                const int32_t a = __ldg(p.kv.table + b * p.kv.ld_table + (src[u] >> p.kv.page_shift));
                to_page[u] = __ldg(p.dst + b * p.ld_dst + (i >> p.kv.page_shift));
                if (a < 0 || a >= p.kv.n_pages || to_page[u] < 0 || to_page[u] >= p.kv.n_pages) {
                    raise_error(DEVERR_ARG);
                    continue;
                }
                page[u] = a;
            }
        };
        look_up(0);
        for (int i0 = 0; i0 < n; i0 += step) {  // the same turns in every block of a cluster
            uint4 v[ROUNDS];
            uint8_t* to[ROUNDS];
#pragma unroll
            for (int u = 0; u < ROUNDS; ++u) {
                const int i = i0 + (part * ROUNDS + u) * rows + row;
                to[u] = nullptr;
                if (page[u] < 0) continue;
                const int64_t from = page[u] * p.kv.page_stride + (src[u] & mask) * p.kv.token_stride;
                v[u] = *reinterpret_cast<const uint4*>(base + 2 * from);
                to[u] = base + 2 * (to_page[u] * p.kv.page_stride + (i & mask) * p.kv.token_stride);
            }
            if (i0 + step < n) look_up(i0 + step);
            if (csize > 1) cluster_sync();  // a turn's reads precede its writes
            else __syncthreads();
#pragma unroll
            for (int u = 0; u < ROUNDS; ++u)
                if (to[u]) *reinterpret_cast<uint4*>(to[u]) = v[u];
        }
    } else {
        for (int i0 = 0; i0 < n; i0 += step) {  // the same turns in every block of a cluster
            uint4 v[ROUNDS];
            int to_page[ROUNDS];  // below 0: nothing to copy (a page takes one register where an address takes two)
            int src[ROUNDS];
#pragma unroll
            for (int u = 0; u < ROUNDS; ++u) {
                const int i = i0 + (part * ROUNDS + u) * rows + row;
                src[u] = i < n ? __ldg(keep + i) : -2;
            }
#pragma unroll
            for (int u = 0; u < ROUNDS; ++u) {
                const int i = i0 + (part * ROUNDS + u) * rows + row;
                to_page[u] = -1;
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
                const int64_t from = a * p.kv.page_stride + (src[u] & mask) * p.kv.token_stride;
                v[u] = *reinterpret_cast<const uint4*>(base + 2 * from);
                to_page[u] = d;
            }
            if (p.in_place) {  // a turn's reads precede its writes
                if (csize > 1) cluster_sync();
                else __syncthreads();
            }
#pragma unroll
            for (int u = 0; u < ROUNDS; ++u) {
                const int i = i0 + (part * ROUNDS + u) * rows + row;
                if (to_page[u] >= 0)
                    *reinterpret_cast<uint4*>(base + 2 * (to_page[u] * p.kv.page_stride + (i & mask) * p.kv.token_stride)) = v[u];
            }
        }
    }
}

}  // namespace hsi
