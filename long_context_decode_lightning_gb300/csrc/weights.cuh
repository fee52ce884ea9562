// The attention weights of a chunk of many rows: exp(scale q.k - lse) summed
// over the rows, per entry, on the tensor cores.
//
// S^T = K Q^T with the entries as the rows of the accumulator: a thread of the
// epilogue owns one entry (one lane of tensor memory), walks the columns (the
// query rows) and adds up in its own registers; nothing is exchanged, and the
// order of the sum is fixed. Rows of a tile: whole tokens with their group of
// query heads (row = token * group + head), one TMA box each 64 dims, so that
// every group size fills a tile of 128 up to its last whole token.
//
// Per 128 x 128 tile of S: 128 x 128 x D multiply-adds (512 cycles at D = 128)
// and 16384 exponentials (512 cycles of the SM's special-function units): both
// bound it together. A CTA keeps 256 entries of K in shared memory and streams
// the query tiles past them (one 32 KB tile per 1024 tensor cycles; 128 entries
// would ask twice the L2 rate), two accumulators per 128 entries, and
// four warpgroups, each for every other tile of its 128 entries.
// Few entries: a cluster shares a unit's query tiles and adds up the partial
// sums through distributed shared memory, in rank order.
//
// Measured: 2 x up to 1024 tokens over up to 16384 entries, 32 query and 8 KV heads
// of 128 in bf16, 170 us (1230 TFLOP/s, 64% of the measured bf16 rate); without the
// exponentials 161, without the columns' work 156, with a quarter of the products 158:
// products (A and B from shared memory, 81 to 107 cycles each for 64) and epilogue
// bound it together.
#pragma once
#include <cstdint>
#include <type_traits>

#include "attend.cuh"
#include "common.cuh"
#include "evict.cuh"
#include "paged.cuh"

namespace hsi {

constexpr int WC_KEYS = 256;                 // entries of a unit: two accumulator tiles of 128
constexpr int WC_ROWS = 128;                 // query rows of a tile
constexpr int WC_THREADS = 32 * 19;          // 16 epilogue warps, MMA, query producer, key producer

template <int D>
struct WeightsCfg {
    static constexpr int HALF_BYTES = 128 * 128;            // 64 dims of 128 rows
    static constexpr int Q_BYTES = HALF_BYTES * (D / 64);
    static constexpr int K_BYTES = 2 * Q_BYTES;             // of a unit
    static constexpr int K_STAGES = 2;
    static constexpr int Q_STAGES = D == 128 ? 3 : 6;
    static constexpr int NL_STAGES = 3;
    static constexpr int RING_BYTES = K_STAGES * K_BYTES + Q_STAGES * Q_BYTES;
    struct Tail {
        float nl[NL_STAGES][WC_ROWS];  // -lse (base 2) of a tile's rows
        float part[2][128];            // per 128 entries: one warpgroup's sums, then the block's
        uint64_t k_full[K_STAGES], k_empty[K_STAGES], q_full[Q_STAGES], q_empty[Q_STAGES];
        uint64_t nl_full[NL_STAGES], nl_empty[NL_STAGES], s_full[2][2], s_empty[2][2], done;
        uint32_t tmem;
        int abort;
    };
    static constexpr int SMEM_BYTES = RING_BYTES + (int)sizeof(Tail);
    static_assert(SMEM_BYTES <= 232448, "shared memory of an SM");
};

// A walk over the units (sequence, KV head, 256 entries), u ascending.
struct WeightsWalk {
    int b, len, m, at, nt;
    int64_t first;
    __device__ __forceinline__ void load(const AttendParams& p) {
        len = paged_len(p.kv, b, p.max_kv);
        m = paged_new(p.q_start, b, p.max_q, p.T, &at);
        nt = (len + WC_KEYS - 1) / WC_KEYS;
    }
    // false when u lies past the last unit
    __device__ __forceinline__ bool seek(const AttendParams& p, int64_t u) {
        while (b < p.kv.B && u >= first + (int64_t)nt * p.kv.H) {
            first += (int64_t)nt * p.kv.H;
            if (++b < p.kv.B) load(p);
        }
        return b < p.kv.B;
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(WC_THREADS, 1)
    weights_chunk_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap qmap, int csize, int tpt) {
    using C = WeightsCfg<D>;
    extern __shared__ __align__(1024) uint8_t ring[];
    uint8_t* const k_ring = ring;
    uint8_t* const q_ring = ring + C::K_STAGES * C::K_BYTES;
    typename C::Tail& s = *reinterpret_cast<typename C::Tail*>(ring + C::RING_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rpt = tpt * p.group;  // rows of a tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::K_STAGES; ++i) mbar_init(&s.k_full[i], 1), mbar_init(&s.k_empty[i], 1);
        for (int i = 0; i < C::Q_STAGES; ++i) mbar_init(&s.q_full[i], 1), mbar_init(&s.q_empty[i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&s.s_full[i >> 1][i & 1], 1), mbar_init(&s.s_empty[i >> 1][i & 1], 4);
        for (int i = 0; i < C::NL_STAGES; ++i) mbar_init(&s.nl_full[i], 1), mbar_init(&s.nl_empty[i], 8);
        mbar_init(&s.done, 1);
        fence_mbar_init();
        s.abort = 0;
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&qmap);
    }
    if (warp == 16) tmem_alloc(&s.tmem, 512);
    // the rows past a tile's last whole token are never loaded: zeros, so that their products are
    for (int i = threadIdx.x; i < C::Q_STAGES * (D / 64) * (WC_ROWS - rpt) * 8; i += WC_THREADS) {
        const int ch = i & 7, r = (i >> 3) % (WC_ROWS - rpt), half = (i >> 3) / (WC_ROWS - rpt);
        *reinterpret_cast<uint4*>(q_ring + half * C::HALF_BYTES + (rpt + r) * 128 + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = s.tmem;

    const int rank = csize > 1 ? (int)cluster_ctarank() : 0;
    const int64_t step = gridDim.x / csize;
    WeightsWalk w;
    w.b = 0;
    w.first = 0;
    w.load(p);
    bool ok = true;
    int kf = 0, qf = 0;  // fills (or uses) of the key and query rings so far
    int row_tok[4], row_head[4];  // the query producer's rows of a tile: token (-1: none) and head
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = lane + 32 * i;
        row_tok[i] = row < rpt ? row / p.group : -1;
        row_head[i] = row % p.group;
    }
    int q_st = 0;        // the products' query stage and its phase
    uint32_t q_ph = 0;
    for (int64_t u = blockIdx.x / csize; w.seek(p, u); u += step) {
        const int local = (int)(u - w.first), head = local / w.nt, k0 = (local % w.nt) * WC_KEYS;
        // query tiles that see any of the unit's entries
        const int past = w.len - w.m, t_first = p.causal && k0 > past ? k0 - past : 0;
        const int j0 = t_first / tpt + rank, j1 = (w.m + tpt - 1) / tpt;

        if (warp == 18) {  // keys: a lane per box
            const int box = p.kv.page_shift < 7 ? 1 << p.kv.page_shift : 128;
            const int halves = D / 64, nbox = WC_KEYS / box * halves;
            const int n = min(w.len - k0, WC_KEYS), live = (n + box - 1) / box * halves;
            if (j0 < j1) {
                const int st = kf % C::K_STAGES;
                ok = ok && __all_sync(~0u, wait_bounded(&s.k_empty[st], (kf / C::K_STAGES & 1) ^ 1, &s.abort));
                if (ok) {
                    if (lane == 0) mbar_arrive_expect_tx(&s.k_full[st], live * box * 128);
                    __syncwarp();
                    for (int i = lane; i < nbox; i += 32) {
                        const int e = (i / halves) * box, half = i % halves;
                        if (e >= n) continue;
                        const int page = paged_page(p.kv, w.b, (k0 + e) >> p.kv.page_shift);
                        tma_page_box(k_ring + st * C::K_BYTES + (e >> 7) * C::Q_BYTES + half * C::HALF_BYTES +
                                         (e & 127) * 128,
                                     &kmap, half * 64, (k0 + e) & ((1 << p.kv.page_shift) - 1), head, page,
                                     &s.k_full[st]);
                    }
                    ++kf;
                }
            }
        } else if (warp == 17) {  // query tiles, and their rows' lse
            const float* lse = p.lse_in + (int64_t)w.at * p.Hq + head * p.group;
            for (int j = j0; j < j1; j += csize) {
                const int st = qf % C::Q_STAGES, nst = qf % C::NL_STAGES;
                float v[4];  // of rows lane, lane + 32, ..
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = j * tpt + row_tok[i];
                    v[i] = -INFINITY;
                    if (row_tok[i] >= 0 && t < w.m) v[i] = __ldg(lse + (int64_t)t * p.Hq + row_head[i]);
                }
                ok = __all_sync(~0u, ok && wait_bounded(&s.q_empty[st], (qf / C::Q_STAGES & 1) ^ 1, &s.abort));
                if (!ok) break;
                if (lane == 0 && !(qf == 0 && *(volatile int*)&g_hsi_skip_first_copy)) {
                    mbar_arrive_expect_tx(&s.q_full[st], rpt * 128 * (D / 64));
                    for (int half = 0; half < D / 64; ++half)
                        tma_rows_box(q_ring + st * C::Q_BYTES + half * C::HALF_BYTES, &qmap, half * 64, head * p.group,
                                     w.at + j * tpt, &s.q_full[st]);
                }
                ++qf;
                ok = __all_sync(~0u, wait_bounded(&s.nl_empty[nst], ((qf - 1) / C::NL_STAGES & 1) ^ 1, &s.abort));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s.nl[nst][lane + 32 * i] = v[i] == -INFINITY ? -INFINITY : -v[i] * LOG2E;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.nl_full[nst]);
            }
        } else if (warp == 16) {  // products: the warp waits, one lane issues
            if (j0 < j1) {
                constexpr uint32_t idesc = idesc_f16(is_bf16<T>, 128, WC_ROWS, false);
                const int kst = kf % C::K_STAGES;
                const uint32_t tm = uniform(tmem);
                const uint32_t kd = uniform(smem_desc_sw128(smem_u32(k_ring + kst * C::K_BYTES)));
                ok = ok && wait_bounded(&s.k_full[kst], kf / C::K_STAGES & 1, &s.abort);
                for (int j = j0; j < j1 && __all_sync(~0u, ok); j += csize) {
                    const int buf = qf & 1;
                    ok = wait_bounded(&s.q_full[q_st], q_ph, &s.abort);
                    const uint32_t qd = uniform(smem_desc_sw128(smem_u32(q_ring + q_st * C::Q_BYTES)));
                    const uint32_t d0 = uniform(tm + buf * 128);
                    ok = ok && wait_bounded(&s.s_empty[0][buf], (qf >> 1 & 1) ^ 1, &s.abort) &&
                         wait_bounded(&s.s_empty[1][buf], (qf >> 1 & 1) ^ 1, &s.abort);
                    if (!__all_sync(~0u, ok)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        // step by step for both accumulators in turn: a chain into one of them waits for
                        // itself (104 cycles a product in two groups, 81 in turn, 64 at the tensor rate)
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t off = ((ks >> 2) * C::HALF_BYTES + (ks & 3) * 32) >> 4;
#pragma unroll
                            for (int kt = 0; kt < 2; ++kt) {
                                const uint32_t a = kd + kt * (C::Q_BYTES >> 4) + off;
                                if (ks == 0) mma_f16_ss(d0 + kt * 256, a, qd, idesc);
                                else mma_f16_ss_add(d0 + kt * 256, a, qd + off, idesc);
                            }
                        }
                        tc_commit(&s.s_full[0][buf]);
                        tc_commit(&s.s_full[1][buf]);
                        tc_commit(&s.q_empty[q_st]);
                    }
                    __syncwarp();
                    ++qf;
                    if (++q_st == C::Q_STAGES) {
                        q_st = 0;
                        q_ph ^= 1;
                    }
                }
                if (elect_one()) tc_commit(&s.k_empty[kst]);
                __syncwarp();
                ++kf;
            }
        } else {  // weights: a thread per entry, a warpgroup for every other tile of it
            const int wg = warp >> 2, kt = wg >> 1, par = wg & 1, tid = threadIdx.x & 127;
            const int key = k0 + kt * 128 + tid;
            // first token that sees this entry
            const int t_min = p.causal ? key - past : 0;
            const uint64_t sl2 = f2_pack(p.sl2, p.sl2);
            const uint32_t ta = tmem + (uint32_t)((warp & 3) * 32 << 16) + (kt * 2 + par) * 128;
            float total = 0.f;
            for (int j = j0; j < j1 && ok; j += csize, ++qf) {
                if ((qf & 1) != par) continue;
                const int nst = qf % C::NL_STAGES;
                ok = wait_bounded(&s.nl_full[nst], qf / C::NL_STAGES & 1, &s.abort);
                ok = __all_sync(~0u, ok && wait_bounded(&s.s_full[kt][par], qf >> 1 & 1, &s.abort));
                if (!ok) break;
                tc_fence_after();
                // columns [c_lo, rows) count; tiles where all do need no comparison
                // (in tokens of the tile first: entries times heads may pass 31 bits)
                const int t0 = j * tpt;
                const bool whole = w.m - t0 >= tpt && (!p.causal || t0 >= k0 + kt * 128 + 127 - past);
                int rows = rpt, c_lo = 0;
                if (!whole) {
                    rows = min(tpt, w.m - t0) * p.group;
                    c_lo = min(max(t_min - t0, 0), tpt) * p.group;
                }
                uint64_t add[4] = {0, 0, 0, 0};
                auto columns = [&](auto masked) {
                    uint32_t r[2][32];
                    tmem_ld32_issue(ta, r[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld_wait(r[c & 1]);
                        if (c < 3) tmem_ld32_issue(ta + (c + 1) * 32, r[(c + 1) & 1]);
                        const ulonglong2* nlv = reinterpret_cast<const ulonglong2*>(&s.nl[nst][c * 32]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const ulonglong2 l2 = nlv[i];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int n = 4 * i + 2 * h;
                                const uint64_t x = f2_fma(
                                    f2_pack(__uint_as_float(r[c & 1][n]), __uint_as_float(r[c & 1][n + 1])), sl2,
                                    h ? l2.y : l2.x);
                                float a, b;
                                f2_unpack(x, a, b);
                                a = ex2(a);
                                b = ex2(b);
                                if (masked.value) {
                                    const int col = c * 32 + n;
                                    a = col >= c_lo && col < rows ? a : 0.f;
                                    b = col + 1 >= c_lo && col + 1 < rows ? b : 0.f;
                                }
                                add[n / 2 & 3] = f2_add(add[n / 2 & 3], f2_pack(a, b));
                            }
                        }
                    }
                };
                if (whole) columns(std::false_type{});
                else columns(std::true_type{});
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s.s_empty[kt][par]);
                    mbar_arrive(&s.nl_empty[nst]);
                }
                float a, b, c, d;
                f2_unpack(f2_add(add[0], add[1]), a, b);
                f2_unpack(f2_add(add[2], add[3]), c, d);
                total += (a + b) + (c + d);
            }
            // the two warpgroups' sums, then the ranks'
            float* part = &s.part[kt][tid];
            if (par == 1) *part = total;
            bar_sync(1 + kt, 256);
            if (par == 0) total += *part;
            if (csize > 1) {
                bar_sync(1 + kt, 256);
                if (par == 0) *part = total;
                cluster_sync();
                if (rank == 0 && par == 0) {
                    total = 0.f;
                    for (int r = 0; r < csize; ++r)
                        total += __uint_as_float(dsmem_load(reinterpret_cast<const uint32_t*>(part), r));
                }
            } else {
                bar_sync(1 + kt, 256);  // read, before the next unit's
            }
            if (rank == 0 && par == 0 && key < w.len && ok) {
                const int64_t at = (int64_t)w.b * p.kv.H + head;
                const float old = p.acc_in ? p.decay * p.acc_in[at * p.ld_acc_in + key] : 0.f;
                p.acc_out[at * p.ld_acc_out + key] = old + total;
            }
        }
        if (csize > 1) {
            if (warp >= 16) cluster_sync();
            cluster_sync();  // the sums have been read
        }
    }
    // nothing of this block may be in flight when it goes
    __syncwarp();
    if (warp == 16 && elect_one()) {
        tc_commit(&s.done);
        wait_drain(&s.done, 0);
    }
    if (warp == 17 && lane == 0)
        for (int i = qf > C::Q_STAGES ? qf - C::Q_STAGES : 0; i < qf; ++i)
            wait_drain(&s.q_full[i % C::Q_STAGES], i / C::Q_STAGES & 1);
    if (warp == 18 && lane == 0)
        for (int i = kf > C::K_STAGES ? kf - C::K_STAGES : 0; i < kf; ++i)
            wait_drain(&s.k_full[i % C::K_STAGES], i / C::K_STAGES & 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 16) tmem_dealloc(tmem, 512);
}

}  // namespace hsi
