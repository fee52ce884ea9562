// Attention of a few new tokens over a paged cache, and the attention weights
// of its entries, for up to a few rows per KV head (a row: one new token and
// one query head). Rows of one KV head share its K and V tiles: with r rows an
// entry costs 4 D bytes and 4 D r flops, far below the tensor rate for r <= 16,
// so the bound is HBM and the work is to keep it busy:
//
//  - The (sequence, row tile, KV head) units, each ceil(length / 64) tiles of 64
//    entries, form one line of tiles that is cut into equal runs, one per CTA, two CTAs
//    an SM. Long and short sequences mix freely and no SM waits for another; a
//    unit that spans CTAs is joined from their partial sums by a second kernel.
//    Short sequences go without the line and the second kernel: a cluster a unit,
//    its tiles in equal parts, joined through distributed shared memory.
//  - A producer warp fetches tiles with one TMA box per page (or 64 entries of
//    it) into a ring of shared-memory stages, a lane per box.
//  - Each of four warps owns 16 entries of a tile: S = Q K^T by mma.sync
//    (16 rows x 16 entries), its own running maximum and sum, P V into its own
//    16 x D accumulator. Nothing is exchanged between warps before the unit's end.
//
// mma.sync suffices here: a 64-entry tile needs 128 of them in the ~1400
// cycles its 32 KB take at the SM's share of HBM. P is rounded to the cache's
// type for the second product (error 2^-9 relative per term in bf16, averaged by
// the sum; fp16: see P_SHIFT); maxima, sums and the output stay in fp32.
//
// Measured (32 query and 8 KV heads of 128, bf16): one token over 16 sequences of
// up to 65536 entries 475 to 500 us, 97 to 102% of the measured copy rate; over one
// of 8000 entries 13 us (floor 5), the start, a tile's chain of 700 cycles and the
// join; three short sequences of up to 777 entries (16 / 2 heads of 64) 7.1 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"
#include "paged.cuh"

namespace hsi {

constexpr int AT_ROWS = 16;      // rows of a unit
constexpr int AT_KT = 64;        // entries of a tile
constexpr int AT_CLUSTER = 8;    // most blocks of a short unit
constexpr int AT_WARPS = 4;      // consumer warps, 16 entries of a tile each
constexpr int AT_THREADS = 32 * (AT_WARPS + 1);

struct AttendParams {
    PagedView kv;
    const void* q;
    int64_t qt, qh;  // token and head strides (elements)
    const int32_t* q_start;
    int64_t T;       // tokens of q
    int max_q, max_kv, Hq, group;  // host bounds of new tokens and entries; query heads, per KV head
    float sl2;       // scale * log2(e) (attend_chunk_kernel: its size, above 0, and its sign)
    int causal, negate;
    void* out;
    int64_t ot, oh;
    float* lse;      // [T][Hq] or null
    // partial sums: slot s holds AT_ROWS x D accumulators, AT_ROWS maxima (base 2), AT_ROWS sums
    float* part;
    uint32_t* base;  // attend_chunk_kernel: [B + 1] first tile of each sequence on the line
    // weights only
    const float* lse_in;
    const float* acc_in;
    float* acc_out;
    int64_t ld_acc_in, ld_acc_out;
    float decay;
};

// A value of rank c's part (this block's own where there is no cluster).
__device__ __forceinline__ float cluster_load(const float* mine, int c, int csize) {
    return csize > 1 ? __uint_as_float(dsmem_load(reinterpret_cast<const uint32_t*>(mine), c)) : *mine;
}
__device__ __forceinline__ float4 cluster_load4(const float* mine, int c, int csize) {
    if (csize <= 1) return *reinterpret_cast<const float4*>(mine);
    uint32_t addr;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(c));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int D>
__host__ __device__ constexpr int attend_slot_floats(int rows) { return rows * (D + 2); }

// A line of `total` tiles (below 2^31, the host's bound) cut into at most
// `grid` runs, none empty: the first `rest` of them one tile longer.
struct Line {
    uint32_t total, G, q, rest;
    __device__ __forceinline__ Line(uint32_t total_, uint32_t grid) : total(total_), G(min(grid, total_)) {
        q = G ? total / G : 0u;
        rest = total - q * G;
    }
    // first tile of run c
    __device__ __forceinline__ uint32_t cut(uint32_t c) const { return c * q + min(c, rest); }
    // the run that holds tile x
    __device__ __forceinline__ uint32_t run(uint32_t x) const {
        const uint32_t longer = rest * (q + 1);
        return x < longer ? x / (q + 1) : rest + (x - longer) / q;
    }
};

// ---------------------------------------------------------------- mma.sync --

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__half>(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// fp16 ends at 2^-24, where p of many entries far below a row's largest still
// add up (a million of 2^-25 hold 3% of a row). So p is taken as 2^(x - m + 15),
// up to half the largest fp16 number, and reaches 2^-39 of the largest; as the sums
// have the same factor, it is a maximum m - 15 to all that follows. bf16 has
// fp32's exponents.
template <typename T>
constexpr float P_SHIFT = is_bf16<T> ? 0.f : 15.f;

// The factor that takes sums by the maximum mine (base 2) to those by the
// maximum m >= mine of all parts. A part whose maximum is -inf has seen nothing
// (sums of 0) or nothing but NaN (which a maximum passes over): its sums stay as
// they are, so that the NaN come through.
__device__ __forceinline__ float part_factor(float mine, float m) { return mine == -INFINITY ? 1.f : ex2(mine - m); }

// --------------------------------------------------------------- the kernel --

template <int D, bool WEIGHTS>
struct AttendCfg {
    static constexpr int HALF_BYTES = AT_KT * 128;                 // 64 values of every entry of a tile
    static constexpr int K_BYTES = HALF_BYTES * (D / 64);
    static constexpr int STAGE_BYTES = WEIGHTS ? K_BYTES : 2 * K_BYTES;
    // CTAs an SM, and stages that fill its shared memory. The weights' tiles are half the bytes
    // at the same latency of a tile's work: two CTAs reach 72% of the copy rate, three 90%.
    static constexpr int CTAS = WEIGHTS ? 3 : 2;
    static constexpr int STAGES = (WEIGHTS ? 65536 : 98304) / STAGE_BYTES;
    static constexpr int RED_BYTES = WEIGHTS ? 0 : AT_WARPS * AT_ROWS * 32 * 4;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + RED_BYTES;
};

// Where a walk along the line stands: the sequence, its tiles and what is left.
struct LineWalk {
    int b;
    int first;        // first tile of sequence b
    int32_t len, m, at;  // entries, new tokens, first new token
    int nt, units;    // tiles of a unit, units of the sequence (row tiles x KV heads)
};

template <bool WEIGHTS>
__device__ __forceinline__ void walk_load(const AttendParams& p, LineWalk& w) {
    w.len = paged_len(p.kv, w.b, p.max_kv);
    w.m = paged_new(p.q_start, w.b, p.max_q, p.T, &w.at);
    w.nt = (w.len + AT_KT - 1) / AT_KT;
    const int rt = (w.m * p.group + AT_ROWS - 1) / AT_ROWS;
    w.units = (WEIGHTS ? 1 : rt) * p.kv.H;  // the weights' units take every row of a KV head
}
__device__ __forceinline__ int walk_tiles(const LineWalk& w) { return w.nt * w.units; }

template <typename T, int D, bool WEIGHTS>
__global__ void __launch_bounds__(AT_THREADS, AttendCfg<D, WEIGHTS>::CTAS)
    attend_token_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, int csize) {
    using C = AttendCfg<D, WEIGHTS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[C::STAGES], empty[C::STAGES];
    __shared__ uint32_t s_lo, s_hi;
    __shared__ int s_b, s_first, s_abort;
    __shared__ float s_m[AT_WARPS][AT_ROWS], s_l[AT_WARPS][AT_ROWS];
    uint8_t* const stage0 = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float* const red = reinterpret_cast<float*>(stage0 + C::STAGES * C::STAGE_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], AT_WARPS);
        }
        fence_mbar_init();
        s_abort = 0;
        tma_prefetch_map(&kmap);
        if (!WEIGHTS) tma_prefetch_map(&vmap);
    }
    griddep_wait();
    griddep_launch_dependents();

    LineWalk w;
    int x, hi;  // the tiles of this block: of the line, or (short) of its unit
    if (!WEIGHTS && csize) {
        // short: a cluster of csize blocks a unit, the unit's tiles in equal parts
        const int u = blockIdx.x / csize, rank = csize > 1 ? (int)cluster_ctarank() : 0;
        const int rts = (p.max_q * p.group + AT_ROWS - 1) / AT_ROWS;
        w.b = u / (rts * p.kv.H);
        w.first = -(u % (rts * p.kv.H));
        walk_load<WEIGHTS>(p, w);
        const int per = (w.nt + csize - 1) / csize;
        const int t0 = min(w.nt, rank * per), t1 = min(w.nt, t0 + per);
        const bool there = -w.first < w.units;  // the row tile has rows
        w.first *= w.nt;
        x = there ? t0 : 0;
        hi = there ? t1 : 0;
        if (x == hi && threadIdx.x < AT_ROWS) {
            float* slot = reinterpret_cast<float*>(stage0);
            slot[AT_ROWS * D + threadIdx.x] = -INFINITY;
            slot[AT_ROWS * (D + 1) + threadIdx.x] = 0.f;
        }
        __syncthreads();
    } else {
        // the line: total tiles, then the sequence that holds this run's first tile (up to 32
        // sequences, a lane each, are looked at once)
        if (warp == 0) {
            auto tiles_of = [&](int b) {
                if (b >= p.kv.B) return 0u;
                LineWalk w;
                w.b = b;
                walk_load<WEIGHTS>(p, w);
                return (uint32_t)walk_tiles(w);
            };
            auto upto = [&](uint32_t n) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t up = __shfl_up_sync(~0u, n, o);
                    if (lane >= o) n += up;
                }
                return n;
            };
            uint32_t total = 0, n = 0;
            for (int b0 = 0; b0 < p.kv.B; b0 += 32) {
                n = tiles_of(b0 + lane);
                total += __reduce_add_sync(~0u, n);
            }
            const Line line(total, gridDim.x);
            const uint32_t lo = line.cut(blockIdx.x);
            uint32_t before = 0;
            for (int b0 = 0; b0 < p.kv.B && before <= lo; b0 += 32) {
                if (p.kv.B > 32) n = tiles_of(b0 + lane);
                const uint32_t sum = upto(n), f = before + sum - n;
                if (lo >= f && lo < f + n) {
                    s_b = b0 + lane;
                    s_first = f;
                }
                before += __shfl_sync(~0u, sum, 31);
            }
            if (lane == 0) {
                s_lo = blockIdx.x < line.G ? lo : 0u;
                s_hi = blockIdx.x < line.G ? line.cut(blockIdx.x + 1) : 0u;
            }
        }
        __syncthreads();
        x = s_lo;
        hi = s_hi;
        if (x >= hi) return;  // more blocks than tiles
        w.b = s_b;
        w.first = s_first;
        walk_load<WEIGHTS>(p, w);
    }
    int stage = 0, fills = 0;
    uint32_t phase = 0;
    bool ok = true;  // false once a wait has run out: no more copies or results, but every barrier is kept

    while (x < hi) {
        while (x >= w.first + walk_tiles(w)) {
            w.first += walk_tiles(w);
            ++w.b;
            walk_load<WEIGHTS>(p, w);
        }
        const int unit = (x - w.first) / w.nt, tile0 = (x - w.first) % w.nt;
        const int n_tiles = min(hi - x, w.nt - tile0);
        const int head = unit % p.kv.H, rt = unit / p.kv.H;
        x += n_tiles;

        if (warp == AT_WARPS) {  // producer: a lane per box
            const int box = p.kv.page_shift < 6 ? 1 << p.kv.page_shift : AT_KT;  // entries of a box
            const int nbox = AT_KT / box, halves = D / 64;
            const int per = nbox * halves;
            const int bi = lane % per, kind = lane / per;  // box; 0: K, 1: V
            const int e = (bi / halves) * box, dim = (bi % halves) * 64;
            for (int i = 0; i < n_tiles; ++i) {
                const int e0 = (tile0 + i) * AT_KT;
                const int live = (min(w.len - e0, AT_KT) + box - 1) / box * halves;  // boxes with entries
                const bool mine = kind < (WEIGHTS ? 1 : 2) && e0 + e < w.len;
                int page = 0;
                if (mine) page = paged_page(p.kv, w.b, (e0 + e) >> p.kv.page_shift);
                ok = wait_bounded(&empty[stage], phase ^ 1, &s_abort);
                ok = __all_sync(~0u, ok);
                if (!ok) {  // let the copies in flight land before the block goes
                    for (int k = fills > C::STAGES ? fills - C::STAGES : 0; k < fills; ++k)
                        wait_drain(&full[k % C::STAGES], (k / C::STAGES) & 1);
                    break;
                }
                ++fills;
                if (fills == 1 && *(volatile int*)&g_hsi_skip_first_copy) goto next;
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], live * box * 128 * (WEIGHTS ? 1 : 2));
                __syncwarp();
                if (mine) {
                    uint8_t* dst = stage0 + stage * C::STAGE_BYTES + kind * C::K_BYTES + (dim / 64) * C::HALF_BYTES +
                                   e * 128;
                    tma_page_box(dst, kind ? &vmap : &kmap, dim, (e0 + e) & ((1 << p.kv.page_shift) - 1), head, page,
                                 &full[stage]);
                }
            next:
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            continue;
        }

        // ---- consumers ----
        const int rows = w.m * p.group;
        const int r_lo = lane >> 2, kq = (lane & 3) * 2;
        const int rt_end = WEIGHTS ? (rows + AT_ROWS - 1) / AT_ROWS : rt + 1;
        uint32_t qf[D / 16][4];
        int lim[2];         // entries that rows r_lo, r_lo + 8 see
        float lse2[2] = {}; // weights: log-sum-exp (base 2)
        auto load_rows = [&](int rtile) {
            const uint32_t* src[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = rtile * AT_ROWS + r_lo + 8 * j;
                src[j] = nullptr;
                lim[j] = 0;
                if (r >= rows) continue;
                const int t = r / p.group, h = head * p.group + r % p.group;
                src[j] = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) + (w.at + t) * p.qt + h * p.qh);
                lim[j] = p.causal ? min(w.len, w.len - w.m + t + 1) : w.len;
                if (WEIGHTS) {
                    const float v = __ldg(p.lse_in + (int64_t)(w.at + t) * p.Hq + h);
                    if (v == -INFINITY) lim[j] = 0;
                    lse2[j] = v * LOG2E;
                }
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    qf[k][j] = src[j & 1] ? __ldg(src[j & 1] + k * 8 + (j >> 1) * 4 + (lane & 3)) : 0u;
            }
        };
        load_rows(WEIGHTS ? 0 : rt);

        float o[WEIGHTS ? 1 : D / 8][4] = {};
        float m2[2] = {-INFINITY, -INFINITY}, l[2] = {};
        // shared-memory addresses of this lane's ldmatrix rows, within a tile
        const int mat = lane >> 3, mrow = lane & 7;
        const int krow = warp * 16 + (mat >> 1) * 8 + mrow;  // K: matrices (entries 0-7, 0-7, 8-15, 8-15) x (chunk, +1)
        const int vrow = warp * 16 + (mat & 1) * 8 + mrow;   // V: matrices (0-7, 8-15) x (chunk, chunk, +1, +1)

        // weights: lanes 0 .. 15 write an entry each, the one whose sum they hold after the
        // shuffles; its old weight is loaded a tile ahead
        const int mine = (lane >> 3 & 1) * 8 + (lane & 3) * 2 + (lane >> 2 & 1);
        const int64_t acc_row = (int64_t)w.b * p.kv.H + head;
        const float* acc_in = WEIGHTS && p.acc_in ? p.acc_in + acc_row * p.ld_acc_in : nullptr;
        float* acc_out = WEIGHTS ? p.acc_out + acc_row * p.ld_acc_out : nullptr;
        float old = 0.f;
        if (WEIGHTS && acc_in && lane < 16 && tile0 * AT_KT + warp * 16 + mine < w.len)
            old = acc_in[tile0 * AT_KT + warp * 16 + mine];

        for (int i = 0; i < n_tiles; ++i) {
            ok = ok && __all_sync(~0u, wait_bounded(&full[stage], phase, &s_abort));
            const uint32_t kbase = smem_u32(stage0 + stage * C::STAGE_BYTES);
            const int e0 = (tile0 + i) * AT_KT + warp * 16;
            float next = 0.f;
            if (WEIGHTS && acc_in && lane < 16 && e0 + AT_KT + mine < w.len) next = acc_in[e0 + AT_KT + mine];
            float add[4] = {};  // weights of entries kq, kq + 1, 8 + kq, 9 + kq
            for (int rr = WEIGHTS ? 0 : rt; ok && rr < rt_end; ++rr) {
                if (WEIGHTS && rt_end > 1) {
                    load_rows(rr);
                    __syncwarp();
                }
                float s[2][4] = {};
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t kf[4];
                    const int chunk = 2 * k + (mat & 1);
                    ldmatrix_x4(kbase + (chunk >> 3) * C::HALF_BYTES + krow * 128 + (((chunk & 7) ^ (krow & 7)) << 4), kf);
                    mma_16816<T>(s[0], qf[k], kf[0], kf[1]);
                    mma_16816<T>(s[1], qf[k], kf[2], kf[3]);
                }
                if (WEIGHTS) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int j = c >> 1, key = e0 + n * 8 + kq + (c & 1);
                            const float pr = key < lim[j] ? ex2(fmaf(s[n][c], p.sl2, -lse2[j])) : 0.f;
                            add[n * 2 + (c & 1)] += pr;
                        }
                    }
                    continue;
                }
                float mx[2] = {m2[0], m2[1]};
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int j = c >> 1, key = e0 + n * 8 + kq + (c & 1);
                        s[n][c] = key < lim[j] ? s[n][c] * p.sl2 : -INFINITY;
                        mx[j] = fmaxf(mx[j], s[n][c]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[j] = fmaxf(mx[j], __shfl_xor_sync(~0u, mx[j], 1));
                    mx[j] = fmaxf(mx[j], __shfl_xor_sync(~0u, mx[j], 2));
                }
                if (__any_sync(~0u, mx[0] > m2[0] || mx[1] > m2[1])) {
                    float f[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        f[j] = mx[j] == -INFINITY ? 1.f : ex2(m2[j] - mx[j]);
                        m2[j] = mx[j];
                        l[j] *= f[j];
                    }
#pragma unroll
                    for (int d = 0; d < (WEIGHTS ? 1 : D / 8); ++d) {
                        o[d][0] *= f[0];
                        o[d][1] *= f[0];
                        o[d][2] *= f[1];
                        o[d][3] *= f[1];
                    }
                }
                float base[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) base[j] = m2[j] == -INFINITY ? 0.f : m2[j] - P_SHIFT<T>;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        s[n][c] = ex2(s[n][c] - base[c >> 1]);
                        l[c >> 1] += s[n][c];
                    }
                }
                const uint32_t pf[4] = {pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]),
                                        pack2<T>(s[1][0], s[1][1]), pack2<T>(s[1][2], s[1][3])};
                const uint32_t vbase = kbase + C::K_BYTES;
                if (e0 + 16 > w.len) {
                    // entries past the length hold whatever the page holds (or nothing was
                    // loaded): 0 * NaN would reach every row, so they become zeros
                    for (int idx = lane; idx < 16 * (D / 8); idx += 32) {
                        const int r = warp * 16 + idx / (D / 8), ch = idx % (D / 8);
                        if ((tile0 + i) * AT_KT + r >= w.len)
                            *reinterpret_cast<uint4*>(stage0 + stage * C::STAGE_BYTES + C::K_BYTES +
                                                      (ch >> 3) * C::HALF_BYTES + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int d = 0; d < (WEIGHTS ? 0 : D / 16); ++d) {
                    uint32_t vf[4];
                    const int chunk = 2 * d + (mat >> 1);
                    ldmatrix_x4_trans(
                        vbase + (chunk >> 3) * C::HALF_BYTES + vrow * 128 + (((chunk & 7) ^ (vrow & 7)) << 4), vf);
                    mma_16816<T>(o[2 * d], pf, vf[0], vf[1]);
                    mma_16816<T>(o[2 * d + 1], pf, vf[2], vf[3]);
                }
            }
            fence_proxy_async_smem();  // what this warp wrote or read precedes the next TMA into the stage
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1;
            }
            if (WEIGHTS && ok) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    add[c] += __shfl_xor_sync(~0u, add[c], 4);
                    add[c] += __shfl_xor_sync(~0u, add[c], 8);
                    add[c] += __shfl_xor_sync(~0u, add[c], 16);
                }
                if (e0 + mine < w.len && lane < 16) {
                    const float sum = lane < 8 ? (lane < 4 ? add[0] : add[1]) : (lane < 12 ? add[2] : add[3]);
                    acc_out[e0 + mine] = p.decay * old + sum;
                }
                old = next;
            }
        }
        if constexpr (!WEIGHTS) {  // join the four warps
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[j] += __shfl_xor_sync(~0u, l[j], 1);
                l[j] += __shfl_xor_sync(~0u, l[j], 2);
                m2[j] -= P_SHIFT<T>;  // what the sums are by
            }
            if ((lane & 3) == 0) {
                s_m[warp][r_lo] = m2[0];
                s_m[warp][r_lo + 8] = m2[1];
                s_l[warp][r_lo] = l[0];
                s_l[warp][r_lo + 8] = l[1];
            }
            bar_sync(1, 32 * AT_WARPS);
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = r_lo + 8 * j;
                float m = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
                f[j] = part_factor(m2[j], m);
            }
            const bool whole = !csize && tile0 == 0 && n_tiles == w.nt;
            float* slot = csize ? reinterpret_cast<float*>(stage0)  // every tile has been read
                                : p.part + (int64_t)(2 * blockIdx.x + (tile0 > 0 ? 0 : 1)) * attend_slot_floats<D>(AT_ROWS);
            // 32 dims at a time: thread -> row tid / 8, dims (tid % 8) * 4 .. + 3
            const int orow = threadIdx.x >> 3, od = (threadIdx.x & 7) * 4;
            const float rm = fmaxf(fmaxf(s_m[0][orow], s_m[1][orow]), fmaxf(s_m[2][orow], s_m[3][orow]));
            float rl = 0.f;
#pragma unroll
            for (int i = 0; i < AT_WARPS; ++i)
                rl += s_l[i][orow] * part_factor(s_m[i][orow], rm);
            const int r = rt * AT_ROWS + orow;
            const int64_t tok = w.at + (r < rows ? r / p.group : 0);
            const int h = head * p.group + (r < rows ? r % p.group : 0);
            const float inv = rl > 0.f || rl != rl ? 1.f / rl : 0.f;
#pragma unroll
            for (int c = 0; c < (WEIGHTS ? 0 : D / 32); ++c) {
                float* mine = red + warp * AT_ROWS * 32;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const float(&v)[4] = o[4 * c + d];
                    *reinterpret_cast<float2*>(mine + r_lo * 32 + d * 8 + kq) = make_float2(v[0] * f[0], v[1] * f[0]);
                    *reinterpret_cast<float2*>(mine + (r_lo + 8) * 32 + d * 8 + kq) = make_float2(v[2] * f[1], v[3] * f[1]);
                }
                bar_sync(1, 32 * AT_WARPS);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < AT_WARPS; ++i) {
                    const float4 v = *reinterpret_cast<const float4*>(red + i * AT_ROWS * 32 + orow * 32 + od);
                    sum.x += v.x;
                    sum.y += v.y;
                    sum.z += v.z;
                    sum.w += v.w;
                }
                if (!whole) {
                    *reinterpret_cast<float4*>(slot + orow * D + c * 32 + od) = sum;
                } else if (r < rows) {
                    uint2 v = make_uint2(pack2<T>(sum.x * inv, sum.y * inv), pack2<T>(sum.z * inv, sum.w * inv));
                    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + tok * p.ot + h * p.oh + c * 32 + od) = v;
                }
                bar_sync(1, 32 * AT_WARPS);
            }
            if ((threadIdx.x & 7) == 0) {
                if (!whole) {
                    slot[AT_ROWS * D + orow] = rm;
                    slot[AT_ROWS * D + AT_ROWS + orow] = rl;
                } else if (r < rows && p.lse) {
                    p.lse[tok * p.Hq + h] = rl == 0.f ? -INFINITY : (rm + log2f(rl)) * LN2;
                }
            }
        }
    }

    if constexpr (!WEIGHTS) {
        if (!csize) return;
        // short: the cluster's parts are joined through distributed shared memory, each block a
        // share of the outputs
        if (csize > 1) cluster_sync();
        else __syncthreads();
        const int rank = csize > 1 ? (int)cluster_ctarank() : 0;
        const int rts = (p.max_q * p.group + AT_ROWS - 1) / AT_ROWS, unit = blockIdx.x / csize % (rts * p.kv.H);
        const int head = unit % p.kv.H, rt = unit / p.kv.H;
        const float* slot = reinterpret_cast<const float*>(stage0);
        for (int i = rank * AT_THREADS + threadIdx.x; i < AT_ROWS * (D / 4); i += csize * AT_THREADS) {
            const int row = i / (D / 4), d = (i % (D / 4)) * 4, r = rt * AT_ROWS + row;
            if (r >= w.m * p.group) break;
            float mc[AT_CLUSTER], lc[AT_CLUSTER], m = -INFINITY, l = 0.f;
#pragma unroll
            for (int c = 0; c < AT_CLUSTER; ++c) {
                mc[c] = -INFINITY;
                lc[c] = 0.f;
                if (c < csize) {
                    mc[c] = cluster_load(slot + AT_ROWS * D + row, c, csize);
                    lc[c] = cluster_load(slot + AT_ROWS * (D + 1) + row, c, csize);
                }
                m = fmaxf(m, mc[c]);
            }
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int c = 0; c < AT_CLUSTER; ++c) {
                if (lc[c] == 0.f) continue;  // a part without tiles has no sums
                const float f = part_factor(mc[c], m);
                const float4 v = cluster_load4(slot + row * D + d, c, csize);
                o.x += f * v.x;
                o.y += f * v.y;
                o.z += f * v.z;
                o.w += f * v.w;
                l += f * lc[c];
            }
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const int64_t tok = w.at + r / p.group;
            const int h = head * p.group + r % p.group;
            *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + tok * p.ot + h * p.oh + d) =
                make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
            if (d == 0 && p.lse) p.lse[tok * p.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
        }
        if (csize > 1) cluster_sync();  // nobody leaves while its part is read
    }
}

// Where unit `unit` of sequence b lies on the line: its first run, and how many
// runs hold it. Whole warp; sets w to sequence b.
__device__ __forceinline__ int line_runs_of(const AttendParams& p, int b, int unit, int grid, LineWalk& w, int& c0) {
    const int lane = threadIdx.x & 31;
    uint32_t total = 0, before = 0;
    for (int b0 = 0; b0 < p.kv.B; b0 += 32) {
        uint32_t n = 0;
        if (b0 + lane < p.kv.B) {
            w.b = b0 + lane;
            walk_load<false>(p, w);
            n = walk_tiles(w);
        }
        total += __reduce_add_sync(~0u, n);
        before += __reduce_add_sync(~0u, b0 + lane < b ? n : 0u);
    }
    w.b = b;
    walk_load<false>(p, w);
    c0 = 0;
    if (!w.nt || unit >= w.units) return 0;
    const Line line(total, grid);
    const uint32_t s0 = before + (uint32_t)unit * w.nt;
    c0 = line.run(s0);
    return (int)line.run(s0 + w.nt - 1) - c0 + 1;
}

// Joins the units that several runs hold: a block per (sequence, row tile, KV
// head) and DIMS dims (all where there are many units). Runs of a unit lie side by side: the first wrote
// its CTA's slot 1, the others their slots 0. A warp takes a row's maxima and
// sums, a lane a run, and leaves each run's factor in shared memory; then
// groups of threads, one per four output values, add up every so many runs (a
// long sequence alone has up to 304 runs a unit) and the groups' sums are added.
// Which runs those are needs only
// the lengths, which were there before the kernel that writes the parts: that
// comes before the wait for it. Sequences without entries get zeros and lse -inf
// here.
constexpr int AT_MAX_RUNS = 512;  // CTAs of the kernel above
constexpr int AT_JOIN_THREADS = 256;

template <typename T, int D, int DIMS>
__global__ void __launch_bounds__(AT_JOIN_THREADS) attend_join_kernel(const __grid_constant__ AttendParams p, int grid) {
    __shared__ float s_f[AT_ROWS][AT_MAX_RUNS];  // a run's factor for a row, over the row's sum
    __shared__ float4 s_o[AT_JOIN_THREADS];
    const int b = blockIdx.z, head = blockIdx.y, rt = blockIdx.x / (D / DIMS);
    const int d0 = blockIdx.x % (D / DIMS) * DIMS, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    LineWalk w;
    int c0;
    const int runs = line_runs_of(p, b, rt * p.kv.H + head, grid, w, c0);
    griddep_wait();
    griddep_launch_dependents();
    const int rows = min(AT_ROWS, w.m * p.group - rt * AT_ROWS);
    if (rows <= 0 || runs == 1) return;  // no rows, or written whole
    constexpr int SLOT = attend_slot_floats<D>(AT_ROWS);
    const float* first = p.part + (int64_t)(2 * c0 + 1) * SLOT;
    const float* rest = p.part + (int64_t)2 * c0 * SLOT;  // run i > 0: rest + 2 i SLOT
    for (int row = warp; row < rows; row += AT_JOIN_THREADS / 32) {
        float mc[AT_MAX_RUNS / 32], lc[AT_MAX_RUNS / 32], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < AT_MAX_RUNS / 32; ++k) {  // all loads at once
            const int i = lane + 32 * k;
            mc[k] = -INFINITY;
            lc[k] = 0.f;
            if (i < runs) {
                const float* slot = i ? rest + 2 * i * SLOT : first;
                mc[k] = slot[AT_ROWS * D + row];
                lc[k] = slot[AT_ROWS * (D + 1) + row];
            }
        }
#pragma unroll
        for (int k = 0; k < AT_MAX_RUNS / 32; ++k) m = fmaxf(m, mc[k]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
#pragma unroll
        for (int k = 0; k < AT_MAX_RUNS / 32; ++k) {
            mc[k] = part_factor(mc[k], m);
            l += mc[k] * lc[k];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
        for (int k = 0; k < AT_MAX_RUNS / 32; ++k)
            if (lane + 32 * k < runs) s_f[row][lane + 32 * k] = mc[k] * inv;
        if (lane == 0 && p.lse && d0 == 0) {
            const int r = rt * AT_ROWS + row;
            p.lse[(w.at + r / p.group) * (int64_t)p.Hq + head * p.group + r % p.group] =
                l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
        }
    }
    __syncthreads();
    const int items = rows * (DIMS / 4);
    const int groups = items < AT_JOIN_THREADS ? min(AT_JOIN_THREADS / items, 32) : 1;
    const int group = items < AT_JOIN_THREADS ? threadIdx.x / items : 0;
    for (int i = threadIdx.x - group * items; group < groups && i < items; i += AT_JOIN_THREADS) {
        const int row = i / (DIMS / 4), d = d0 + (i % (DIMS / 4)) * 4, r = rt * AT_ROWS + row;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int c = group; c < runs; c += groups) {
            const float f = s_f[row][c];
            const float4 v = *reinterpret_cast<const float4*>((c ? rest + 2 * c * SLOT : first) + row * D + d);
            o.x += f * v.x;
            o.y += f * v.y;
            o.z += f * v.z;
            o.w += f * v.w;
        }
        if (groups > 1) {
            s_o[group * items + i] = o;
            break;
        }
        const int64_t tok = w.at + r / p.group;
        const int h = head * p.group + r % p.group;
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + tok * p.ot + h * p.oh + d) =
            make_uint2(pack2<T>(o.x, o.y), pack2<T>(o.z, o.w));
    }
    if (groups == 1) return;
    __syncthreads();
    if (group) return;
    const int i = threadIdx.x, row = i / (DIMS / 4), d = d0 + (i % (DIMS / 4)) * 4, r = rt * AT_ROWS + row;
    float4 o = s_o[i];
    for (int c = 1; c < groups; ++c) {
        const float4 v = s_o[c * items + i];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
    }
    const int64_t tok = w.at + r / p.group;
    const int h = head * p.group + r % p.group;
    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + tok * p.ot + h * p.oh + d) =
        make_uint2(pack2<T>(o.x, o.y), pack2<T>(o.z, o.w));
}

}  // namespace hsi
