// Attention of a chunk of new tokens over a paged cache on the tensor cores.
//
// A unit is (sequence, KV head, 256 query rows): two accumulator tiles of 128
// rows, row = token * group + head, so that a KV head's K and V tiles of 128
// entries serve all of its query heads. Each tile has a warpgroup, a thread per
// row. One thread issues the products:
//   S_w = Q_w K^T            (Q, K from shared memory, S in tensor memory)
//   O_w += P_w V             (P in tensor memory over S, V from shared memory)
// and while warpgroup 0 turns S_0 into P_0, the tensor cores work for tile 1:
// 2 x 512 cycles a tile at D = 128 for the products against 512 for the
// exponentials. P becomes visible in two halves, so that the second product
// starts while the second half is still being exponentiated.
//
// The running maximum is lazy: O is rescaled only where a row's maximum has
// grown by more than 2^8 since the last time (p stays below 256, or 2^15 where
// fp16 is shifted), which after the first tiles hardly happens; the row sum
// is taken from the fp32 p in the shadow of the exponentials (the exponentials of
// half a tile by the old maximum, before the new one is known, were no faster).
//
// The units' key tiles (causal: only those that some row of the unit sees)
// form one line that is cut into equal runs, one per SM, as for single tokens;
// a unit that spans runs is joined by a second kernel from fp32 partial sums.
//
// Measured (32 query and 8 KV heads of 128, bf16): 2048 tokens over 32768 entries
// 735 us alone, 1450 TFLOP/s or 75% of the measured burst rate, and 780 to 800 us back
// to back under the power limit, 80% of the sustained rate; heads of 64 600 us, half
// the products for the same exponentials. A pair of tiles takes 3300
// cycles, 2200 of products: the rest is the chain of a tile's S, softmax and P V
// (1250 cycles from S to P) and the issuing warp's waits. Short units add 8000
// cycles of start and end each: four chunks of up to 1001 tokens over 5003 entries
// (28 / 4 heads) 165 us for a floor of 92.
#pragma once
#include <cstdint>

#include "attend.cuh"
#include "common.cuh"
#include "paged.cuh"

namespace hsi {

constexpr int CH_ROWS = 128;               // rows of a tile; a unit has two
constexpr int CH_KEYS = 128;               // entries of a key tile
constexpr int CH_THREADS = 32 * 12;        // two softmax warpgroups; one of MMA, copies and two idle warps
constexpr float CH_LAZY = 8.f;             // growth of a maximum (base 2) that O takes without rescaling

// Lengths of sequence b and what follows from them.
struct ChunkSeq {
    int len, m, at, past, n_rt;
    __device__ __forceinline__ void load(const AttendParams& p, int b, int tpt) {
        len = paged_len(p.kv, b, p.max_kv);
        m = paged_new(p.q_start, b, p.max_q, p.T, &at);
        past = len - m;
        n_rt = (m + 2 * tpt - 1) / (2 * tpt);
    }
    // key tiles that the rows of unit rt see
    __device__ __forceinline__ int tiles(const AttendParams& p, int rt, int tpt) const {
        const int seen = p.causal ? min(len, past + min(m, (rt + 1) * 2 * tpt)) : len;
        return seen > 0 ? (seen + CH_KEYS - 1) / CH_KEYS : 0;
    }
};

template <int D>
struct ChunkCfg {
    static constexpr int HALF_BYTES = 128 * 128;
    static constexpr int TILE_BYTES = HALF_BYTES * (D / 64);  // 128 rows of Q, K or V
    static constexpr int Q_STAGES = D == 128 ? 1 : 2;
    static constexpr int KV_STAGES = D == 128 ? 5 : 8;
    static constexpr int RING_BYTES = (2 * Q_STAGES + KV_STAGES) * TILE_BYTES;
    struct Tail {
        uint64_t q_full[Q_STAGES], q_empty[Q_STAGES], kv_full[KV_STAGES], kv_empty[KV_STAGES];
        uint64_t s_full[2], p_full[2][2], o_full[2], o_empty[2], done;
        uint32_t tmem;
        int abort;
        int left, b, g, rt, tile;  // this block's run: key tiles, and where it starts
        ChunkSeq q;
    };
    static constexpr int SMEM_BYTES = RING_BYTES + (int)sizeof(Tail);
    static_assert(SMEM_BYTES <= 232448, "shared memory of an SM");
};

// A cut of the line this near to a unit's end moves there. A part of a unit
// costs its own start and end and two partial sums, some four tiles' time; a
// longer run costs its tiles. So it pays where runs are short, a few units
// each: 2048 tokens over themselves (14 tiles a run, 8 a unit) 62 us against 73;
// runs of 73 tiles lost 4% by it.
__device__ __forceinline__ uint32_t chunk_snap(const Line& line) { return line.q < 32 ? min(4u, line.q / 4) : 0u; }

__host__ __device__ constexpr int64_t chunk_slot_floats(int D) { return 2 * CH_ROWS * (int64_t)(D + 2); }

// A walk along a block's run of the line: segment by segment, each a unit or the part of one that the run holds.
struct ChunkWalk {
    int left, b, g, rt, tile0;
    ChunkSeq q;
    int n, tok0, tiles;  // key tiles of the segment, the unit's first token, row tiles that hold tokens
    bool whole;

    __device__ __forceinline__ void step(const AttendParams& p, int tpt) {
        if (++rt < q.n_rt) return;
        rt = 0;
        if (++g < p.kv.H) return;
        g = 0;
        do q.load(p, ++b, tpt);
        while (q.n_rt == 0);
    }
    // The segment here; false at the run's end.
    __device__ __forceinline__ bool begin(const AttendParams& p, int tpt) {
        if (left <= 0) return false;
        int nt = q.tiles(p, rt, tpt);
        while (nt == 0) {  // there are tiles left, so a unit that has some follows
            step(p, tpt);
            nt = q.tiles(p, rt, tpt);
        }
        n = min(left, nt - tile0);
        whole = tile0 == 0 && n == nt;
        tok0 = rt * 2 * tpt;
        tiles = q.m - tok0 > tpt ? 2 : 1;
        return true;
    }
    __device__ __forceinline__ void advance(const AttendParams& p, int tpt) {
        left -= n;
        tile0 = 0;
        if (left > 0) step(p, tpt);
    }
};

// 32 columns of 32-bit values into this warp's 32 lanes.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <typename T, int D>
__global__ void __launch_bounds__(CH_THREADS, 1)
    attend_chunk_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap, int tpt) {
    using C = ChunkCfg<D>;
    extern __shared__ __align__(1024) uint8_t ring[];
    uint8_t* const q_ring = ring;
    uint8_t* const kv_ring = ring + 2 * C::Q_STAGES * C::TILE_BYTES;
    typename C::Tail& s = *reinterpret_cast<typename C::Tail*>(ring + C::RING_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rpt = tpt * p.group;  // rows of a tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::Q_STAGES; ++i) mbar_init(&s.q_full[i], 1), mbar_init(&s.q_empty[i], 1);
        for (int i = 0; i < C::KV_STAGES; ++i) mbar_init(&s.kv_full[i], 1), mbar_init(&s.kv_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i][0], 4), mbar_init(&s.p_full[i][1], 4);
            mbar_init(&s.o_full[i], 1), mbar_init(&s.o_empty[i], 4);
        }
        mbar_init(&s.done, 1);
        fence_mbar_init();
        s.abort = 0;
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
        tma_prefetch_map(&qmap);
    }
    if (warp == 8) tmem_alloc(&s.tmem, 512);
    // rows past a tile's last whole token are never loaded; finite, so that nothing of them is odd
    for (int i = threadIdx.x; i < 2 * C::Q_STAGES * (D / 64) * (CH_ROWS - rpt) * 8; i += CH_THREADS) {
        const int ch = i & 7, r = (i >> 3) % (CH_ROWS - rpt), half = (i >> 3) / (CH_ROWS - rpt);
        *reinterpret_cast<uint4*>(q_ring + half * C::HALF_BYTES + (rpt + r) * 128 + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 0) {  // the line: its length, then this block's run
        // tiles of a KV head's units of sequence b0 + lane: few sequences one by one with a lane per
        // unit, many with a lane each
        ChunkSeq mine;  // sequence b0 + lane: loaded at once, handed around by shuffles
        auto load = [&](int b0) {
            mine.len = mine.m = mine.at = mine.past = mine.n_rt = 0;
            if (b0 + lane < p.kv.B) mine.load(p, b0 + lane, tpt);
        };
        auto seq = [&](int l) {
            ChunkSeq q;
            q.len = __shfl_sync(~0u, mine.len, l);
            q.m = __shfl_sync(~0u, mine.m, l);
            q.past = q.len - q.m;
            q.n_rt = __shfl_sync(~0u, mine.n_rt, l);
            return q;
        };
        auto tiles_of = [&](int b0) {
            load(b0);
            uint32_t n = 0;
            if (p.kv.B >= 32) {
                for (int rt = 0; rt < mine.n_rt; ++rt) n += mine.tiles(p, rt, tpt);
                return n;
            }
            for (int i = 0; i < p.kv.B; ++i) {
                const ChunkSeq q = seq(i);
                uint32_t sum = 0;
                for (int rt = lane; rt < q.n_rt; rt += 32) sum += q.tiles(p, rt, tpt);
                sum = __reduce_add_sync(~0u, sum);
                if (lane == i) n = sum;
            }
            return n;
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
            n = tiles_of(b0);
            const uint32_t sum = upto(n * p.kv.H);
            if (blockIdx.x == 0 && b0 + lane < p.kv.B) p.base[b0 + lane + 1] = total + sum;
            total += __shfl_sync(~0u, sum, 31);
        }
        if (blockIdx.x == 0 && lane == 0) p.base[0] = 0;
        const Line line(total, gridDim.x);
        const uint32_t snap = chunk_snap(line);
        int cut[2] = {0, 0};  // the run's start and end
        for (int e = 0; e < 2 && blockIdx.x < line.G; ++e) {
            const uint32_t x = line.cut(blockIdx.x + e);
            cut[e] = (int)x;
            uint32_t before = 0;
            bool found = e == 1 && (x == total || snap == 0);  // as it is
            for (int b0 = 0; b0 < p.kv.B && !found; b0 += 32) {
                if (p.kv.B > 32) n = tiles_of(b0);
                const uint32_t sum = upto(n * p.kv.H), f = before + sum - n * p.kv.H;
                const uint32_t has = __ballot_sync(~0u, x >= f && x < f + n * p.kv.H);
                before += __shfl_sync(~0u, sum, 31);
                if (!has) continue;
                found = true;
                // the sequence, its KV head, then the unit, a lane per unit
                const int at = __ffs(has) - 1;
                const uint32_t nb = __shfl_sync(~0u, n, at), off = x - __shfl_sync(~0u, f, at);
                uint32_t rem = off % nb;
                const ChunkSeq q = seq(at);
                for (int r0 = 0; r0 < q.n_rt; r0 += 32) {
                    const uint32_t t = r0 + lane < q.n_rt ? q.tiles(p, r0 + lane, tpt) : 0;
                    const uint32_t u = upto(t), all = __shfl_sync(~0u, u, 31);
                    if (rem >= all) {
                        rem -= all;
                        continue;
                    }
                    const int l = __ffs(__ballot_sync(~0u, rem < u)) - 1;
                    const uint32_t nt = __shfl_sync(~0u, t, l), tile = rem - __shfl_sync(~0u, u - t, l);
                    const uint32_t to = tile <= snap ? 0 : nt - tile <= snap ? nt : tile;
                    cut[e] = (int)(x + to - tile);
                    if (e == 0 && lane == at) {
                        s.q = mine;
                        s.b = b0 + at;
                        s.g = off / nb;
                        s.rt = r0 + l;
                        s.tile = to;
                    }
                    break;
                }
            }
        }
        if (lane == 0) s.left = cut[1] - cut[0];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    ChunkWalk k;
    k.left = s.left;
    if (k.left > 0) {
        k.b = s.b;
        k.g = s.g;
        k.rt = s.rt;
        k.tile0 = s.tile;
        k.q = s.q;
        if (k.tile0 == k.q.tiles(p, k.rt, tpt)) {  // the cut moved to the unit's end
            k.tile0 = 0;
            k.step(p, tpt);
        }
    }
    bool ok = true;  // false once a wait has run out: the role ends, after what it has in flight

    // The softmax holds a row of S in registers: 216 a thread of the 168 x 12 warps that the
    // block was launched with (8 x 216 + 4 x 72 = 12 x 168).
    if (warp < 8) {  // softmax, a thread per row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        constexpr float SHIFT = P_SHIFT<T> ? P_SHIFT<T> - CH_LAZY : 0.f;  // p up to 2^CH_LAZY of its own
        int kvn = 0, seg = 0, it = 0;
        const int w = warp >> 2, row = threadIdx.x & 127;
        for (; ok && k.begin(p, tpt); k.advance(p, tpt)) {
            if (w >= k.tiles) {
                kvn += 2 * k.n;
                continue;
            }
            const int rtok = row / p.group, tok = k.tok0 + w * tpt + rtok, h = k.g * p.group + row % p.group;
            const bool valid = row < rpt && tok < k.q.m;
            const int lim = !valid ? 0 : p.causal ? min(k.q.len, k.q.past + tok + 1) : k.q.len;
            // entries that every row of the tile sees
            const int lim_all = p.causal ? min(k.q.len, k.q.past + k.tok0 + w * tpt + 1) : k.q.len;
            const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t ts = tmem + lane_base + w * 128, to = tmem + lane_base + 256 + w * 128;
            float m_used = -INFINITY, l = 0.f;
            for (int i = 0; i < k.n && ok; ++i) {
                const int k0 = (k.tile0 + i) * CH_KEYS;
                ok = __all_sync(~0u, wait_bounded(&s.s_full[w], (it + i) & 1, &s.abort));
                if (!ok) break;
                tc_fence_after();
                uint32_t r[4][32];
                float mx = -INFINITY;
                const bool full = k0 + CH_KEYS <= lim_all;
                const int edge = lim - k0;  // columns below it are seen
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld32_issue(ts + c * 32, r[c]);
                }
                tmem_ld_wait(r[0]);
#pragma unroll
                for (int c = 1; c < 4; ++c) tmem_ld_waited(r[c]);
                if (!full) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[c][j] = c * 32 + j < edge ? r[c][j] : 0xFF800000u;
                }
                float top[4];  // four chains of three-way maxima
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    top[c] = max3(__uint_as_float(r[c][0]), __uint_as_float(r[c][1]), __uint_as_float(r[c][2]));
#pragma unroll
                    for (int j = 3; j < 31; j += 2)
                        top[c] = max3(top[c], __uint_as_float(r[c][j]), __uint_as_float(r[c][j + 1]));
                    top[c] = fmaxf(top[c], __uint_as_float(r[c][31]));
                }
                mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
                const float mt = mx * p.sl2;  // p.sl2 > 0
                if (__any_sync(~0u, mt > m_used + CH_LAZY)) {
                    const float m_new = fmaxf(m_used, mt);
                    const float f = m_new == -INFINITY ? 1.f : ex2(m_used - m_new);
                    l *= f;
                    if (i > 0) {  // the last product into O came before this S
                        uint32_t o[32];
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            tmem_ld32_issue(to + c * 32, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st32(to + c * 32, o);
                        }
                        tmem_st_wait();
                    }
                    m_used = m_new;
                }
                const float base = m_used == -INFINITY ? 0.f : m_used - SHIFT;
                const uint64_t sl2 = f2_pack(p.sl2, p.sl2), nb = f2_pack(-base, -base);
                if (w == 0 && k0 + CH_KEYS > k.q.len) {
                    // entries past the length hold whatever the page holds (or nothing was loaded):
                    // 0 * NaN would reach every row, so V's become zeros
                    const int st = (kvn + 2 * i + 1) % C::KV_STAGES;
                    ok = __all_sync(~0u, wait_bounded(&s.kv_full[st], (kvn + 2 * i + 1) / C::KV_STAGES & 1, &s.abort));
                    if (!ok) break;
                    const int e0 = k.q.len - k0;
                    for (int i0 = 0; i0 < (CH_KEYS - e0) * (D / 8); i0 += 128) {
                        const int idx = i0 + row;
                        if (idx >= (CH_KEYS - e0) * (D / 8)) continue;
                        *reinterpret_cast<uint4*>(kv_ring + st * C::TILE_BYTES + (idx / 8 % (D / 64)) * C::HALF_BYTES +
                                                  (e0 + idx / (D / 8)) * 128 + (idx & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const uint64_t x =
                                f2_fma(f2_pack(__uint_as_float(r[c][j]), __uint_as_float(r[c][j + 1])), sl2, nb);
                            float a, e;
                            f2_unpack(x, a, e);
                            a = ex2(a);
                            e = ex2(e);
                            sum[j >> 1 & 1] = f2_add(sum[j >> 1 & 1], f2_pack(a, e));
                            pk[(c - 2 * hf) * 16 + j / 2] = pack2<T>(a, e);
                        }
                    }
                    tmem_st32(ts + hf * 32, pk);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.p_full[w][hf]);
                }
                float a, e, c2, d2;
                f2_unpack(sum[0], a, e);
                f2_unpack(sum[1], c2, d2);
                l += (a + e) + (c2 + d2);
            }
            ok = ok && __all_sync(~0u, wait_bounded(&s.o_full[w], seg & 1, &s.abort));
            m_used -= SHIFT;  // what the sums are by
            if (ok) {
                tc_fence_after();
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
                float* slot = p.part + (2 * (int64_t)blockIdx.x + (k.tile0 > 0 ? 0 : 1)) * chunk_slot_floats(D);
                T* out = static_cast<T*>(p.out) + (int64_t)(k.q.at + tok) * p.ot + (int64_t)h * p.oh;
                uint32_t all[D / 32][32];  // whole warps load, before some lanes store
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tmem_ld32_issue(to + c * 32, all[c]);
                tmem_ld_wait(all[0]);
#pragma unroll
                for (int c = 1; c < D / 32; ++c) tmem_ld_waited(all[c]);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const uint32_t(&o)[32] = all[c];
                    if (!k.whole) {  // four dims of 32 rows lie side by side; rows that hold nothing are not read
                        if (valid)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                reinterpret_cast<uint4*>(slot)[(c * 8 + j) * 2 * CH_ROWS + w * CH_ROWS + row] =
                                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    } else if (valid) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t v[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                v[x] = pack2<T>(__uint_as_float(o[8 * j + 2 * x]) * inv,
                                                __uint_as_float(o[8 * j + 2 * x + 1]) * inv);
                            *reinterpret_cast<uint4*>(out + c * 32 + j * 8) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.o_empty[w]);
                if (!k.whole) {
                    slot[2 * CH_ROWS * D + w * CH_ROWS + row] = m_used;
                    slot[2 * CH_ROWS * (D + 1) + w * CH_ROWS + row] = l;
                } else if (valid && p.lse) {
                    p.lse[(int64_t)(k.q.at + tok) * p.Hq + h] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * LN2;
                }
            }
            kvn += 2 * k.n;
            ++seg;
            it += k.n;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 9) {  // copies: Q, then K and V in turn
            int qn = 0, kvn = 0;  // fills of the query ring, and of the key and value ring, so far
            for (; ok && k.begin(p, tpt); k.advance(p, tpt)) {
                {
                    const int st = qn % C::Q_STAGES;
                    ok = ok && __all_sync(~0u, wait_bounded(&s.q_empty[st], (qn / C::Q_STAGES & 1) ^ 1, &s.abort));
                    if (ok) {
                        ++qn;
                        if (lane == 0 && !(qn == 1 && *(volatile int*)&g_hsi_skip_first_copy)) {
                            mbar_arrive_expect_tx(&s.q_full[st], k.tiles * rpt * 128 * (D / 64));
                            for (int i = 0; i < k.tiles * (D / 64); ++i) {
                                const int t = i / (D / 64), half = i % (D / 64);
                                tma_rows_box(q_ring + (st * 2 + t) * C::TILE_BYTES + half * C::HALF_BYTES, &qmap, half * 64,
                                             k.g * p.group, k.q.at + k.tok0 + t * tpt, &s.q_full[st]);
                            }
                        }
                    }
                }
                const int box = p.kv.page_shift < 7 ? 1 << p.kv.page_shift : CH_KEYS;
                const int halves = D / 64, nbox = CH_KEYS / box * halves;
                for (int i = 0; i < k.n && ok; ++i) {
                    const int k0 = (k.tile0 + i) * CH_KEYS, have = min(k.q.len - k0, CH_KEYS);
                    const int live = (have + box - 1) / box * halves;
                    for (int kind = 0; kind < 2 && ok; ++kind) {
                        const int st = kvn % C::KV_STAGES;
                        const int e0 = (lane / halves) * box;
                        int page = lane < nbox && e0 < have ? paged_page(p.kv, k.b, (k0 + e0) >> p.kv.page_shift) : 0;
                        ok = __all_sync(~0u, wait_bounded(&s.kv_empty[st], (kvn / C::KV_STAGES & 1) ^ 1, &s.abort));
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&s.kv_full[st], live * box * 128);
                        __syncwarp();
                        if (lane < nbox && e0 < have)
                            tma_page_box(kv_ring + st * C::TILE_BYTES + (lane % halves) * C::HALF_BYTES + e0 * 128,
                                         kind ? &vmap : &kmap, (lane % halves) * 64,
                                         (k0 + e0) & ((1 << p.kv.page_shift) - 1), k.g,
                                         page, &s.kv_full[st]);
                        ++kvn;
                    }
                }
            }
            if (lane == 0) {  // no copy may be in flight when the block goes
                for (int i = qn > C::Q_STAGES ? qn - C::Q_STAGES : 0; i < qn; ++i)
                    wait_drain(&s.q_full[i % C::Q_STAGES], i / C::Q_STAGES & 1);
                for (int i = kvn > C::KV_STAGES ? kvn - C::KV_STAGES : 0; i < kvn; ++i)
                    wait_drain(&s.kv_full[i % C::KV_STAGES], i / C::KV_STAGES & 1);
            }
        } else if (warp == 8) {  // products: the warp waits, one lane issues
            constexpr uint32_t id_o = idesc_f16(is_bf16<T>, 128, D, true);
            const uint32_t id_s = idesc_f16(is_bf16<T>, 128, CH_KEYS, false) | (p.negate ? 1u << 13 : 0u);  // of -Q
            constexpr uint32_t TILE16 = C::TILE_BYTES >> 4;
            const uint32_t tm = uniform(tmem);
            const uint32_t q_desc = smem_desc_sw128(smem_u32(q_ring)), k_desc = smem_desc_sw128(smem_u32(kv_ring)),
                           v_desc = smem_desc_sw128(smem_u32(kv_ring), C::HALF_BYTES);
            int qst = 0, st = 0;          // the query stage, the stage of the next K or V
            uint32_t qph = 0, ph = 0;     // and their phases
            uint32_t it = 0, seg = 0;     // of row tile w, in bit w: parities of its key tiles and segments so far
            auto product_s = [&](int w) {
                const uint32_t a = uniform(q_desc + (qst * 2 + w) * TILE16), b = uniform(k_desc + st * TILE16);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = ((ks >> 2) * C::HALF_BYTES + (ks & 3) * 32) >> 4;
                        if (ks == 0) mma_f16_ss(tm + w * 128, a, b, id_s);
                        else mma_f16_ss_add(tm + w * 128, a + off, b + off, id_s);
                    }
                    tc_commit(&s.s_full[w]);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) tc_commit(bar);
                __syncwarp();
            };
            auto next = [&]() {
                if (++st == C::KV_STAGES) {
                    st = 0;
                    ph ^= 1;
                }
            };
            for (; k.begin(p, tpt); k.advance(p, tpt)) {
                // S of the first key tile
                ok = wait_bounded(&s.q_full[qst], qph, &s.abort) && wait_bounded(&s.kv_full[st], ph, &s.abort);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                product_s(0);
                if (k.tiles == 2) product_s(1);
                commit(&s.kv_empty[st]);
                if (k.n == 1) commit(&s.q_empty[qst]);
                next();
                for (int i = 0; i < k.n; ++i) {
                    const int vst = st;
                    const uint32_t v = uniform(v_desc + vst * TILE16);
                    const uint32_t more = uniform((uint32_t)i);
                    ok = wait_bounded(&s.kv_full[st], ph, &s.abort);
                    next();  // to the next K
                    auto tile = [&](int w) {
                        if (i == 0) ok = ok && wait_bounded(&s.o_empty[w], (seg >> w & 1) ^ 1, &s.abort);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ok = ok && wait_bounded(&s.p_full[w][h], (it >> w ^ i) & 1, &s.abort);
                            if (!__all_sync(~0u, ok)) return;
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int ks = 4 * h; ks < 4 * h + 4; ++ks) {
                                    const uint32_t d = tm + 256 + w * 128, a = tm + w * 128 + ks * 8;
                                    if (ks == 0) mma_f16_ts(d, a, v, id_o, more);
                                    else mma_f16_ts_add(d, a, v + ks * 128, id_o);
                                }
                            }
                            __syncwarp();
                        }
                        if (i + 1 < k.n) {
                            if (w == 0) ok = wait_bounded(&s.kv_full[st], ph, &s.abort);
                            if (!__all_sync(~0u, ok)) return;
                            tc_fence_after();
                            product_s(w);
                        } else {
                            commit(&s.o_full[w]);
                        }
                    };
                    tile(0);
                    if (k.tiles == 2) tile(1);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    commit(&s.kv_empty[vst]);
                    if (i + 1 < k.n) {
                        commit(&s.kv_empty[st]);
                        if (i + 2 == k.n) commit(&s.q_empty[qst]);
                        next();
                    }
                }
                if (!ok) break;
                if (++qst == C::Q_STAGES) {
                    qst = 0;
                    qph ^= 1;
                }
                const uint32_t both = k.tiles == 2 ? 3 : 1;
                seg ^= both;
                if (k.n & 1) it ^= both;
            }
            if (elect_one()) {
                tc_commit(&s.done);
                wait_drain(&s.done, 0);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// Joins the units that several runs hold, as attend_join_kernel does: a block
// per unit and DIMS dims (fewer where there are few units), a thread per row. Rows that see no entry get
// zeros and lse -inf here.
template <typename T, int D, int DIMS>
__global__ void __launch_bounds__(2 * CH_ROWS)
    attend_chunk_join_kernel(const __grid_constant__ AttendParams p, int grid, int tpt) {
    const int b = blockIdx.z, g = blockIdx.y, row = threadIdx.x, lane = row & 31;
    const int rt = blockIdx.x / (D / DIMS), d0 = blockIdx.x % (D / DIMS) * DIMS;
    // the lengths were there before the kernel that is waited for
    ChunkSeq q;
    q.load(p, b, tpt);
    const int nt = rt < q.n_rt ? q.tiles(p, rt, tpt) : 0;
    uint32_t before = 0;
    for (int i = lane; i < rt; i += 32) before += q.tiles(p, i, tpt);
    before = __reduce_add_sync(~0u, before);
    griddep_wait();
    griddep_launch_dependents();
    if (rt >= q.n_rt) return;
    int c0 = 0, c1 = -1;
    if (nt) {
        const Line line(p.base[p.kv.B], grid);
        const uint32_t s0 = p.base[b] + (p.base[b + 1] - p.base[b]) / p.kv.H * g + before;
        // the runs that the cuts which stayed inside the unit make of it
        const uint32_t snap = chunk_snap(line);
        c0 = line.run(min(s0 + snap, line.total - 1));
        c1 = line.run(max(s0, s0 + nt - min((uint32_t)nt, snap + 1)));
        if (c0 >= c1) return;  // written whole
    }
    const int w = row / CH_ROWS, r = row % CH_ROWS;
    const int tok = rt * 2 * tpt + w * tpt + r / p.group, h = g * p.group + r % p.group;
    if (r >= tpt * p.group || tok >= q.m) return;
    constexpr int SLOT = (int)chunk_slot_floats(D), V = DIMS / 4, AT_ONCE = 16 / V;  // runs whose loads are in flight
    const int runs = c1 - c0 + 1;
    const float* first = p.part + (int64_t)(2 * c0 + 1) * SLOT;
    const float* rest = p.part + (int64_t)2 * c0 * SLOT;  // run i > 0: rest + 2 i SLOT
    float m = -INFINITY, l = 0.f;
    float4 o[V] = {};
    for (int i0 = 0; i0 < runs; i0 += AT_ONCE) {
        float mc[AT_ONCE], lc[AT_ONCE];
        float4 oc[AT_ONCE][V];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int i = i0 + k;
            const float* slot = i ? rest + (int64_t)2 * i * SLOT : first;
            mc[k] = -INFINITY;
            lc[k] = 0.f;
            if (i >= runs) continue;
            mc[k] = slot[2 * CH_ROWS * D + row];
            lc[k] = slot[2 * CH_ROWS * (D + 1) + row];
#pragma unroll
            for (int j = 0; j < V; ++j)
                oc[k][j] = reinterpret_cast<const float4*>(slot)[(d0 / 4 + j) * 2 * CH_ROWS + row];
        }
        float m_new = m;
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) m_new = fmaxf(m_new, mc[k]);
        const float keep = part_factor(m, m_new);
        m = m_new;
        l *= keep;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            o[j].x *= keep;
            o[j].y *= keep;
            o[j].z *= keep;
            o[j].w *= keep;
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            if (lc[k] == 0.f) continue;  // past the runs, or a part that this row does not see
            const float f = part_factor(mc[k], m);
            l += f * lc[k];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j].x += f * oc[k][j].x;
                o[j].y += f * oc[k][j].y;
                o[j].z += f * oc[k][j].z;
                o[j].w += f * oc[k][j].w;
            }
        }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    uint32_t v[2 * V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        v[2 * j] = pack2<T>(o[j].x * inv, o[j].y * inv);
        v[2 * j + 1] = pack2<T>(o[j].z * inv, o[j].w * inv);
    }
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (int64_t)(q.at + tok) * p.ot + (int64_t)h * p.oh + d0);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) out[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    if (d0 == 0 && p.lse) p.lse[(int64_t)(q.at + tok) * p.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

}  // namespace hsi
