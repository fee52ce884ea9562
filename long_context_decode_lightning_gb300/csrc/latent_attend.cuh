// Attention over a latent cache, absorbed form: every query head's key is the
// whole entry and its value the entry's first 512 dims.
//   s_e = scale q.c_e,  out = sum p_e c_e[:512] / sum p_e,  p_e = exp(s_e - max)
// over the entries that a token sees, or those of a list it brings.
//
// A unit is up to 64 rows (row = token * heads + head) over the same entries: a
// token's heads (or an even share of them, at most 64), several tokens of few heads
// where there are no lists. Its entries come in tiles of 64, kept in shared memory
// once, 64 dims of the tile to a chunk, and used twice by the tensor cores:
//   S = Q K^T       64 rows x 64 entries, K-major chunks
//   O^T += V^T P^T  512 dims x 64 rows, the same chunks MN-major
// O is kept transposed, as 64 rows x 512 dims in place take all of tensor
// memory and leave nothing for S: transposed they are four accumulators of 128
// dims by 64 columns. A row's rescaling (lazy, as in attend_chunk.cuh) is one of
// columns then, by all softmax warps together; they agree on it by a vote.
//
// Bytes and products are near balance: an entry of 1152 bytes costs 128 rows 22 ns
// of an SM's tensor rate and 26 ns of its share of HBM. 64 rows cost the tensor
// cores 1920 cycles a tile, which is what shared memory can feed (S 36 products of
// 64 x 64 x 16 at 32 cycles, P V 16 of 128 x 64 x 16 at 48, both measured alone).
//
// Warps: four turn S into P and write results, two issue products (S and P V each
// wait for others, and from one warp each held the other up: 455 us against 417 on
// the prompt below), one looks entries up (lists, pages) up to three tiles ahead, one
// brings the queries, and four bring the entries by 16-byte asynchronous copies, which
// take any address and any order of rows and fill with zeros what is not there (or
// sixteen by loads, decoding FP8 and FP4). The tensor-map gather of four rows was
// measured at 5.0 us a tile and SM from L2 against 0.7 us, one box of 64 rows at 1.6 us.
// P stands in the place of the dims past the value, which S is done with.
//
// The units' tiles form one line that is cut into equal runs, one per CTA; a unit that
// spans runs is joined by a second kernel from fp32 partial sums. Where that would cost
// more than it gains, units go to blocks whole, though SMs may stay idle then (64 lists
// of 512 entries: 88 of 152); latent_whole has the rule and both sides of it.
//
// Measured: 1024 tokens of 64 heads over 2048 listed bf16 entries of 576 each 372 us, 784
// TFLOP/s (41% of the measured burst rate); one token of 16 x 32768 entries at 128 heads 153
// us (3.05 TB/s, 730 TFLOP/s); of 8 x 65536 FP8 entries at 64 heads 117 us (2.3 TB/s). A tile
// of 16-bit entries takes 1.3 to 1.7 us where 1920 cycles are 1.0: two stages leave the chain
// of a stage (its copies 2000 cycles, S 1200 to 2000 beside the other stage's P V, softmax 1000,
// P V until the first dims are free 700) as the bound. One of FP8 entries takes 2.5 us (42 an
// SM in the 117): a stage is decoded after the P V before it, so that decoding is part of the
// chain. A first tile comes 5 us after the start, partial sums leave at 32 bytes a cycle and
// SM (2 us), the join takes 5 to 10 us.
#pragma once
#include <cstdint>

#include "attend.cuh"
#include "attend_chunk.cuh"
#include "common.cuh"
#include "latent.cuh"

namespace hsi {

constexpr int LA_ROWS = 64;   // rows of a unit
constexpr int LA_KEYS = 64;   // entries of a tile
__host__ __device__ constexpr bool latent_plain(int fmt) { return fmt == LF_BF16 || fmt == LF_FP16; }  // copied as they are
// Warps that bring entries: four that copy (eight: 448 us against 435 on chunks, the rest within 2%), or two times eight
// that decode.
__host__ __device__ constexpr int latent_loaders(int fmt) { return latent_plain(fmt) ? 4 : 16; }
__host__ __device__ constexpr int latent_threads(int fmt) { return 32 * (8 + latent_loaders(fmt)); }
constexpr int LA_CHUNK = LA_KEYS * 128;  // bytes of 64 dims of a tile, of a unit's queries, and of P
constexpr int LA_ADDR = 3;    // tiles whose entries are looked up ahead

struct LatentAttendParams {
    LatentView c;
    const void* q;
    int64_t qt, qh;  // token and head strides (elements)
    const int32_t* q_start;
    int64_t T;
    int max_q, max_kv, H;  // host bounds of new tokens and entries; query heads
    int nht, hp, tpt;      // head tiles of a token, heads of one, tokens of a unit
    int inv_hp;            // 2^16 / hp + 1: row / hp is row * inv_hp >> 16 for the rows of a unit
    const int32_t* idx;    // [T][ld_idx], k entries a token, or null
    int64_t ld_idx;
    int k;
    float sl2;             // |scale| * log2(e), above 0
    int causal, negate;    // negate: scale is negative
    void* out;
    int64_t ot, oh;
    float* lse;            // [T][H] or null
    int runs;              // runs that the line is cut into, at most
    int whole, n_rt;       // short form: no unit is split; units of a sequence at most
    int4* desc;            // [runs][nht]: the unit that begins in this run and ends in another: runs, first token, tokens
    float* part;           // partial sums, latent_slot below
};

// floats: four rows of a dim side by side, [row / 4][512][4], then maxima (base 2) and sums
constexpr int LA_SLOT = LA_ROWS * (LT_VALUE + 2);
// A run's partial sums: of a unit that began before it (0) and of one that goes on after it (1).
__device__ __forceinline__ float* latent_slot(const LatentAttendParams& p, int run, int ht, int last) {
    return p.part + (((int64_t)run * 2 + last) * p.nht + ht) * LA_SLOT;
}

// Partial sums of four rows by two dims.
struct LatentSums {
    float m[4], l[4], o[4][2];
    __device__ __forceinline__ LatentSums() {
#pragma unroll
        for (int r = 0; r < 4; ++r) m[r] = -INFINITY, l[r] = o[r][0] = o[r][1] = 0.f;
    }
    // a part: maxima, sums and the two dims of the four rows
    __device__ __forceinline__ void add(const float4& mc, const float4& lc, const float4& a, const float4& b) {
        const float mr[4] = {mc.x, mc.y, mc.z, mc.w}, lr[4] = {lc.x, lc.y, lc.z, lc.w};
        const float ar[4] = {a.x, a.y, a.z, a.w}, br[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (lr[r] == 0.f) continue;  // a part that this row does not see
            const float top = fmaxf(m[r], mr[r]), keep = part_factor(m[r], top), f = part_factor(mr[r], top);
            l[r] = l[r] * keep + lr[r] * f;
            o[r][0] = o[r][0] * keep + ar[r] * f;
            o[r][1] = o[r][1] * keep + br[r] * f;
            m[r] = top;
        }
    }
    // rows row0 .. row0 + 3 of a unit of ntok tokens from tok0 on, dims d and d + 1
    template <typename T>
    __device__ __forceinline__ void store(const LatentAttendParams& p, int tok0, int ntok, int ht, int row0, int d) const {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = (row0 + r) * p.inv_hp >> 16, h = ht * p.hp + row0 + r - i * p.hp;
            if (i >= ntok || h >= p.H) continue;
            const float inv = l[r] > 0.f || l[r] != l[r] ? 1.f / l[r] : 0.f;
            const int64_t t = tok0 + i;
            *reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + t * p.ot + (int64_t)h * p.oh + d) =
                pack2<T>(o[r][0] * inv, o[r][1] * inv);
            if (d == 0 && p.lse) p.lse[t * p.H + h] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * LN2;
        }
    }
};

// Lengths of sequence b and what follows from them.
struct LatentSeq {
    int len, m, at, past, n_rt;
    __device__ __forceinline__ void load(const LatentAttendParams& p, int b) {
        len = latent_len(p.c, b, p.max_kv);
        m = paged_new(p.q_start, b, p.max_q, p.T, &at);
        past = len - m;
        n_rt = (m + p.tpt - 1) / p.tpt;
    }
    // entries that some row of unit rt sees, and tiles of them: one where there are none, so that somebody writes its rows
    __device__ __forceinline__ int seen(const LatentAttendParams& p, int rt) const {
        return p.causal ? max(0, min(len, past + min(m, (rt + 1) * p.tpt))) : len;
    }
    __device__ __forceinline__ int tiles(const LatentAttendParams& p, int rt) const {
        return max(1, (seen(p, rt) + LA_KEYS - 1) / LA_KEYS);
    }
    // tiles of the units before rt (rt <= n_rt)
    __device__ __forceinline__ uint32_t before(const LatentAttendParams& p, int rt) const {
        if (rt == 0) return 0u;
        if (!p.causal) return (uint32_t)rt * tiles(p, 0);
        // unit j - 1 sees past + j tpt entries, the last unit of all len
        uint32_t sum = rt == n_rt ? tiles(p, rt - 1) : 0u;
        const int n = rt == n_rt ? rt - 1 : rt;
        const int none = past >= 0 ? 0 : min(n, -past / p.tpt);  // see nothing: a tile each
        sum += none;
        // sum over j of ceil((past + j tpt) / 64) for j = none + 1 .. n: the sum of (a j + b) less that of its
        // residues, which go round the multiples of a's power of two
        const int a = p.tpt, g = a & -a, sh = 6 - (__ffs(g) - 1), per = 1 << sh;  // per = 64 / g
        const uint64_t cnt = n - none, b = (uint64_t)(past + (int64_t)(none + 1) * a + LA_KEYS - 1);
        uint64_t all = b * cnt + (cnt ? cnt * (cnt - 1) / 2 : 0) * a;
        all -= (cnt >> sh) * (uint64_t)(per * (int)(b & (g - 1)) + LA_KEYS / 2 * (per - 1));
        for (uint32_t i = (uint32_t)cnt & ~(per - 1u); i < (uint32_t)cnt; ++i) all -= ((uint32_t)b + i * a) & (LA_KEYS - 1);
        return sum + (uint32_t)(all / LA_KEYS);
    }
};

// A walk along a block's run of the line: segment by segment, each a unit or the part of one that the run holds.
// Whole warps.
struct LatentWalk {
    int left, b, rt, tile0;  // with lists rt is the token
    LatentSeq q;
    int n, nt, tok0, ntok;   // tiles of the segment and of the unit; its first token and its tokens
    int seen;                // entries that some row of the unit sees

    __device__ __forceinline__ bool begin(const LatentAttendParams& p) {
        if (p.idx) {
            for (;; left -= n, tile0 = 0, ++rt) {
                if (left <= 0) return false;
                nt = (p.k + LA_KEYS - 1) / LA_KEYS;
                n = min(left, nt - tile0);
                int32_t first, past;
                b = token_seq_warp(p.q_start, p.c.B, rt, p.T, &first, &past);
                if (b < 0) continue;  // a token of no sequence: its tiles are passed over
                q.len = latent_len(p.c, b, p.max_kv);
                q.past = q.len - (past - rt);
                seen = p.causal ? max(0, min(q.len, q.past + 1)) : q.len;
                tok0 = rt;
                ntok = 1;
                return true;
            }
        }
        if (left <= 0) return false;
        nt = q.tiles(p, rt);
        n = min(left, nt - tile0);
        seen = q.seen(p, rt);
        tok0 = q.at + rt * p.tpt;
        ntok = min(p.tpt, q.m - rt * p.tpt);
        return true;
    }
    __device__ __forceinline__ void advance(const LatentAttendParams& p) {
        left -= n;
        tile0 = 0;
        if (left <= 0) return;
        ++rt;
        if (p.idx || rt < q.n_rt) return;
        rt = 0;
        do q.load(p, ++b);  // there are tiles left, so a sequence that has some follows
        while (q.n_rt == 0 && b + 1 < p.c.B);
    }
    __device__ __forceinline__ bool whole() const { return tile0 == 0 && n == nt; }
    // entries that the unit's token i sees
    __device__ __forceinline__ int sees(const LatentAttendParams& p, int i) const {
        return p.idx ? seen : p.causal ? max(0, min(q.len, q.past + rt * p.tpt + i + 1)) : q.len;
    }
};

template <int DIM, int FMT>
struct LatentCfg {
    static constexpr int CHUNKS = DIM / 64, PAIRS = LT_VALUE / 128;
    // a stage holds a tile: eight chunks of the value, then one of the dims past it, in whose place P comes once S is done
    static constexpr int STAGE_BYTES = (2 * PAIRS + 1) * LA_CHUNK, P_OFF = 2 * PAIRS * LA_CHUNK;
    static constexpr int KV_OFF = CHUNKS * LA_CHUNK, RING_BYTES = KV_OFF + 2 * STAGE_BYTES;
    // S is issued by groups of chunks: as soon as half of a tile's dims are there; decoded tiles come whole
    static constexpr int GROUPS = latent_plain(FMT) ? 2 : 1, GROUP = (CHUNKS + GROUPS - 1) / GROUPS;
    __host__ __device__ static constexpr int in_group(int g) { return g + 1 < GROUPS ? GROUP : CHUNKS - g * GROUP; }
    struct Tail {
        uint64_t q_full, q_empty, s_full[2], p_full[2], o_empty, done[2];
        uint64_t full[2][GROUPS];      // the entries' dims of a group are there
        uint64_t empty[2][PAIRS];      // 128 dims of a tile have been used (with the last: all of it, and O is at rest)
        uint64_t addr_full[LA_ADDR], addr_empty[LA_ADDR];
        const uint8_t* entry[LA_ADDR][LA_KEYS];  // null: no such entry
        uint32_t live[LA_ADDR][2];     // entries that there are
        int end[LA_ADDR];              // no tile follows
        int64_t row_out[LA_ROWS];      // where a row's result goes (elements), -1: nowhere
        float factor[LA_ROWS];
        uint32_t vote[2][4];
        uint32_t tmem, total;
        int abort;
        int none;                      // q_start descends: no tile is this block's
        int left, b, rt, tile;         // this block's run: tiles, and where it starts
        LatentSeq q;
    };
    static constexpr int SMEM_BYTES = RING_BYTES + (int)sizeof(Tail);
    static_assert(SMEM_BYTES <= 232448, "shared memory of an SM");
};

// Accumulators' columns of tensor memory: O^T in four of 64, S in two of 64.
constexpr uint32_t LA_S_COL = 256;

// 64 columns of 16 lanes, as matrix fragments: register 4 g + 2 h + x is column 8 g + 2 (lane & 3) + x of row
// (lane >> 2) + 8 h.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
    tmem_ld_wait(r);
}

__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Loads that stay where they are written, far ahead of their use (the compiler would move them down to it).
__device__ __forceinline__ uint4 load_ahead16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t load_ahead1(const void* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t load_ahead2(const void* p) {
    uint16_t v;
    asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

// 16 bytes into shared memory without waiting, zeros where src is null.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, const void* any) {
    const int bytes = src ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src ? src : any), "r"(bytes) : "memory");
}
// An arrival on `bar` once all copies of this thread so far are there.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The line: its length, then where this block's run starts. One warp.
template <typename Tail>
__device__ __forceinline__ void latent_line(const LatentAttendParams& p, int run, Tail& s) {
    const int lane = threadIdx.x & 31;
    if (p.idx) {
        const uint32_t nt = (p.k + LA_KEYS - 1) / LA_KEYS;
        const Line line((uint32_t)p.T * (p.whole ? 1 : nt), p.runs);
        if (lane == 0) {
            s.total = line.total;
            const uint32_t x = line.cut(run);
            s.left = run < (int)line.G ? (int)(line.cut(run + 1) - x) * (p.whole ? nt : 1) : 0;
            s.rt = p.whole ? x : x / nt;
            s.tile = p.whole ? 0 : x % nt;
        }
        return;
    }
    if (p.whole) {  // a unit a block
        LatentSeq q;
        const int b = run / p.n_rt, rt = run % p.n_rt;
        q.load(p, b);
        if (lane == 0) {
            s.left = rt < q.n_rt ? q.tiles(p, rt) : 0;
            s.b = b;
            s.rt = rt;
            s.tile = 0;
            s.q = q;
        }
        return;
    }
    LatentSeq mine;
    const auto load = [&](int b0) {  // tiles of sequence b0 + lane
        mine.n_rt = 0;
        if (b0 + lane < p.c.B) mine.load(p, b0 + lane);
        return mine.n_rt ? mine.before(p, mine.n_rt) : 0u;
    };
    const auto upto = [&](uint32_t n) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(~0u, n, o);
            if (lane >= o) n += up;
        }
        return n;
    };
    uint32_t total = 0, n = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        n = load(b0);
        total += __reduce_add_sync(~0u, n);
    }
    const Line line(total, p.runs);
    const uint32_t x = line.cut(run);
    if (lane == 0) {
        s.total = total;
        s.left = run < (int)line.G ? (int)(line.cut(run + 1) - x) : 0;
    }
    if (run >= (int)line.G) return;
    uint32_t first = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        if (p.c.B > 32) n = load(b0);
        const uint32_t sum = upto(n), f = first + sum - n;
        const uint32_t has = __ballot_sync(~0u, x >= f && x < f + n);
        first += __shfl_sync(~0u, sum, 31);
        if (!has) continue;
        const int at = __ffs(has) - 1;
        LatentSeq q;
        q.len = __shfl_sync(~0u, mine.len, at);
        q.m = __shfl_sync(~0u, mine.m, at);
        q.at = __shfl_sync(~0u, mine.at, at);
        q.past = __shfl_sync(~0u, mine.past, at);
        q.n_rt = __shfl_sync(~0u, mine.n_rt, at);
        const uint32_t off = x - __shfl_sync(~0u, f, at);
        // the last unit that starts at or before the tile, by 32 guesses at a time
        int lo = 0, hi = q.n_rt;  // before(lo) <= off < before(hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, guess = lo + step * lane;
            const uint32_t ok = __ballot_sync(~0u, guess < hi && (lane == 0 || q.before(p, guess) <= off));
            lo += step * (31 - __clz(ok));
            hi = min(hi, lo + step);
        }
        const uint32_t start = q.before(p, lo);
        if (lane == 0) {
            s.b = b0 + at;
            s.rt = lo;
            s.tile = (int)(off - start);
            s.q = q;
        }
        return;
    }
}

// Whether q_start descends (which paged_new reports). Sequences claim the same tokens then: more units than tokens,
// which the host's bounds do not cover, and two results for a row; so that no row is written without lists. A warp other
// than that which looks for the run's start (nine sequences of 8191 entries, four tokens each: 34.8 us without the look,
// 35.0 with it, 36.3 where that warp has it among its lengths).
__device__ __forceinline__ bool latent_falls(const LatentAttendParams& p) {
    bool falls = false;
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < p.c.B; i += 32) falls = falls || __ldg(p.q_start + i) > __ldg(p.q_start + i + 1);
    return __any_sync(~0u, falls);
}

template <typename T, int DIM, int FMT>
__global__ void __launch_bounds__(latent_threads(FMT), 1) latent_attend_kernel(const __grid_constant__ LatentAttendParams p) {
    using C = LatentCfg<DIM, FMT>;
    extern __shared__ __align__(1024) uint8_t ring[];
    typename C::Tail& s = *reinterpret_cast<typename C::Tail*>(ring + C::RING_BYTES);
    uint8_t* const q_smem = ring;
    uint8_t* const kv_smem = ring + C::KV_OFF;
    // (put into a uniform register, so that the roles' code is known not to part a warp's lanes)
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int run = blockIdx.x / p.nht, ht = blockIdx.x % p.nht;
    constexpr int LOADERS = latent_loaders(FMT);
    constexpr bool PLAIN = latent_plain(FMT);

    if (threadIdx.x == 0) {
        mbar_init(&s.q_full, 32), mbar_init(&s.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.s_full[i], 1), mbar_init(&s.p_full[i], 4);
            for (int g = 0; g < C::GROUPS; ++g) mbar_init(&s.full[i][g], PLAIN ? 32 * C::in_group(g) : LOADERS / 2);
            for (int c = 0; c < C::PAIRS; ++c) mbar_init(&s.empty[i][c], 1);
        }
        mbar_init(&s.o_empty, 4);
        for (int i = 0; i < LA_ADDR; ++i) mbar_init(&s.addr_full[i], 1), mbar_init(&s.addr_empty[i], 4 + (PLAIN ? LOADERS : LOADERS / 2));
        mbar_init(&s.done[0], 1), mbar_init(&s.done[1], 1);
        fence_mbar_init();
        s.abort = 0;
    }
    if (warp == 4) tmem_alloc(&s.tmem, 512);
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x == 0 && !p.whole) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (warp == 0) latent_line(p, run, s);
    if (warp == 1) {
        const bool none = !p.idx && latent_falls(p);
        if (lane == 0) s.none = none;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    LatentWalk k;
    k.left = s.none ? 0 : s.left;
    k.b = s.b;
    k.rt = s.rt;
    k.tile0 = s.tile;
    k.q = s.q;
    bool ok = true;  // false once a wait has run out: the role ends, after what it has in flight

    if (warp < 4) {  // softmax: rows ra and ra + 8, a quarter of their columns each lane
        constexpr float SHIFT = P_SHIFT<T> ? P_SHIFT<T> - CH_LAZY : 0.f;  // p up to 2^CH_LAZY of its own
        const int ra = 16 * warp + (lane >> 2), c0 = 2 * (lane & 3);
        const uint32_t quarter = (uint32_t)(warp * 32) << 16;
        uint32_t it = 0, seg = 0, votes = 0;  // tiles, segments and votes so far
        // The four warps come together, each with a wait that it has won or lost and a question: whether all have won
        // (they go on or leave together, so that none stays behind at the barrier), and in *any whether one says yes.
        const auto vote = [&](bool yes, bool* any) {
            const uint32_t mine = (__any_sync(~0u, yes) ? 1u : 0u) | (ok ? 0u : 2u);
            uint32_t* const all = s.vote[votes++ & 1];
            if (lane == 0) all[warp] = mine;
            bar_sync(1, 128);
            const uint32_t sum = all[0] | all[1] | all[2] | all[3];
            *any = __any_sync(~0u, sum & 1u);
            ok = !__any_sync(~0u, sum & 2u);
            return ok;
        };
        bool any;
        for (; __all_sync(~0u, ok && k.begin(p)); k.advance(p), ++seg) {
            const int n = (int)uniform(k.n);
            if (threadIdx.x < LA_ROWS) {
                const int i = (int)threadIdx.x * p.inv_hp >> 16, h = ht * p.hp + threadIdx.x - i * p.hp;
                s.row_out[threadIdx.x] = i < k.ntok && h < p.H ? (int64_t)(k.tok0 + i) * p.ot + (int64_t)h * p.oh : -1;
            }
            int lim[2];
            float m_used[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = (ra + 8 * h) * p.inv_hp >> 16;
                lim[h] = p.idx ? INT32_MAX : k.sees(p, min(i, k.ntok - 1));
            }
            const int lim_all = p.idx ? INT32_MAX : k.sees(p, 0);  // entries that every row sees
            for (int i = 0; i < n; ++i, ++it) {
                const int k0 = (k.tile0 + i) * LA_KEYS, a = it % LA_ADDR;
                ok = ok && __all_sync(~0u, wait_bounded(&s.addr_full[a], it / LA_ADDR & 1, &s.abort) &&
                                         wait_bounded(&s.s_full[it & 1], it / 2 & 1, &s.abort));
                const uint32_t live[2] = {s.live[a][0], s.live[a][1]};
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.addr_empty[a]);
                __syncwarp();
                tc_fence_after();
                uint32_t r[32];
                tmem_ld_16x64(tmem + quarter + LA_S_COL + (it & 1) * LA_KEYS, r);
                if ((live[0] & live[1]) != ~0u || k0 + LA_KEYS > lim_all) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int col = 8 * (j >> 2) + c0 + (j & 1);
                        const bool sees = (live[j >> 4] >> (col & 31) & 1) && (p.idx || k0 + col < lim[j >> 1 & 1]);
                        r[j] = sees ? r[j] : 0xFF800000u;
                    }
                }
                float mt[2];
                bool grew = false;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float top = fmaxf(__uint_as_float(r[2 * h]), __uint_as_float(r[2 * h + 1]));
#pragma unroll
                    for (int g = 1; g < 8; ++g)
                        top = max3(top, __uint_as_float(r[4 * g + 2 * h]), __uint_as_float(r[4 * g + 2 * h + 1]));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    mt[h] = top * p.sl2;  // p.sl2 > 0
                    grew = grew || mt[h] > m_used[h] + CH_LAZY;
                }
                // a row whose maximum has grown: all warps rescale O's columns, as each holds all rows of its dims
                bool some;
                if (!vote(grew, &some)) break;
                if (some) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float m_new = mt[h] > m_used[h] + CH_LAZY ? mt[h] : m_used[h];
                        const float f = m_new == -INFINITY ? 1.f : ex2(m_used[h] - m_new);
                        l[h] *= f;
                        m_used[h] = m_new;
                        if ((lane & 3) == 0) s.factor[ra + 8 * h] = f;
                    }
                }
                uint32_t pk[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float base = m_used[h] == -INFINITY ? 0.f : m_used[h] - SHIFT;
                    float sum = 0.f;
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        const float x = ex2(fmaf(__uint_as_float(r[4 * g + 2 * h]), p.sl2, -base));
                        const float y = ex2(fmaf(__uint_as_float(r[4 * g + 2 * h + 1]), p.sl2, -base));
                        sum += x + y;
                        pk[2 * g + h] = pack2<T>(x, y);
                    }
                    l[h] += sum;
                }
                if (some) {
                    // O is at rest once the last tile's product is done
                    if (i > 0) ok = __all_sync(~0u, wait_bounded(&s.empty[(it & 1) ^ 1][C::PAIRS - 1], (it - 1) / 2 & 1, &s.abort));
                    if (!vote(false, &any)) break;
                    if (i > 0) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[32];
                            tmem_ld32_issue(tmem + quarter + c * 32, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                o[j] = __float_as_uint(__uint_as_float(o[j]) * s.factor[(c & 1) * 32 + j]);
                            tmem_st32(tmem + quarter + c * 32, o);
                        }
                        tmem_st_wait();
                    }
                    if (!vote(false, &any)) break;  // the factors have been read
                }
                const int row = 16 * warp + (lane & 15), g1 = lane >> 4;
                const uint32_t dst = smem_u32(kv_smem) + (it & 1) * C::STAGE_BYTES + C::P_OFF + row * 128;
#pragma unroll
                for (int g = 0; g < 8; g += 2)
                    stmatrix_x4(dst + (((g + g1) ^ (row & 7)) << 4), pk[2 * g], pk[2 * g + 1], pk[2 * g + 2], pk[2 * g + 3]);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full[it & 1]);
                __syncwarp();
            }
            if (!vote(false, &any)) break;  // (a warp may have lost its last wait)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(~0u, l[h], 1);
                l[h] += __shfl_xor_sync(~0u, l[h], 2);
                m_used[h] -= SHIFT;  // what the sums are by
                if ((lane & 3) == 0) s.factor[ra + 8 * h] = l[h] > 0.f || l[h] != l[h] ? 1.f / l[h] : 0.f;
            }
            const bool whole = k.whole();
            float* slot = latent_slot(p, run, ht, k.tile0 == 0);
            if (!whole && k.tile0 == 0 && threadIdx.x == 0) {  // the unit goes on in later runs
                const Line line(s.total, p.runs);
                const int last = (int)line.run(line.cut(run + 1) + (k.nt - k.n) - 1);
                p.desc[blockIdx.x] = make_int4(last - run + 1, k.tok0, k.ntok, 0);
            }
            ok = __all_sync(~0u, wait_bounded(&s.empty[(it - 1) & 1][C::PAIRS - 1], (it - 1) / 2 & 1, &s.abort));
            if (!vote(false, &any)) break;  // factors and rows are there
            tc_fence_after();
            if ((lane & 3) == 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = ra + 8 * h;
                    if (!whole) {
                        slot[LA_ROWS * LT_VALUE + row] = m_used[h];
                        slot[LA_ROWS * (LT_VALUE + 1) + row] = l[h];
                    } else if (p.lse && s.row_out[row] >= 0) {
                        const int i = row * p.inv_hp >> 16;
                        p.lse[(int64_t)(k.tok0 + i) * p.H + ht * p.hp + row - i * p.hp] =
                            l[h] == 0.f ? -INFINITY : (m_used[h] + log2f(l[h])) * LN2;
                    }
                }
            }
            const int rows = k.ntok * p.hp;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                const int col0 = (c & 1) * 32, d = (c >> 1) * 128 + warp * 32 + lane;
                if (col0 >= rows) continue;
                __syncwarp();
                uint32_t o[32];
                tmem_ld32_issue(tmem + quarter + c * 32, o);
                tmem_ld_wait(o);
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        if (col0 + j < rows)
                            reinterpret_cast<uint4*>(slot)[(col0 + j) / 4 * LT_VALUE + d] =
                                make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                } else {
                    // two rows at a time: an even lane stores two dims of the first, an odd one of the second
                    T* const out = static_cast<T*>(p.out) + (d & ~1);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float x = __uint_as_float(o[j]) * s.factor[col0 + j];
                        const float y = __uint_as_float(o[j + 1]) * s.factor[col0 + j + 1];
                        const float z = __shfl_xor_sync(~0u, lane & 1 ? x : y, 1);
                        const uint32_t v = lane & 1 ? pack2<T>(z, y) : pack2<T>(x, z);
                        const int64_t to = s.row_out[col0 + j + (lane & 1)];
                        if (to >= 0) *reinterpret_cast<uint32_t*>(out + to) = v;
                    }
                }
            }
            tc_fence_before();
            if (!vote(false, &any)) break;  // rows and factors have been read
            if (lane == 0) mbar_arrive(&s.o_empty);
        }
    } else if (warp == 4) {  // S: the warp waits, one lane issues
        const uint32_t id_s = idesc_f16(is_bf16<T>, LA_ROWS, LA_KEYS, false) | (p.negate ? 1u << 13 : 0u);  // of -Q
        constexpr uint32_t CHUNK16 = LA_CHUNK >> 4, STAGE16 = C::STAGE_BYTES >> 4;
        const uint32_t q_desc = uniform(smem_desc_sw128(smem_u32(q_smem))), tm = uniform(tmem),
                       k_desc = uniform(smem_desc_sw128(smem_u32(kv_smem)));
        uint32_t it = 0, seg = 0;  // tiles and segments so far
        for (; __all_sync(~0u, ok && k.begin(p)); k.advance(p), ++seg) {
            const int n = (int)uniform(k.n);
            ok = __all_sync(~0u, wait_bounded(&s.q_full, seg & 1, &s.abort));
            for (int i = 0; i < n && __all_sync(~0u, ok); ++i, ++it) {
                // a stage is filled again when its last tile's P V is done, so its S has been read, too
                const uint32_t st = it & 1, d = tm + LA_S_COL + st * LA_KEYS, kd = k_desc + st * STAGE16;
                const bool end = i + 1 == n;
#pragma unroll
                for (int g = 0; g < C::GROUPS; ++g) {
                    ok = ok && wait_bounded(&s.full[st][g], it / 2 & 1, &s.abort);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    fence_proxy_async_smem();  // copies of other warps, then the tensor cores
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < C::in_group(g) * 4; ++x) {
                            const uint32_t off = (g * C::GROUP + (x >> 2)) * CHUNK16 + (x & 3) * 2;
                            if (g == 0 && x == 0) mma_f16_ss(d, q_desc, kd, id_s);
                            else mma_f16_ss_add(d, q_desc + off, kd + off, id_s);
                        }
                        if (g + 1 == C::GROUPS) {
                            tc_commit(&s.s_full[st]);
                            if (end) tc_commit(&s.q_empty);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (elect_one()) {
            tc_commit(&s.done[0]);
            wait_drain(&s.done[0], 0);
        }
    } else if (warp == 6) {  // P V, from a warp of its own: each issues while the other waits
        constexpr uint32_t id_o = idesc_f16(is_bf16<T>, 128, LA_ROWS, false) | 1u << 15;  // A = V^T, MN-major
        constexpr uint32_t CHUNK16 = LA_CHUNK >> 4, STAGE16 = C::STAGE_BYTES >> 4;
        const uint32_t tm = uniform(tmem), v_desc = uniform(smem_desc_sw128(smem_u32(kv_smem), LA_CHUNK)),
                       p_desc = uniform(smem_desc_sw128(smem_u32(kv_smem) + C::P_OFF));
        uint32_t it = 0, seg = 0;
        for (; __all_sync(~0u, ok && k.begin(p)); k.advance(p), ++seg) {
            const int n = (int)uniform(k.n);
            ok = __all_sync(~0u, wait_bounded(&s.o_empty, (seg & 1) ^ 1, &s.abort));
            for (int i = 0; i < n && __all_sync(~0u, ok); ++i, ++it) {
                const uint32_t st = it & 1, vd = v_desc + st * STAGE16, pd = p_desc + st * STAGE16, more = i;
                ok = __all_sync(~0u, wait_bounded(&s.p_full[st], it / 2 & 1, &s.abort));
                if (!ok) break;
                fence_proxy_async_smem();  // the entries' copies as well, which the softmax of their S came after
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int m = 0; m < C::PAIRS; ++m) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint32_t a = vd + 2 * m * CHUNK16 + ks * 128, b = pd + ks * 2;
                            if (ks == 0) mma_f16_ss_acc(tm + m * 64, a, b, id_o, more);
                            else mma_f16_ss_add(tm + m * 64, a, b, id_o);
                        }
                        tc_commit(&s.empty[st][m]);
                    }
                }
                __syncwarp();
            }
        }
        if (elect_one()) {
            tc_commit(&s.done[1]);
            wait_drain(&s.done[1], 0);
        }
    } else if (warp == 5) {  // entries: where the tiles' rows are
        uint32_t it = 0;
        for (; __all_sync(~0u, ok && k.begin(p)); k.advance(p)) {
            const int n = (int)uniform(k.n);
            for (int i = 0; i < n && __all_sync(~0u, ok); ++i, ++it) {
                const int k0 = (k.tile0 + i) * LA_KEYS, a = it % LA_ADDR;
                const uint8_t* at[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int j = k0 + 32 * h + lane;
                    int e = j < k.seen ? j : -1;
                    if (p.idx) {
                        e = j < p.k ? __ldg(p.idx + (int64_t)k.tok0 * p.ld_idx + j) : -1;
                        if (e >= k.seen) {
                            raise_error(DEVERR_ARG);
                            e = -1;
                        }
                    }
                    at[h] = e >= 0 ? latent_entry(p.c, k.b, e) : nullptr;
                }
                ok = __all_sync(~0u, wait_bounded(&s.addr_empty[a], (it / LA_ADDR & 1) ^ 1, &s.abort));
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s.entry[a][32 * h + lane] = at[h];
                    const uint32_t live = __ballot_sync(~0u, at[h] != nullptr);
                    if (lane == 0) s.live[a][h] = live;
                }
                if (lane == 0) s.end[a] = 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.addr_full[a]);
            }
        }
        for (int i = 0; ok && i < 2; ++i, ++it) {  // two ends: the loaders of even and odd tiles look for one each
            const int a = it % LA_ADDR;
            ok = __all_sync(~0u, wait_bounded(&s.addr_empty[a], (it / LA_ADDR & 1) ^ 1, &s.abort));
            if (ok && lane == 0) {
                s.end[a] = 1;
                mbar_arrive(&s.addr_full[a]);
            }
            __syncwarp();
        }
    } else if (warp == 7) {  // queries, a unit at a time
        const T* const q = static_cast<const T*>(p.q);
        uint32_t seg = 0;
        for (; __all_sync(~0u, ok && k.begin(p)); k.advance(p), ++seg) {
            ok = __all_sync(~0u, wait_bounded(&s.q_empty, (seg & 1) ^ 1, &s.abort));
            if (!ok) break;
            const int r0 = lane >> 3, j = lane & 7;
#pragma unroll 4
            for (int x = 0; x < LA_ROWS / 4; ++x) {
                const int r = 4 * x + r0, i = r * p.inv_hp >> 16, h = ht * p.hp + r - i * p.hp;
                const T* src = i < k.ntok && h < p.H ? q + (int64_t)(k.tok0 + i) * p.qt + (int64_t)h * p.qh + 8 * j : nullptr;
                const uint32_t dst = smem_u32(q_smem) + r * 128 + ((j ^ (r & 7)) << 4);
#pragma unroll
                for (int c = 0; c < C::CHUNKS; ++c) cp_async16(dst + c * LA_CHUNK, src ? src + c * 64 : nullptr, q);
            }
            if (!(seg == 0 && *(volatile int*)&g_hsi_skip_first_copy)) cp_async_arrive(&s.q_full);
        }
        cp_async_wait_all();
    } else {  // entries' values
        const int w = warp - 8;
        uint32_t it = 0;
        if constexpr (PLAIN) {
            uint32_t n = 0;  // chunks so far: the warps take them in turn
            for (;; ++it) {
                const int a = it % LA_ADDR, st = it & 1;
                ok = __all_sync(~0u, wait_bounded(&s.addr_full[a], it / LA_ADDR & 1, &s.abort));
                if (__any_sync(~0u, !ok || s.end[a])) break;
                const uint8_t* e[LA_KEYS / 4];  // of rows 4 x + lane / 8, this lane's 16 bytes of a chunk
#pragma unroll
                for (int x = 0; x < LA_KEYS / 4; ++x) {
                    e[x] = s.entry[a][4 * x + (lane >> 3)];
                    if (e[x]) e[x] += (lane & 7) * 16;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.addr_empty[a]);
#pragma unroll 1
                for (int c = 0; c < C::CHUNKS; ++c, ++n) {
                    if ((int)(n % LOADERS) != w) continue;
                    ok = __all_sync(~0u, wait_bounded(&s.empty[st][min(c >> 1, C::PAIRS - 1)], (it / 2 & 1) ^ 1, &s.abort));
                    if (!ok) break;
                    const uint32_t dst = smem_u32(kv_smem) + st * C::STAGE_BYTES + c * LA_CHUNK + (lane >> 3) * 128;
#pragma unroll
                    for (int x = 0; x < LA_KEYS / 4; ++x) {
                        cp_async16(dst + x * 512 + (((lane & 7) ^ (lane >> 3) ^ (x & 1) * 4) << 4),
                                   e[x] ? e[x] + c * 128 : nullptr, p.c.data);
                    }
                    cp_async_arrive(&s.full[st][c / C::GROUP]);
                }
                if (!ok) break;
            }
            cp_async_wait_all();
        } else {
            // Eight warps take the even tiles and eight the odd ones: a tile's loads are all issued, then waited for,
            // while the other half decodes. (Loads for the next tile among the steps of this one, by eight warps,
            // were waited for at every step: a warp has few counters of loads in flight, and waits for all on one.)
            // A warp takes eight whole rows, 512 bytes of one row (FP4: 256 of two) to a load: a row is no multiple of
            // 128 bytes, so that 128 bytes of four rows each were eight lines and twelve turns of the data path.
            const int half = w >> 3, r0 = (w & 7) * 8, st = half;
            constexpr int CODES = FMT == LF_FP8 ? DIM - LT_TAIL : DIM;
            constexpr int R = FMT == LF_FP8 ? 8 : 4;  // loads of codes
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t base = smem_u32(kv_smem) + st * C::STAGE_BYTES;
            const auto put = [&](int r, int m, const uint32_t (&o)[4]) {  // eight values from dim m on
                const uint32_t dst = base + (m >> 6) * LA_CHUNK + r * 128 + (((m >> 3 & 7) ^ (r & 7)) << 4);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                             : "memory");
            };
            for (it = half;; it += 2) {
                const int a = it % LA_ADDR;
                ok = __all_sync(~0u, wait_bounded(&s.addr_full[a], it / LA_ADDR & 1, &s.abort));
                if (__any_sync(~0u, !ok || s.end[a])) break;
                uint4 v[R], tail[2];
                uint32_t scale[R];
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    if constexpr (FMT == LF_FP8) {
                        const uint8_t* const e = lane < CODES / 16 ? s.entry[a][r0 + x] : nullptr;
                        v[x] = e ? load_ahead16(e + 16 * lane) : zero;
                        scale[x] = e ? load_ahead1(e + CODES + 2 * LT_TAIL + (lane >> 2)) : 0u;
                    } else {
                        const uint8_t* const e = s.entry[a][r0 + 2 * x + (lane >> 4)];
                        v[x] = e ? load_ahead16(e + 16 * (lane & 15)) : zero;
                        scale[x] = e ? load_ahead2(e + 256 + 2 * (lane & 15)) : 0u;
                    }
                }
                if constexpr (FMT == LF_FP8)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint8_t* const e = s.entry[a][r0 + 4 * y + (lane >> 3)];
                        tail[y] = e ? load_ahead16(e + CODES + 16 * (lane & 7)) : zero;
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.addr_empty[a]);
                // the whole stage: a row has all its dims
                ok = __all_sync(~0u, wait_bounded(&s.empty[st][C::PAIRS - 1], (it / 2 & 1) ^ 1, &s.abort));
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    uint32_t o[4];
                    if constexpr (FMT == LF_FP8) {
                        if (lane < CODES / 16) {
                            // lanes of odd chunks store their halves the other way round: eight lanes reach all banks
                            const bool swap = lane & 4;
                            const uint2 lo = make_uint2(v[x].x, v[x].y), hi = make_uint2(v[x].z, v[x].w);
                            decode8_fp8(swap ? hi : lo, scale[x], o);
                            put(r0 + x, 16 * lane + (swap ? 8 : 0), o);
                            decode8_fp8(swap ? lo : hi, scale[x], o);
                            put(r0 + x, 16 * lane + (swap ? 0 : 8), o);
                        }
                    } else {
                        // (here the four parts of a lane go round by its chunk)
                        const int c = lane >> 1 & 3, r = r0 + 2 * x + (lane >> 4), m = 32 * (lane & 15);
                        const uint32_t s0 = e4m3_pair(scale[x] & 0xFFu), s1 = e4m3_pair(scale[x] >> 8);
                        const uint32_t p0 = c & 2 ? v[x].z : v[x].x, p1 = c & 2 ? v[x].w : v[x].y;
                        const uint32_t p2 = c & 2 ? v[x].x : v[x].z, p3 = c & 2 ? v[x].y : v[x].w;
                        const uint32_t lo = c & 2 ? s1 : s0, hi = c & 2 ? s0 : s1;
                        decode8_fp4(c & 1 ? p1 : p0, lo, o);
                        put(r, m + 8 * c, o);
                        decode8_fp4(c & 1 ? p0 : p1, lo, o);
                        put(r, m + 8 * (c ^ 1), o);
                        decode8_fp4(c & 1 ? p3 : p2, hi, o);
                        put(r, m + 8 * (c ^ 2), o);
                        decode8_fp4(c & 1 ? p2 : p3, hi, o);
                        put(r, m + 8 * (c ^ 3), o);
                    }
                }
                if constexpr (FMT == LF_FP8)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t t[4] = {tail[y].x, tail[y].y, tail[y].z, tail[y].w};
                        put(r0 + 4 * y + (lane >> 3), CODES + 8 * (lane & 7), t);
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane < C::GROUPS) mbar_arrive(&s.full[st][lane]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, 512);
}

// Joins the units that several runs hold: a block per run, head tile, four rows and 512 / G dims, two dims a thread;
// its G groups of threads take every G-th part and are joined through shared memory. G = 8 where units are few and
// of many parts. Bound by latency: two parts' loads in flight at four blocks an SM beat four at two (nine units of 17
// parts: 5 us less), one at six and three at three.
constexpr int LJ_THREADS = 256;
template <typename T, int G>
__global__ void __launch_bounds__(LJ_THREADS, 4) latent_join_kernel(const __grid_constant__ LatentAttendParams p) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int PER = LJ_THREADS / G;
    const int row0 = blockIdx.x / G * 4;
    int at = blockIdx.y;  // the unit's place in desc
    if constexpr (G > 1) {  // few units: block y takes the y-th that there is
        const int lane = threadIdx.x & 31, places = p.runs * p.nht;
        int left = at;
        at = -1;
        for (int i0 = 0; i0 < places && at < 0; i0 += 160) {
            bool is[5];
#pragma unroll
            for (int x = 0; x < 5; ++x) is[x] = i0 + 32 * x + lane < places && p.desc[i0 + 32 * x + lane].x != 0;
#pragma unroll
            for (int x = 0; x < 5; ++x) {
                uint32_t has = __ballot_sync(~0u, is[x]);
                const int n = __popc(has);
                if (at < 0 && left < n) {
                    for (; left > 0; --left) has &= has - 1;
                    at = i0 + 32 * x + __ffs(has) - 1;
                }
                left -= n;
            }
        }
        if (at < 0) return;
    }
    const int run = at / p.nht, ht = at % p.nht;
    const int g = threadIdx.x / PER, t = threadIdx.x % PER, d = 2 * (blockIdx.x % G * PER + t);
    const int4 unit = p.desc[at];
    if (unit.x == 0 || row0 >= unit.z * p.hp) return;
    constexpr int AT_ONCE = 2;  // parts whose loads are in flight
    LatentSums sum;
    for (int c0 = g; c0 < unit.x; c0 += G * AT_ONCE) {
        float4 mc[AT_ONCE], lc[AT_ONCE], a[AT_ONCE], b[AT_ONCE];
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x) {
            const int c = c0 + x * G;
            lc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c >= unit.x) continue;
            const float* slot = latent_slot(p, run + c, ht, c == 0);
            mc[x] = *reinterpret_cast<const float4*>(slot + LA_ROWS * LT_VALUE + row0);
            lc[x] = *reinterpret_cast<const float4*>(slot + LA_ROWS * (LT_VALUE + 1) + row0);
            const float4* v = reinterpret_cast<const float4*>(slot) + row0 / 4 * LT_VALUE + d;
            a[x] = v[0];
            b[x] = v[1];
        }
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x)
            if (c0 + x * G < unit.x) sum.add(mc[x], lc[x], a[x], b[x]);
    }
    if constexpr (G > 1) {
        __shared__ float4 s_part[G - 1][4][PER];
        if (g > 0) {
            s_part[g - 1][0][t] = make_float4(sum.m[0], sum.m[1], sum.m[2], sum.m[3]);
            s_part[g - 1][1][t] = make_float4(sum.l[0], sum.l[1], sum.l[2], sum.l[3]);
            s_part[g - 1][2][t] = make_float4(sum.o[0][0], sum.o[1][0], sum.o[2][0], sum.o[3][0]);
            s_part[g - 1][3][t] = make_float4(sum.o[0][1], sum.o[1][1], sum.o[2][1], sum.o[3][1]);
        }
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int x = 0; x < G - 1; ++x) sum.add(s_part[x][0][t], s_part[x][1][t], s_part[x][2][t], s_part[x][3][t]);
    }
    sum.store<T>(p, unit.y, unit.z, ht, row0, d);
}

}  // namespace hsi
