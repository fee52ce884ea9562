// C-ABI entry points of the rotary positions and the paged cache: host-side
// validation, tensor maps, launch shapes. Included by hsi.cu after its helpers.
#pragma once
#include <cudaTypedefs.h>

#include <cmath>

#include "attend.cuh"
#include "attend_chunk.cuh"
#include "evict.cuh"
#include "paged.cuh"
#include "rope.cuh"
#include "weights.cuh"

namespace {

// cuTensorMapEncodeTiled through the runtime, so that the library links no
// driver library of its own. Null where the driver lacks it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode() {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &res) != cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// {dim, entry, head, page} map of one of the cache's tensors; a box is 64 dims
// of `box` entries, its rows swizzled over 128 bytes.
hsi_status paged_map(const hsi_paged_kv& c, const PagedView& v, void* base, int box, CUtensorMap* map) {
    const auto encode = tensor_map_encode();
    if (!encode) return HSI_ERR_CUDA;
    const cuuint64_t dims[4] = {(cuuint64_t)v.D, (cuuint64_t)c.page_size, (cuuint64_t)v.H, (cuuint64_t)v.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)v.token_stride * 2, (cuuint64_t)v.head_stride * 2,
                                   (cuuint64_t)v.page_stride * 2};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)(c.page_size < box ? c.page_size : box), 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, c.dtype == HSI_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                              4, base, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? HSI_OK : HSI_ERR_INVALID_ARG;
}

// {dim, head, token} map of the query rows; a box is 64 dims of `tpt` tokens'
// heads of one group. INVALID_ARG where a stride has no map (a broadcast axis).
hsi_status rows_map(hsi_dtype dt, const void* q, int64_t qt, int64_t qh, int64_t T, int Hq, int D, int group, int tpt,
                    CUtensorMap* map) {
    const auto encode = tensor_map_encode();
    if (!encode) return HSI_ERR_CUDA;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)(Hq > 1 ? qh : D) * 2, (cuuint64_t)(T > 1 ? qt : D) * 2};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)group, (cuuint32_t)tpt};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = encode(map, dt == HSI_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                              const_cast<void*>(q), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? HSI_OK : HSI_ERR_INVALID_ARG;
}

// Many rows per KV head go to the tensor-memory kernels, whose tiles hold
// whole tokens of 128 rows (groups of at most 128 heads, no broadcast axis of q).
// Measured, few-row kernel against theirs, 32 query and 8 KV heads of 128: 8
// sequences of 8000 entries 65 and 66 us at 20 rows, 67 and 66 at 32, 133 and 67
// at 40; 32 of 2000 94 and 68 at 20; two of 1000 9.7 and 11.9 at 20, 10.7 and 12.1
// at 48: few units alone would have the few-row kernel, by 2 us.
bool chunk_rows(const AttendParams& p) {
    return (int64_t)p.max_q * p.group > AT_ROWS && p.group <= 128 && (p.qt > 0 || p.T == 1) && (p.qh > 0 || p.Hq == 1);
}

// A launch in clusters of `csize` blocks, in the programmatic chain.
template <typename... KArgs, typename... Args>
hsi_status launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int csize, cudaStream_t s,
                          Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cuda_ok(e);
}

hsi_status paged_view(const hsi_paged_kv* c, PagedView* v) {
    if (!c || !c->k || !c->v || !c->table || !c->kv_len || c->B <= 0 || c->heads <= 0 || c->n_pages <= 0 ||
        c->n_pages >= INT32_MAX || c->ld_table <= 0 || c->page_size <= 0 || c->table_width < 0 ||
        c->table_width > c->ld_table)
        return HSI_ERR_INVALID_ARG;
    if (c->dtype == HSI_FP32) return HSI_ERR_UNSUPPORTED;
    if (c->dtype != HSI_BF16 && c->dtype != HSI_FP16) return HSI_ERR_INVALID_ARG;
    if ((c->dim != 64 && c->dim != 128) || c->page_size < 8 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) ||
        c->B > 65535 || c->heads > 65535)
        return HSI_ERR_UNSUPPORTED;
    v->k = c->k;
    v->v = c->v;
    v->page_stride = c->page_stride;
    v->token_stride = c->token_stride;
    v->head_stride = c->head_stride;
    // the stride of an axis of one element is never used: any valid value stands in
    if (c->heads == 1) v->head_stride = c->dim;
    if (c->n_pages == 1) v->page_stride = c->dim;
    for (int64_t s : {v->page_stride, v->token_stride, v->head_stride})
        if (s < c->dim || s % 8 || s >= (int64_t(1) << 38)) return HSI_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return HSI_ERR_INVALID_ARG;
    v->n_pages = c->n_pages;
    v->table = c->table;
    v->ld_table = c->ld_table;
    const int64_t width = c->table_width ? c->table_width : c->ld_table, most = INT32_MAX / c->page_size;
    v->capacity = width > most ? INT32_MAX : (int)(width * c->page_size);  // lengths are 32-bit
    v->kv_len = c->kv_len;
    v->B = c->B;
    v->H = c->heads;
    v->D = c->dim;
    v->page_shift = 0;
    while ((1 << v->page_shift) < c->page_size) ++v->page_shift;
    return HSI_OK;
}

bool rows_ok(const void* p, int64_t token_stride, int64_t head_stride) {
    return p && aligned(p, 16) && token_stride % 8 == 0 && head_stride % 8 == 0 && token_stride >= 0 && head_stride >= 0;
}

bool turn_ok(int32_t D, int32_t rot, int32_t off) { return rot >= 2 && rot % 2 == 0 && off >= 0 && off + rot <= D; }

template <typename T>
hsi_status launch_rope(const RopeParams& p0, cudaStream_t s) {
    RopeParams p = p0;
    constexpr int V = Vec16<T>::N;
    const bool pairs = p.r.pairs;
    const bool vec = aligned(p.x, 16) && aligned(p.y, 16) && p.xt % V == 0 && p.xh % V == 0 && p.yt % V == 0 &&
                     p.yh % V == 0 && p.D % V == 0 && p.r.off % V == 0 && p.r.rot % (pairs ? V : 2 * V) == 0 &&
                     p.r.rot / 2 <= ROPE_CS;
    if (!vec) {
        const int64_t items = p.T * p.H * (p.D - p.r.rot / 2);
        const int64_t blocks = (items + ROPE_THREADS - 1) / ROPE_THREADS;
        const unsigned grid = (unsigned)(blocks < 65536 ? blocks : 65536);
        return launch(rope_scalar_kernel<T>, dim3(grid), dim3(ROPE_THREADS), 0, s, p);
    }
    // tokens per block: enough for every thread's loads in flight, but every SM two blocks first
    const int sms = sm_count();
    if (sms <= 0) return HSI_ERR_CUDA;
    const int64_t per = (int64_t)p.H * rope_spans<V>(p.D, p.r.rot, p.r.pairs);
    int64_t tb = (ROPE_THREADS * ROPE_UNROLL + per - 1) / per;
    const int64_t fair = p.T / (2 * sms);
    if (tb > fair) tb = fair;
    if (tb > ROPE_CS / (p.r.rot / 2)) tb = ROPE_CS / (p.r.rot / 2);
    p.tb = (int)(tb < 1 ? 1 : tb);
    return launch(rope_kernel<T>, dim3((unsigned)((p.T + p.tb - 1) / p.tb)), dim3(ROPE_THREADS), 0, s, p);
}

// CTAs of the few-row kernels: what the SMs hold, no more than there can be tiles.
int64_t attend_grid(int32_t B, int32_t heads, int32_t group, int32_t max_q, int64_t max_kv, bool weights) {
    const int64_t rt = weights ? 1 : ((int64_t)max_q * group + AT_ROWS - 1) / AT_ROWS;
    const int64_t tiles = (int64_t)B * heads * rt * ((max_kv + AT_KT - 1) / AT_KT);
    static_assert(AttendCfg<64, false>::CTAS * 160 <= AT_MAX_RUNS, "the join's runs");
    const int64_t most = (weights ? AttendCfg<64, true>::CTAS : AttendCfg<64, false>::CTAS) * (int64_t)sm_count();
    return tiles < most ? tiles : most;
}

// Workspace of the attention: the chunks' line, then the partial sums' slots.
size_t attend_base_bytes(int32_t B) { return align_up(((size_t)B + 1) * 4, 256); }

// Blocks of a unit in the short form (0: the line): up to eight while all units'
// blocks run at once, each with at most AT_SHORT_TILES tiles. Units so few that
// twice the blocks would still run at once leave SMs idle that the line would
// use: they take it past AT_FEW_TILES. Measured, one token, 8 KV heads of 128, us
// short against line: 16 sequences of 1500 entries 20 and 26, four of 6000 20 and
// 20; two of 1100 8.8 and 9.9, of 5100 13.9 and 12.4; one of 4600 11.8 and 11.2, of
// 8000 16 and 13. Both bounds are below where the line wins: 32 of 1000 26 and 32
// (lengths from half of that 21 and 23, of any 17 and 32), of 2500 54 and 63 (46
// and 50, 36 and 50), 16 of 3000 35 and 44, four of 9000 29 and 33, one of 3000 9.8
// and 12 take the line. Clusters of sixteen: two of 1100 17.2 (they do not seem to
// run all at once).
constexpr int AT_SHORT_TILES = 12, AT_FEW_TILES = 4;
int attend_short(const AttendParams& p) {
    const int64_t rt = ((int64_t)p.max_q * p.group + AT_ROWS - 1) / AT_ROWS, units = rt * p.kv.H * p.kv.B;
    const int64_t tiles = (p.max_kv + AT_KT - 1) / AT_KT, room = 2 * (int64_t)sm_count();
    int csize = 1;
    while (csize < AT_CLUSTER && 2 * csize <= tiles && 2 * csize * units <= room) csize *= 2;
    const int most = 2 * csize * units <= room ? AT_FEW_TILES : AT_SHORT_TILES;
    return csize * units <= room && tiles <= most * csize ? csize : 0;
}

template <typename T, int D, bool WEIGHTS>
hsi_status launch_attend_token(const AttendParams& p, const CUtensorMap& km, const CUtensorMap& vm, int64_t grid,
                               cudaStream_t s) {
    using C = AttendCfg<D, WEIGHTS>;
    static std::atomic<bool> attr_set[kMaxDevices];
    if (smem_attr_once(attend_token_kernel<T, D, WEIGHTS>, C::SMEM_BYTES, attr_set) != HSI_OK) return HSI_ERR_CUDA;
    const unsigned rt = (unsigned)(((int64_t)p.max_q * p.group + AT_ROWS - 1) / AT_ROWS);
    const int csize = WEIGHTS ? 0 : attend_short(p);
    if (csize)
        return launch_cluster(attend_token_kernel<T, D, WEIGHTS>, dim3(rt * p.kv.H * p.kv.B * csize), dim3(AT_THREADS),
                              C::SMEM_BYTES, csize, s, p, km, vm, csize);
    const hsi_status st = launch(attend_token_kernel<T, D, WEIGHTS>, dim3((unsigned)grid), dim3(AT_THREADS),
                                 C::SMEM_BYTES, s, p, km, vm, 0);
    if (st != HSI_OK || WEIGHTS) return st;
    if ((int64_t)rt * p.kv.H * p.kv.B * 2 >= grid)  // blocks for every SM without splitting a unit's dims
        return launch(attend_join_kernel<T, D, D>, dim3(rt, p.kv.H, p.kv.B), dim3(AT_JOIN_THREADS), 0, s, p, (int)grid);
    return launch(attend_join_kernel<T, D, 16>, dim3(rt * (D / 16), p.kv.H, p.kv.B), dim3(AT_JOIN_THREADS), 0, s, p,
                  (int)grid);
}

template <bool WEIGHTS>
hsi_status run_attend_token(const AttendParams& p, hsi_dtype dt, const CUtensorMap& km, const CUtensorMap& vm,
                            int64_t grid, cudaStream_t s) {
    if (dt == HSI_BF16)
        return p.kv.D == 128 ? launch_attend_token<__nv_bfloat16, 128, WEIGHTS>(p, km, vm, grid, s)
                             : launch_attend_token<__nv_bfloat16, 64, WEIGHTS>(p, km, vm, grid, s);
    return p.kv.D == 128 ? launch_attend_token<__half, 128, WEIGHTS>(p, km, vm, grid, s)
                         : launch_attend_token<__half, 64, WEIGHTS>(p, km, vm, grid, s);
}

template <typename T, int D>
hsi_status launch_attend_chunk(const AttendParams& p, const CUtensorMap& km, const CUtensorMap& vm,
                               const CUtensorMap& qm, int tpt, int64_t grid, cudaStream_t s) {
    using C = ChunkCfg<D>;
    static std::atomic<bool> attr_set[kMaxDevices];
    if (smem_attr_once(attend_chunk_kernel<T, D>, C::SMEM_BYTES, attr_set) != HSI_OK) return HSI_ERR_CUDA;
    const hsi_status st = launch(attend_chunk_kernel<T, D>, dim3((unsigned)grid), dim3(CH_THREADS), C::SMEM_BYTES, s, p, km,
                                 vm, qm, tpt);
    if (st != HSI_OK) return st;
    const unsigned rt = (unsigned)((p.max_q + 2 * tpt - 1) / (2 * tpt));
    if ((int64_t)rt * p.kv.H * p.kv.B >= grid)
        return launch(attend_chunk_join_kernel<T, D, 32>, dim3(rt * (D / 32), p.kv.H, p.kv.B), dim3(2 * CH_ROWS), 0, s, p,
                      (int)grid, tpt);
    return launch(attend_chunk_join_kernel<T, D, 8>, dim3(rt * (D / 8), p.kv.H, p.kv.B), dim3(2 * CH_ROWS), 0, s, p,
                  (int)grid, tpt);
}

// CTAs of the chunk kernel: one an SM, no more than there can be key tiles.
int64_t chunk_grid(int32_t B, int32_t heads, int32_t group, int32_t max_q, int64_t max_kv) {
    const int tpt = CH_ROWS / group;
    const int64_t tiles =
        (int64_t)B * heads * ((max_q + 2 * tpt - 1) / (2 * tpt)) * ((max_kv + CH_KEYS - 1) / CH_KEYS);
    const int64_t most = sm_count();
    return tiles < most ? tiles : most;
}

template <typename T, int D>
hsi_status launch_weights_chunk(const AttendParams& p, const CUtensorMap& km, const CUtensorMap& qm, int tpt,
                                cudaStream_t s) {
    using C = WeightsCfg<D>;
    static std::atomic<bool> attr_set[kMaxDevices];
    if (smem_attr_once(weights_chunk_kernel<T, D>, C::SMEM_BYTES, attr_set) != HSI_OK) return HSI_ERR_CUDA;
    const int sms = sm_count();
    if (sms <= 0) return HSI_ERR_CUDA;
    const int64_t units = (int64_t)p.kv.B * p.kv.H * (((int64_t)p.max_kv + WC_KEYS - 1) / WC_KEYS);
    const int64_t tiles = (p.max_q + tpt - 1) / tpt;
    // units that leave SMs idle are shared by clusters, no CTA without a query tile
    int csize = 1;
    while (csize < EV_MAX_CLUSTER && 2 * csize * units <= sms && 2 * csize <= tiles) csize *= 2;
    const int64_t grid = csize > 1 || units < sms ? units * csize : sms;
    return launch_cluster(weights_chunk_kernel<T, D>, dim3((unsigned)grid), dim3(WC_THREADS), C::SMEM_BYTES, csize, s, p,
                          km, qm, csize, tpt);
}

// The checks that attention and weights share.
hsi_status attend_params(const hsi_paged_kv* cache, const void* q, int64_t qt, int64_t qh, int32_t q_heads,
                         const int32_t* q_start, int64_t T, int32_t max_q, int64_t max_kv, float scale, int32_t causal,
                         AttendParams* p) {
    const hsi_status st = paged_view(cache, &p->kv);
    if (st != HSI_OK) return st;
    if (!q_start || T <= 0 || T > INT32_MAX || max_q <= 0 || max_kv <= 0 || max_kv > INT32_MAX || q_heads <= 0 ||
        q_heads % cache->heads || !rows_ok(q, qt, qh) || !(scale == scale))
        return HSI_ERR_INVALID_ARG;
    p->max_kv = (int)(max_kv < p->kv.capacity ? max_kv : p->kv.capacity);
    p->q = q;
    p->qt = qt;
    p->qh = qh;
    p->q_start = q_start;
    p->T = T;
    p->max_q = (int)(max_q < T ? max_q : T);
    p->Hq = q_heads;
    p->group = q_heads / cache->heads;
    p->sl2 = scale * LOG2E;
    p->causal = causal != 0;
    // the kernels count entries, rounded up to whole tiles, and a KV head's rows in 31 bits
    if (p->max_kv > INT32_MAX - 4096 || (int64_t)p->max_q * p->group > INT32_MAX - 4096) return HSI_ERR_UNSUPPORTED;
    return HSI_OK;
}

// Whether the tiles of a kernel's line, `keys` entries each of B x heads x row_tiles units, can be counted in 31 bits
// (at the host's bounds, as the lengths are the device's). No factor is above 2^31 and heads, B are below 2^16.
bool line_ok(int64_t row_tiles, int64_t heads, int64_t B, int64_t max_kv, int64_t keys) {
    const int64_t units = row_tiles * heads;
    return units <= INT32_MAX && units * B <= INT32_MAX / ((max_kv + keys - 1) / keys);
}

}  // namespace

extern "C" {

hsi_status hsi_rope_steps(int32_t rot, double base, hsi_rope_scaling scaling, double factor, double original_len,
                          double beta_fast, double beta_slow, uint64_t* steps, float* gain) {
    if (!steps || !gain || rot < 2 || rot % 2 || rot > 2 * ROPE_CS || !(base > 1.0)) return HSI_ERR_INVALID_ARG;
    if (scaling < HSI_ROPE_PLAIN || scaling > HSI_ROPE_YARN) return HSI_ERR_INVALID_ARG;
    if (scaling != HSI_ROPE_PLAIN && !(factor >= 1.0)) return HSI_ERR_INVALID_ARG;
    if (scaling == HSI_ROPE_NTK && rot == 2) return HSI_ERR_INVALID_ARG;
    if (scaling == HSI_ROPE_YARN && !(original_len > 0.0 && beta_fast >= beta_slow && beta_slow > 0.0))
        return HSI_ERR_INVALID_ARG;
    const double pi2 = 6.283185307179586476925;
    const int half = rot / 2;
    if (scaling == HSI_ROPE_NTK) base *= std::pow(factor, (double)rot / (rot - 2));
    double lo = 0.0, hi = 0.0;
    if (scaling == HSI_ROPE_YARN) {
        // the pair whose wave turns `beta` times over the original length
        const auto at = [&](double beta) { return rot * std::log(original_len / (beta * pi2)) / (2.0 * std::log(base)); };
        lo = std::fmax(std::floor(at(beta_fast)), 0.0);
        hi = std::fmin(std::ceil(at(beta_slow)), rot - 1.0);
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == HSI_ROPE_LINEAR) f /= factor;
        if (scaling == HSI_ROPE_YARN) {
            const double ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
            f = f * (1.0 - ramp) + f / factor * ramp;
        }
        steps[i] = (uint64_t)std::nearbyint(f / pi2 * 0x1p64);  // f <= 1: below 2^62
    }
    *gain = scaling == HSI_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return HSI_OK;
}

hsi_status hsi_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, hsi_dtype dtype, int64_t T, int32_t H,
                    int32_t D, const int32_t* positions, const uint64_t* steps, int32_t rot, int32_t rot_offset,
                    int32_t interleaved, float gain, int32_t inverse, void* y, int64_t y_token_stride,
                    int64_t y_head_stride, cudaStream_t stream) {
    if (!x || !y || !positions || !steps || T <= 0 || H <= 0 || D <= 0 || T > INT32_MAX || (int64_t)H * D > INT32_MAX ||
        dtype < HSI_BF16 || dtype > HSI_FP32)
        return HSI_ERR_INVALID_ARG;
    if (!turn_ok(D, rot, rot_offset) || !(gain == gain)) return HSI_ERR_INVALID_ARG;
    if (x_token_stride < 0 || x_head_stride < 0 || y_token_stride < 0 || y_head_stride < 0) return HSI_ERR_INVALID_ARG;
    const size_t es = dtype == HSI_FP32 ? 4 : 2;
    if (!aligned(x, es) || !aligned(y, es) || !aligned(positions, 4) || !aligned(steps, 8)) return HSI_ERR_INVALID_ARG;
    if (x == y && (x_token_stride != y_token_stride || x_head_stride != y_head_stride)) return HSI_ERR_INVALID_ARG;
    // two results in one place
    if ((T > 1 && y_token_stride < D) || (H > 1 && y_head_stride < D)) return HSI_ERR_INVALID_ARG;
    RopeParams p{};
    p.r = {reinterpret_cast<const unsigned long long*>(steps), positions, rot, rot_offset, interleaved != 0, gain,
           inverse ? -1.f : 1.f};
    p.x = x;
    p.y = y;
    p.xt = x_token_stride;
    p.xh = x_head_stride;
    p.yt = y_token_stride;
    p.yh = y_head_stride;
    p.T = T;
    p.H = H;
    p.D = D;
    if (dtype == HSI_BF16) return launch_rope<__nv_bfloat16>(p, stream);
    if (dtype == HSI_FP16) return launch_rope<__half>(p, stream);
    return launch_rope<float>(p, stream);
}

hsi_status hsi_paged_append(const hsi_paged_kv* cache, const void* k_new, int64_t k_token_stride, int64_t k_head_stride,
                            const void* v_new, int64_t v_token_stride, int64_t v_head_stride, const int32_t* q_start,
                            int64_t T, const int32_t* positions, const uint64_t* steps, int32_t rot, int32_t rot_offset,
                            int32_t interleaved, float gain, const void* q, int64_t q_token_stride,
                            int64_t q_head_stride, int32_t q_heads, void* q_out, int64_t o_token_stride,
                            int64_t o_head_stride, cudaStream_t stream) {
    PagedAppendParams p{};
    const hsi_status st = paged_view(cache, &p.kv);
    if (st != HSI_OK) return st;
    if (!q_start || T <= 0 || T > INT32_MAX || !rows_ok(k_new, k_token_stride, k_head_stride) ||
        !rows_ok(v_new, v_token_stride, v_head_stride))
        return HSI_ERR_INVALID_ARG;
    if (steps) {
        if (!positions || !aligned(positions, 4) || !aligned(steps, 8) || !turn_ok(cache->dim, rot, rot_offset) ||
            !(gain == gain))
            return HSI_ERR_INVALID_ARG;
        if (rot % 16 || rot_offset % 8) return HSI_ERR_UNSUPPORTED;
        p.r = {reinterpret_cast<const unsigned long long*>(steps), positions, rot, rot_offset, interleaved != 0, gain, 1.f};
    }
    if (q) {
        if (!steps || q_heads <= 0 || (int64_t)q_heads * cache->dim > INT32_MAX || !rows_ok(q, q_token_stride, q_head_stride) ||
            !rows_ok(q_out, o_token_stride, o_head_stride))
            return HSI_ERR_INVALID_ARG;
        if (q == q_out && (q_token_stride != o_token_stride || q_head_stride != o_head_stride)) return HSI_ERR_INVALID_ARG;
        if ((T > 1 && o_token_stride < cache->dim) || (q_heads > 1 && o_head_stride < cache->dim))
            return HSI_ERR_INVALID_ARG;
    }
    p.q_start = q_start;
    p.q = q;
    p.k = k_new;
    p.v = v_new;
    p.q_out = q_out;
    p.qt = q_token_stride;
    p.qh = q_head_stride;
    p.ot = o_token_stride;
    p.oh = o_head_stride;
    p.kt = k_token_stride;
    p.kh = k_head_stride;
    p.vt = v_token_stride;
    p.vh = v_head_stride;
    p.T = T;
    p.Hq = q_heads;
    // as many tokens a block as leave every SM the blocks that it holds at once
    const int64_t room = APPEND_CTAS * (int64_t)sm_count();
    if (room <= 0) return HSI_ERR_CUDA;
    const int64_t tb = (T + room - 1) / room;
    p.tb = (int)(tb > APPEND_TOKENS ? APPEND_TOKENS : tb);
    const dim3 grid((unsigned)((T + p.tb - 1) / p.tb));
    if (cache->dtype == HSI_BF16)
        return launch(paged_append_kernel<__nv_bfloat16>, grid, dim3(ROPE_THREADS), 0, stream, p);
    return launch(paged_append_kernel<__half>, grid, dim3(ROPE_THREADS), 0, stream, p);
}

size_t hsi_paged_attention_ws(int32_t B, int32_t kv_heads, int32_t q_heads, int32_t dim, int32_t max_q, int64_t max_kv) {
    if (B <= 0 || kv_heads <= 0 || q_heads <= 0 || q_heads % kv_heads || dim <= 0 || max_q <= 0 || max_kv <= 0) return 0;
    const int group = q_heads / kv_heads;
    size_t floats = (size_t)attend_grid(B, kv_heads, group, max_q, max_kv, false) * 2 * AT_ROWS * (dim + 2);
    if ((int64_t)max_q * group > AT_ROWS && group <= 128) {
        const size_t chunk = (size_t)chunk_grid(B, kv_heads, group, max_q, max_kv) * 2 * chunk_slot_floats(dim);
        if (chunk > floats) floats = chunk;
    }
    return attend_base_bytes(B) + align_up(floats * 4, 256);
}

hsi_status hsi_paged_attention(const hsi_paged_kv* cache, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                               int32_t q_heads, const int32_t* q_start, int64_t T, int32_t max_q, int64_t max_kv,
                               float scale, int32_t causal, void* out, int64_t o_token_stride, int64_t o_head_stride,
                               float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
    AttendParams p{};
    hsi_status st = attend_params(cache, q, q_token_stride, q_head_stride, q_heads, q_start, T, max_q, max_kv, scale,
                                  causal, &p);
    if (st != HSI_OK) return st;
    if (!rows_ok(out, o_token_stride, o_head_stride) || out == q || (T > 1 && o_token_stride < cache->dim) ||
        (q_heads > 1 && o_head_stride < cache->dim))
        return HSI_ERR_INVALID_ARG;
    const bool chunk = chunk_rows(p);
    const int64_t tile = chunk ? 2 * (CH_ROWS / p.group) : AT_ROWS, rows = chunk ? p.max_q : p.max_q * p.group;
    if (!line_ok((rows + tile - 1) / tile, cache->heads, cache->B, p.max_kv, chunk ? CH_KEYS : AT_KT))
        return HSI_ERR_UNSUPPORTED;
    const size_t need = hsi_paged_attention_ws(cache->B, cache->heads, q_heads, cache->dim, p.max_q, p.max_kv);
    if (!ws || ws_bytes < need || !aligned(ws, 256)) return HSI_ERR_WORKSPACE;
    p.out = out;
    p.ot = o_token_stride;
    p.oh = o_head_stride;
    p.lse = lse;
    p.base = static_cast<uint32_t*>(ws);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + attend_base_bytes(cache->B));
    CUtensorMap km, vm;
    if (chunk) {
        const int tpt = CH_ROWS / p.group;
        CUtensorMap qm;
        if ((st = paged_map(*cache, p.kv, cache->k, CH_KEYS, &km)) != HSI_OK) return st;
        if ((st = paged_map(*cache, p.kv, cache->v, CH_KEYS, &vm)) != HSI_OK) return st;
        if ((st = rows_map(cache->dtype, q, q_token_stride, q_head_stride, T, q_heads, cache->dim, p.group, tpt, &qm)) !=
            HSI_OK)
            return st;
        p.negate = p.sl2 < 0.f;
        p.sl2 = std::fmax(std::fabs(p.sl2), 1e-30f);  // above 0, so that -inf stays -inf: at scale 0 every p is 1
        const int64_t grid = chunk_grid(cache->B, cache->heads, p.group, p.max_q, p.max_kv);
        if (grid <= 0) return HSI_ERR_CUDA;
        if (cache->dtype == HSI_BF16)
            return cache->dim == 128 ? launch_attend_chunk<__nv_bfloat16, 128>(p, km, vm, qm, tpt, grid, stream)
                                     : launch_attend_chunk<__nv_bfloat16, 64>(p, km, vm, qm, tpt, grid, stream);
        return cache->dim == 128 ? launch_attend_chunk<__half, 128>(p, km, vm, qm, tpt, grid, stream)
                                 : launch_attend_chunk<__half, 64>(p, km, vm, qm, tpt, grid, stream);
    }
    if ((st = paged_map(*cache, p.kv, cache->k, AT_KT, &km)) != HSI_OK) return st;
    if ((st = paged_map(*cache, p.kv, cache->v, AT_KT, &vm)) != HSI_OK) return st;
    const int64_t grid = attend_grid(cache->B, cache->heads, p.group, p.max_q, p.max_kv, false);
    if (grid <= 0) return HSI_ERR_CUDA;
    return run_attend_token<false>(p, cache->dtype, km, vm, grid, stream);
}

hsi_status hsi_attention_weights(const hsi_paged_kv* cache, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                 int32_t q_heads, const float* lse, const int32_t* q_start, int64_t T, int32_t max_q,
                                 int64_t max_kv, float scale, int32_t causal, float decay, const float* acc_in,
                                 int64_t ld_acc_in, float* acc_out, int64_t ld_acc_out, cudaStream_t stream) {
    AttendParams p{};
    hsi_status st = attend_params(cache, q, q_token_stride, q_head_stride, q_heads, q_start, T, max_q, max_kv, scale,
                                  causal, &p);
    if (st != HSI_OK) return st;
    if (!lse || !acc_out || ld_acc_out < p.max_kv || (acc_in && ld_acc_in < p.max_kv) || !(decay == decay))
        return HSI_ERR_INVALID_ARG;
    // in place with other rows' distances, a row's results would lie on another row's inputs
    if (acc_in == acc_out && ld_acc_in != ld_acc_out && (int64_t)cache->B * cache->heads > 1) return HSI_ERR_INVALID_ARG;
    const bool chunk = chunk_rows(p);
    // a unit takes every row; the chunk kernel counts the units of all sequences in 64 bits
    if (!line_ok(1, cache->heads, chunk ? 1 : cache->B, p.max_kv, chunk ? WC_KEYS : AT_KT)) return HSI_ERR_UNSUPPORTED;
    p.lse_in = lse;
    p.acc_in = acc_in;
    p.acc_out = acc_out;
    p.ld_acc_in = ld_acc_in;
    p.ld_acc_out = ld_acc_out;
    p.decay = decay;
    CUtensorMap km;
    if (chunk) {
        const int tpt = WC_ROWS / p.group;
        CUtensorMap qm;
        if ((st = paged_map(*cache, p.kv, cache->k, 128, &km)) != HSI_OK) return st;
        if ((st = rows_map(cache->dtype, q, q_token_stride, q_head_stride, T, q_heads, cache->dim, p.group, tpt, &qm)) !=
            HSI_OK)
            return st;
        if (cache->dtype == HSI_BF16)
            return cache->dim == 128 ? launch_weights_chunk<__nv_bfloat16, 128>(p, km, qm, tpt, stream)
                                     : launch_weights_chunk<__nv_bfloat16, 64>(p, km, qm, tpt, stream);
        return cache->dim == 128 ? launch_weights_chunk<__half, 128>(p, km, qm, tpt, stream)
                                 : launch_weights_chunk<__half, 64>(p, km, qm, tpt, stream);
    }
    if ((st = paged_map(*cache, p.kv, cache->k, AT_KT, &km)) != HSI_OK) return st;
    const int64_t grid = attend_grid(cache->B, cache->heads, p.group, p.max_q, p.max_kv, true);
    if (grid <= 0) return HSI_ERR_CUDA;
    return run_attend_token<true>(p, cache->dtype, km, km, grid, stream);
}

hsi_status hsi_evict_select(const float* acc, int64_t ld_acc, const int32_t* kv_len, int32_t B, int32_t heads,
                            int64_t max_len, int32_t budget, int32_t sink, int32_t recent, int32_t* keep,
                            int64_t ld_keep, int32_t* new_len, float* acc_out, int64_t ld_out, cudaStream_t stream) {
    if (!acc || !kv_len || !keep || !new_len || B <= 0 || heads <= 0 || max_len <= 0 || max_len > INT32_MAX ||
        ld_acc < max_len || budget <= 0 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget || ld_keep < budget)
        return HSI_ERR_INVALID_ARG;
    if (acc_out && ld_out < budget) return HSI_ERR_INVALID_ARG;
    int csize = 1;
    // a CTA a row up to 16384 entries: a cluster's barriers and remote counts, 10000 cycles in all,
    // cost two CTAs what they save there; slices of 16384 beyond
    while (csize < EV_MAX_CLUSTER && max_len > (int64_t)csize * 16384) csize *= 2;
    // past the clusters' shared memory, weights are read while others are written
    if (acc_out == acc && (max_len + csize - 1) / csize > EV_CAP) return HSI_ERR_UNSUPPORTED;
    if ((int64_t)B * heads * csize > INT32_MAX) return HSI_ERR_UNSUPPORTED;
    // what a row's blocks write, other rows' blocks may not have read yet
    if (new_len == kv_len || (acc_out == acc && ld_out != ld_acc && (int64_t)B * heads > 1)) return HSI_ERR_INVALID_ARG;
    EvictParams p{};
    p.acc = acc;
    p.ld_acc = ld_acc;
    p.kv_len = kv_len;
    p.B = B;
    p.H = heads;
    p.max_len = max_len;
    p.budget = budget;
    p.sink = sink;
    p.recent = recent;
    p.keep = keep;
    p.ld_keep = ld_keep;
    p.acc_out = acc_out;
    p.ld_out = ld_out;
    p.n_out = acc_out == acc ? (ld_out < max_len ? ld_out : max_len) : budget;
    p.new_len = new_len;
    static std::atomic<bool> attr_set[kMaxDevices];
    if (smem_attr_once(evict_select_kernel, (int)sizeof(EvictSmem), attr_set) != HSI_OK) return HSI_ERR_CUDA;
    return launch_cluster(evict_select_kernel, dim3((unsigned)(B * heads * csize)), dim3(EV_THREADS), sizeof(EvictSmem),
                          csize, stream, p, csize);
}

hsi_status hsi_paged_compact(const hsi_paged_kv* cache, const int32_t* keep, int64_t ld_keep, const int32_t* new_len,
                             int32_t budget, const int32_t* dst_table, int64_t ld_dst, cudaStream_t stream) {
    CompactParams p{};
    const hsi_status st = paged_view(cache, &p.kv);
    if (st != HSI_OK) return st;
    if (!keep || !new_len || !dst_table || budget <= 0 || ld_keep < budget || ld_dst <= 0 ||
        ld_dst * cache->page_size < budget)
        return HSI_ERR_INVALID_ARG;
    // places are counted in 31 bits up to a turn of all blocks past the budget (256 of up to 16 blocks an SM)
    if (budget > INT32_MAX - (1 << 20)) return HSI_ERR_UNSUPPORTED;
    p.keep = keep;
    p.ld_keep = ld_keep;
    p.new_len = new_len;
    p.budget = budget;
    p.dst = dst_table;
    p.ld_dst = ld_dst;
    p.in_place = dst_table == cache->table;
    if (p.in_place && (budget > p.kv.capacity || (ld_dst != cache->ld_table && cache->B > 1))) return HSI_ERR_INVALID_ARG;
    // blocks of a (sequence, KV head, K or V): until every SM has sixteen (four at a time), none
    // without a turn's entries
    const int64_t rows = (int64_t)cache->B * cache->heads * 2, sms = sm_count();
    if (sms <= 0) return HSI_ERR_CUDA;
    const int64_t round = CP_THREADS / (cache->dim / 8);
    const bool few = rows * ((budget + 8 * round - 1) / (8 * round)) < 2 * sms;
    const int64_t turn = round * (few ? 2 : 8), most = (budget + turn - 1) / turn;
    int64_t split = 1;
    while (split * rows < 16 * sms && 2 * split <= most && (!p.in_place || split < EV_MAX_CLUSTER)) split *= 2;
    if (rows * split > INT32_MAX) return HSI_ERR_UNSUPPORTED;
    const int csize = p.in_place ? (int)split : 1;
    const dim3 grid((unsigned)(rows * split));
    const auto kernel = few                                        ? paged_compact_kernel<2, false>
                        : p.in_place && rows * split <= 2 * sms ? paged_compact_kernel<8, true>
                                                                : paged_compact_kernel<8, false>;
    return launch_cluster(kernel, grid, dim3(CP_THREADS), 0, csize, stream, p, (int)split, csize);
}

}  // extern "C"
