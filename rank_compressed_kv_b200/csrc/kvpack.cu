// kvpack.cu -- the C ABI of libkvpack (see include/kvpack.h): argument
// validation, workspace planning and kernel launches.  Everything that
// computes runs in the kernels of decode.cuh, rstream.cuh, select.cuh,
// compress.cuh, rope.cuh and paged.cuh.
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <utility>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kvpack.h"
#include "common.cuh"
#include "decode.cuh"
#include "rstream.cuh"
#include "baseline.cuh"
#include "select.cuh"
#include "compress.cuh"
#include "rope.cuh"
#include "paged.cuh"

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxT = KVPACK_MAX_T;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

kvpack_status check_dims(const kvpack_dims *d, int32_t n_layers) {
    if (d == nullptr || n_layers <= 0) return KVPACK_ERR_INVALID_ARG;
    if (d->batch <= 0 || d->n_q_heads <= 0 || d->n_kv_heads <= 0 || d->T_vis <= 0 || d->L_text_cap < 0)
        return KVPACK_ERR_INVALID_ARG;
    if (d->group != KVPACK_GROUP || d->head_dim != KVPACK_HEAD_DIM || d->rank != KVPACK_RANK ||
        (d->rank_lo != KVPACK_RANK_LO && d->rank_lo != 0))
        return KVPACK_ERR_UNSUPPORTED;
    if (d->n_kv_heads % KVPACK_GROUP != 0 || d->n_q_heads % d->n_kv_heads != 0) return KVPACK_ERR_UNSUPPORTED;
    if ((d->n_q_heads / d->n_kv_heads) * KVPACK_GROUP > 32) return KVPACK_ERR_UNSUPPORTED;
    if (d->T_vis > kMaxT || d->L_text_cap > KVPACK_MAX_TEXT) return KVPACK_ERR_UNSUPPORTED;
    const long long units = (long long)n_layers * d->batch * (d->n_kv_heads / KVPACK_GROUP);
    if (units > (1LL << 30)) return KVPACK_ERR_UNSUPPORTED;
    return KVPACK_OK;
}

inline int n_units(const kvpack_dims *d, int32_t n_layers) {
    return n_layers * d->batch * (d->n_kv_heads / KVPACK_GROUP);
}

inline int hg(const kvpack_dims *d) { return (d->n_q_heads / d->n_kv_heads) * KVPACK_GROUP; }

// Text tail: work items of kTextChunk tokens per (unit, KV head).
constexpr int kTextChunk = 64;
// The visual passes are sized for a full B200 (148 SMs) whatever the device, so the
// workspace, the work split and hence the results depend on the shapes alone.
constexpr int kPlanSMs = 148;

namespace rs = kvpack::decode::rs;

struct DecodePlan {
    int units, Hg, NH, tpu, nwords, Sc_max;
    long long ntiles;
    int cta_s, cta_v, nslot_s, nslot_v;
    size_t off_qt, off_tp, off_sp, off_ustat, off_vp, off_counter, off_hipos, off_hicnt, total;
    int Tp;   // stride of a unit's list of full-rank positions (T rounded up to 8)
    // the text tokens' own rank-space passes (text compressed too); absent when L_c = 0
    int L_c, tpu2, nwords2, cta2, nslot2, Tp2;
    long long ntiles2;
    size_t off_qt2, off_sp2, off_vp2, off_mask2, off_hipos2, off_hicnt2;
};

inline int round_heads(int Hg) { return Hg <= 4 ? 4 : Hg <= 8 ? 8 : Hg <= 16 ? 16 : Hg <= 28 ? 28 : 32; }

// Most partial slots any unit gets when NT tiles are split over C CTAs (tpu tiles per unit).
inline int max_slots(long long NT, long long C, int tpu) { return (int)(((long long)tpu * C + NT - 1) / NT) + 1; }

DecodePlan plan_decode(const kvpack_dims *d, int32_t n_layers, int L_c = 0, bool paged_text = false) {
    DecodePlan pl{};
    pl.Hg = hg(d);
    pl.NH = round_heads(pl.Hg);
    pl.units = n_units(d, n_layers);
    const int T = d->T_vis;
    pl.tpu = (T + rs::kTile - 1) / rs::kTile;
    pl.nwords = (T + 31) / 32;
    pl.ntiles = (long long)pl.units * pl.tpu;
    const int blocks = pl.NH <= 16 ? 2 : 1;     // resident CTAs per SM of both visual passes
    pl.cta_s = (int)(pl.ntiles < (long long)kPlanSMs * blocks ? pl.ntiles : (long long)kPlanSMs * blocks);
    pl.cta_v = pl.cta_s;
    pl.nslot_s = max_slots(pl.ntiles, pl.cta_s, pl.tpu);
    pl.nslot_v = max_slots(pl.ntiles, pl.cta_v, pl.tpu);
    pl.Sc_max = paged_text ? 1 : (d->L_text_cap + kTextChunk - 1) / kTextChunk;   // paged: joined to one partial
    size_t off = 0;
    pl.off_qt = off;
    off = align256(off + (size_t)pl.units * kvpack::decode::qblock_bytes(pl.Hg));
    pl.off_tp = off;
    off = align256(off + (size_t)pl.units * pl.Sc_max * pl.Hg * kvpack::decode::kTxtPart * sizeof(float));
    pl.off_sp = off;
    off = align256(off + (size_t)pl.units * pl.nslot_s * pl.Hg * 2 * sizeof(float));
    pl.off_ustat = off;
    off = align256(off + (size_t)pl.units * pl.Hg * 2 * sizeof(float));
    pl.off_vp = off;
    off = align256(off + (size_t)pl.units * pl.nslot_v * pl.Hg * 64 * sizeof(float));
    pl.off_counter = off;   // work counter of the text kernel
    off = align256(off + 4 * sizeof(unsigned int));
    pl.Tp = (T + 7) & ~7;
    pl.off_hipos = off;
    off = align256(off + (size_t)pl.units * pl.Tp * sizeof(uint16_t));
    pl.off_hicnt = off;
    off = align256(off + (size_t)pl.units * pl.tpu * sizeof(int));
    pl.L_c = L_c;
    if (L_c > 0) {
        pl.tpu2 = (L_c + rs::kTile - 1) / rs::kTile;
        pl.nwords2 = (L_c + 31) / 32;
        pl.ntiles2 = (long long)pl.units * pl.tpu2;
        pl.cta2 = (int)(pl.ntiles2 < (long long)kPlanSMs * blocks ? pl.ntiles2 : (long long)kPlanSMs * blocks);
        pl.nslot2 = max_slots(pl.ntiles2, pl.cta2, pl.tpu2);
        pl.off_qt2 = off;
        off = align256(off + (size_t)pl.units * kvpack::decode::qblock_bytes(pl.Hg));
        pl.off_sp2 = off;
        off = align256(off + (size_t)pl.units * pl.nslot2 * pl.Hg * 2 * sizeof(float));
        pl.off_vp2 = off;
        off = align256(off + (size_t)pl.units * pl.nslot2 * pl.Hg * 64 * sizeof(float));
        pl.off_mask2 = off;     // every text token at the full rank
        off = align256(off + (size_t)pl.units * pl.nwords2 * sizeof(uint32_t));
        pl.Tp2 = (L_c + 7) & ~7;
        pl.off_hipos2 = off;
        off = align256(off + (size_t)pl.units * pl.Tp2 * sizeof(uint16_t));
        pl.off_hicnt2 = off;
        off = align256(off + (size_t)pl.units * pl.tpu2 * sizeof(int));
    }
    pl.total = off;
    return pl;
}

struct DeviceInfo {
    bool ready = false;
    unsigned long long ctx_id = 0;       // the context the attributes below were set in
    int sms = 0;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

template <int NH, bool VALUE, bool Q4>
bool rs_attr() {
    const void *fn = (const void *)rs::rs_kernel<NH, VALUE, Q4>;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)rs::smem_bytes<NH, VALUE>()) ==
               cudaSuccess &&
           cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess;
}
bool rs_attrs() {
    return rs_attr<4, false, false>() && rs_attr<4, true, false>() && rs_attr<8, false, false>() &&
           rs_attr<8, true, false>() && rs_attr<16, false, false>() && rs_attr<16, true, false>() &&
           rs_attr<28, false, false>() && rs_attr<28, true, false>() && rs_attr<32, false, false>() &&
           rs_attr<32, true, false>() && rs_attr<4, false, true>() && rs_attr<4, true, true>() &&
           rs_attr<8, false, true>() && rs_attr<8, true, true>() && rs_attr<16, false, true>() &&
           rs_attr<16, true, true>() && rs_attr<28, false, true>() && rs_attr<28, true, true>() &&
           rs_attr<32, false, true>() && rs_attr<32, true, true>();
}

bool paged_attrs() {
    namespace pg = kvpack::paged;
    return cudaFuncSetAttribute(pg::attend_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess &&
           cudaFuncSetAttribute(pg::short_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess &&
           cudaFuncSetAttribute(pg::unit_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                pg::kWarps * pg::kRingBytes) == cudaSuccess;
}

// Launch on `st` with programmatic stream serialization: the kernel may start while the
// previous kernel on the stream drains, and waits for it (griddep_wait) before reading its
// outputs.
template <typename... Args, typename... Params>
cudaError_t launch_pdl(void (*kernel)(Params...), int grid, int threads, size_t smem, cudaStream_t st,
                       Args &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <bool VALUE, bool Q4>
cudaError_t launch_rs_q(int NH, const rs::Params &rp, int grid, cudaStream_t st) {
    switch (NH) {
        case 4:
            return launch_pdl(rs::rs_kernel<4, VALUE, Q4>, grid, rs::Cfg<4, VALUE>::kThreads, rs::smem_bytes<4, VALUE>(),
                              st, rp);
        case 8:
            return launch_pdl(rs::rs_kernel<8, VALUE, Q4>, grid, rs::Cfg<8, VALUE>::kThreads, rs::smem_bytes<8, VALUE>(),
                              st, rp);
        case 16:
            return launch_pdl(rs::rs_kernel<16, VALUE, Q4>, grid, rs::Cfg<16, VALUE>::kThreads, rs::smem_bytes<16, VALUE>(),
                              st, rp);
        case 28:
            return launch_pdl(rs::rs_kernel<28, VALUE, Q4>, grid, rs::Cfg<28, VALUE>::kThreads, rs::smem_bytes<28, VALUE>(),
                              st, rp);
        default:
            return launch_pdl(rs::rs_kernel<32, VALUE, Q4>, grid, rs::Cfg<32, VALUE>::kThreads, rs::smem_bytes<32, VALUE>(),
                              st, rp);
    }
}
template <bool VALUE>
cudaError_t launch_rs(int NH, const rs::Params &rp, int grid, cudaStream_t st) {
    return rp.QK_lo != nullptr ? launch_rs_q<VALUE, true>(NH, rp, grid, st) : launch_rs_q<VALUE, false>(NH, rp, grid, st);
}

// finish_kernel is instantiated for 1..8 query heads per KV head, and for a whole unit per
// block (many units) or one KV head per block (few units)
template <int PK>
cudaError_t launch_finish_pk(const rs::FinishParams &fp, int units, int sms, cudaStream_t st) {
    if (units >= 2 * sms) return launch_pdl(rs::finish_kernel<PK, 4>, units, 256, 0, st, fp);
    return launch_pdl(rs::finish_kernel<PK, 1>, units * 4, 64, 0, st, fp);
}
cudaError_t launch_finish(int per_kv, const rs::FinishParams &fp, int units, int sms, cudaStream_t st) {
    switch (per_kv) {
        case 1: return launch_finish_pk<1>(fp, units, sms, st);
        case 2: return launch_finish_pk<2>(fp, units, sms, st);
        case 3: return launch_finish_pk<3>(fp, units, sms, st);
        case 4: return launch_finish_pk<4>(fp, units, sms, st);
        case 5: return launch_finish_pk<5>(fp, units, sms, st);
        case 6: return launch_finish_pk<6>(fp, units, sms, st);
        case 7: return launch_finish_pk<7>(fp, units, sms, st);
        default: return launch_finish_pk<8>(fp, units, sms, st);
    }
}

// Unique id of the calling thread's current context (cuCtxGetId, looked up once through the
// runtime).  Kernel attributes belong to a context: one torn down and created again
// (cudaDeviceReset) needs them set afresh.
kvpack_status current_context_id(unsigned long long *id) {
    using GetCtx = CUresult (*)(CUcontext *);
    using GetId = CUresult (*)(CUcontext, unsigned long long *);
    static GetCtx get_ctx = nullptr;
    static GetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f1 = nullptr, *f2 = nullptr;
        cudaDriverEntryPointQueryResult q1, q2;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &f1, cudaEnableDefault, &q1) == cudaSuccess &&
            q1 == cudaDriverEntryPointSuccess &&
            cudaGetDriverEntryPoint("cuCtxGetId", &f2, cudaEnableDefault, &q2) == cudaSuccess &&
            q2 == cudaDriverEntryPointSuccess) {
            get_ctx = reinterpret_cast<GetCtx>(f1);
            get_id = reinterpret_cast<GetId>(f2);
        }
    });
    if (get_ctx == nullptr || get_id == nullptr) return KVPACK_ERR_CUDA;
    CUcontext ctx = nullptr;
    if (get_ctx(&ctx) != CUDA_SUCCESS) return KVPACK_ERR_CUDA;
    if (ctx == nullptr) {   // a thread without a current context: bind the device's primary context
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return KVPACK_ERR_CUDA;
        if (get_ctx(&ctx) != CUDA_SUCCESS || ctx == nullptr) return KVPACK_ERR_CUDA;
    }
    if (get_id(ctx, id) != CUDA_SUCCESS) return KVPACK_ERR_CUDA;
    return KVPACK_OK;
}

kvpack_status device_info(DeviceInfo **out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return KVPACK_ERR_CUDA;
    unsigned long long ctx_id = 0;
    if (current_context_id(&ctx_id) != KVPACK_OK) return KVPACK_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    DeviceInfo &di = g_dev[dev];
    if (!di.ready || di.ctx_id != ctx_id) {
        di.ready = false;
        di.ctx_id = ctx_id;
        if (cudaDeviceGetAttribute(&di.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return KVPACK_ERR_CUDA;
        namespace dc = kvpack::decode;
        if (cudaFuncSetAttribute(dc::text::text_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)dc::text::smem_bytes()) != cudaSuccess ||
            cudaFuncSetAttribute(dc::text::text_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) !=
                cudaSuccess ||
            !rs_attrs() || !paged_attrs() ||
            cudaFuncSetAttribute(kvpack::baseline::decompress_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(kvpack::baseline::DecSmem)) != cudaSuccess)
            return KVPACK_ERR_CUDA;
        kvpack_status cs = kvpack::compress::prepare_device();
        if (cs != KVPACK_OK) return cs;
        di.ready = true;
    }
    *out = &di;
    return KVPACK_OK;
}

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::mutex g_encode_mu;

kvpack_status tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000 *out) {
    std::lock_guard<std::mutex> lk(g_encode_mu);
    if (g_encode == nullptr) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || fn == nullptr)
            return KVPACK_ERR_CUDA;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    *out = g_encode;
    return KVPACK_OK;
}

// bf16 tensor map of `rank` dims (innermost first), byte strides of dims 1.., box, swizzle
bool encode_bf16(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, const void *ptr, int rank,
                 const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle sw) {
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KPT>
cudaError_t launch_select_warp(const kvpack::select::Params &p, cudaStream_t st) {
    kvpack::select::select_warp_kernel<KPT><<<(p.n_units + 7) / 8, 256, 0, st>>>(p);
    return cudaGetLastError();
}

template <int KPT>
cudaError_t launch_select_block(const kvpack::select::Params &p, cudaStream_t st) {
    kvpack::select::select_block_kernel<KPT><<<p.n_units, kvpack::select::kBlockThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <int KPT>
cudaError_t launch_select_cluster(const kvpack::select::Params &p, cudaStream_t st) {
    namespace sl = kvpack::select;
    sl::select_cluster_kernel<KPT><<<p.n_units * sl::kClusterCtas, sl::kClusterThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

extern "C" {

int32_t kvpack_version(void) { return KVPACK_VERSION; }

const char *kvpack_status_string(kvpack_status s) {
    switch (s) {
        case KVPACK_OK: return "KVPACK_OK";
        case KVPACK_ERR_INVALID_ARG: return "KVPACK_ERR_INVALID_ARG";
        case KVPACK_ERR_ALIGNMENT: return "KVPACK_ERR_ALIGNMENT";
        case KVPACK_ERR_UNSUPPORTED: return "KVPACK_ERR_UNSUPPORTED";
        case KVPACK_ERR_WORKSPACE: return "KVPACK_ERR_WORKSPACE";
        case KVPACK_ERR_CUDA: return "KVPACK_ERR_CUDA";
        case KVPACK_ERR_NOCONVERGE: return "KVPACK_ERR_NOCONVERGE";
        case KVPACK_ERR_TIMEOUT: return "KVPACK_ERR_TIMEOUT";
        case KVPACK_ERR_PAGE: return "KVPACK_ERR_PAGE";
    }
    return "KVPACK_ERR_UNKNOWN";
}

kvpack_status kvpack_last_device_status(void *stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return KVPACK_ERR_CUDA;
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, kvpack::g_error_word, sizeof(v)) != cudaSuccess) return KVPACK_ERR_CUDA;
    if (cudaMemcpyToSymbol(kvpack::g_error_word, &zero, sizeof(zero)) != cudaSuccess) return KVPACK_ERR_CUDA;
    return static_cast<kvpack_status>(v);
}

kvpack_status kvpack_footprint(const kvpack_dims *d, int32_t n_layers, int32_t L_text, uint64_t out[3]) {
    kvpack_status s = check_dims(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (out == nullptr || L_text < 0) return KVPACK_ERR_INVALID_ARG;
    const uint64_t units = (uint64_t)n_units(d, n_layers);
    const uint64_t T = (uint64_t)d->T_vis, L = (uint64_t)L_text, n = KVPACK_GROUP * KVPACK_HEAD_DIM;
    out[0] = units * (T + L) * n * 2 * 2;
    out[1] = units * (T * KVPACK_RANK * 2 * 2 + L * n * 2 * 2);
    out[2] = units * (uint64_t)KVPACK_RANK * n * 2 * 2;
    return KVPACK_OK;
}

// ------------------------------------------------------------------ decode

size_t kvpack_decode_workspace(const kvpack_dims *d, int32_t n_layers) {
    if (check_dims(d, n_layers) != KVPACK_OK) return 0;
    return plan_decode(d, n_layers).total;
}

}  // extern "C"

namespace {

// ------------------------------------------------------------------ paged cache

namespace pg = kvpack::paged;

kvpack_status check_paged(const kvpack_paged_dims *d, int32_t n_layers) {
    if (d == nullptr || n_layers <= 0) return KVPACK_ERR_INVALID_ARG;
    if (d->batch <= 0 || d->n_q_heads <= 0 || d->n_kv_heads <= 0 || d->page_size <= 0 || d->n_pages <= 0 ||
        d->max_pages <= 0)
        return KVPACK_ERR_INVALID_ARG;
    if (d->head_dim != KVPACK_HEAD_DIM || d->n_q_heads % d->n_kv_heads != 0) return KVPACK_ERR_UNSUPPORTED;
    if (d->n_q_heads / d->n_kv_heads > 8 || d->n_kv_heads > 1024) return KVPACK_ERR_UNSUPPORTED;
    if (d->batch > KVPACK_MAX_PAGED_BATCH) return KVPACK_ERR_UNSUPPORTED;
    if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)) != 0)
        return KVPACK_ERR_UNSUPPORTED;
    if ((long long)d->max_pages * d->page_size > KVPACK_MAX_PAGED_TOKENS) return KVPACK_ERR_UNSUPPORTED;
    if ((long long)n_layers * d->batch * d->n_q_heads > (1LL << 30)) return KVPACK_ERR_UNSUPPORTED;
    const long long units = (long long)n_layers * d->batch * d->n_kv_heads;
    if (units * ((long long)d->max_pages * d->page_size / 16) > (1LL << 40)) return KVPACK_ERR_UNSUPPORTED;   // tiles
    return KVPACK_OK;
}

inline int log2_exact(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

struct PagedPlan {
    long long units;
    int per_kv, slots;
    int cluster, shorts;         // blocks per unit, or blocks that take whole units; both 0 where runs cross units
    size_t off_stat, off_acc, total;
};

// Three forms, by the number of units and the tables' capacity (the lengths are on the device).  Measured, bf16, us:
//   a cluster of blocks per unit, one wave of blocks      few units, caches of up to kUnitTiles tiles a warp
//     1 x 1024 tokens (8 units) 5.3, runs 6.9; 32 x 1024 (256 units) 24.7, 29.5; ragged up to 2048: 34.4, 31.3
//   a warp per unit                                       units for 85 % of the warps, up to kShortTiles tiles
//     1024 units of 16 tokens 4.0, runs 7.5; of 512 44, 48; of 1024 83, 89; ragged up to 1024: 69, 53
//     also few tiles on units past one wave of clusters: 512 units of 64 tokens 7.0, 11.0
//   even runs over all units, joined                      the rest: one long sequence keeps every warp busy
// The limits keep a long sequence among short ones, which only the runs share out, to some tens of us.  Short
// caches behind a table for long ones take the runs too: 1 x 64 tokens 4.1 us behind a table for 64, 6.0 for 32768.
constexpr int kUnitTiles = 32;
constexpr int kShortTiles = 64;

// Runs for a full B200, fewer where the tables' capacity cannot fill them.
PagedPlan plan_paged(const kvpack_paged_dims *d, int32_t n_layers) {
    PagedPlan pl{};
    pl.units = (long long)n_layers * d->batch * d->n_kv_heads;
    pl.per_kv = d->n_q_heads / d->n_kv_heads;
    const long long places = pl.units * ((long long)d->max_pages * d->page_size / pg::kTile + 1);
    const long long runs = (places + pg::kMinPlaces - 1) / pg::kMinPlaces;
    // as many runs for each of a few units, so that the ends of equal units are ends of runs: 4 x 66560 tokens
    // (32 units) 165 us with 1024 runs, 171 with 1036 or, eight an SM, 1184
    long long most = (long long)kPlanSMs * pg::kSlotsPerSM;
    if (pl.units * 8 <= most) most -= most % pl.units;
    pl.slots = (int)(runs < most ? runs : most);
    const long long wave = kPlanSMs * pg::kUnitBlocksPerSM, cap = (long long)d->max_pages * d->page_size / pg::kTile;
    int S = 8;
    while (S > 1 && (pl.units * S > wave || cap * 2 <= (long long)S * pg::kWarps)) S >>= 1;   // one wave; two warps a tile are too many
    const long long warps = kPlanSMs * pg::kShortPerSM;
    if (pl.units > wave && cap <= (pl.units * 20 >= warps * 17 ? kShortTiles : 4))
        pl.shorts = (int)(pl.units < warps ? pl.units : warps);
    // past two waves of blocks the runs are level or ahead (1024 units of 256 tokens: 32.8, 27.3)
    else if (pl.units <= 2 * wave && cap <= (long long)S * pg::kWarps * kUnitTiles) pl.cluster = S;
    const size_t slots = pl.cluster > 0 || pl.shorts > 0 ? 0 : 2 * (size_t)pl.slots;
    size_t off = 0;
    pl.off_stat = off;
    off = align256(off + slots * 8 * 2 * sizeof(float));
    pl.off_acc = off;
    off = align256(off + slots * pl.per_kv * 128 * sizeof(float));
    pl.total = off > 0 ? off : 256;
    return pl;
}

cudaError_t launch_unit(const pg::Params &p, const PagedPlan &pl, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(pl.units * pl.cluster));
    cfg.blockDim = dim3(pg::kThreads);
    cfg.dynamicSmemBytes = pg::kWarps * pg::kRingBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)pl.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, pg::unit_kernel, p, pl.cluster);
}

// out and lse of every unit, or (out null) the softmax parts of every query head in the text tail's
// partial layout
kvpack_status launch_paged_attend(const kvpack_paged_dims *d, int32_t n_layers, const uint16_t *q, const uint16_t *K,
                                  const uint16_t *V, const int32_t *table, const int32_t *lens, float softmax_scale,
                                  uint16_t *out, float *lse, float *tpart, void *ws, cudaStream_t st) {
    const PagedPlan pl = plan_paged(d, n_layers);
    unsigned char *w = static_cast<unsigned char *>(ws);
    pg::Params p{};
    p.q = q; p.K = K; p.V = V; p.table = table; p.lens = lens; p.out = out; p.lse = lse; p.tpart = tpart;
    p.stat = reinterpret_cast<float *>(w + pl.off_stat);
    p.acc = reinterpret_cast<float *>(w + pl.off_acc);
    p.layers = n_layers; p.batch = d->batch; p.n_kv = d->n_kv_heads; p.per_kv = pl.per_kv;
    p.n_pages = d->n_pages; p.max_pages = d->max_pages; p.page_shift = log2_exact(d->page_size);
    p.slots = pl.slots;
    p.scale2 = softmax_scale * 1.4426950408889634f;
    if (pl.cluster > 0) return launch_unit(p, pl, st) == cudaSuccess ? KVPACK_OK : KVPACK_ERR_CUDA;
    if (pl.shorts > 0)
        return launch_pdl(pg::short_kernel, pl.shorts, 32, pg::kRingBytes, st, p, (int)pl.units) == cudaSuccess
                   ? KVPACK_OK : KVPACK_ERR_CUDA;
    if (launch_pdl(pg::attend_kernel, pl.slots, 32, pg::kRingBytes, st, p) != cudaSuccess)
        return KVPACK_ERR_CUDA;
    const long long rows = pl.units * pl.per_kv;
    // warps per row: so many that each has about four parts
    const long long parts = pl.slots / pl.units + 1;
    cudaError_t e;
    if (parts > 64) e = launch_pdl(pg::join_kernel<32>, (int)rows, 1024, 0, st, p, rows);
    else if (parts > 16) e = launch_pdl(pg::join_kernel<8>, (int)rows, 256, 0, st, p, rows);
    else if (parts > 8) e = launch_pdl(pg::join_kernel<4>, (int)((rows + 1) / 2), 256, 0, st, p, rows);
    else if (parts > 4) e = launch_pdl(pg::join_kernel<2>, (int)((rows + 3) / 4), 256, 0, st, p, rows);
    else {
        const long long blocks = (rows + 7) / 8, most = kPlanSMs * 4;
        e = launch_pdl(pg::join_kernel<1>, (int)(blocks < most ? blocks : most), 256, 0, st, p, rows);
    }
    return e == cudaSuccess ? KVPACK_OK : KVPACK_ERR_CUDA;
}

kvpack_status check_paged_pointers(const void *K, const void *V, const void *table, const void *lens) {
    const void *ptrs[] = {K, V, table, lens};
    for (const void *ptr : ptrs) {
        if (ptr == nullptr) return KVPACK_ERR_INVALID_ARG;
        if (!aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
    }
    return KVPACK_OK;
}

// A text tail in pages (decode_impl's K_text, V_text are then null)
struct PagedText {
    const kvpack_paged_dims *pd;
    const uint16_t *K, *V;
    const int32_t *table, *lens;
};

// 4-bit visual coefficients (quant.cuh) in place of the 16-bit planes
struct Q4Planes {
    const uint8_t *QK_lo, *QK_hi, *QV_lo, *QV_hi;
    const int8_t *EK, *EV;
};

// The decode step; tb (the text tokens compressed with a basis of their own), q4 (4-bit visual
// coefficients, when CK_lo .. CV_hi are null) and pt (the uncompressed tail in pages, when K_text
// and V_text are null) may be null.
kvpack_status decode_impl(const kvpack_dims *d, int32_t n_layers, const uint16_t *q, const uint16_t *CK_lo,
                          const uint16_t *CK_hi, const uint16_t *BK, const uint16_t *CV_lo, const uint16_t *CV_hi,
                          const uint16_t *BV, const Q4Planes *q4, const kvpack_text_basis *tb, const uint16_t *K_text,
                          const uint16_t *V_text, int32_t L_text, const uint32_t *mask, float softmax_scale,
                          uint16_t *out, float *mass, void *ws, size_t ws_bytes, void *stream,
                          const PagedText *pt = nullptr) {
    kvpack_status s = check_dims(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (pt != nullptr) {
        if ((s = check_paged(pt->pd, n_layers)) != KVPACK_OK) return s;
        if (pt->pd->batch != d->batch || pt->pd->n_q_heads != d->n_q_heads || pt->pd->n_kv_heads != d->n_kv_heads)
            return KVPACK_ERR_INVALID_ARG;
        if ((s = check_paged_pointers(pt->K, pt->V, pt->table, pt->lens)) != KVPACK_OK) return s;
    }
    const int L_c = tb != nullptr ? tb->L_c : 0;
    if (tb != nullptr) {
        if (L_c < 0 || L_c > kMaxT) return KVPACK_ERR_INVALID_ARG;
        if (L_c > 0) {
            const void *tp[] = {tb->CK_lo, tb->CK_hi, tb->BK, tb->CV_lo, tb->CV_hi, tb->BV};
            for (const void *ptr : tp) {
                if (ptr == nullptr) return KVPACK_ERR_INVALID_ARG;
                if (!aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
            }
        }
    }
    if (L_text < 0 || L_text > d->L_text_cap) return KVPACK_ERR_INVALID_ARG;
    if (!q || !BK || !BV || !mask || !out) return KVPACK_ERR_INVALID_ARG;
    if (q4 == nullptr && (!CK_lo || !CK_hi || !CV_lo || !CV_hi)) return KVPACK_ERR_INVALID_ARG;
    if (q4 != nullptr) {
        const void *qp[] = {q4->QK_lo, q4->QK_hi, q4->QV_lo, q4->QV_hi, q4->EK, q4->EV};
        for (const void *ptr : qp) {
            if (ptr == nullptr) return KVPACK_ERR_INVALID_ARG;
            if (!aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
        }
    }
    if (L_text > 0 && (!K_text || !V_text)) return KVPACK_ERR_INVALID_ARG;
    if (!(softmax_scale == softmax_scale) || softmax_scale <= 0.f) return KVPACK_ERR_INVALID_ARG;
    const void *ptrs[] = {q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, mask, out, mass, ws,
                          L_text > 0 ? K_text : nullptr, L_text > 0 ? V_text : nullptr};
    for (const void *ptr : ptrs)
        if (ptr && !aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
    const DecodePlan pl = plan_decode(d, n_layers, L_c, pt != nullptr);
    if ((long long)pl.units * d->T_vis * 3 >= (1LL << 31)) return KVPACK_ERR_UNSUPPORTED;   // int32 rows
    if ((long long)pl.units * L_c * 3 >= (1LL << 31)) return KVPACK_ERR_UNSUPPORTED;
    const size_t need = pl.total + (pt != nullptr ? plan_paged(pt->pd, n_layers).total : 0);
    if (ws == nullptr || ws_bytes < need) return KVPACK_ERR_WORKSPACE;
    DeviceInfo *di = nullptr;
    if ((s = device_info(&di)) != KVPACK_OK) return s;

    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if ((s = tensor_map_encoder(&enc)) != KVPACK_OK) return s;
    namespace dc = kvpack::decode;

    const int T = d->T_vis, Hg = pl.Hg, per_kv = d->n_q_heads / d->n_kv_heads;
    const int groups = d->n_kv_heads / KVPACK_GROUP;
    // text chunks: 64 tokens, doubled (up to 1024) while the items would still fill the GPU twice
    // over (148 SMs x 8 warps), so that a long tail on few units keeps many items and a short tail
    // on many units writes one partial per (unit, KV head)
    int ct = kTextChunk;
    while (ct < 1024 && (long long)pl.units * 4 * ((L_text + 2 * ct - 1) / (2 * ct)) >= 2LL * kPlanSMs * 8 * 2) ct <<= 1;
    const int Sc_dense = (L_text + ct - 1) / ct;         // partials the text kernel writes
    const int Sc = pt != nullptr ? 1 : Sc_dense;         // partials that are combined
    const float scale2 = softmax_scale * 1.4426950408889634f;
    unsigned char *w = static_cast<unsigned char *>(ws);
    unsigned char *qt = w + pl.off_qt;
    float *tpart = reinterpret_cast<float *>(w + pl.off_tp);
    float *spart = reinterpret_cast<float *>(w + pl.off_sp);
    float *ustat = reinterpret_cast<float *>(w + pl.off_ustat);
    float *vpart = reinterpret_cast<float *>(w + pl.off_vp);
    unsigned int *counter = reinterpret_cast<unsigned int *>(w + pl.off_counter);
    unsigned char *qt2 = L_c > 0 ? w + pl.off_qt2 : nullptr;
    float *spart2 = L_c > 0 ? reinterpret_cast<float *>(w + pl.off_sp2) : nullptr;
    float *vpart2 = L_c > 0 ? reinterpret_cast<float *>(w + pl.off_vp2) : nullptr;
    uint32_t *mask2 = L_c > 0 ? reinterpret_cast<uint32_t *>(w + pl.off_mask2) : nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);

    // 0. a paged tail's softmax parts, joined to one partial per unit.  The text kernel is a plain
    // launch: it starts after the join has ended, and so does all that reads the partials.
    if (pt != nullptr && (s = launch_paged_attend(pt->pd, n_layers, q, pt->K, pt->V, pt->table, pt->lens, softmax_scale,
                                                  nullptr, nullptr, tpart, w + pl.total, st)) != KVPACK_OK)
        return s;

    // the text kernel's work counter starts at zero; the text tokens' own mask is all ones
    if (cudaMemsetAsync(counter, 0, 4 * sizeof(unsigned int), st) != cudaSuccess) return KVPACK_ERR_CUDA;
    if (L_c > 0 && cudaMemsetAsync(mask2, 0xFF, (size_t)pl.units * pl.nwords2 * sizeof(uint32_t), st) != cudaSuccess)
        return KVPACK_ERR_CUDA;

    // 1. q~ per (unit, KV head) and the text tail partials, one persistent launch
    {
        dc::text::Params tp;
        std::memset(&tp, 0, sizeof(tp));
        if (L_text > 0) {
            const cuuint64_t dims[4] = {128, 4, (cuuint64_t)L_text, (cuuint64_t)pl.units};
            const cuuint64_t strides[3] = {256, 1024, (cuuint64_t)d->L_text_cap * 1024};
            const cuuint32_t box[4] = {64, 1, 16, 1};
            if (!encode_bf16(enc, &tp.tm_k, K_text, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
                !encode_bf16(enc, &tp.tm_v, V_text, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
                return KVPACK_ERR_CUDA;
        }
        {
            const cuuint64_t dims[3] = {512, 64, (cuuint64_t)pl.units};
            const cuuint64_t strides[2] = {1024, 64 * 1024};
            const cuuint32_t box[3] = {64, 64, 1};
            if (!encode_bf16(enc, &tp.tm_bk, BK, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
                return KVPACK_ERR_CUDA;
            if (L_c > 0 && !encode_bf16(enc, &tp.tm_bk2, tb->BK, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
                return KVPACK_ERR_CUDA;
        }
        tp.q = q; tp.part = tpart; tp.qt = qt; tp.qt2 = qt2; tp.counter = counter;
        tp.qsplit = pl.NH == 28 ? 14 : 1 << 30;
        tp.n_units = pl.units; tp.L = L_text; tp.Hg = Hg; tp.per_kv = per_kv; tp.n_q = d->n_q_heads;
        tp.groups = groups; tp.Sc = Sc_dense; tp.ct = ct; tp.n_qitems = pl.units * 4 * (L_c > 0 ? 2 : 1);
        tp.n_items = tp.n_qitems + pl.units * 4 * Sc_dense; tp.scale2 = scale2;
        const int grid = tp.n_items < di->sms ? tp.n_items : di->sms;
        dc::text::text_kernel<<<grid, dc::text::kThreads, dc::text::smem_bytes(), st>>>(tp);
        if (cudaGetLastError() != cudaSuccess) return KVPACK_ERR_CUDA;
    }

    // 2-4. the visual tokens (and the text tokens' own rank space): softmax statistics, the
    // unit-wide statistics, then the value passes
    rs::Params rp;
    std::memset(&rp, 0, sizeof(rp));
    if (q4 != nullptr) {
        rp.QK_lo = q4->QK_lo; rp.QK_hi = q4->QK_hi; rp.QV_lo = q4->QV_lo; rp.QV_hi = q4->QV_hi;
        rp.EK = q4->EK; rp.EV = q4->EV;
    } else {
        const cuuint64_t dims[3] = {16, (cuuint64_t)T, (cuuint64_t)pl.units};
        const cuuint64_t strides[2] = {32, (cuuint64_t)T * 32};
        const cuuint32_t box[3] = {16, 256, 1};
        if (!encode_bf16(enc, &rp.tm_ck, CK_lo, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_32B) ||
            !encode_bf16(enc, &rp.tm_cv, CV_lo, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_32B))
            return KVPACK_ERR_CUDA;
    }
    rp.CK_lo = CK_lo; rp.CK_hi = CK_hi; rp.CV_lo = CV_lo; rp.CV_hi = CV_hi;
    rp.qt = qt; rp.mask = mask; rp.ustat = ustat;
    uint16_t *hipos = reinterpret_cast<uint16_t *>(w + pl.off_hipos);
    int *hicnt = reinterpret_cast<int *>(w + pl.off_hicnt);
    uint16_t *hipos2 = L_c > 0 ? reinterpret_cast<uint16_t *>(w + pl.off_hipos2) : nullptr;
    int *hicnt2 = L_c > 0 ? reinterpret_cast<int *>(w + pl.off_hicnt2) : nullptr;
    rp.hipos = hipos; rp.hicnt = hicnt; rp.Tp = pl.Tp;
    rp.units = pl.units; rp.T = T; rp.Hg = Hg; rp.nwords = pl.nwords; rp.tpu = pl.tpu;
    rp.rank0 = d->rank_lo == 0 ? 1 : 0; rp.ntiles = pl.ntiles;
    rs::Params rp2;
    std::memset(&rp2, 0, sizeof(rp2));
    if (L_c > 0) {
        const cuuint64_t dims[3] = {16, (cuuint64_t)L_c, (cuuint64_t)pl.units};
        const cuuint64_t strides[2] = {32, (cuuint64_t)L_c * 32};
        const cuuint32_t box[3] = {16, 256, 1};
        if (!encode_bf16(enc, &rp2.tm_ck, tb->CK_lo, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_32B) ||
            !encode_bf16(enc, &rp2.tm_cv, tb->CV_lo, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_32B))
            return KVPACK_ERR_CUDA;
        rp2.CK_lo = tb->CK_lo; rp2.CK_hi = tb->CK_hi; rp2.CV_lo = tb->CV_lo; rp2.CV_hi = tb->CV_hi;
        rp2.qt = qt2; rp2.mask = mask2; rp2.ustat = ustat;
        rp2.hipos = hipos2; rp2.hicnt = hicnt2; rp2.Tp = pl.Tp2;
        rp2.units = pl.units; rp2.T = L_c; rp2.Hg = Hg; rp2.nwords = pl.nwords2; rp2.tpu = pl.tpu2;
        rp2.rank0 = 0; rp2.ntiles = pl.ntiles2;
    }
    {
        // each unit's full-rank positions, for the HI tiles of both passes
        // with two consumer groups (28 or 32 heads) the value pass adds the groups' shares of a
        // token's attention mass into the zeroed output
        float *mass0 = pl.NH >= 28 ? mass : nullptr;
        const rs::HiposParams ha{mask, hipos, hicnt, mass0, pl.units, T, pl.nwords, pl.tpu, pl.Tp,
                                 rs::hipos_group(pl.nwords)};
        const rs::HiposParams hb = L_c > 0 ? rs::HiposParams{mask2, hipos2, hicnt2, nullptr, pl.units, L_c, pl.nwords2,
                                                             pl.tpu2, pl.Tp2, rs::hipos_group(pl.nwords2)}
                                           : ha;
        // 256-thread blocks unless a unit's group is larger; enough blocks for the set with the fewer
        // units per block
        const int tpg = ha.tpg > hb.tpg ? ha.tpg : hb.tpg, threads = tpg > 256 ? tpg : 256, upb = threads / tpg;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)((pl.units + upb - 1) / upb), L_c > 0 ? 2u : 1u);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, rs::hipos_kernel, ha, hb) != cudaSuccess) return KVPACK_ERR_CUDA;
    }
    rp.part = spart; rp.nslot = pl.nslot_s; rp.mass = nullptr;
    if (launch_rs<false>(pl.NH, rp, pl.cta_s, st) != cudaSuccess) return KVPACK_ERR_CUDA;
    if (L_c > 0) {
        rp2.part = spart2; rp2.nslot = pl.nslot2; rp2.mass = nullptr;
        if (launch_rs<false>(pl.NH, rp2, pl.cta2, st) != cudaSuccess) return KVPACK_ERR_CUDA;
    }
    const rs::Segs sv{spart, pl.nslot_s, pl.tpu, pl.cta_s, pl.ntiles};
    const rs::Segs s2{spart2, pl.nslot2, pl.tpu2, pl.cta2, pl.ntiles2};
    if (launch_pdl(rs::combine_kernel, (pl.units + 7) / 8, 256, 0, st, sv, s2, (const float *)tpart, ustat, pl.units,
                   Hg, Sc) != cudaSuccess)
        return KVPACK_ERR_CUDA;
    rp.part = vpart; rp.nslot = pl.nslot_v; rp.mass = mass;
    if (launch_rs<true>(pl.NH, rp, pl.cta_v, st) != cudaSuccess) return KVPACK_ERR_CUDA;
    if (L_c > 0) {
        rp2.part = vpart2; rp2.nslot = pl.nslot2; rp2.mass = nullptr;
        if (launch_rs<true>(pl.NH, rp2, pl.cta2, st) != cudaSuccess) return KVPACK_ERR_CUDA;
    }

    // 5. combine the partials and project through B_V (and the text tokens' B_V)
    rs::FinishParams fp{};
    fp.BV = BV; fp.vpart = vpart; fp.tpart = Sc > 0 ? tpart : nullptr; fp.ustat = ustat; fp.out = out;
    fp.Hg = Hg; fp.per_kv = per_kv; fp.n_q = d->n_q_heads; fp.groups = groups; fp.Sc = Sc;
    fp.nslot = pl.nslot_v; fp.tpu = pl.tpu; fp.cta_v = pl.cta_v; fp.ntiles = pl.ntiles;
    if (L_c > 0) {
        fp.BV2 = tb->BV; fp.vpart2 = vpart2; fp.nslot2 = pl.nslot2; fp.tpu2 = pl.tpu2; fp.cta_v2 = pl.cta2;
        fp.ntiles2 = pl.ntiles2;
    }
    if (launch_finish(per_kv, fp, pl.units, di->sms, st) != cudaSuccess) return KVPACK_ERR_CUDA;
    return KVPACK_OK;
}

}  // namespace

extern "C" {

kvpack_status kvpack_decode_attn(const kvpack_dims *d, int32_t n_layers, const uint16_t *q,
                                 const uint16_t *CK_lo, const uint16_t *CK_hi, const uint16_t *BK,
                                 const uint16_t *CV_lo, const uint16_t *CV_hi, const uint16_t *BV,
                                 const uint16_t *K_text, const uint16_t *V_text, int32_t L_text,
                                 const uint32_t *mask, float softmax_scale, uint16_t *out, float *mass,
                                 void *ws, size_t ws_bytes, void *stream) {
    return decode_impl(d, n_layers, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, nullptr, nullptr, K_text, V_text, L_text,
                       mask, softmax_scale, out, mass, ws, ws_bytes, stream);
}

size_t kvpack_decode_tb_workspace(const kvpack_dims *d, int32_t n_layers, int32_t L_c) {
    if (check_dims(d, n_layers) != KVPACK_OK || L_c < 0 || L_c > kMaxT) return 0;
    return plan_decode(d, n_layers, L_c).total;
}

kvpack_status kvpack_decode_attn_tb(const kvpack_dims *d, int32_t n_layers, const uint16_t *q,
                                    const uint16_t *CK_lo, const uint16_t *CK_hi, const uint16_t *BK,
                                    const uint16_t *CV_lo, const uint16_t *CV_hi, const uint16_t *BV,
                                    const kvpack_text_basis *tb, const uint16_t *K_text, const uint16_t *V_text,
                                    int32_t L_text, const uint32_t *mask, float softmax_scale, uint16_t *out,
                                    float *mass, void *ws, size_t ws_bytes, void *stream) {
    if (tb == nullptr) return KVPACK_ERR_INVALID_ARG;
    return decode_impl(d, n_layers, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, nullptr, tb, K_text, V_text, L_text, mask,
                       softmax_scale, out, mass, ws, ws_bytes, stream);
}

kvpack_status kvpack_quantize4(const kvpack_dims *d, int32_t n_layers, int32_t T, const uint16_t *C_lo,
                               const uint16_t *C_hi, uint8_t *Q_lo, uint8_t *Q_hi, int8_t *E, void *stream) {
    kvpack_status s = check_dims(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (T < 1 || T > kMaxT) return KVPACK_ERR_INVALID_ARG;
    if (!C_lo || !C_hi || !Q_lo || !Q_hi || !E) return KVPACK_ERR_INVALID_ARG;
    const void *ptrs[] = {C_lo, C_hi, Q_lo, Q_hi, E};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
    const long long rows = (long long)n_units(d, n_layers) * T;
    const long long blocks = (rows + 255) / 256;
    kvpack::quant::quantize4_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        C_lo, C_hi, Q_lo, Q_hi, E, rows);
    return cudaGetLastError() == cudaSuccess ? KVPACK_OK : KVPACK_ERR_CUDA;
}

kvpack_status kvpack_decode_attn_q4(const kvpack_dims *d, int32_t n_layers, const uint16_t *q,
                                    const uint8_t *QK_lo, const uint8_t *QK_hi, const int8_t *EK, const uint16_t *BK,
                                    const uint8_t *QV_lo, const uint8_t *QV_hi, const int8_t *EV, const uint16_t *BV,
                                    const uint16_t *K_text, const uint16_t *V_text, int32_t L_text,
                                    const uint32_t *mask, float softmax_scale, uint16_t *out, float *mass, void *ws,
                                    size_t ws_bytes, void *stream) {
    const Q4Planes q4{QK_lo, QK_hi, QV_lo, QV_hi, EK, EV};
    return decode_impl(d, n_layers, q, nullptr, nullptr, BK, nullptr, nullptr, BV, &q4, nullptr, K_text, V_text, L_text,
                       mask, softmax_scale, out, mass, ws, ws_bytes, stream);
}

}  // extern "C"

// ------------------------------------------------------------------ decode without allocation
//
// For callers that cannot give the library device memory (a framework-owned
// plugin with no workspace hook, a serving loop that bans allocator calls):
// the decode scratch lives in this fixed device array, which every GPU holds
// from the library's first use there until exit.  Host code must not pass the
// array's name to a kernel -- on the host it is only a stand-in -- so its
// device address is looked up with the caller's device current.  The lookup
// runs on every call and is not cached: a context torn down and created
// again (cudaDeviceReset) places the array at a new address.

namespace {

static __device__ __align__(256) unsigned char g_noalloc_scratch[KVPACK_NOALLOC_SCRATCH_BYTES];

kvpack_status noalloc_scratch(void **out) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) return KVPACK_ERR_CUDA;
    *out = p;
    return KVPACK_OK;
}

}  // namespace

extern "C" {

size_t kvpack_noalloc_scratch_bytes(void) { return KVPACK_NOALLOC_SCRATCH_BYTES; }

kvpack_status kvpack_decode_attn_noalloc(const kvpack_dims *d, int32_t n_layers, const uint16_t *q,
                                         const uint16_t *CK_lo, const uint16_t *CK_hi, const uint16_t *BK,
                                         const uint16_t *CV_lo, const uint16_t *CV_hi, const uint16_t *BV,
                                         const uint16_t *K_text, const uint16_t *V_text, int32_t L_text,
                                         const uint32_t *mask, float softmax_scale, uint16_t *out, float *mass,
                                         void *stream) {
    kvpack_status s = check_dims(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (plan_decode(d, n_layers).total > KVPACK_NOALLOC_SCRATCH_BYTES) return KVPACK_ERR_WORKSPACE;
    void *ws = nullptr;
    if ((s = noalloc_scratch(&ws)) != KVPACK_OK) return s;
    return kvpack_decode_attn(d, n_layers, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, K_text, V_text, L_text, mask,
                              softmax_scale, out, mass, ws, KVPACK_NOALLOC_SCRATCH_BYTES, stream);
}

// ------------------------------------------------------------------ baselines

namespace {

size_t dense_workspace(int units, int Hg, int L_cap) {
    const int Sc = (L_cap + kvpack::baseline::kDenseChunk - 1) / kvpack::baseline::kDenseChunk;
    return align256((size_t)units * (Sc > 0 ? Sc : 1) * Hg * kvpack::decode::kTxtPart * sizeof(float)) + 256;
}

cudaError_t launch_dense_finish(int per_kv, const kvpack::baseline::DenseFinishParams &fp, int units, cudaStream_t st) {
    namespace bl = kvpack::baseline;
    const int grid = units * 4;
    switch (per_kv) {
        case 1: bl::dense_finish_kernel<1><<<grid, 128, 0, st>>>(fp); break;
        case 2: bl::dense_finish_kernel<2><<<grid, 128, 0, st>>>(fp); break;
        case 3: bl::dense_finish_kernel<3><<<grid, 128, 0, st>>>(fp); break;
        case 4: bl::dense_finish_kernel<4><<<grid, 128, 0, st>>>(fp); break;
        case 5: bl::dense_finish_kernel<5><<<grid, 128, 0, st>>>(fp); break;
        case 6: bl::dense_finish_kernel<6><<<grid, 128, 0, st>>>(fp); break;
        case 7: bl::dense_finish_kernel<7><<<grid, 128, 0, st>>>(fp); break;
        default: bl::dense_finish_kernel<8><<<grid, 128, 0, st>>>(fp); break;
    }
    return cudaGetLastError();
}

}  // namespace

extern "C" {

size_t kvpack_dense_decode_workspace(const kvpack_dims *d, int32_t n_layers, int32_t L_cap) {
    if (check_dims(d, n_layers) != KVPACK_OK || L_cap < 1) return 0;
    return dense_workspace(n_units(d, n_layers), hg(d), L_cap);
}

kvpack_status kvpack_dense_decode_attn(const kvpack_dims *d, int32_t n_layers, const uint16_t *q, const uint16_t *K,
                                       const uint16_t *V, int32_t L_cap, int32_t L, float softmax_scale,
                                       uint16_t *out, void *ws, size_t ws_bytes, void *stream) {
    kvpack_status s = check_dims(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (L_cap < 1 || L < 1 || L > L_cap || (long long)L_cap > 4LL * KVPACK_MAX_T) return KVPACK_ERR_INVALID_ARG;
    if (!q || !K || !V || !out) return KVPACK_ERR_INVALID_ARG;
    if (!(softmax_scale == softmax_scale) || softmax_scale <= 0.f) return KVPACK_ERR_INVALID_ARG;
    const void *ptrs[] = {q, K, V, out, ws};
    for (const void *ptr : ptrs)
        if (ptr && !aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
    const int units = n_units(d, n_layers), Hg = hg(d), per_kv = d->n_q_heads / d->n_kv_heads;
    const size_t need = dense_workspace(units, Hg, L_cap);
    if (ws == nullptr || ws_bytes < need) return KVPACK_ERR_WORKSPACE;
    DeviceInfo *di = nullptr;
    if ((s = device_info(&di)) != KVPACK_OK) return s;
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if ((s = tensor_map_encoder(&enc)) != KVPACK_OK) return s;
    namespace dc = kvpack::decode;
    const int ct = kvpack::baseline::kDenseChunk, Sc = (L + ct - 1) / ct;
    unsigned char *w = static_cast<unsigned char *>(ws);
    float *tpart = reinterpret_cast<float *>(w);
    unsigned int *counter = reinterpret_cast<unsigned int *>(w + need - 256);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(counter, 0, 4 * sizeof(unsigned int), st) != cudaSuccess) return KVPACK_ERR_CUDA;
    dc::text::Params tp;
    std::memset(&tp, 0, sizeof(tp));
    {
        const cuuint64_t dims[4] = {128, 4, (cuuint64_t)L, (cuuint64_t)units};
        const cuuint64_t strides[3] = {256, 1024, (cuuint64_t)L_cap * 1024};
        const cuuint32_t box[4] = {64, 1, 16, 1};
        if (!encode_bf16(enc, &tp.tm_k, K, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_bf16(enc, &tp.tm_v, V, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return KVPACK_ERR_CUDA;
    }
    tp.q = q; tp.part = tpart; tp.qt = nullptr; tp.counter = counter;
    tp.qsplit = 1 << 30;
    tp.n_units = units; tp.L = L; tp.Hg = Hg; tp.per_kv = per_kv; tp.n_q = d->n_q_heads;
    tp.groups = d->n_kv_heads / KVPACK_GROUP; tp.Sc = Sc; tp.ct = ct; tp.n_qitems = 0;
    tp.n_items = units * 4 * Sc; tp.scale2 = softmax_scale * 1.4426950408889634f;
    const int grid = tp.n_items < di->sms ? tp.n_items : di->sms;
    dc::text::text_kernel<<<grid, dc::text::kThreads, dc::text::smem_bytes(), st>>>(tp);
    if (cudaGetLastError() != cudaSuccess) return KVPACK_ERR_CUDA;
    kvpack::baseline::DenseFinishParams fp{tpart, out, Hg, d->n_q_heads, d->n_kv_heads / KVPACK_GROUP, Sc};
    return launch_dense_finish(per_kv, fp, units, st) == cudaSuccess ? KVPACK_OK : KVPACK_ERR_CUDA;
}

kvpack_status kvpack_decompress(const kvpack_dims *d, int32_t n_layers, const uint16_t *CK_lo, const uint16_t *CK_hi,
                                const uint16_t *BK, const uint16_t *CV_lo, const uint16_t *CV_hi, const uint16_t *BV,
                                const uint32_t *mask, uint16_t *K_out, uint16_t *V_out, int32_t L_cap, void *stream) {
    kvpack_status s = check_dims(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (L_cap < d->T_vis) return KVPACK_ERR_INVALID_ARG;
    if (!CK_lo || !CK_hi || !BK || !CV_lo || !CV_hi || !BV || !mask || !K_out || !V_out) return KVPACK_ERR_INVALID_ARG;
    const void *ptrs[] = {CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, mask, K_out, V_out};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
    DeviceInfo *di = nullptr;
    if ((s = device_info(&di)) != KVPACK_OK) return s;
    namespace bl = kvpack::baseline;
    bl::DecompressParams p{};
    p.C_lo[0] = CK_lo; p.C_hi[0] = CK_hi; p.B[0] = BK;
    p.C_lo[1] = CV_lo; p.C_hi[1] = CV_hi; p.B[1] = BV;
    p.mask = mask; p.out[0] = K_out; p.out[1] = V_out;
    p.T = d->T_vis; p.L_cap = L_cap; p.nwords = (d->T_vis + 31) / 32;
    p.tiles = (d->T_vis + bl::kDecTok - 1) / bl::kDecTok; p.rank_lo = d->rank_lo;
    const long long grid = (long long)n_units(d, n_layers) * p.tiles;
    if (grid >= (1LL << 31)) return KVPACK_ERR_UNSUPPORTED;
    bl::decompress_kernel<<<(unsigned)grid, bl::kDecThreads, sizeof(bl::DecSmem), static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? KVPACK_OK : KVPACK_ERR_CUDA;
}

}  // extern "C"

// ------------------------------------------------------------------ bounded-wait self-test

namespace {

// One thread announces a 16-byte transfer on a fresh barrier and waits for it; no copy is
// issued, so the library's bounded wait must give up after `cycles`, record
// KVPACK_ERR_TIMEOUT in the error word and return.
__global__ void wait_selftest_kernel(long long cycles) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        kvpack::mbar_init(&bar, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        kvpack::mbar_arrive_tx(&bar, 16u);
        kvpack::mbar_wait_for(&bar, 0u, &abort_flag, cycles);
    }
}

}  // namespace

extern "C" kvpack_status kvpack_selftest_bounded_wait(int64_t cycles, void *stream) {
    if (cycles < 1 || cycles > kvpack::kWaitCycles) return KVPACK_ERR_INVALID_ARG;
    wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>((long long)cycles);
    return cudaGetLastError() == cudaSuccess ? KVPACK_OK : KVPACK_ERR_CUDA;
}

// ------------------------------------------------------------------ select

kvpack_status kvpack_select(const kvpack_dims *d, int32_t n_layers, const float *mass, float *score, float alpha,
                            int32_t k_hi, uint32_t *mask_out, void *stream) {
    kvpack_status s = check_dims(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (!mass || !mask_out) return KVPACK_ERR_INVALID_ARG;
    if (k_hi < 0 || k_hi > d->T_vis) return KVPACK_ERR_INVALID_ARG;
    if (!(alpha >= 0.f && alpha < 1.f)) return KVPACK_ERR_INVALID_ARG;
    if (alpha != 0.f && score == nullptr) return KVPACK_ERR_INVALID_ARG;
    if (!aligned16(mass) || !aligned16(mask_out) || (score && !aligned16(score))) return KVPACK_ERR_ALIGNMENT;
    DeviceInfo *di = nullptr;
    if ((s = device_info(&di)) != KVPACK_OK) return s;
    kvpack::select::Params p{};
    p.mass = mass; p.score = score; p.alpha = alpha; p.k = k_hi; p.T = d->T_vis;
    p.nwords = (d->T_vis + 31) / 32; p.n_units = n_units(d, n_layers); p.mask = mask_out;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const int T = d->T_vis;
    namespace sl = kvpack::select;
    if (T <= 32 * 64) {
        // rows of 32 tokens, rounded up to an instantiated count
        const int rows = (T + 31) / 32;
        if (rows <= 1) e = launch_select_warp<1>(p, st);
        else if (rows <= 2) e = launch_select_warp<2>(p, st);
        else if (rows <= 4) e = launch_select_warp<4>(p, st);
        else if (rows <= 8) e = launch_select_warp<8>(p, st);
        else if (rows <= 12) e = launch_select_warp<12>(p, st);
        else if (rows <= 16) e = launch_select_warp<16>(p, st);
        else if (rows <= 18) e = launch_select_warp<18>(p, st);
        else if (rows <= 24) e = launch_select_warp<24>(p, st);
        else if (rows <= 32) e = launch_select_warp<32>(p, st);
        else if (rows <= 48) e = launch_select_warp<48>(p, st);
        else e = launch_select_warp<64>(p, st);
    } else if (T <= sl::kBlockThreads * 32) {
        // rows of 256 tokens (9 to 32 here), rounded up to an instantiated count
        const int rows = (T + sl::kBlockThreads - 1) / sl::kBlockThreads;
        if (rows <= 9) e = launch_select_block<9>(p, st);
        else if (rows <= 12) e = launch_select_block<12>(p, st);
        else if (rows <= 16) e = launch_select_block<16>(p, st);
        else if (rows <= 20) e = launch_select_block<20>(p, st);
        else if (rows <= 25) e = launch_select_block<25>(p, st);
        else e = launch_select_block<32>(p, st);
    } else {
        int kpt = 1;
        while (sl::kClusterCtas * sl::kClusterThreads * kpt < T) kpt <<= 1;
        switch (kpt) {
            case 1: e = launch_select_cluster<1>(p, st); break;
            case 2: e = launch_select_cluster<2>(p, st); break;
            case 4: e = launch_select_cluster<4>(p, st); break;
            case 8: e = launch_select_cluster<8>(p, st); break;
            case 16: e = launch_select_cluster<16>(p, st); break;
            default: e = launch_select_cluster<32>(p, st); break;
        }
    }
    return (e == cudaSuccess) ? KVPACK_OK : KVPACK_ERR_CUDA;
}

// ------------------------------------------------------------------ compress

size_t kvpack_compress_workspace(const kvpack_dims *d, int32_t n_layers) {
    if (check_dims(d, n_layers) != KVPACK_OK) return 0;
    return kvpack::compress::workspace_bytes(n_units(d, n_layers), d->T_vis);
}

kvpack_status kvpack_compress(const kvpack_dims *d, int32_t n_layers, const uint16_t *X, uint16_t *C_lo,
                              uint16_t *C_hi, uint16_t *B, float *sigma, void *ws, size_t ws_bytes, void *stream) {
    kvpack_status s = check_dims(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (!X || !C_lo || !C_hi || !B) return KVPACK_ERR_INVALID_ARG;
    const void *ptrs[] = {X, C_lo, C_hi, B, sigma, ws};
    for (const void *ptr : ptrs)
        if (ptr && !aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
    const int units = n_units(d, n_layers);
    if (ws == nullptr || ws_bytes < kvpack::compress::workspace_bytes(units, d->T_vis)) return KVPACK_ERR_WORKSPACE;
    DeviceInfo *di = nullptr;
    if ((s = device_info(&di)) != KVPACK_OK) return s;
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if ((s = tensor_map_encoder(&enc)) != KVPACK_OK) return s;
    CUtensorMap tm_x;
    {
        const cuuint64_t dims[3] = {512, (cuuint64_t)d->T_vis, (cuuint64_t)units};
        const cuuint64_t strides[2] = {1024, (cuuint64_t)d->T_vis * 1024};
        const cuuint32_t box[3] = {64, 64, 1};
        if (!encode_bf16(enc, &tm_x, X, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return KVPACK_ERR_CUDA;
    }
    // KVPACK_EIG_MAX_ITER (1 .. the built-in cap) lowers the eigen-solver's iteration cap: a test
    // knob that drives the KVPACK_ERR_NOCONVERGE path without any change to the inputs
    int max_iter = kvpack::compress::kMaxIter;
    if (const char *e = std::getenv("KVPACK_EIG_MAX_ITER")) {
        const int v = std::atoi(e);
        if (v >= 1 && v < max_iter) max_iter = v;
    }
    return kvpack::compress::run(units, d->T_vis, X, tm_x, C_lo, C_hi, B, sigma, ws, di->sms, max_iter,
                                 static_cast<cudaStream_t>(stream));
}

}  // extern "C"

// ------------------------------------------------------------------ positions and the paged cache

namespace {

namespace rp = kvpack::rope;

kvpack_status check_spec(const kvpack_rope_spec *r) {
    if (r->rotary_dim <= 0 || r->n_axes <= 0 || (r->adjacent != 0 && r->adjacent != 1)) return KVPACK_ERR_INVALID_ARG;
    if (r->rotary_dim % 16 != 0 || r->rotary_dim > KVPACK_HEAD_DIM || r->n_axes > KVPACK_MAX_AXES)
        return KVPACK_ERR_UNSUPPORTED;
    for (int i = 0; i < r->rotary_dim / 2; ++i)
        if (r->axis[i] >= r->n_axes) return KVPACK_ERR_INVALID_ARG;
    return KVPACK_OK;
}

kvpack_status check_heads(const kvpack_heads *v) {
    if (v == nullptr || v->data == nullptr) return KVPACK_ERR_INVALID_ARG;
    if (!aligned16(v->data) || v->outer_stride % 8 != 0 || v->row_stride % 8 != 0 || v->group_stride % 8 != 0)
        return KVPACK_ERR_ALIGNMENT;
    return KVPACK_OK;
}

// An output is its input (rotation in place) only with the same strides, and its rows do not share memory.
kvpack_status check_pair(const kvpack_heads *in, const kvpack_heads *out, int32_t outer, int32_t rows, int32_t n) {
    kvpack_status s = check_heads(in);
    if (s == KVPACK_OK) s = check_heads(out);
    if (s != KVPACK_OK) return s;
    if (in->data == out->data && (in->outer_stride != out->outer_stride || in->row_stride != out->row_stride ||
                                  in->group_stride != out->group_stride))
        return KVPACK_ERR_INVALID_ARG;
    if ((outer > 1 && out->outer_stride == 0) || (rows > 1 && out->row_stride == 0) || (n > 4 && out->group_stride == 0))
        return KVPACK_ERR_INVALID_ARG;
    return KVPACK_OK;
}

inline rp::View view(const kvpack_heads *v) {
    return rp::View{v->data, v->outer_stride, v->row_stride, v->group_stride};
}

void set_spec(rp::Params &p, const kvpack_rope_spec *r, const double *freq, const int32_t *pos, bool inverse) {
    p.sign = inverse ? -1.f : 1.f;
    if (r == nullptr) return;
    p.freq = freq;
    p.pos = pos;
    p.rot8 = r->rotary_dim / 16;
    for (int i = 0; i < r->rotary_dim / 2; ++i) p.axis2[i >> 4] |= (uint32_t)r->axis[i] << (2 * (i & 15));
}

template <bool APPEND, int U>
cudaError_t launch_rope_u(const rp::Params &p, long long grid, bool adjacent, cudaStream_t st) {
    return adjacent ? launch_pdl(rp::rope_kernel<APPEND, true, U>, (int)grid, rp::kThreads, 0, st, p)
                    : launch_pdl(rp::rope_kernel<APPEND, false, U>, (int)grid, rp::kThreads, 0, st, p);
}

// A row's quads of heads are split over warps while the rows leave warps of the GPU free: one each where all
// fit at once, else shares of two and more, up to two waves (2500 rows of 64 heads 16.6 us; 21.3 with a warp
// per row), or three where a warp per row would half fill the second (6000 rows 34.0 us; 36.1).  Quads on the way at a time: four in the rotation of many rows (100352 rows of 32 heads 247 us;
// 258 with three, 263 with two), three in the append, whose stores scatter (53 k rows of 36 heads 151 us; 155
// with two, 162 with four), fewer where a warp has few.
template <bool APPEND>
kvpack_status launch_rope(rp::Params &p, long long orows, bool adjacent, cudaStream_t st) {
    const long long warps = (long long)kPlanSMs * rp::kWarpsPerSM;
    long long splits = 2 * warps / orows;
    if (splits == 1 && orows > warps && 3 * warps >= 2 * orows && p.quads >= 6) splits = 2;
    if (orows * p.quads <= warps) splits = p.quads;
    else if (splits > p.quads / 2) splits = p.quads / 2;
    if (splits < 1) splits = 1;
    p.qpw = (int)((p.quads + splits - 1) / splits);
    p.splits = (p.quads + p.qpw - 1) / p.qpw;
    p.items = orows * p.splits;
    const long long grid = (p.items + rp::kThreads / 32 - 1) / (rp::kThreads / 32);
    if (grid > 0x7fffffffLL) return KVPACK_ERR_UNSUPPORTED;
    const int most = APPEND ? (p.splits > 1 ? 2 : 3) : (p.splits > 1 ? 3 : 4);
    cudaError_t e;
    if (most == 2 || p.qpw < 3 || (APPEND && p.quads < 6)) e = launch_rope_u<APPEND, 2>(p, grid, adjacent, st);
    else if (most == 3 || p.qpw < 4) e = launch_rope_u<APPEND, 3>(p, grid, adjacent, st);
    else e = launch_rope_u<APPEND, APPEND ? 3 : 4>(p, grid, adjacent, st);
    return e == cudaSuccess ? KVPACK_OK : KVPACK_ERR_CUDA;
}

}  // namespace

extern "C" {

kvpack_status kvpack_rope(const kvpack_rope_spec *spec, const double *freq, const int32_t *pos, int32_t n_outer,
                          int32_t n_rows, int32_t n_q, const kvpack_heads *q, const kvpack_heads *q_out, int32_t n_k,
                          const kvpack_heads *k, const kvpack_heads *k_out, int32_t inverse, void *stream) {
    if (spec == nullptr || n_outer <= 0 || n_rows < 0 || n_q < 0 || n_k < 0 || (n_q == 0 && n_k == 0))
        return KVPACK_ERR_INVALID_ARG;
    kvpack_status s = check_spec(spec);
    if (s != KVPACK_OK) return s;
    if (n_q > 1024 || n_k > 1024) return KVPACK_ERR_UNSUPPORTED;
    if (n_rows == 0) return KVPACK_OK;
    if (!freq || !pos) return KVPACK_ERR_INVALID_ARG;
    if (!aligned16(freq) || !aligned16(pos)) return KVPACK_ERR_ALIGNMENT;
    if (n_q > 0 && (s = check_pair(q, q_out, n_outer, n_rows, n_q)) != KVPACK_OK) return s;
    if (n_k > 0 && (s = check_pair(k, k_out, n_outer, n_rows, n_k)) != KVPACK_OK) return s;
    rp::Params p{};
    if (n_q > 0) { p.q = view(q); p.q_out = view(q_out); }
    if (n_k > 0) { p.k = view(k); p.k_out = view(k_out); }
    set_spec(p, spec, freq, pos, inverse != 0);
    p.rows = n_rows;
    p.pos_outer = n_rows;
    p.pos_axis = (long long)n_outer * n_rows;
    p.n_q = n_q; p.n_k = n_k;
    p.quads_q = (n_q + 3) / 4; p.quads_k = (n_k + 3) / 4; p.quads = p.quads_q + p.quads_k;
    return launch_rope<false>(p, (long long)n_outer * n_rows, spec->adjacent != 0, static_cast<cudaStream_t>(stream));
}

kvpack_status kvpack_paged_append(const kvpack_paged_dims *d, int32_t n_layers, const kvpack_rope_spec *spec,
                                  const double *freq, const int32_t *pos, int32_t n_rows, const kvpack_heads *q,
                                  const kvpack_heads *k, const kvpack_heads *v, const int32_t *row_offsets,
                                  const int32_t *seq_lens, const int32_t *block_table, const kvpack_heads *q_out,
                                  uint16_t *K_pages, uint16_t *V_pages, void *stream) {
    kvpack_status s = check_paged(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (n_rows < 0 || (row_offsets == nullptr && n_rows != d->batch)) return KVPACK_ERR_INVALID_ARG;
    if (spec != nullptr && (s = check_spec(spec)) != KVPACK_OK) return s;
    if (n_rows == 0) return KVPACK_OK;
    if (spec != nullptr && (!freq || !pos)) return KVPACK_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr)) return KVPACK_ERR_INVALID_ARG;
    if ((s = check_heads(k)) != KVPACK_OK || (s = check_heads(v)) != KVPACK_OK) return s;
    if (q != nullptr && (s = check_pair(q, q_out, n_layers, n_rows, d->n_q_heads)) != KVPACK_OK) return s;
    if ((s = check_paged_pointers(K_pages, V_pages, block_table, seq_lens)) != KVPACK_OK) return s;
    const void *ptrs[] = {freq, pos, row_offsets};
    for (const void *ptr : ptrs)
        if (ptr && !aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
    rp::Params p{};
    if (q != nullptr) { p.q = view(q); p.q_out = view(q_out); }
    p.k = view(k);
    p.v = view(v);
    set_spec(p, spec, freq, pos, false);
    p.rows = n_rows;
    p.pos_axis = n_rows;
    p.pos_outer = 0;
    p.n_q = q != nullptr ? d->n_q_heads : 0;
    p.n_k = d->n_kv_heads;
    p.quads_q = (p.n_q + 3) / 4; p.quads_k = (p.n_k + 3) / 4; p.quads = p.quads_q + 2 * p.quads_k;
    p.K = K_pages; p.V = V_pages; p.table = block_table; p.lens = seq_lens; p.offsets = row_offsets;
    p.batch = d->batch; p.n_pages = d->n_pages; p.max_pages = d->max_pages; p.page_shift = log2_exact(d->page_size);
    return launch_rope<true>(p, (long long)n_layers * n_rows, spec != nullptr && spec->adjacent != 0,
                             static_cast<cudaStream_t>(stream));
}

size_t kvpack_paged_decode_workspace(const kvpack_paged_dims *d, int32_t n_layers) {
    if (check_paged(d, n_layers) != KVPACK_OK) return 0;
    return plan_paged(d, n_layers).total;
}

kvpack_status kvpack_paged_decode_attn(const kvpack_paged_dims *d, int32_t n_layers, const uint16_t *q,
                                       const uint16_t *K_pages, const uint16_t *V_pages, const int32_t *block_table,
                                       const int32_t *seq_lens, float softmax_scale, uint16_t *out, float *lse, void *ws,
                                       size_t ws_bytes, void *stream) {
    kvpack_status s = check_paged(d, n_layers);
    if (s != KVPACK_OK) return s;
    if (!q || !out) return KVPACK_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.f) || softmax_scale > 3.402823466e38f) return KVPACK_ERR_INVALID_ARG;
    if ((s = check_paged_pointers(K_pages, V_pages, block_table, seq_lens)) != KVPACK_OK) return s;
    const void *ptrs[] = {q, out, lse, ws};
    for (const void *ptr : ptrs)
        if (ptr && !aligned16(ptr)) return KVPACK_ERR_ALIGNMENT;
    if (ws == nullptr || ws_bytes < plan_paged(d, n_layers).total) return KVPACK_ERR_WORKSPACE;
    DeviceInfo *di = nullptr;                            // kernel attributes of the device
    if ((s = device_info(&di)) != KVPACK_OK) return s;
    return launch_paged_attend(d, n_layers, q, K_pages, V_pages, block_table, seq_lens, softmax_scale, out, lse, nullptr,
                               ws, static_cast<cudaStream_t>(stream));
}

size_t kvpack_decode_paged_workspace(const kvpack_dims *d, const kvpack_paged_dims *pd, int32_t n_layers) {
    if (check_dims(d, n_layers) != KVPACK_OK || check_paged(pd, n_layers) != KVPACK_OK) return 0;
    return plan_decode(d, n_layers, 0, true).total + plan_paged(pd, n_layers).total;
}

kvpack_status kvpack_decode_attn_paged(const kvpack_dims *d, const kvpack_paged_dims *pd, int32_t n_layers,
                                       const uint16_t *q, const uint16_t *CK_lo, const uint16_t *CK_hi,
                                       const uint16_t *BK, const uint16_t *CV_lo, const uint16_t *CV_hi,
                                       const uint16_t *BV, const uint16_t *K_pages, const uint16_t *V_pages,
                                       const int32_t *block_table, const int32_t *seq_lens, const uint32_t *mask,
                                       float softmax_scale, uint16_t *out, float *mass, void *ws, size_t ws_bytes,
                                       void *stream) {
    const PagedText pt{pd, K_pages, V_pages, block_table, seq_lens};
    return decode_impl(d, n_layers, q, CK_lo, CK_hi, BK, CV_lo, CV_hi, BV, nullptr, nullptr, nullptr, nullptr, 0, mask,
                       softmax_scale, out, mass, ws, ws_bytes, stream, &pt);
}

}  // extern "C"
