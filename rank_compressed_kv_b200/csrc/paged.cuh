// paged.cuh -- attention of one new token per sequence over a paged cache, split over the
// cache's length and joined.
//
// Per (layer, sequence b, KV head) unit and query head h, over the sequence's len_b tokens:
//   s_t = scale q_h . K_t,   out_h = sum_t e^(s_t - m) V_t / l,   l = sum_t e^(s_t - m),
//   lse_h = m + ln l          (logits in the log2 domain: the scale folds log2 e)
// One pass keeps the running maximum and sum.  The tokens of all units are cut into tiles of 16
// (a page holds whole tiles) and the tiles, in unit order, into equal runs, one per warp, whatever
// the lengths: ragged batches keep every warp busy to the end.  A unit inside one run is finished
// by its warp; of the others each warp leaves its part (m, l, sum p V), and join_kernel adds the
// parts in their order.  The runs depend on the lengths alone, so repeated calls give equal bits.
#pragma once

#include "common.cuh"
#include "decode.cuh"

namespace kvpack {
namespace paged {

constexpr int kTile = 16;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlocksPerSM = 3;
constexpr int kMinTiles = 2;        // shortest run of a warp
constexpr int kMaxBatch = 4096;
constexpr float kLn2 = 0.69314718055994531f;

struct Params {
    const uint16_t *q, *K, *V;      // [layers * batch][n_q][128], [layers][n_pages][n_kv][page][128]
    const int32_t *table, *lens;
    uint16_t *out;                  // [layers * batch][n_q][128], or null: tpart
    float *lse;                     // [layers * batch][n_q] or null
    float *tpart;                   // [layers * batch][n_q][kTxtPart]: (m, l, sum p V) of each head, or null
    float *stat;                    // [2 * warps][8][2]: m, l of a run's part; slot 2 w for the unit that an
    float *acc;                     // [2 * warps][per_kv][128]     earlier warp began, 2 w + 1 for the one it leaves
    int2 *desc;                     // [units]: first warp and number of parts
    int layers, batch, n_kv, per_kv, n_pages, max_pages, page_shift, warps;
    float scale2;
};

struct Cursor {
    int b, lk, t, nt, len;          // sequence, layer * n_kv + KV head, tile, tiles and length of the sequence
};

// Tiles of every sequence, summed up: pre[b] tiles (of one layer and KV head) before sequence b.
__device__ __forceinline__ int clamped_len(const Params &p, int b, bool report) {
    const long long cap = (long long)p.max_pages << p.page_shift;
    int len = __ldg(p.lens + b);
    if (len < 0 || len > cap) {
        if (report) report_error(KVPACK_ERR_PAGE);
        len = len < 0 ? 0 : (int)cap;
    }
    return len;
}

__device__ __forceinline__ void scan_tiles(const Params &p, long long *pre) {
    __shared__ long long wsum[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long carry = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
        const int b = b0 + tid;
        long long v = b < p.batch ? (clamped_len(p, b, blockIdx.x == 0) + kTile - 1) / kTile : 0;
        #pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += o;
        }
        if (lane == 31) wsum[warp] = v;
        __syncthreads();
        long long before = carry;
        for (int w = 0; w < warp; ++w) before += wsum[w];
        if (b < p.batch) pre[b + 1] = before + v;
        for (int w = 0; w < kWarps; ++w) carry += wsum[w];
        __syncthreads();
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
}

__device__ __forceinline__ uint4 ldg_stream(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// No shared memory holds keys or values: the order of the 128 entries of q . K is free as long as
// q and K share it, and so is the order of the output's entries, so a lane's 16-byte loads are the
// operands of the matrix instructions as they are (K), or after one byte permutation that pairs
// two tokens (V).  Lane 4 g + t:
//   S (16 tokens x 8 heads) = K q^T: row g of K, entries 32 i + 8 t .. + 7 for k-steps 2 i, 2 i + 1
//   O^T (128 x 8 heads) += V^T P: tokens 2t, 2t + 1, 2t + 8, 2t + 9, entries 8 g .. 8 g + 7 (+ 64)
// P goes in as bf16 hi + lo (two products): rounding it to bf16 once would add as much error as
// the rounding of the output.
__global__ void __launch_bounds__(kThreads, kBlocksPerSM) attend_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) long long pre[];     // [batch + 1]
    griddep_launch_dependents();
    scan_tiles(p, pre);
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    const int LK = p.layers * p.n_kv;
    const long long total = pre[p.batch] * LK;
    const long long most = total / kMinTiles;
    const long long W = most < 1 ? 1 : most < p.warps ? most : p.warps;
    // neighbouring runs go to different SMs, so that few runs spread over all of them
    const long long w = (long long)(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
    if (w >= W) return;
    const long long x0 = w * total / W, x1 = (w + 1) * total / W;
    if (x0 >= x1) return;

    Cursor ld{};
    {
        int lo = 0, hi = p.batch;                        // the sequence with pre[b] LK <= x0 < pre[b + 1] LK
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] * LK <= x0) lo = mid; else hi = mid;
        }
        ld.b = lo;
        ld.nt = (int)(pre[lo + 1] - pre[lo]);
        ld.len = clamped_len(p, lo, false);
        const long long rem = x0 - pre[lo] * LK;
        ld.lk = (int)(rem / ld.nt);
        ld.t = (int)(rem % ld.nt);
    }
    const int page_mask = (1 << p.page_shift) - 1;
    auto advance = [&](Cursor &c) {
        if (++c.t < c.nt) return;
        c.t = 0;
        if (++c.lk < LK) return;
        c.lk = 0;
        do ++c.b; while (c.b < p.batch && pre[c.b + 1] == pre[c.b]);
        if (c.b < p.batch) {
            c.nt = (int)(pre[c.b + 1] - pre[c.b]);
            c.len = clamped_len(p, c.b, false);
        }
    };
    auto page_of = [&](const Cursor &c) {
        return __ldg(p.table + (long long)c.b * p.max_pages + ((c.t * kTile) >> p.page_shift));
    };
    // element offset of a tile's first row; n = its valid tokens (none where the page is out of range)
    auto tile_at = [&](const Cursor &c, int page, int &n) {
        n = min(kTile, c.len - c.t * kTile);
        if (page < 0 || page >= p.n_pages) {
            if (lane == 0) report_error(KVPACK_ERR_PAGE);
            n = 0;
            page = 0;
        }
        const int layer = c.lk / p.n_kv, kvh = c.lk - layer * p.n_kv;
        return (((((long long)layer * p.n_pages + page) * p.n_kv + kvh) << p.page_shift) + ((c.t * kTile) & page_mask)) * 128;
    };
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 kr[2][4], vr[4][2], qr[4];
    auto load_k = [&](long long at, int n) {
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint16_t *src = p.K + at + (g + 8 * r) * 128 + 8 * tig;
            #pragma unroll
            for (int i = 0; i < 4; ++i) kr[r][i] = g + 8 * r < n ? ldg_stream(src + 32 * i) : zero;
        }
    };
    auto load_v = [&](long long at, int n) {
        #pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = 2 * tig + (r & 1) + 8 * (r >> 1);
            const uint16_t *src = p.V + at + tok * 128 + 8 * g;
            #pragma unroll
            for (int i = 0; i < 2; ++i) vr[r][i] = tok < n ? ldg_stream(src + 64 * i) : zero;
        }
    };

    Cursor cu = ld;                                      // the tile being computed; ld runs one ahead
    int n_cu, n_ld = 0;
    long long at_cu = tile_at(cu, page_of(cu), n_cu), at_ld = 0;
    load_k(at_cu, n_cu);
    int page_ld = 0;
    advance(ld);
    if (x0 + 1 < x1) page_ld = page_of(ld);

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, wt[8][4];
    #pragma unroll
    for (int e = 0; e < 8; ++e) wt[e][0] = wt[e][1] = wt[e][2] = wt[e][3] = 0.f;
    bool fresh = true;                                   // q of cu's unit not loaded yet
    bool head = cu.t != 0;                               // an earlier warp began cu's unit

    for (long long x = x0; x < x1; ++x) {
        const int layer = cu.lk / p.n_kv, kvh = cu.lk - layer * p.n_kv;
        const long long lb = (long long)layer * p.batch + cu.b;
        load_v(at_cu, n_cu);
        if (fresh) {
            const uint16_t *src = p.q + (lb * p.n_kv + kvh) * p.per_kv * 128 + (g < p.per_kv ? g : 0) * 128 + 8 * tig;
            #pragma unroll
            for (int i = 0; i < 4; ++i)
                qr[i] = g < p.per_kv ? __ldg(reinterpret_cast<const uint4 *>(src + 32 * i)) : zero;
            fresh = false;
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a0[4] = {kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y};
            mma_bf16(s, a0, qr[i].x, qr[i].y);
            const uint32_t a1[4] = {kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w};
            mma_bf16(s, a1, qr[i].z, qr[i].w);
        }
        const int n = n_cu;
        if (x + 1 < x1) {
            at_ld = tile_at(ld, page_ld, n_ld);
            load_k(at_ld, n_ld);
        }
        // s[0], s[1]: token g, heads 2 tig, 2 tig + 1; s[2], s[3]: token g + 8
        s[0] = g < n ? s[0] * p.scale2 : -INFINITY;
        s[1] = g < n ? s[1] * p.scale2 : -INFINITY;
        s[2] = g + 8 < n ? s[2] * p.scale2 : -INFINITY;
        s[3] = g + 8 < n ? s[3] * p.scale2 : -INFINITY;
        float mx0 = fmaxf(s[0], s[2]), mx1 = fmaxf(s[1], s[3]);
        #pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
        }
        const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
        // no finite logit so far: exponents against 0, so that -inf - -inf does not appear
        const float r0 = mn0 == -INFINITY ? 0.f : mn0, r1 = mn1 == -INFINITY ? 0.f : mn1;
        const float f0 = ex2(m[0] - r0), f1 = ex2(m[1] - r1);
        const float p0 = ex2(s[0] - r0), p1 = ex2(s[1] - r1), p2 = ex2(s[2] - r0), p3 = ex2(s[3] - r1);
        l[0] = l[0] * f0 + (p0 + p2);
        l[1] = l[1] * f1 + (p1 + p3);
        m[0] = mn0;
        m[1] = mn1;
        uint32_t h0, h1, q0, q1;
        split2(p0, p1, h0, q0);
        split2(p2, p3, h1, q1);
        h0 = movmatrix_t(h0);
        h1 = movmatrix_t(h1);
        q0 = movmatrix_t(q0);
        q1 = movmatrix_t(q1);
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            wt[e][0] *= f0; wt[e][1] *= f1; wt[e][2] *= f0; wt[e][3] *= f1;
            const uint32_t sel = e & 1 ? 0x7632u : 0x5410u;
            const uint32_t a[4] = {__byte_perm(word(vr[0][0], e >> 1), word(vr[1][0], e >> 1), sel),
                                   __byte_perm(word(vr[0][1], e >> 1), word(vr[1][1], e >> 1), sel),
                                   __byte_perm(word(vr[2][0], e >> 1), word(vr[3][0], e >> 1), sel),
                                   __byte_perm(word(vr[2][1], e >> 1), word(vr[3][1], e >> 1), sel)};
            mma_bf16(wt[e], a, h0, h1);
            mma_bf16(wt[e], a, q0, q1);
        }

        const bool ends = cu.t + 1 == cu.nt;             // the unit ends with this tile
        if (ends || x + 1 == x1) {
            #pragma unroll
            for (int e = 0; e < 2; ++e)
                #pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
            const long long row = (lb * p.n_kv + kvh) * p.per_kv;
            const bool whole = ends && !head;
            if (!head && lane == 0) {                    // this warp began the unit: where its parts are
                const long long last = x + (cu.nt - 1 - cu.t);
                const long long w1 = ((last + 1) * W - 1) / total;
                p.desc[lb * p.n_kv + kvh] = make_int2((int)w, (int)(w1 - w) + 1);
            }
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hh = 2 * tig + e;
                if (hh >= p.per_kv) continue;
                if (whole && p.tpart == nullptr) {
                    const float il = 1.f / l[e];
                    uint32_t o[2][4];
                    #pragma unroll
                    for (int i = 0; i < 2; ++i)
                        #pragma unroll
                        for (int k = 0; k < 4; ++k)
                            o[i][k] = pack_bf16(wt[2 * k][2 * i + e] * il, wt[2 * k + 1][2 * i + e] * il);
                    uint16_t *dst = p.out + (row + hh) * 128 + 8 * g;
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
                    *reinterpret_cast<uint4 *>(dst + 64) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
                    if (p.lse != nullptr && g == 0) p.lse[row + hh] = (m[e] + log2f(l[e])) * kLn2;
                } else {
                    const long long slot = 2 * w + (head ? 0 : 1);
                    float *st = whole ? p.tpart + (row + hh) * decode::kTxtPart : p.stat + (slot * 8 + hh) * 2;
                    float *dst = whole ? st + 2 : p.acc + (slot * p.per_kv + hh) * 128;
                    if (g == 0) *reinterpret_cast<float2 *>(st) = make_float2(m[e], l[e]);
                    #pragma unroll
                    for (int i = 0; i < 2; ++i)
                        #pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<float2 *>(dst + 64 * i + 8 * g + 2 * k) =
                                make_float2(wt[2 * k][2 * i + e], wt[2 * k + 1][2 * i + e]);
                }
            }
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.f;
            #pragma unroll
            for (int e = 0; e < 8; ++e) wt[e][0] = wt[e][1] = wt[e][2] = wt[e][3] = 0.f;
            head = false;
            fresh = true;
        }
        cu = ld;
        at_cu = at_ld;
        n_cu = n_ld;
        if (x + 2 < x1) {
            advance(ld);
            page_ld = page_of(ld);
        }
    }
}

// One block per (unit, query head): the parts of a unit that several warps share, in their order,
//   M = max m_k, out = sum 2^(m_k - M) acc_k / sum 2^(m_k - M) l_k,
// and the rows of sequences without tokens (out 0, lse -inf).
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ Params p) {
    __shared__ float red[kJoinWarps][128];
    __shared__ float ml[kJoinWarps][2];
    griddep_wait();
    const int hh = blockIdx.x % p.per_kv;
    const long long unit = blockIdx.x / p.per_kv;
    const int b = (int)((unit / p.n_kv) % p.batch);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = unit * p.per_kv + hh;
    float M = -INFINITY, L = 0.f, v = 0.f;
    if (__ldg(p.lens + b) > 0) {
        const int2 d = p.desc[unit];
        if (d.y == 1) return;                            // its warp finished it
        auto slot = [&](int k) { return k == 0 ? 2LL * d.x + 1 : 2LL * (d.x + k); };
        for (int k = tid; k < d.y; k += kJoinWarps * 32) M = fmaxf(M, p.stat[(slot(k) * 8 + hh) * 2]);
        #pragma unroll
        for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
        if (lane == 0) ml[warp][0] = M;
        __syncthreads();
        #pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) M = fmaxf(M, ml[i][0]);
        const float R = M == -INFINITY ? 0.f : M;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float lw = 0.f;
        #pragma unroll 4
        for (int k = warp; k < d.y; k += kJoinWarps) {
            const long long s = slot(k);
            const float2 st = *reinterpret_cast<const float2 *>(p.stat + (s * 8 + hh) * 2);
            const float f = ex2(st.x - R);
            const float4 c = *reinterpret_cast<const float4 *>(p.acc + (s * p.per_kv + hh) * 128 + 4 * lane);
            lw = fmaf(st.y, f, lw);
            a.x = fmaf(c.x, f, a.x);
            a.y = fmaf(c.y, f, a.y);
            a.z = fmaf(c.z, f, a.z);
            a.w = fmaf(c.w, f, a.w);
        }
        *reinterpret_cast<float4 *>(&red[warp][4 * lane]) = a;
        if (lane == 0) ml[warp][1] = lw;
        __syncthreads();
        if (tid < 128) {
            #pragma unroll
            for (int i = 0; i < kJoinWarps; ++i) {
                v += red[i][tid];
                L += ml[i][1];
            }
        }
    }
    if (tid >= 128) return;
    if (p.tpart != nullptr) {
        float *dst = p.tpart + row * decode::kTxtPart;
        if (tid == 0) { dst[0] = M; dst[1] = L; }
        dst[2 + tid] = v;
        return;
    }
    const bool none = __ldg(p.lens + b) <= 0;
    p.out[row * 128 + tid] = float_to_bf16_bits(none ? 0.f : v / L);
    if (p.lse != nullptr && tid == 0) p.lse[row] = (M + log2f(L)) * kLn2;
}

}  // namespace paged
}  // namespace kvpack
