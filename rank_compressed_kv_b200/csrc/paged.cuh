// paged.cuh -- attention of one new token per sequence over a paged cache, split over the
// cache's length and joined.
//
// Per (layer, sequence b, KV head) unit and query head h, over the sequence's len_b tokens:
//   s_t = scale q_h . K_t,   out_h = sum_t e^(s_t - m) V_t / l,   l = sum_t e^(s_t - m),
//   lse_h = m + ln l          (logits in the log2 domain: the scale folds log2 e)
// One pass keeps the running maximum and sum.  A page holds whole tiles of 16 tokens; walk() takes a
// warp over tiles.  Every byte of the cache is read once, 512 bytes a token and KV head, for at most
// 8 query heads x 512 flops: memory bounds it.  Three forms share the walk:
//   unit_kernel    a cluster of blocks per unit                    few units, short caches: latency
//   short_kernel   a warp per unit, several in turn                many units
//   attend_kernel  the tiles of all units in even runs, one per    long or few sequences of any lengths;
//                  warp, parts joined by join_kernel               ragged batches keep every warp busy
// Which, goes by the shapes (launch_paged_attend's plan); how tiles are shared goes by the lengths alone,
// so repeated calls give equal bits.
//
// Measured (one B200, launches in a graph; a plain copy runs at 6549 GB/s, a read-only kernel at 7240; calls from
// Python one behind the other take 0 to 3 us more):
//   64 x 704 tokens, 32 KV heads, 739 MB         114 us   6480 GB/s   (short_kernel)
//   4 x 66560 tokens, 8 KV heads, 1.09 GB        164 us   6650 GB/s   (attend_kernel + join_kernel)
//   32 ragged sequences up to 2561, 8 KV heads    37 us   4650 GB/s   (the same: 6 us of launches, ramp and join)
//   1 x 608 tokens, 32 KV heads, 10 MB           5.6 us               (unit_kernel: four dependent loads and a barrier)
#pragma once

#include "common.cuh"
#include "decode.cuh"

namespace kvpack {
namespace paged {

constexpr int kTile = 16;
constexpr int kWarps = 4;           // of unit_kernel's blocks
constexpr int kThreads = kWarps * 32;
constexpr int kSlotsPerSM = 7;      // runs, and so warps, per SM: one less than it holds
constexpr int kShortPerSM = 8;      // warps of short_kernel per SM
constexpr int kUnitBlocksPerSM = 2; // of unit_kernel
constexpr int kSlots = 3;           // tiles of a warp in shared memory
constexpr int kMinPlaces = 2;       // shortest run
constexpr int kMaxCluster = 8;
constexpr float kLn2 = 0.69314718055994531f;

struct Params {
    const uint16_t *q, *K, *V;      // [layers * batch][n_q][128], [layers][n_pages][n_kv][page][128]
    const int32_t *table, *lens;
    uint16_t *out;                  // [layers * batch][n_q][128], or null: tpart
    float *lse;                     // [layers * batch][n_q] or null
    float *tpart;                   // [layers * batch][n_q][kTxtPart]: (m, l, sum p V) of each head, or null
    float *stat;                    // [2 * runs][8][2]: m, l of a run's part; slot 2 w for the unit that an
    float *acc;                     // [2 * runs][per_kv][128]     earlier run began, 2 w + 1 for the one it leaves
    int layers, batch, n_kv, per_kv, n_pages, max_pages, page_shift, slots;   // slots: runs at most
    float scale2;
};

struct Cursor {
    int b, lk, t, nt, len;          // sequence, layer * n_kv + KV head, tile, tiles and length of the sequence
    long long x;                    // place among all (attend_kernel)
};

__device__ __forceinline__ int clamped_len(const Params &p, int b, bool report) {
    const long long cap = (long long)p.max_pages << p.page_shift;
    int len = p.lens[b];                                 // a plain load: the kernel may start before its writer ends
    if (len < 0 || len > cap) {
        if (report) report_error(KVPACK_ERR_PAGE);
        len = len < 0 ? 0 : (int)cap;
    }
    return len;
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint16_t *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// x, y >= 0 as three pairs of bf16 that sum to x and y: the upper eight bits of the value, of what that leaves, and
// the rest.  With their lowest bits set (2^-23 of the value at most) no term of a value from 2^-102 on is zero, and
// none is negative: times an infinite V each gives the infinity that the whole gives, and not a NaN.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&w)[3]) {
    x = __uint_as_float(__float_as_uint(x) | 1u);
    y = __uint_as_float(__float_as_uint(y) | 1u);
    #pragma unroll
    for (int i = 0; i < 3; ++i) {
        w[i] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
        x -= __uint_as_float(w[i] << 16);
        y -= __uint_as_float(w[i] & 0xffff0000u);
    }
    w[2] |= __vminu2(w[0], 0x00010001u);                 // and none of 0 is above it
}

// The softmax state of a run's current unit, as the matrix instructions lay it out.  Lane 4 g + t:
// m, l of heads 2t, 2t + 1; o[c / 2][2 (c % 2) + e]: entry 8 c + g of head 2t + e (c < 16).
struct State {
    float m[2], l[2], o[8][4];

    __device__ __forceinline__ void clear() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
        #pragma unroll
        for (int e = 0; e < 8; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
    }
    // every lane's share of the sums
    __device__ __forceinline__ void sum_lanes() {
        #pragma unroll
        for (int e = 0; e < 2; ++e)
            #pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
    }
    // head 2t + e unnormalised: dst[0 .. 127]
    __device__ __forceinline__ void store(int e, int g, float *dst) const {
        #pragma unroll
        for (int c = 0; c < 16; ++c) dst[8 * c + g] = o[c >> 1][2 * (c & 1) + e];
    }
};

// The rows of a unit that one warp has walked from end to end
__device__ __forceinline__ void finish_unit(const Params &p, long long row, const State &st, int g, int tig) {
    #pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int hh = 2 * tig + e;
        if (hh >= p.per_kv) continue;
        if (p.tpart != nullptr) {
            float *dst = p.tpart + (row + hh) * decode::kTxtPart;
            if (g == 0) *reinterpret_cast<float2 *>(dst) = make_float2(st.m[e], st.l[e]);
            st.store(e, g, dst + 2);
        } else if (p.lse != nullptr && g == 0) {
            p.lse[row + hh] = (st.m[e] + log2f(st.l[e])) * kLn2;
        }
    }
    if (p.tpart != nullptr) return;
    // transposed: lane 4 g + t has entries 8 c + 2 t, + 1 of head g
    const float i0 = 1.f / st.l[0], i1 = 1.f / st.l[1];
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + (row + g) * 128) + tig;
    #pragma unroll
    for (int c = 0; c < 16; ++c) {
        const uint32_t v = movmatrix_t(pack_bf16(st.o[c >> 1][2 * (c & 1)] * i0, st.o[c >> 1][2 * (c & 1) + 1] * i1));
        if (g < p.per_kv) dst[4 * c] = v;
    }
}

// A warp's ring of tiles in shared memory: 16 rows of K, then 16 of V, 256 bytes each, 16-byte chunk
// c of row r at c ^ (r & 7), so that eight rows of one chunk lie in different banks.
constexpr int kTileBytes = 2 * kTile * 256;
constexpr int kRingBytes = kSlots * kTileBytes;          // of a warp

// A warp's walk over the tiles from cursor `ld` on; advance(c) moves a cursor to the next tile and says
// whether it still belongs to the walk.  done(cu, ends, state) is called at the end of a unit (ends) or
// of the walk, and the state starts afresh.
//   S (16 tokens x 8 heads) = K q^T,   O^T (128 x 8 heads) += V^T P      (mma.sync, fp32 sums)
// P goes in whole, as three bf16 terms: of two, 16 bits, values that nearly cancel leave what those lack.  The
// matrix instruction cuts its sums off instead of rounding them, so it adds up one tile alone, and the running
// sum takes the tile with a rounded fma: over 4 x 66560 tokens 0.05 % of the outputs are then not the nearest bf16,
// 0.25 % with sums that stay in the accumulators.  Both cost the short caches 2 % (64 x 704: 112 to 114 us), the
// long ones nothing.  Rows past the sequence's end are not read; the copy writes zeros.
// Loads are asynchronous copies of 512 contiguous bytes a warp (two rows): register loads in the
// operand layout of K, 64 bytes of each of eight rows, stream 3 % slower (6949 against 7162 GB/s over
// 1.09 GB, loads alone).  Three slots: two tiles on their way, 112 KB an SM with attend_kernel's seven warps and
// 128 KB with the other kernels' eight, more than the 56 KB that its part of the bandwidth needs at 1.2 us of
// latency; with two slots the whole is 20 % slower.
template <typename Advance, typename Done>
__device__ __forceinline__ void walk(const Params &p, unsigned char *ring, Cursor ld, Advance advance, Done done) {
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    const int page_mask = (1 << p.page_shift) - 1;
    const uint32_t sb = smem_u32(ring);
    auto page_of = [&](const Cursor &c) {
        return p.table[(long long)c.b * p.max_pages + ((c.t * kTile) >> p.page_shift)];
    };
    // copy of lane: row 2 i + lane / 16, chunk lane % 16, i < 8
    const int row2 = lane >> 4, chunk = lane & 15;
    uint32_t dst[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = (2 * i + row2) * 256 + ((chunk ^ ((2 * i + row2) & 7)) << 4);
    auto fetch = [&](const Cursor &c, int page, int slot) {
        int n = min(kTile, c.len - c.t * kTile);
        if (page < 0 || page >= p.n_pages) {             // out of range: as if it held no tokens
            if (lane == 0) report_error(KVPACK_ERR_PAGE);
            n = 0;
            page = 0;
        }
        const int layer = c.lk / p.n_kv, kvh = c.lk - layer * p.n_kv;
        const long long at =
            (((((long long)layer * p.n_pages + page) * p.n_kv + kvh) << p.page_shift) + ((c.t * kTile) & page_mask)) * 128 +
            row2 * 128 + chunk * 8;
        const uint32_t to = sb + slot * kTileBytes;
        #pragma unroll
        for (int i = 0; i < 8; ++i)
            copy16(to + dst[i & 3] + (i >> 2) * 2048, p.K + at + i * 256, 2 * i + row2 < n);
        #pragma unroll
        for (int i = 0; i < 8; ++i)
            copy16(to + 4096 + dst[i & 3] + (i >> 2) * 2048, p.V + at + i * 256, 2 * i + row2 < n);
        return n;
    };

    // Cursors: cu is the tile being computed, ld the one to fetch (kSlots - 1 ahead), nx the one after, whose
    // page number is on its way while ld is fetched.  A unit's queries are loaded with its first tile.
    Cursor cu = ld, nx = ld;
    int n[kSlots], ahead = 0;                            // tiles' valid rows; tiles fetched and not computed yet
    uint32_t qn[kSlots][8][2];
    int page_ld = page_of(ld), page_nx = 0;
    bool more = true, more_nx = advance(nx), begins = true;          // ld, nx are tiles of the walk; ld begins a unit
    if (more_nx) page_nx = page_of(nx);
    auto fetch_next = [&](int &nn, uint32_t (&qs)[8][2], int slot) {
        if (more) {
            nn = fetch(ld, page_ld, slot);
            if (begins) {
                const int layer = ld.lk / p.n_kv, kvh = ld.lk - layer * p.n_kv;
                const long long row = (((long long)layer * p.batch + ld.b) * p.n_kv + kvh) * p.per_kv;
                const bool ok = g < p.per_kv;
                const uint32_t *src = reinterpret_cast<const uint32_t *>(p.q + (row + (ok ? g : 0)) * 128) + tig;
                #pragma unroll
                for (int k = 0; k < 8; ++k) {
                    qs[k][0] = ok ? src[8 * k] : 0u;
                    qs[k][1] = ok ? src[8 * k + 4] : 0u;
                }
            }
            ++ahead;
            begins = ld.t + 1 == ld.nt;
            more = more_nx;
            ld = nx;
            page_ld = page_nx;
            if (more) {
                more_nx = advance(nx);
                if (more_nx) page_nx = page_of(nx);
            }
        }
        copy_commit();
    };
    #pragma unroll
    for (int i = 0; i < kSlots; ++i) n[i] = 0;
    #pragma unroll
    for (int i = 0; i < kSlots - 1; ++i) fetch_next(n[i], qn[i], i);
    const int kx = (lane >> 4) ^ (lane & 7), vx = ((lane >> 3) & 1) ^ (lane & 7);
    const uint32_t krow = (lane & 15) * 256, vrow = 4096 + ((lane & 7) + ((lane >> 4) << 3)) * 256;
    State st;
    st.clear();
    uint32_t qf[8][2];
    bool fresh = true;                                   // cu is its unit's first tile of the walk

    auto step = [&](int slot, int &nt, const uint32_t (&qs)[8][2], int &nn, uint32_t (&qq)[8][2]) {
        copy_wait<kSlots - 2>();                         // the tile has landed
        __syncwarp();                                    // for every lane, and all are done with the one before
        if (fresh) {
            #pragma unroll
            for (int k = 0; k < 8; ++k) { qf[k][0] = qs[k][0]; qf[k][1] = qs[k][1]; }
            fresh = false;
        }
        fetch_next(nn, qq, (slot + kSlots - 1) % kSlots);
        const uint32_t tb = sb + slot * kTileBytes;
        // two sums of four products each: half the chain of dependent instructions, which bounds a lone warp
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
        #pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t a[4];
            ldsm_x4(tb + krow + (((2 * k) ^ kx) << 4), a[0], a[1], a[2], a[3]);
            mma_bf16(k & 1 ? s2 : s, a, qf[k][0], qf[k][1]);
        }
        // s[0], s[1]: token g, heads 2 tig, 2 tig + 1; s[2], s[3]: token g + 8
        s[0] = g < nt ? (s[0] + s2[0]) * p.scale2 : -INFINITY;
        s[1] = g < nt ? (s[1] + s2[1]) * p.scale2 : -INFINITY;
        s[2] = g + 8 < nt ? (s[2] + s2[2]) * p.scale2 : -INFINITY;
        s[3] = g + 8 < nt ? (s[3] + s2[3]) * p.scale2 : -INFINITY;
        float mx0 = fmaxf(s[0], s[2]), mx1 = fmaxf(s[1], s[3]);
        #pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
        }
        const float mn0 = fmaxf(st.m[0], mx0), mn1 = fmaxf(st.m[1], mx1);
        // no finite logit so far: exponents against 0, so that -inf - -inf does not appear
        const float r0 = mn0 == -INFINITY ? 0.f : mn0, r1 = mn1 == -INFINITY ? 0.f : mn1;
        const float f0 = ex2(st.m[0] - r0), f1 = ex2(st.m[1] - r1);
        const float p0 = ex2(s[0] - r0), p1 = ex2(s[1] - r1), p2 = ex2(s[2] - r0), p3 = ex2(s[3] - r1);
        st.l[0] = st.l[0] * f0 + (p0 + p2);
        st.l[1] = st.l[1] * f1 + (p1 + p3);
        st.m[0] = mn0;
        st.m[1] = mn1;
        uint32_t w0[3], w1[3];
        split3(p0, p1, w0);
        split3(p2, p3, w1);
        #pragma unroll
        for (int i = 0; i < 3; ++i) {
            w0[i] = movmatrix_t(w0[i]);
            w1[i] = movmatrix_t(w1[i]);
        }
        // two accumulators' products side by side: each is a chain of three
        #pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float d[2][4] = {};
            uint32_t a[2][4];
            #pragma unroll
            for (int k = 0; k < 2; ++k)
                ldsm_x4_t(tb + vrow + (((2 * (e + k)) ^ vx) << 4), a[k][0], a[k][1], a[k][2], a[k][3]);
            #pragma unroll
            for (int i = 0; i < 3; ++i) {
                mma_bf16(d[0], a[0], w0[i], w1[i]);
                mma_bf16(d[1], a[1], w0[i], w1[i]);
            }
            #pragma unroll
            for (int k = 0; k < 2; ++k) {
                float (&o)[4] = st.o[e + k];
                o[0] = fmaf(o[0], f0, d[k][0]); o[1] = fmaf(o[1], f1, d[k][1]);
                o[2] = fmaf(o[2], f0, d[k][2]); o[3] = fmaf(o[3], f1, d[k][3]);
            }
        }
        --ahead;
        const bool ends = cu.t + 1 == cu.nt;             // the unit ends with this tile
        if (ends || ahead == 0) {
            st.sum_lanes();
            done(cu, ends, st);
            st.clear();
            fresh = true;
        }
        if (ahead > 0) advance(cu);
    };
    while (ahead > 0) {
        #pragma unroll
        for (int i = 0; i < kSlots; ++i)
            if (ahead > 0) step(i, n[i], qn[i], n[(i + kSlots - 1) % kSlots], qn[(i + kSlots - 1) % kSlots]);
    }
}

// The places, `total` of them, in W even runs: the first `more` have base + 1 places, the others base.
struct Runs {
    long long W, base, more;

    __device__ __forceinline__ Runs(long long total, int slots) {
        const long long most = total / kMinPlaces;
        W = most < 1 ? 1 : most < slots ? most : slots;
        base = quotient(total, W);
        more = total - base * W;
    }
    __device__ __forceinline__ long long first(long long w) const { return w * base + (w < more ? w : more); }
    __device__ __forceinline__ long long of(long long x) const {
        const long long longer = more * (base + 1);
        return x < longer ? quotient(x, base + 1) : more + quotient(x - longer, base);
    }
};

// -------------------------------------------------------------------------- runs over all units

__device__ __forceinline__ long long warp_sums(long long v, int lane) {
    #pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Places of all sequences, in the sequences' order, by a warp.  A unit of nt tiles has nt + 1 places: its
// end costs about as much as a tile (the queries' load, the sums over lanes, the output), so that runs of
// short units would end late if only tiles counted.  Lane i has the places of the `per` groups of 32
// sequences from i * per on, and the sum up to their end.
struct Lengths {
    const Params &p;
    int lane, per;
    long long mine, upto, total;     // total: of one layer and KV head

    __device__ __forceinline__ int places_of(int b) const {
        const int len = b < p.batch ? clamped_len(p, b, false) : 0;
        return len > 0 ? (len + kTile - 1) / kTile + 1 : 0;
    }
    __device__ __forceinline__ Lengths(const Params &p_, int lane_) : p(p_), lane(lane_) {
        const int groups = (p.batch + 31) / 32;
        per = (groups + 31) / 32;
        mine = 0;
        #pragma unroll 8
        for (int i = 0; i < groups; ++i) {
            const unsigned sum = __reduce_add_sync(0xffffffffu, (unsigned)places_of(32 * i + lane));
            if (i / per == lane) mine += sum;
        }
        upto = warp_sums(mine, lane);
        total = __shfl_sync(0xffffffffu, upto, 31);
    }
    // the sequence whose places, times LK, hold place x: b, its places, and those before it
    __device__ __forceinline__ void find(long long x, int LK, int &b, int &own, long long &before) const {
        const int at = __popc(__ballot_sync(0xffffffffu, upto * LK <= x));
        before = __shfl_sync(0xffffffffu, upto - mine, at);
        b = own = 0;
        for (int i = at * per; i < (at + 1) * per; ++i) {
            const long long t = places_of(32 * i + lane), end = before + warp_sums(t, lane);
            const uint32_t past = __ballot_sync(0xffffffffu, end * LK > x);
            if (past != 0) {
                const int s = __ffs(past) - 1;
                b = 32 * i + s;
                own = (int)__shfl_sync(0xffffffffu, t, s);
                before = __shfl_sync(0xffffffffu, end, s) - own;
                return;
            }
            before = __shfl_sync(0xffffffffu, end, 31);
        }
    }
    // places before sequence b
    __device__ __forceinline__ long long before(int b) const {
        const int at = b / (32 * per);
        long long n = __shfl_sync(0xffffffffu, upto - mine, at);
        for (int i = at * per; 32 * i < b; ++i)
            n += __reduce_add_sync(0xffffffffu, (unsigned)(32 * i + lane < b ? places_of(32 * i + lane) : 0));
        return n;
    }
};

// A block is one warp and takes one run; the runs fill the GPU once, seven an SM (eight: 4 x 66560 tokens
// 171 us instead of 165, ragged batches level).  SMs do not get equal parts of
// the memory's bandwidth, so the last warp ends 10 to 15 % after the median; shorter runs that go where an SM
// is done even that out, but each end of a run costs about a tile and they gain nothing.
__global__ void __launch_bounds__(32) attend_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) unsigned char smem[];
    // in this order: the join may then read the lengths, which a kernel before this one may write
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x, g = lane >> 2, tig = lane & 3;
    const int LK = p.layers * p.n_kv;
    const Lengths lens(p, lane);
    const long long total = lens.total * LK, w = blockIdx.x;   // places
    if (blockIdx.x == 0)
        for (int b = lane; b < p.batch; b += 32) clamped_len(p, b, true);
    if (total == 0) return;
    const Runs runs(total, p.slots);
    if (w >= runs.W) return;
    const long long x0 = runs.first(w), x1 = runs.first(w + 1);

    auto advance = [&](Cursor &c) {
        ++c.x;
        if (++c.t < c.nt) return c.x < x1;
        if (++c.x >= x1) return false;                   // past the unit's last place
        c.t = 0;
        if (++c.lk < LK) return true;
        c.lk = 0;
        do c.len = clamped_len(p, ++c.b, false); while (c.len == 0);   // x < total: there is one
        c.nt = (c.len + kTile - 1) / kTile;
        return true;
    };
    Cursor first{};
    {
        long long before;
        int own;
        lens.find(x0, LK, first.b, own, before);
        first.x = x0;
        first.nt = own - 1;
        first.len = clamped_len(p, first.b, false);
        const long long rem = x0 - before * LK;
        first.lk = (int)quotient(rem, own);
        first.t = (int)(rem - (long long)first.lk * own);
        if (first.t == first.nt) {                       // the place that has no tile: on to the next unit
            --first.t;
            --first.x;
            if (!advance(first)) return;
        }
    }
    bool head = first.t != 0;                            // an earlier run began the current unit
    walk(p, smem, first, advance, [&](const Cursor &cu, bool ends, const State &st) {
        const int layer = cu.lk / p.n_kv, kvh = cu.lk - layer * p.n_kv;
        const long long unit = ((long long)layer * p.batch + cu.b) * p.n_kv + kvh, row = unit * p.per_kv;
        const bool whole = ends && !head;
        if (whole) {
            finish_unit(p, row, st, g, tig);
        } else {
            const long long slot = 2 * w + (head ? 0 : 1);
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hh = 2 * tig + e;
                if (hh >= p.per_kv) continue;
                if (g == 0) *reinterpret_cast<float2 *>(p.stat + (slot * 8 + hh) * 2) = make_float2(st.m[e], st.l[e]);
                st.store(e, g, p.acc + (slot * p.per_kv + hh) * 128);
            }
        }
        head = false;
    });
}

// What a joined row (unit, head) becomes: M and L of all its tokens, v = entry tid of sum 2^(s - M) V
__device__ __forceinline__ void write_row(const Params &p, long long row, bool none, float M, float L, float4 v, int lane) {
    if (p.tpart != nullptr) {
        float *dst = p.tpart + row * decode::kTxtPart;
        if (lane == 0) *reinterpret_cast<float2 *>(dst) = make_float2(M, L);
        *reinterpret_cast<float2 *>(dst + 2 + 4 * lane) = make_float2(v.x, v.y);
        *reinterpret_cast<float2 *>(dst + 4 + 4 * lane) = make_float2(v.z, v.w);
        return;
    }
    const float il = none ? 0.f : 1.f / L;
    *reinterpret_cast<uint2 *>(p.out + row * 128 + 4 * lane) =
        make_uint2(pack_bf16(v.x * il, v.y * il), pack_bf16(v.z * il, v.w * il));
    if (p.lse != nullptr && lane == 0) p.lse[row] = (M + log2f(L)) * kLn2;
}

// Many units of few tokens: a warp takes whole units, every gridDim.x-th, its copies running from one into the
// next.  Nothing to scan and nothing to join.
__global__ void __launch_bounds__(32) short_kernel(const __grid_constant__ Params p, int units) {
    extern __shared__ __align__(128) unsigned char smem[];
    griddep_launch_dependents();
    const int lane = threadIdx.x, g = lane >> 2, tig = lane & 3;
    // unit u as a cursor's sequence, head and length; x = u
    auto enter = [&](Cursor &c, int u) {
        const int lb = u / p.n_kv, layer = lb / p.batch;
        c.x = u;
        c.b = lb - layer * p.batch;
        c.lk = layer * p.n_kv + u - lb * p.n_kv;
        c.t = 0;
        c.len = clamped_len(p, c.b, c.lk == 0);
        c.nt = (c.len + kTile - 1) / kTile;
    };
    // the first unit from u on that has tokens
    auto seek = [&](Cursor &c, int u) {
        for (; u < units; u += gridDim.x) {
            enter(c, u);
            if (c.len > 0) return true;
        }
        return false;
    };
    griddep_wait();
    Cursor first{};
    for (int u = blockIdx.x; u < units; u += gridDim.x) {             // rows of sequences without tokens
        enter(first, u);
        if (first.len == 0)
            for (int h = 0; h < p.per_kv; ++h)
                write_row(p, (long long)u * p.per_kv + h, true, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f), lane);
    }
    if (!seek(first, blockIdx.x)) return;
    auto advance = [&](Cursor &c) { return ++c.t < c.nt || seek(c, (int)c.x + (int)gridDim.x); };
    walk(p, smem, first, advance, [&](const Cursor &cu, bool, const State &st) {
        finish_unit(p, cu.x * p.per_kv, st, g, tig);
    });
}

// The parts of the units that several runs share, in their order,
//   M = max m_k, out = sum 2^(m_k - M) acc_k / sum 2^(m_k - M) l_k,
// and the rows of sequences without tokens (out 0, lse -inf).  JW warps take a row (unit, query head),
// and with JW = 1 a warp takes rows in turn.  Where a unit's parts are follows from the lengths: the
// sums over them are taken while the attention still runs.  (With 32 warps a block 64 registers a thread are
// all there are, and 76 bytes of join_kernel<32> are spilled.)
constexpr int join_warps(int JW) { return JW > 8 ? JW : 8; }         // of a block

template <int JW>
__global__ void __launch_bounds__(join_warps(JW) * 32) join_kernel(const __grid_constant__ Params p, long long rows) {
    constexpr int kAhead = 4;                            // parts a warp loads at a time
    constexpr int kRows = join_warps(JW) / JW;           // rows of a block
    __shared__ float4 red[JW > 1 ? join_warps(JW) : 1][32];
    __shared__ float ml[join_warps(JW)][2];
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, jw = warp % JW;
    const int LK = p.layers * p.n_kv;
    // the lengths are inputs, complete when attend_kernel let this kernel start
    const Lengths lens(p, lane);
    const Runs runs(lens.total > 0 ? lens.total * LK : 1, p.slots);
    bool waited = false;
    for (long long row = (long long)blockIdx.x * kRows + warp / JW; row < rows || (JW > 1 && !waited);
         row += (long long)gridDim.x * kRows) {
        const bool in = row < rows;
        const long long unit = quotient(in ? row : 0, p.per_kv), lb = quotient(unit, p.n_kv);
        const int hh = (int)(row - unit * p.per_kv);
        const int layer = (int)quotient(lb, p.batch), b = (int)(lb - (long long)layer * p.batch);
        const int len = clamped_len(p, b, false), nt = (len + kTile - 1) / kTile;
        int parts = 0;
        long long w0 = 0;
        if (in && len > 0) {
            const long long x = lens.before(b) * LK + (layer * p.n_kv + (unit - lb * p.n_kv)) * (nt + 1);
            w0 = runs.of(x);
            parts = (int)(runs.of(x + nt - 1) - w0) + 1;
        }
        if (!waited) griddep_wait();
        waited = true;
        if (JW == 1 && parts == 1) continue;             // its warp finished it
        auto slot = [&](int k) { return k == 0 ? 2 * w0 + 1 : 2 * (w0 + k); };
        float M = -INFINITY, L = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = jw; k0 < parts && parts > 1; k0 += JW * kAhead) {
            float2 st[kAhead];
            float4 c[kAhead];
            float top = M;
            #pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = k0 + i * JW;
                st[i] = make_float2(-INFINITY, 0.f);
                c[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < parts) {
                    st[i] = *reinterpret_cast<const float2 *>(p.stat + (slot(k) * 8 + hh) * 2);
                    c[i] = *reinterpret_cast<const float4 *>(p.acc + (slot(k) * p.per_kv + hh) * 128 + 4 * lane);
                }
                top = fmaxf(top, st[i].x);
            }
            const float R = top == -INFINITY ? 0.f : top, f = ex2(M - R);
            L *= f;
            a.x *= f; a.y *= f; a.z *= f; a.w *= f;
            M = top;
            #pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float f = ex2(st[i].x - R);
                L = fmaf(st[i].y, f, L);
                a.x = fmaf(c[i].x, f, a.x);
                a.y = fmaf(c[i].y, f, a.y);
                a.z = fmaf(c[i].z, f, a.z);
                a.w = fmaf(c[i].w, f, a.w);
            }
        }
        if constexpr (JW > 1) {
            red[warp][lane] = a;
            if (lane == 0) { ml[warp][0] = M; ml[warp][1] = L; }
            __syncthreads();
            if (jw != 0) return;                         // one row a block
            const float own = M;
            #pragma unroll
            for (int i = 1; i < JW; ++i) M = fmaxf(M, ml[warp + i][0]);
            const float R = M == -INFINITY ? 0.f : M, f = ex2(own - R);
            L *= f;
            a.x *= f; a.y *= f; a.z *= f; a.w *= f;
            #pragma unroll
            for (int i = 1; i < JW; ++i) {
                const float f = ex2(ml[warp + i][0] - R);
                const float4 c = red[warp + i][lane];
                L = fmaf(ml[warp + i][1], f, L);
                a.x = fmaf(c.x, f, a.x);
                a.y = fmaf(c.y, f, a.y);
                a.z = fmaf(c.z, f, a.z);
                a.w = fmaf(c.w, f, a.w);
            }
        }
        if (in && parts != 1) write_row(p, row, len <= 0, M, L, a, lane);
        if (JW > 1) return;
    }
    if (!waited) griddep_wait();
}

// ------------------------------------------------------------------ a cluster of blocks per unit

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

// Short caches of few units: a cluster takes one unit, its warps equal shares of the unit's tiles,
// and the parts meet in the blocks' shared memories.  One launch, nothing to scan, no workspace:
// 1 x 608 tokens of 32 heads 5.6 us, 7.0 as runs and join.
__global__ void __launch_bounds__(kThreads, kUnitBlocksPerSM) unit_kernel(const __grid_constant__ Params p, int S) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) float2 pml[kWarps][8];
    __shared__ __align__(16) float sum[8][128];
    __shared__ __align__(16) float2 ml[8];
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tig = lane & 3;
    const int rank = (int)(blockIdx.x % S);
    const long long unit = blockIdx.x / S;
    const long long lb = unit / p.n_kv;
    const int layer = (int)(lb / p.batch), b = (int)(lb - (long long)layer * p.batch), kvh = (int)(unit - lb * p.n_kv);
    griddep_wait();
    const int len = clamped_len(p, b, blockIdx.x % S == 0);
    const long long row = unit * p.per_kv;
    if (len == 0) {                                      // the same for the whole cluster
        if (rank == 0)
            for (int h = warp; h < p.per_kv; h += kWarps)
                write_row(p, row + h, true, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f), lane);
        return;
    }
    const int nt = (len + kTile - 1) / kTile, n_warps = S * kWarps, w = rank * kWarps + warp;
    const int base = nt / n_warps, more = nt - base * n_warps;
    const int t0 = w * base + min(w, more), count = base + (w < more ? 1 : 0);
    unsigned char *ring = smem + warp * kRingBytes;
    if (count > 0) {
        const Cursor first{b, layer * p.n_kv + kvh, t0, nt, len, 0};
        walk(p, ring, first, [&](Cursor &c) { return ++c.t < t0 + count; }, [&](const Cursor &, bool, const State &st) {
            __syncwarp();                                // the ring has been read: the part goes there
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hh = 2 * tig + e;
                if (hh >= p.per_kv) continue;
                if (g == 0) pml[warp][hh] = make_float2(st.m[e], st.l[e]);
                st.store(e, g, reinterpret_cast<float *>(ring) + hh * 128);
            }
        });
    }
    __syncthreads();
    // the block's parts, in the warps' order (warps without tiles are the last ones)
    const int live = base > 0 ? kWarps : max(0, min(kWarps, nt - rank * kWarps));
    for (int h = warp; h < p.per_kv; h += kWarps) {
        float M = -INFINITY, L = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < live; ++i) M = fmaxf(M, pml[i][h].x);
        const float R = M == -INFINITY ? 0.f : M;
        for (int i = 0; i < live; ++i) {
            const float f = ex2(pml[i][h].x - R);
            const float4 c = *reinterpret_cast<const float4 *>(smem + i * kRingBytes + h * 512 + 16 * lane);
            L = fmaf(pml[i][h].y, f, L);
            a.x = fmaf(c.x, f, a.x);
            a.y = fmaf(c.y, f, a.y);
            a.z = fmaf(c.z, f, a.z);
            a.w = fmaf(c.w, f, a.w);
        }
        *reinterpret_cast<float4 *>(&sum[h][4 * lane]) = a;
        if (lane == 0) ml[h] = make_float2(M, L);
    }
    cluster_arrive();
    cluster_wait();
    // head h of the unit is joined by warp h / S of block h % S
    for (int h = warp * S + rank; h < p.per_kv; h += kWarps * S) {
        const uint32_t at = smem_u32(&sum[h][4 * lane]), at_ml = smem_u32(&ml[h]);
        float M = -INFINITY, L = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float2 st[kMaxCluster];
        float4 c[kMaxCluster];
        #pragma unroll
        for (int i = 0; i < kMaxCluster; ++i)
            if (i < S) {
                st[i] = cluster_ld2(cluster_map(at_ml, i));
                c[i] = cluster_ld4(cluster_map(at, i));
                M = fmaxf(M, st[i].x);
            }
        const float R = M == -INFINITY ? 0.f : M;
        #pragma unroll
        for (int i = 0; i < kMaxCluster; ++i)
            if (i < S) {
                const float f = ex2(st[i].x - R);
                L = fmaf(st[i].y, f, L);
                a.x = fmaf(c[i].x, f, a.x);
                a.y = fmaf(c[i].y, f, a.y);
                a.z = fmaf(c[i].z, f, a.z);
                a.w = fmaf(c[i].w, f, a.w);
            }
        write_row(p, row + h, false, M, L, a, lane);
    }
    cluster_arrive();                                    // no block leaves while another reads its sums
    cluster_wait();
}

}  // namespace paged
}  // namespace kvpack
