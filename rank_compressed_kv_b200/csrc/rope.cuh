// rope.cuh -- rotary positions with one or several axes (time, height, width): rotation of
// queries and keys, and the append to a paged cache that rotates on the way.
//
// Pair p < R/2 of a head of 128 values turns by the angle t = pos[axis(p)][row] * freq[p]:
//   (x, y) -> (x cos t - y sin t, y cos t + x sin t),   the inverse by -t (also the gradient);
// entries R .. 127 pass unchanged.  Angles of far positions need more than 32 bits: the number of
// turns, pos * freq / 2 pi, is taken in fp64, its whole part dropped, and sine and cosine of what
// is left are fp32, as is the rotation; one rounding to bf16.  What is left, at most half a turn, is off by
// 2^-26 of a turn (its rounding to fp32) and 2^-52 of all the turns: 2^-23.4 together at position 2^31 and freq 1.
#pragma once

#include "common.cuh"

namespace kvpack {
namespace rope {

// bf16 heads of 128 values: head h of row r of outer row o at
// o * outer + r * row + (h / 4) * group + (h % 4) * 128 elements
struct View {
    uint16_t *data;
    long long outer, row, group;
};

// Inputs are read with plain loads: the kernel may start before the kernel that writes them ends.
struct Params {
    View q, q_out, k, k_out, v;     // append: k_out is not used, k and v go into the pages
    const int32_t *pos;             // [axes][outers][rows], append: [axes][rows]
    const double *freq;             // [R / 2]
    long long pos_axis, pos_outer;  // elements between axes, between outer rows
    long long items;                // outers * rows * splits
    int rows, splits, qpw;          // splits warps per row, qpw quads of heads each
    int n_q, n_k, quads_q, quads_k, quads;   // quads: ceil(heads / 4) of q, of k (and of v), of all
    int rot8;                       // R / 16: lanes with a rotated pair of 16-byte chunks
    float sign;                     // of the sine
    uint32_t axis2[4];              // two bits a pair
    // append
    uint16_t *K, *V;                // [outers][n_pages][n_k][page][128]
    const int32_t *table, *lens, *offsets;
    int batch, n_pages, max_pages, page_shift;
};

// The slot a row's key and value go to: (page, offset in it), the page's number unchecked, < 0 for an index
// out of range.  found: the row belongs to a sequence (rows behind the last one, and idle sequences of
// length 0, do not).
__device__ __forceinline__ void find_slot(const Params &p, int row, int lane, bool &found, int &page, int &at) {
    found = false;
    page = -1;
    at = 0;
    int seq, index;
    if (p.offsets == nullptr) {
        seq = row;
        const int len = p.lens[row];
        if (len == 0) return;
        index = len - 1;
    } else {
        // the last sequence that starts at or before the row, 32 starts at a time
        int lo = 0, hi = p.batch + 1;            // the answer is lo - 1 + something below hi
        int last = -1;
        while (lo < hi) {
            const int step = (hi - lo + 31) >> 5, at32 = lo + lane * step;
            const bool le = at32 < hi && p.offsets[at32] <= row;
            const int cnt = __popc(__ballot_sync(0xffffffffu, le));
            if (cnt == 0) break;
            last = lo + (cnt - 1) * step;
            lo = last + 1;
            hi = min(hi, last + step);
        }
        if (last < 0 || last >= p.batch) return;
        seq = last;
        const int o1 = p.offsets[seq + 1];
        if (row >= o1) return;
        index = p.lens[seq] - (o1 - row);
    }
    found = true;
    const long long cap = (long long)p.max_pages << p.page_shift;
    if (index >= 0 && index < cap) page = p.table[(long long)seq * p.max_pages + (index >> p.page_shift)];
    at = index & ((1 << p.page_shift) - 1);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two 16-byte chunks of a lane: x of pairs 0..7 in a, y in b (halves), or pairs 0..3 in a and 4..7
// in b, x and y side by side (adjacent).
template <bool ADJ>
__device__ __forceinline__ void turn(uint4 &a, uint4 &b, const float (&c)[8], const float (&s)[8]) {
    uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (ADJ) {
            const float x0 = bf_lo(x[e]), y0 = bf_hi(x[e]), x1 = bf_lo(y[e]), y1 = bf_hi(y[e]);
            x[e] = pack_bf16(x0 * c[e] - y0 * s[e], y0 * c[e] + x0 * s[e]);
            y[e] = pack_bf16(x1 * c[e + 4] - y1 * s[e + 4], y1 * c[e + 4] + x1 * s[e + 4]);
        } else {
            const float x0 = bf_lo(x[e]), x1 = bf_hi(x[e]), y0 = bf_lo(y[e]), y1 = bf_hi(y[e]);
            x[e] = pack_bf16(x0 * c[2 * e] - y0 * s[2 * e], x1 * c[2 * e + 1] - y1 * s[2 * e + 1]);
            y[e] = pack_bf16(y0 * c[2 * e] + x0 * s[2 * e], y1 * c[2 * e + 1] + x1 * s[2 * e + 1]);
        }
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
    b = make_uint4(y[0], y[1], y[2], y[3]);
}

constexpr int kThreads = 128;
constexpr int kBlocks = 8;          // per SM: 64 registers a thread (four quads at a time spill 12 bytes)
constexpr int kWarpsPerSM = kBlocks * kThreads / 32;

// A warp takes a row's heads (or a share of them) four at a time: lane 8 s + c holds head s of the
// four and two 16-byte chunks of it, for c < R/16 the two halves of pairs 8c .. 8c + 7.  A lane
// evaluates two of the row's angles; the eight it needs come from the four lanes of the same c.
// U quads are loaded at a time, the first before the angles are worked out.  Memory bounds long calls:
// 16 x 6272 rows of 32 heads move 1.65 GB in 247 us (a plain copy of as much takes 251).
template <bool APPEND, bool ADJ, int U>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const __grid_constant__ Params p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, c = lane & 7, sub = lane >> 3;
    const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= p.items) return;
    const int split = (int)(item % p.splits);
    const long long orow = item / p.splits;
    const int row = (int)(orow % p.rows), outer = (int)(orow / p.rows);
    const int q0 = split * p.qpw, q1 = min(q0 + p.qpw, p.quads);
    const bool rotated = c < p.rot8;
    const int e0 = ADJ ? 16 * c : rotated ? 8 * c : 16 * c;
    const int e1 = ADJ ? e0 + 8 : rotated ? 8 * (p.rot8 + c) : e0 + 8;

    // the quad's tensor (0 q, 1 k, 2 v) and its number in it
    auto part = [&](int qd, int &g) {
        const int t = qd < p.quads_q ? 0 : !APPEND || qd < p.quads_q + p.quads_k ? 1 : 2;
        g = qd - (t == 0 ? 0 : t == 1 ? p.quads_q : p.quads_q + p.quads_k);
        return t;
    };
    uint4 a[U], b[U];
    auto load = [&](int qd0) {
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            int g;
            const int t = part(qd0 + u, g);
            const View &s = t == 0 ? p.q : t == 1 ? p.k : p.v;
            if (qd0 + u < q1 && 4 * g + sub < (t == 0 ? p.n_q : p.n_k)) {
                const uint16_t *src = s.data + outer * s.outer + row * s.row + g * s.group + sub * 128;
                a[u] = *reinterpret_cast<const uint4 *>(src + e0);
                b[u] = *reinterpret_cast<const uint4 *>(src + e1);
            }
        }
    };
    load(q0);                                   // on their way while the angles and the slot are worked out

    const int p0 = 8 * c + 2 * sub;             // the lane's two pairs
    auto position = [&](int i) {
        const uint32_t w = p0 < 16 ? p.axis2[0] : p0 < 32 ? p.axis2[1] : p0 < 48 ? p.axis2[2] : p.axis2[3];
        const int ax = (w >> (2 * ((p0 + i) & 15))) & 3;
        return p.pos[ax * p.pos_axis + outer * p.pos_outer + row];
    };
    // before the slot's chain of loads; without one they only cost registers there
    int early_pos[2] = {0, 0};
    double early_freq[2] = {0., 0.};
    if (APPEND && rotated) {
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            early_pos[i] = position(i);
            early_freq[i] = p.freq[p0 + i];
        }
    }
    bool found = true;
    int page = 0, at = 0;
    if constexpr (APPEND) {
        find_slot(p, row, lane, found, page, at);
        if (!found) return;
    }

    float cs[8], sn[8];
    if (p.rot8 > 0) {
        float c2[2] = {1.f, 1.f}, s2[2] = {0.f, 0.f};
        if (rotated) {
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at_pos = APPEND ? early_pos[i] : position(i);
                const double freq = APPEND ? early_freq[i] : p.freq[p0 + i];
                const double turns = (double)at_pos * (freq * 0.15915494309189535);
                const float part = (float)(turns - rint(turns));
                sincospif(2.f * part, &s2[i], &c2[i]);
            }
        }
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            cs[j] = __shfl_sync(0xffffffffu, c2[j & 1], (j >> 1) * 8 + c);
            sn[j] = __shfl_sync(0xffffffffu, s2[j & 1], (j >> 1) * 8 + c) * p.sign;
        }
    }

    if constexpr (APPEND) {
        if (page < 0 || page >= p.n_pages) {
            page = -1;
            if (lane == 0) report_error(KVPACK_ERR_PAGE);
        }
    }
    for (int qd0 = q0; qd0 < q1; qd0 += U) {
        if (qd0 > q0) load(qd0);
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            int g;
            const int t = part(qd0 + u, g), h = 4 * g + sub;
            if (qd0 + u < q1 && h < (t == 0 ? p.n_q : p.n_k)) {
                if (rotated && t < 2) turn<ADJ>(a[u], b[u], cs, sn);
                uint16_t *dst = nullptr;
                if (!APPEND || t == 0) {
                    const View &o = t == 0 ? p.q_out : p.k_out;
                    dst = o.data + outer * o.outer + row * o.row + g * o.group + sub * 128;
                } else if (page >= 0) {
                    dst = (t == 1 ? p.K : p.V) +
                          (((((long long)outer * p.n_pages + page) * p.n_k + h) << p.page_shift) + at) * 128;
                }
                if (dst != nullptr) {
                    *reinterpret_cast<uint4 *>(dst + e0) = a[u];
                    *reinterpret_cast<uint4 *>(dst + e1) = b[u];
                }
            }
        }
    }
}

}  // namespace rope
}  // namespace kvpack
