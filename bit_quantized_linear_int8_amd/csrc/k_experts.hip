// k_experts.hip -- the gated feed-forward of the experts a token was routed to,
// on int8 MFMA (gfx950).
//
//   g, u   = s_x[t] s13[e][.] (Xq[t] W13[e]^T)          gate rows 0..F-1, up rows F..2F-1
//   h      = g u / (1 + exp(-g))                        (fp32)
//   s_h    = max|h| / 127 (1 where that is 0), hq = rint(h / s_h)
//   y      = s_h s2[e][.] (hq W2[e]^T)                  (fp32)
//   out[t] = sum_j w[t][j] y[pair t k + j]              (j ascending, fp32)
//
// Rows are the dispatched pairs in expert order ("slots"): offsets[e] ..
// offsets[e + 1] are expert e's, order[slot] names the pair t k + j.
//
// Four launches: the gate and up product (the weight rows alternate between a
// gate row and its up row, so one lane holds both factors of an h), the codes of h, the
// down product, and the sum per token.  h and y pass through memory in fp32: the
// scale of an h row needs the whole row, and fp16 there would move about 1% of
// the codes.
//
// Few rows per expert: the weights are the traffic, so k_experts_stream reads
// each weight byte once per 16 MT rows, straight into MFMA operands, K split
// over the block's waves.  Many rows: k_experts_tile on LDS tiles.
#include "qa_tile.hpp"
#include "qa_launch.hpp"

namespace qa {

namespace {

typedef float v2f __attribute__((ext_vector_type(2)));

struct ExpertArgs {
    const int8_t* A;          // codes: Xq [T x K] (gated) or hq [slots x F]
    const float* sa;          // scale per token or per slot
    const int8_t* W;          // [E x rows x Kc]
    const float* sw;          // [E x rows]
    const int32_t* order;     // [P]
    const int32_t* offsets;   // [E + 1]
    const int32_t* tiles;     // of k_experts_plan
    int32_t* inv;             // [P] slot of a pair
    float* out;               // h [slots x F] or y [slots x K]
    int64_t T, P;
    int32_t E, k;
    int64_t Kc;               // bytes of the contraction
    int64_t N;                // output columns (gated: F)
};

// Expert e's slots, held within [0, P] whatever the offsets say.
__device__ __forceinline__ void slots_of(const ExpertArgs& a, int e, int64_t& s0, int64_t& n) {
    int64_t b = a.offsets[e], c = a.offsets[e + 1];
    b = b < 0 ? 0 : (b > a.P ? a.P : b);
    c = c < b ? b : (c > a.P ? a.P : c);
    s0 = b;
    n = c - b;
}

// Row of A that a slot reads (gated: its token), or -1.
template <bool GATED>
__device__ __forceinline__ int64_t row_of(const ExpertArgs& a, int64_t slot) {
    if constexpr (!GATED) return slot;
    const int p = a.order[slot];
    return p < 0 || p >= a.P ? -1 : p / a.k;
}

__device__ __forceinline__ float gated(float g, float u) { return g * sigmoid(g) * u; }

}  // namespace

// ---------------------------------------------------------------------------
// Few rows: block (n, e) computes 32 weight rows of expert e (16 gate and the
// same 16 up columns, or 32 columns) for all its slots, 16 MT at a time.  Bound by
// the weights' bytes: 8 tokens on 64 experts of 4096 x 1024 (8 each, 42 experts
// hit: 352 and 176 MB) in 62 and 27 us, 5.7 and 6.5 TB/s.  h and y are 5 us each in
// launches of their own (k_experts_codes, k_experts_sum): the scale of an h row
// and the sum of a token need every block's columns.
// ---------------------------------------------------------------------------
template <int MT, bool GATED>
__global__ __launch_bounds__(256) void k_experts_stream(ExpertArgs a) {
    __shared__ v4i part[4][MT][2][64];
    const int lane = threadIdx.x & 63, wave = wave_id();
    if (GATED) {
        const int64_t stride = (int64_t)gridDim.x * gridDim.y * 256;
        for (int64_t p = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x; p < a.P; p += stride)
            a.inv[p] = -1;
    }
    const int e = blockIdx.y;
    int64_t s0, n;
    slots_of(a, e, s0, n);
    if (n == 0) return;
    const int64_t n0 = (int64_t)blockIdx.x * (GATED ? 16 : 32);
    const int64_t wrows = GATED ? 2 * a.N : a.N;
    const rsrc_t rw = make_rsrc(a.W + (int64_t)e * wrows * a.Kc, wrows * a.Kc);
    const int r16 = lane & 15, c16 = (lane >> 4) * 16;
    const int64_t c0 = n0 + r16, c1 = GATED ? c0 : c0 + 16;  // output columns of this lane's weight rows
    const uint32_t o0 = c0 < a.N ? (uint32_t)(c0 * a.Kc) : kOOB;
    const uint32_t o1 = c1 < a.N ? (uint32_t)((GATED ? a.N + c1 : c1) * a.Kc) : kOOB;
    const uint32_t Kc = (uint32_t)a.Kc;
    const int nk = (int)((Kc + 63) / 64);
    for (int64_t m0 = 0; m0 < n; m0 += 16 * MT) {
        const int8_t* A = GATED ? a.A : a.A + (s0 + m0) * a.Kc;
        const rsrc_t ra = make_rsrc(A, GATED ? a.T * a.Kc : (n - m0) * a.Kc);
        uint32_t oa[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int64_t s = m0 + m * 16 + r16;
            const int64_t row = s < n ? (GATED ? row_of<true>(a, s0 + s) : s - m0) : -1;
            oa[m] = row < 0 ? kOOB : (uint32_t)(row * a.Kc);
        }
        v4i acc[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = v4i{0, 0, 0, 0};
        constexpr int U = 4;
        for (int s = wave; s < nk; s += 4 * U) {
            u32x4 w0[U], w1[U], x[U][MT];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const uint32_t kb = (uint32_t)(s + 4 * q) * 64 + c16;
                const bool in = kb < Kc;
                w0[q] = bload16(rw, in ? o0 + kb : kOOB);
                w1[q] = bload16(rw, in ? o1 + kb : kOOB);
#pragma unroll
                for (int m = 0; m < MT; ++m) x[q][m] = bload16(ra, in ? oa[m] + kb : kOOB);
            }
            __builtin_amdgcn_sched_barrier(0);               // every load in flight before the first use
#pragma unroll
            for (int q = 0; q < U; ++q)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const v4i xv = __builtin_bit_cast(v4i, x[q][m]);
                    acc[m][0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, w0[q]), xv, acc[m][0], 0, 0, 0);
                    acc[m][1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, w1[q]), xv, acc[m][1], 0, 0, 0);
                }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            part[wave][m][0][lane] = acc[m][0];
            part[wave][m][1][lane] = acc[m][1];
        }
        __syncthreads();
        for (int it = threadIdx.x; it < MT * (GATED ? 64 : 128); it += 256) {
            const int m = GATED ? it >> 6 : it >> 7, f = GATED ? 0 : (it >> 6) & 1, ln = it & 63;
            const int64_t s = m0 + m * 16 + (ln & 15);
            const int64_t col = n0 + f * 16 + 4 * (ln >> 4);
            if (s < n && col < a.N) {                        // N % 16 == 0: four columns exist together
                const int64_t row = row_of<GATED>(a, s0 + s);
                const float sx = row < 0 ? 0.0f : a.sa[row];
                v4i g = part[0][m][f][ln];
#pragma unroll
                for (int w = 1; w < 4; ++w) g += part[w][m][f][ln];
                v4f o;
                if constexpr (GATED) {
                    v4i u = part[0][m][1][ln];
#pragma unroll
                    for (int w = 1; w < 4; ++w) u += part[w][m][1][ln];
                    const float* sg = a.sw + (int64_t)e * wrows + col;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o[q] = gated((float)g[q] * sx * sg[q], (float)u[q] * sx * sg[a.N + q]);
                } else {
                    const float* sg = a.sw + (int64_t)e * wrows + col;
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[q] = (float)g[q] * sx * sg[q];
                }
                *reinterpret_cast<v4f*>(a.out + (s0 + s) * a.N + col) = o;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Many rows.  tiles[0] = number of row tiles; tiles[8 + 8 i ..] of row tile i: its
// expert, the expert's first row tile and its number of them, its first slot and
// its number of slots.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(1024) void k_experts_plan(ExpertArgs a, int32_t* __restrict__ tiles, int32_t bm,
                                                       int32_t most) {
    __shared__ int32_t pre[1024];
    const int e = threadIdx.x;
    for (int64_t p = (int64_t)blockIdx.x * 1024 + e; p < a.P; p += (int64_t)gridDim.x * 1024) a.inv[p] = -1;
    if (blockIdx.x != 0) return;
    int64_t s0 = 0, n = 0;
    if (e < a.E) slots_of(a, e, s0, n);
    const int mine = (int)((n + bm - 1) / bm);
    pre[e] = mine;
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
        const int v = e >= o ? pre[e - o] : 0;
        __syncthreads();
        pre[e] += v;
        __syncthreads();
    }
    // `most` tiles cover every set of disjoint ranges; overlapping ones (which
    // the caller must not pass) are cut off there
    if (e == 1023) tiles[0] = min(pre[1023], most);
    const int at = pre[e] - mine;
    for (int i = 0; i < mine && at + i < most; ++i) {
        int32_t* t = tiles + 8 + 8 * (at + i);
        t[0] = e;
        t[1] = at;
        t[2] = min(mine, most - at);
        t[3] = (int32_t)s0;
        t[4] = (int32_t)n;
    }
}

// 4099 tokens of 4 experts each, 32 experts, K = 4096, F = 2048: gate and up 340 to
// 385 us (the clock falls under the load), 1.45 to 1.6 POPS of the pairs' own
// operations, an eighth more with the ragged tiles'; down 200 to 220, 1.25 to 1.4:
// bound as the tile product is, then by its epilogue (268 MB).  256 tokens of 8, 64
// experts, F = 1024: 125 and 62 us, 537 and 268 MB of weights, 4.3 TB/s: bound by
// the weights, which 64-row tiles of 32 slots each read once.
template <class C, bool GATED>
__global__ __launch_bounds__(C::THREADS, 4) void k_experts_tile(ExpertArgs a, int32_t tiles_n) {
    extern __shared__ uint8_t smem[];
    const int ntiles = a.tiles[0] * tiles_n;
    // Blocks go round-robin over the 8 XCDs: XCD x walks a contiguous range of
    // tiles, an expert's row tiles in turn for one column tile and then the next,
    // so that weight rows (the larger operand) are fetched once into that L2.
    // With the columns fastest they are fetched once per row tile: 412 us against
    // 380 for the gate and up product of 4099 x 4 rows, 32 experts of 4096 x 4096.
    const int per = (ntiles + 7) >> 3;
    const int slot8 = (int)(blockIdx.x >> 3);
    const int id = (int)(blockIdx.x & 7) * per + slot8;
    if (slot8 >= per || id >= ntiles) return;
    const int32_t* row_tile = a.tiles + 8 + 8 * (id / tiles_n);
    const int e = row_tile[0], local = id - row_tile[1] * tiles_n;
    const int tn = local / row_tile[2];
    const int64_t m0 = (int64_t)(local % row_tile[2]) * C::BM;
    const int64_t s0 = row_tile[3], n = row_tile[4];
    constexpr int NC = GATED ? C::BN / 2 : C::BN;            // output columns of the tile
    const int64_t n0 = (int64_t)tn * NC;
    const int64_t wrows = GATED ? 2 * a.N : a.N;
    const int8_t* A = GATED ? a.A : a.A + (s0 + m0) * a.Kc;
    const rsrc_t ra = make_rsrc(A, GATED ? a.T * a.Kc : (n - m0) * a.Kc);
    const rsrc_t rw = make_rsrc(a.W + (int64_t)e * wrows * a.Kc, wrows * a.Kc);
    // the lane's rows and columns, their scales requested before the product
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t mw = m0 + (wave / C::WN) * C::TM + (lane & 15);
    const int wn = wave % C::WN;
    const float* sw = a.sw + (int64_t)e * wrows;
    float sx[C::FM], sg[C::FN][4];
    int64_t col[C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
        const int64_t s = mw + i * 16, row = s < n ? row_of<GATED>(a, s0 + s) : -1;
        sx[i] = row < 0 ? 0.0f : a.sa[row];
    }
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        col[j] = GATED ? n0 + wn * (C::TN / 2) + (lane >> 4) * (2 * C::FN) + j * 2
                       : n0 + wn * C::TN + j * 16 + 4 * (lane >> 4);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            sg[j][q] = col[j] < a.N ? (GATED ? sw[(q & 1 ? a.N : 0) + col[j] + (q >> 1)] : sw[col[j] + q]) : 0.0f;
    }
    v4i acc[C::FM][C::FN];
    tile::product<C>(
        ra, rw, (uint32_t)a.Kc, smem,
        [&](int r) -> uint32_t {
            if (m0 + r >= n) return kOOB;
            const int64_t row = GATED ? row_of<true>(a, s0 + m0 + r) : r;
            return row < 0 ? kOOB : (uint32_t)(row * a.Kc);
        },
        [&](int r) -> uint32_t {
            // gated: row 4 q + e of a wave's fragment j is the gate (e even) or up (e odd) row of its output column
            // 2 FN q + 2 j + e / 2, so that lane q's outputs of all fragments lie side by side
            const int64_t col = !GATED ? n0 + r
                                       : n0 + r / C::TN * (C::TN / 2) + ((r >> 2) & 3) * (2 * C::FN) +
                                             (r % C::TN) / 16 * 2 + ((r >> 1) & 1);
            if (col >= a.N) return kOOB;
            return (uint32_t)(((GATED && (r & 1) ? a.N : 0) + col) * a.Kc);
        },
        acc);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        if (col[j] >= a.N) continue;                         // N % 16 == 0: a lane's columns exist together
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            if (mw + i * 16 >= n) continue;
            float* o = a.out + (s0 + mw + i * 16) * a.N + col[j];
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = (float)acc[i][j][q] * sx[i] * sg[j][q];
            if constexpr (GATED) *reinterpret_cast<v2f*>(o) = v2f{gated(v[0], v[1]), gated(v[2], v[3])};
            else *reinterpret_cast<v4f*>(o) = v4f{v[0], v[1], v[2], v[3]};
        }
    }
}

// ---------------------------------------------------------------------------
// Codes of h, and the slot of each pair for the sum.  A row is read once, into
// registers: NC quads to a lane of its WPR waves (several rows to a block where
// one wave holds a row).  NC == 0: any F, one block per row, the row read twice,
// the second time from the caches.  Bound by memory: 134 MB in and 34 out at
// 16396 x 2048 in 30 us (5.6 TB/s; 39 with
// the row read twice and a division per element).
// ---------------------------------------------------------------------------
template <int WPR, int NC>
__global__ __launch_bounds__(256) void k_experts_codes(const float* __restrict__ h, const int32_t* __restrict__ order,
                                                       const int32_t* __restrict__ offsets, int32_t E, int64_t P,
                                                       int64_t F, int8_t* __restrict__ q, float* __restrict__ s_h,
                                                       int32_t* __restrict__ inv) {
    static_assert(WPR == 1 || WPR == 4, "waves of a row");
    __shared__ float red[4];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t slot = (int64_t)blockIdx.x * (4 / WPR) + (WPR == 1 ? wave : 0);
    // slots in no expert's range have no h: those past the last range, and those
    // before the first one where the caller holds a part of the experts
    if (slot < offsets[0] || slot >= offsets[E] || slot >= P) return;        // (the whole block with WPR == 4)
    const float* x = h + slot * F;
    constexpr int LANES = 64 * WPR;
    const int lp = WPR == 1 ? lane : (int)threadIdx.x;
    float amax = 0.0f;
    bool nan = false;
    auto look = [&](const v4f& v) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            amax = fmaxf(amax, __builtin_fabsf(v[j]));
            nan |= v[j] != v[j];
        }
    };
    v4f v[NC > 0 ? NC : 1];
    if constexpr (NC > 0) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = ((int64_t)i * LANES + lp) * 4;
            v[i] = c < F ? *reinterpret_cast<const v4f*>(x + c) : v4f{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) look(v[i]);
    } else {
        for (int64_t c = lp * 4; c < F; c += LANES * 4) look(*reinterpret_cast<const v4f*>(x + c));
    }
    if (nan) amax = __builtin_inff();
    amax = wave_max(amax);
    if constexpr (WPR == 4) {
        if (lane == 0) red[wave] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    }
    const bool fine = amax < __builtin_inff();
    float s = amax / 127.0f;
    if (s == 0.0f) s = 1.0f;
    if (!fine) s = __builtin_nanf("");
    if (lp == 0) {
        s_h[slot] = s;
        const int p = order[slot];
        if (p >= 0 && p < P) inv[p] = (int32_t)slot;
    }
    const float r = 1.0f / s;
    auto put = [&](int64_t c, const v4f& w) __attribute__((always_inline)) {
        uint32_t b = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // (the reciprocal of a scale near fp32's smallest normal number is not enough)
            const float n = s >= 0x1p-120f ? quot_rne(w[j], s, r) : __builtin_rintf(w[j] / s);
            b |= (fine ? (uint32_t)(int)n & 0xffu : 0u) << (8 * j);
        }
        *reinterpret_cast<uint32_t*>(q + slot * F + c) = b;
    };
    if constexpr (NC > 0) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = ((int64_t)i * LANES + lp) * 4;
            if (c < F) put(c, v[i]);
        }
    } else {
        for (int64_t c = lp * 4; c < F; c += LANES * 4) put(c, *reinterpret_cast<const v4f*>(x + c));
    }
}

// out[t] = sum_j w[t][j] y[slot of pair t k + j]; pairs without a slot add nothing.
// A thread has four columns of one token, K / 4 threads to a token; eight pairs'
// rows in flight at once.  Bound by memory: 268 MB in and 34 out at 4099 x 4 x
// 4096 in 50 us (6.0 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void k_experts_sum(const float* __restrict__ y, const float* __restrict__ w,
                                                     const int32_t* __restrict__ inv, int64_t T, int32_t k, int32_t K,
                                                     void* __restrict__ out) {
    const uint32_t id = blockIdx.x * 256 + threadIdx.x, quads = (uint32_t)K / 4;         // (T K is below 2^31)
    const int64_t t = id / quads;
    if (t >= T) return;
    const int c = (int)(id % quads) * 4;
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int U = 8;
    for (int j0 = 0; j0 < k; j0 += U) {
        int s[U];
        float wt[U];
        v4f v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            s[j] = j0 + j < k ? inv[t * k + j0 + j] : -1;
            wt[j] = j0 + j < k ? w[t * k + j0 + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (s[j] >= 0) v[j] = *reinterpret_cast<const v4f*>(y + (int64_t)s[j] * K + c);
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (s[j] >= 0)
#pragma unroll
                for (int q = 0; q < 4; ++q) o[q] = __builtin_fmaf(wt[j], v[j][q], o[q]);
    }
    store4(out, t * K + c, DT, o, 4, true);
}

namespace {
constexpr size_t up256(size_t v) { return (v + 255) / 256 * 256; }
struct ExpertLayout { size_t mid, hq, s_h, inv, tiles, total; };
ExpertLayout expert_layout(int64_t P, int64_t K, int64_t E, int64_t F) {
    ExpertLayout L;
    size_t off = 0;
    L.mid = off; off += up256((size_t)P * (size_t)(K > F ? K : F) * 4);      // h, then y
    L.hq = off; off += up256((size_t)P * (size_t)F);
    L.s_h = off; off += up256((size_t)P * 4);
    L.inv = off; off += up256((size_t)P * 4);
    L.tiles = off; off += up256((size_t)(8 + 8 * (P / 64 + E + 1)) * 4);      // tiles of 64 rows or more
    L.total = off;
    return L;
}
}  // namespace

size_t experts_scratch_bytes(int64_t P, int64_t K, int64_t E, int64_t F) { return expert_layout(P, K, E, F).total; }

// Upper bound of the row tiles: the whole ones and one ragged one per expert.
template <class C>
static int64_t most_tiles(const ExpertArgs& a) { return a.P / C::BM + (a.E < a.P ? a.E : a.P); }

template <class C, bool GATED>
static hipError_t run_tile(const ExpertArgs& a, hipStream_t st) {
    const int64_t nc = GATED ? C::BN / 2 : C::BN;
    const int64_t tn = (a.N + nc - 1) / nc;
    const int64_t tm = most_tiles<C>(a);
    const int64_t blocks = ((tm * tn + 7) / 8) * 8;
    hipLaunchKernelGGL((k_experts_tile<C, GATED>), dim3((unsigned)blocks), dim3(C::THREADS), C::LDS, st, a, (int32_t)tn);
    return hipGetLastError();
}

template <bool GATED>
static hipError_t run_stream(const ExpertArgs& a, int mt, hipStream_t st) {
    const dim3 grid((unsigned)((a.N + (GATED ? 15 : 31)) / (GATED ? 16 : 32)), (unsigned)a.E);
    if (mt == 1) hipLaunchKernelGGL((k_experts_stream<1, GATED>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_experts_stream<2, GATED>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <class C, class F>
static hipError_t run_tiles(const ExpertArgs& a1, const ExpertArgs& a2, int32_t* tiles, F&& codes, hipStream_t st) {
    hipLaunchKernelGGL(k_experts_plan, dim3((unsigned)((a1.P + 8191) / 8192)), dim3(1024), 0, st, a1, tiles, C::BM,
                       (int32_t)most_tiles<C>(a1));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (e = run_tile<C, true>(a1, st)) != hipSuccess || (e = codes()) != hipSuccess) return e;
    return run_tile<C, false>(a2, st);
}

hipError_t launch_experts_i8(const int8_t* Xq, const float* s_x, int64_t T, int64_t K, const float* w,
                             const int32_t* order, const int32_t* offsets, int64_t E, int k, const int8_t* W13,
                             const float* s13, int64_t F, const int8_t* W2, const float* s2, void* out, int out_dtype,
                             void* scratch, hipStream_t st) {
    const int64_t P = T * k;
    const ExpertLayout L = expert_layout(P, K, E, F);
    uint8_t* ws = static_cast<uint8_t*>(scratch);
    float* mid = reinterpret_cast<float*>(ws + L.mid);
    int8_t* hq = reinterpret_cast<int8_t*>(ws + L.hq);
    float* s_h = reinterpret_cast<float*>(ws + L.s_h);
    int32_t* inv = reinterpret_cast<int32_t*>(ws + L.inv);
    int32_t* tiles = reinterpret_cast<int32_t*>(ws + L.tiles);
    ExpertArgs a1{Xq, s_x, W13, s13, order, offsets, tiles, inv, mid, T, P, (int32_t)E, k, K, F};
    ExpertArgs a2{hq, s_h, W2, s2, order, offsets, tiles, inv, mid, T, P, (int32_t)E, k, F, K};
    hipError_t e;
    auto codes = [&]() {
#define QA_CODES(WPR, NC)                                                                                            \
    hipLaunchKernelGGL((k_experts_codes<WPR, NC>), dim3((unsigned)((P + 4 / WPR - 1) / (4 / WPR))), dim3(256), 0, st, \
                       mid, order, offsets, (int32_t)E, P, F, hq, s_h, inv)
        if (F <= 256) QA_CODES(1, 1);
        else if (F <= 1024) QA_CODES(1, 4);
        else if (F <= 2048) QA_CODES(4, 2);
        else if (F <= 4096) QA_CODES(4, 4);
        else QA_CODES(4, 0);
#undef QA_CODES
        return hipGetLastError();
    };
    // By rows per expert (64 experts of 8 per token, K = 4096, F = 1024; us of the
    // call).  Streaming 16 or 32 rows at a time, tiles of 64 x 128 (three stages,
    // for weights that come from HBM), tiles of 128 x 192:
    //   rows     1     4     8    16    32    64   125   250
    //   16      99   158   199   285   449   816
    //   32     102   152   180   229   332   555
    //   64     113   166   179   195   219   248   318   569
    //   128    116   197   204   219   239   270   313   486
    const int64_t avg = P / E;
    if (avg < 8) {
        const int mt = avg <= 2 ? 1 : 2;
        if ((e = run_stream<true>(a1, mt, st)) != hipSuccess) return e;
        if ((e = codes()) != hipSuccess) return e;
        if ((e = run_stream<false>(a2, mt, st)) != hipSuccess) return e;
    } else {
        // the large tile needs enough of them for two on every CU
        const int64_t large = (P / 128) * ((2 * F + 191) / 192);
        if (avg < 120 || large < 512) e = run_tiles<tile::Cfg<64, 128, 2, 4, 3>>(a1, a2, tiles, codes, st);
        else e = run_tiles<tile::Cfg<128, 192, 2, 4, 2>>(a1, a2, tiles, codes, st);
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)((T * (K / 4) + 255) / 256));
    if (out_dtype == 0) hipLaunchKernelGGL(k_experts_sum<0>, grid, dim3(256), 0, st, mid, w, inv, T, k, (int32_t)K, out);
    else if (out_dtype == 1) hipLaunchKernelGGL(k_experts_sum<1>, grid, dim3(256), 0, st, mid, w, inv, T, k, (int32_t)K, out);
    else hipLaunchKernelGGL(k_experts_sum<2>, grid, dim3(256), 0, st, mid, w, inv, T, k, (int32_t)K, out);
    return hipGetLastError();
}

}  // namespace qa
