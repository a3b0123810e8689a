// k_linear.hip -- the int8 linear on codes with bias, activation and residual in
// its epilogue, on gfx950.
//
//   out[m][n] = act(s_x[m] s_w[n] sum_k Xq[m][k] Wq[n][k] + bias[n]) + res[m][n]
//
// The product is exact (int32); the rest is fp32 and rounded once.  Three forms: for
// few tokens the weights streamed, straight into MFMA operands in one round of blocks
// or through LDS in many, and for many tokens the tile product of qa_tile.hpp.
//
// The activations need no table and no branch:
//   silu x sigma(x), and gelu's tanh form 0.5 x (1 + tanh u) = x sigma(2 u), by the
//   library's sigma, which keeps its digits in both tails;
//   gelu x Phi(x) = max(x, 0) - |x| erfc(|x| / sqrt 2) / 2, with erfc(z) = exp(-z^2)
//   t P(t), t = 1 / (1 + z / 2): exp(z^2) erfc(z) / t is smooth on 0 < t <= 1, and P
//   of degree 8, fitted to it for the least relative error (4.4e-8), is 3e-7
//   off in fp32.
#include "qa_tile.hpp"
#include "qa_launch.hpp"

namespace qa {

namespace {

struct LinearArgs {
    const int8_t* Xq;
    const float* s_x;
    const int8_t* Wq;
    const float* s_w;
    const float* bias;         // [N] or nullptr
    const void* res;           // [M][ldr] or nullptr, of type dt
    void* out;                 // [M][ldo]
    int64_t M, K, N, ldr, ldo;
    float c1, c3;              // sigma's argument c1 x + c3 x^3
    float least;               // linear: results below it become it (-inf, or relu's 0)
    int32_t dt;
    bool vec, vecr, vecn;      // rows of out, of res, and s_w and bias allow 4-element vectors
};

enum Act { LINEAR = 0, SIGMA = 1, GELU = 2 };

template <int ACT>
__device__ __forceinline__ float activate(const LinearArgs& a, float x) {
    if constexpr (ACT == SIGMA) {
        const float y = __builtin_amdgcn_fmed3f(x, -256.0f, 256.0f);    // (sigma is 0 or 1 there, and c3 times an infinity may be NaN)
        return x * sigmoid(y * __builtin_fmaf(a.c3 * y, y, a.c1));
    }
    if constexpr (ACT == GELU) {
        const float z = __builtin_fabsf(x);
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(z, 0.353553390593273762f, 1.0f));
        float p = -0.05927713f;
        p = __builtin_fmaf(p, t, 0.28559145f);
        p = __builtin_fmaf(p, t, -0.48930627f);
        p = __builtin_fmaf(p, t, 0.28047854f);
        p = __builtin_fmaf(p, t, -0.02828767f);
        p = __builtin_fmaf(p, t, 0.20339027f);
        p = __builtin_fmaf(p, t, 0.242926f);
        p = __builtin_fmaf(p, t, 0.2823997f);
        p = __builtin_fmaf(p, t, 0.28208503f);
        const float e = __builtin_amdgcn_exp2f(x * x * -0.72134752044448170368f);
        return (x < 0.0f ? 0.0f : x) - __builtin_fminf(z, 32.0f) * (0.5f * t * p * e);    // (from 16 on e is 0: no infinity times it)
    }
    return x < a.least ? a.least : x;                        // (a NaN stays)
}

// Sixteen bytes from each lane's offset to LDS, lane after lane.
__device__ __forceinline__ void load_lds16(rsrc_t r, uint32_t off, void* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (tile::lds_void*)lds, 16, off, 0, 0, 0);
}

// Four 16-bit values of type dt (1 fp16, 2 bf16).
__device__ __forceinline__ v4f widen4(u32x2 w, int dt) {
    v4f v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint16_t h = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        v[e] = dt == 1 ? h2f(h) : __builtin_bit_cast(float, (uint32_t)h << 16);
    }
    return v;
}

// Four residuals of type dt at p[at], of which the first n exist.
__device__ __forceinline__ v4f load4(const void* p, int64_t at, int dt, int n, bool vec) {
    v4f v = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (dt == 0) {
        const float* r = static_cast<const float*>(p) + at;
        if (vec && n >= 4) return *reinterpret_cast<const v4f*>(r);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) v[e] = r[e];
        return v;
    }
    const uint16_t* r = static_cast<const uint16_t*>(p) + at;
    uint16_t h[4] = {0, 0, 0, 0};
    if (vec && n >= 4) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(r);
        h[0] = (uint16_t)w[0], h[1] = (uint16_t)(w[0] >> 16), h[2] = (uint16_t)w[1], h[3] = (uint16_t)(w[1] >> 16);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) h[e] = r[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = dt == 1 ? h2f(h[e]) : __builtin_bit_cast(float, (uint32_t)h[e] << 16);
    return v;
}

}  // namespace

// ---------------------------------------------------------------------------
// Few tokens (at most 16 MT) and columns: 16 output columns per block, K split over
// its 8 waves, which bring the weights' rows straight into MFMA operands with every
// load in flight at once.  One round of blocks, bound by latency: 16 x 4096 x 4096 in
// 6.8 us, 2.5 TB/s (the stream below, which has to go through LDS, 7.2; tiles 12.8).
// ---------------------------------------------------------------------------
template <int MT>
__global__ __launch_bounds__(512) void k_linear_stream(LinearArgs a, int act) {
    __shared__ v4i part[8][MT][64];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const uint32_t K = (uint32_t)a.K;
    const int r16 = lane & 15, c16 = (lane >> 4) * 16;
    const int64_t mo = wave * 16 + r16, no = n0 + 4 * (lane >> 4);    // the lane's outputs (waves below MT)
    const bool live = wave < MT && mo < a.M && no < a.N;
    const int cols = live ? (int)(a.N - no < 4 ? a.N - no : 4) : 0;
    // what the epilogue reads is requested before the weights
    float sx = 0.0f, sw[4] = {0.0f, 0.0f, 0.0f, 0.0f}, bi[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    v4f res = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
        sx = a.s_x[mo];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            sw[q] = a.s_w[no + min(q, cols - 1)];
            if (a.bias) bi[q] = a.bias[no + min(q, cols - 1)];
        }
        if (a.res) res = load4(a.res, mo * a.ldr + no, a.dt, cols, a.vecr);
    }
    const rsrc_t rw = make_rsrc(a.Wq + n0 * a.K, (a.N - n0) * a.K);
    const rsrc_t rx = make_rsrc(a.Xq, a.M * a.K);
    const uint32_t ow = n0 + r16 < a.N ? (uint32_t)r16 * K : kOOB;
    uint32_t ox[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) ox[m] = m * 16 + r16 < a.M ? (uint32_t)(m * 16 + r16) * K : kOOB;
    v4i acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4i{0, 0, 0, 0};
    const int nk = (int)((K + 63) / 64);
    constexpr int U = MT == 4 ? 4 : 8;
    u32x4 w[U], x[U][MT];
    auto load = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const uint32_t kb = (uint32_t)(s + 8 * q) * 64 + c16;
            const bool in = kb < K;
            w[q] = bload16(rw, in ? ow + kb : kOOB);
#pragma unroll
            for (int m = 0; m < MT; ++m) x[q][m] = bload16(rx, in ? ox[m] + kb : kOOB);
        }
        __builtin_amdgcn_sched_barrier(0);                   // every load in flight before the first use
    };
    __builtin_amdgcn_sched_barrier(0);
    load(wave);
    for (int s = wave; s < nk;) {
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, w[q]),
                                                               __builtin_bit_cast(v4i, x[q][m]), acc[m], 0, 0, 0);
        s += 8 * U;
        if (s < nk) load(s);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][m][lane] = acc[m];
    __syncthreads();
    if (!live) return;
    v4i c = part[0][wave][lane];
#pragma unroll
    for (int p = 1; p < 8; ++p) c += part[p][wave][lane];
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float y = (float)c[q] * sx * sw[q] + bi[q];
        v[q] = (act == SIGMA ? activate<SIGMA>(a, y) : act == GELU ? activate<GELU>(a, y) : activate<LINEAR>(a, y)) + res[q];
    }
    store4(a.out, mo * a.ldo + no, a.dt, v, cols, a.vec);
}

// Four floats of a vector of n from column c on, as far as there are any.
__device__ __forceinline__ v4f cols4(const float* p, int64_t c, int n, bool vec) {
    if (vec && n >= 4) return *reinterpret_cast<const v4f*>(p + c);
    v4f v = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n) v[e] = p[c + e];
    return v;
}

// ---------------------------------------------------------------------------
// At most 16 tokens and many columns: the stream of the weights is the work.  A block
// takes 16 output columns at a time (gridDim.x apart), its 8 waves a slice of 512
// bytes each of every 4096 of K.  A wave's 16 rows of W come by direct loads of whole
// lines into a stage of LDS of its own (the 16-byte chunk c of row r at c ^ (r & 7)),
// one further stage in flight, so that no barrier drains the stream; its tokens' codes
// are MFMA operands in registers, which stay there from column to column while K is at
// most 4096 and are requested a stage ahead where it is more.  The waves' sums meet in
// LDS, and one wave ends the tile.
// By size (us, graphs of calls; this form, the one above, tiles of 64 x 64):
//   K 4096   1 x 11008     12.0   10.9   13.3      16 x 11008    13.2   14.0   13.2
//            1 x 32000     28.0   26.2   28.4      16 x 32000    29.4   40.8   29.2
//            1 x 128000    95.8   89.3    128      16 x 128000    103    149    129
//   K 11008  1 x 8192      18.3   21.0   33.1      16 x 8192     23.3   27.5   33.1
//            1 x 16384     38.6   44.7   46.2      16 x 16384    48.3   59.6   46.8
// (5.1 TB/s at 16 x 128000.)  The border to the form above goes by columns alone: a
// single token whose K is one part would be 7 to 10% faster there, 16 tokens, and one with
// K of several parts, are slower.  32 tokens in two operands are no faster than tiles from
// 8192 columns on (13.0 and 13.2), 64 slower (their codes' traffic passes the weights').
// ---------------------------------------------------------------------------
template <bool RES16>
__global__ __launch_bounds__(512, 2) void k_linear_few(LinearArgs a, int act) {
    constexpr int SL = 512, STEPS = SL / 64, INS = SL / 64, CH = SL / 16, NW = 8;
    constexpr int STAGE = 16 * SL;
    // one array: beside a second one the compiler takes every stage load for a writer of what is read
    __shared__ __attribute__((aligned(16))) uint8_t smem[NW * 2 * STAGE + NW * 1024];
    v4i* const part = reinterpret_cast<v4i*>(smem + NW * 2 * STAGE);
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r16 = lane & 15, q16 = lane >> 4;
    const uint32_t K = (uint32_t)a.K;
    const int groups = (int)((a.N + 15) / 16), parts = (int)((K + NW * SL - 1) / (NW * SL));
    const rsrc_t rx = make_rsrc(a.Xq, a.M * a.K);
    const uint32_t ox = r16 < a.M ? (uint32_t)r16 * K : kOOB;
    v4i x[STEPS];
    auto load_x = [&](int p) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const uint32_t k = (uint32_t)(p * NW + wave) * SL + s * 64 + q16 * 16;
            x[s] = __builtin_bit_cast(v4i, bload16(rx, k < K ? ox + k : kOOB));
        }
    };
    // a lane's rows and chunks of the loads of a stage
    uint32_t row[INS], chunk[INS];
#pragma unroll
    for (int n = 0; n < INS; ++n) {
        const int P = n * 64 + lane;
        row[n] = P / CH;
        chunk[n] = (uint32_t)(((P % CH) ^ (row[n] & 7)) * 16);
    }
    uint8_t* const mine = smem + wave * 2 * STAGE;
    auto fill = [&](int st, int grp, int p) __attribute__((always_inline)) {
        const int64_t n0 = (int64_t)grp * 16;
        const uint32_t rows = grp < groups ? (uint32_t)(a.N - n0 < 16 ? a.N - n0 : 16) : 0u;
        const rsrc_t rw = make_rsrc(a.Wq + (grp < groups ? n0 : 0) * a.K, (int64_t)rows * K);
        const uint32_t k0 = (uint32_t)(p * NW + wave) * SL;
#pragma unroll
        for (int n = 0; n < INS; ++n)
            load_lds16(rw, row[n] < rows && k0 + chunk[n] < K ? row[n] * K + k0 + chunk[n] : kOOB, mine + st * STAGE + n * 1024);
    };
    const bool ends = wave == 0 && r16 < a.M;                // the lane's row is r16
    const float sx = ends ? a.s_x[r16] : 0.0f;

    // items: the parts of K of one group after the other
    int grp = blockIdx.x, p = 0, ngrp = grp, np = 0, st = 0;
    auto next = [&]() __attribute__((always_inline)) {
        if (++np == parts) np = 0, ngrp += gridDim.x;
    };
    load_x(0);
    fill(0, ngrp, np);
    next();
    fill(1, ngrp, np);
    next();
    v4i acc = v4i{0, 0, 0, 0};
    while (grp < groups) {
        __builtin_amdgcn_s_waitcnt(tile::vmcnt(INS));          // this stage and these codes are there, the next stage may not
        asm volatile("" ::: "memory");
        const uint8_t* from = mine + st * STAGE;
        v4i w[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            w[s] = *reinterpret_cast<const v4i*>(from + r16 * SL + (((4 * s + q16) ^ (r16 & 7)) << 4));
#pragma unroll
        for (int s = 0; s < STEPS; ++s) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s], x[s], acc, 0, 0, 0);
        const bool last = p + 1 == parts;
        const int64_t n = (int64_t)grp * 16 + 4 * q16;
        const int cols = (int)(a.N - n < 4 ? a.N - n : 4);
        // What the end reads is requested before the stream goes on, without a branch (one would wait for it).
        const int64_t n0 = (int64_t)grp * 16;
        const int64_t bytes = last && wave == 0 ? (a.N - n0 < 16 ? a.N - n0 : 16) * 4 : 0;
        const rsrc_t rsw = make_rsrc(a.s_w + n0, bytes), rbi = make_rsrc(a.bias + n0, a.bias ? bytes : 0);
        float sw[4], bi[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            sw[q] = __builtin_bit_cast(float, bload4(rsw, 16 * q16 + 4 * q));
            bi[q] = __builtin_bit_cast(float, bload4(rbi, 16 * q16 + 4 * q));
        }
        u32x2 early;
        if constexpr (RES16)
            early = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.res) + (ends ? r16 : 0) * a.ldr + (cols > 0 ? n : 0));
        if (parts > 1) load_x(last ? 0 : p + 1);
        __builtin_amdgcn_s_waitcnt(0xC07F);                  // lgkmcnt(0): the stage is read
        asm volatile("" ::: "memory");
        fill(st, ngrp, np);
        next();
        st ^= 1;
        if (!last) {
            ++p;
            continue;
        }
        p = 0;
        lds_only_barrier();                                  // the sums before these have been taken
        part[wave * 64 + lane] = acc;
        acc = v4i{0, 0, 0, 0};
        lds_only_barrier();
        if (ends && cols > 0) {
            v4i c = part[lane];
#pragma unroll
            for (int q = 1; q < NW; ++q) c += part[q * 64 + lane];
            v4f res = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (RES16) res = widen4(early, a.dt);
            else if (a.res) res = load4(a.res, r16 * a.ldr + n, a.dt, cols, a.vecr);
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float y = (float)c[q] * sx * sw[q] + bi[q];
                v[q] = (act == SIGMA ? activate<SIGMA>(a, y) : act == GELU ? activate<GELU>(a, y) : activate<LINEAR>(a, y)) + res[q];
            }
            store4(a.out, r16 * a.ldo + n, a.dt, v, cols, a.vec);
        }
        grp += gridDim.x;
    }
    __builtin_amdgcn_s_waitcnt(tile::vmcnt(0));                // no load is left to land in another block's LDS
}

// ---------------------------------------------------------------------------
// Many tokens: one tile of the product per block.
//
// A stage's fragment reads are what a tile of few blocks per CU waits for most: with
// Split the waves are two groups that take half of each stage's K each, so that a
// wave's tile is twice as large and its reads per product half in one direction; the
// groups exchange halves of their sums through LDS at the end.  (us, tiles as below
// without and with it, graphs of calls with gelu and residual)
//   K 4096   128 x 4096  14.1  12.2      512 x 4096   20.7  18.4      200 x 16000  28.9  26.8
//            256 x 4096  15.1  12.9      777 x 4096   28.5  26.5      1024 x 4096  32.1  28.5
//   K 11008  128 x 4096  29.0  24.3      777 x 4096   57.7  52.2
// (4, 5 stages or half of the waves with larger tiles are no faster: 26 to 27 at 777 x
// 4096; of its 26 about 4 are the epilogue's vector instructions, 40 a result with gelu.)
// Tiles that have two blocks on each CU anyway are slower with it (2048 x 4096: 47.2
// and 50.9), and at 128 x 192 their sums pass the registers.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, int STAGES>
struct Whole : tile::Cfg<BM, BN, WM, WN, STAGES> {
    static constexpr int KS = 1;
};
template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct Split {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KS = 2, NW = WM * WN, NWA = KS * NW;
    static constexpr int BK = 128, STAGES = STAGES_, THREADS = 64 * NWA;
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    static constexpr int INS = (BM + BN) / 8 / NWA;          // load instructions of a wave per stage
    static constexpr int STAGE = (BM + BN) * BK, LDS = STAGES * STAGE;
    static_assert(FM % 2 == 0 && TN % 16 == 0, "the groups halve a wave tile's fragments");
    static_assert((BM + BN) % (8 * NWA) == 0 && BM % 8 == 0, "a stage's rows split evenly over the waves");
    static_assert(BM * BN * 4 <= LDS && STAGES >= 3, "both groups' halves fit the stages");
};

// tile::product with each stage's K halved between two groups of waves: on return sum
// holds the first (group 0) or second half of the wave tile's rows of fragments.
template <class C, class RA, class RB>
__device__ __forceinline__ void split_product(rsrc_t rsa, rsrc_t rsb, uint32_t K, uint8_t* smem, RA&& row_a, RB&& row_b,
                                              v4i (&sum)[C::FM / 2][C::FN]) {
    const int lane = threadIdx.x & 63, all = wave_id(), grp = all / C::NW, wave = all % C::NW;
    const int wm = wave / C::WN, wn = wave % C::WN;
    uint32_t off[C::INS], ck[C::INS];
#pragma unroll
    for (int q = 0; q < C::INS; ++q) {
        const int P = (q * C::NWA + all) * 64 + lane;        // 16-byte chunk of the stage
        const int r = P >> 3, c = (P & 7) ^ (r & 7);
        const uint32_t base = r < C::BM ? row_a(r) : row_b(r - C::BM);
        off[q] = base == kOOB ? kOOB : base + c * 16;
        ck[q] = c * 16;
    }
    const int nk = (int)((K + C::BK - 1) / C::BK);
    auto issue = [&](int kt, int st) __attribute__((always_inline)) {    // (zeros past K: always as many loads)
        const uint32_t k0 = (uint32_t)kt * C::BK;
#pragma unroll
        for (int q = 0; q < C::INS; ++q) {
            const bool a = (q * C::NWA + all) * 8 < C::BM;
            load_lds16(a ? rsa : rsb, k0 + ck[q] < K ? off[q] + k0 : kOOB, smem + st * C::STAGE + (q * C::NWA + all) * 1024);
        }
    };
    v4i acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = v4i{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < C::STAGES - 1; ++q) issue(q, q);
    const int c = (lane >> 4) + 4 * grp;
    int st = 0;
    for (int kt = 0; kt < nk; ++kt) {
        // this stage is there, and what this wave read of the one before has arrived: its buffer is filled anew
        __builtin_amdgcn_s_waitcnt(tile::vmcnt(C::INS * (C::STAGES - 2)) & 0xf0ff);
        tile::block_barrier();
        issue(kt + C::STAGES - 1, st == 0 ? C::STAGES - 1 : st - 1);
        const uint8_t* sa = smem + st * C::STAGE;
        const uint8_t* sb = sa + C::BM * C::BK;
        v4i fa[C::FM], fb[C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
            fa[i] = *reinterpret_cast<const v4i*>(sa + tile::swz(wm * C::TM + i * 16 + (lane & 15), c));
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            fb[j] = *reinterpret_cast<const v4i*>(sb + tile::swz(wn * C::TN + j * 16 + (lane & 15), c));
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        st = st + 1 == C::STAGES ? 0 : st + 1;
    }
    __builtin_amdgcn_s_waitcnt(tile::vmcnt(0));
    __syncthreads();                                         // the stages are free
    constexpr int H = C::FM / 2;
    v4i* const mine = reinterpret_cast<v4i*>(smem) + all * (H * C::FN * 64) + lane;
    const v4i* const theirs = reinterpret_cast<const v4i*>(smem) + ((1 - grp) * C::NW + wave) * (H * C::FN * 64) + lane;
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            mine[(i * C::FN + j) * 64] = grp ? acc[i][j] : acc[H + i][j];
            sum[i][j] = grp ? acc[H + i][j] : acc[i][j];
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) sum[i][j] += theirs[(i * C::FN + j) * 64];
}

// RES16: a 16-bit residual whose rows allow vectors is requested before the product
// and waits in registers (24 for the largest tile), so that its bytes come during
// the product instead of after it: 2048 x 11008 x 4096 takes 103 us so against 119.
template <class C, int ACT, bool RES16>
__global__ __launch_bounds__(C::THREADS, 4) void k_linear_tile(LinearArgs a, int32_t tiles_m, int32_t tiles_n) {
    extern __shared__ uint8_t smem[];
    int tm, tn;
    tile::of_block(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * C::BN;
    const rsrc_t ra = make_rsrc(a.Xq + m0 * a.K, (a.M - m0) * a.K);
    const rsrc_t rw = make_rsrc(a.Wq + n0 * a.K, (a.N - n0) * a.K);
    const uint32_t K = (uint32_t)a.K;
    constexpr int FM = C::FM / C::KS;                        // rows of fragments that the wave ends
    const int lane = threadIdx.x & 63, wave = wave_id() % (C::WM * C::WN), grp = wave_id() / (C::WM * C::WN);
    const int64_t mw = m0 + (wave / C::WN) * C::TM + grp * 16 * FM + (lane & 15);
    const int64_t nw = n0 + (wave % C::WN) * C::TN + 4 * (lane >> 4);
    u32x2 early[RES16 ? FM : 1][RES16 ? C::FN : 1];
    if constexpr (RES16) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                const int64_t m = mw + i * 16 < a.M ? mw + i * 16 : a.M - 1, n = nw + j * 16 < a.N ? nw + j * 16 : 0;
                early[i][j] = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.res) + m * a.ldr + n);
            }
    }
    v4i acc[FM][C::FN];
    const auto row_a = [&](int r) -> uint32_t { return m0 + r < a.M ? (uint32_t)r * K : kOOB; };
    const auto row_b = [&](int r) -> uint32_t { return n0 + r < a.N ? (uint32_t)r * K : kOOB; };
    if constexpr (C::KS == 1) tile::product<C>(ra, rw, K, smem, row_a, row_b, acc);
    else split_product<C>(ra, rw, K, smem, row_a, row_b, acc);
    float sx[FM];
    v4f sw[C::FN], bi[C::FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) sx[i] = mw + i * 16 < a.M ? a.s_x[mw + i * 16] : 0.0f;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        const int64_t n = nw + j * 16;
        const int cols = (int)(a.N - n < 4 ? a.N - n : 4);
        sw[j] = cols4(a.s_w, n, cols, a.vecn);
        bi[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        if (a.bias) bi[j] = cols4(a.bias, n, cols, a.vecn);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t m = mw + i * 16;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const int64_t n = nw + j * 16;
            if (n >= a.N) continue;
            const int cols = (int)(a.N - n < 4 ? a.N - n : 4);
            v4f res = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (RES16) res = widen4(early[i][j], a.dt);
            else if (a.res) res = load4(a.res, m * a.ldr + n, a.dt, cols, a.vecr);
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = activate<ACT>(a, (float)acc[i][j][q] * sx[i] * sw[j][q] + bi[j][q]) + res[q];
            store4(a.out, m * a.ldo + n, a.dt, v, cols, a.vec);
        }
    }
}

namespace {

// Whether a 16-bit residual can be read four values at a time.
bool res16(const LinearArgs& a) { return a.res && a.dt != 0 && a.vecr && a.N % 4 == 0; }

template <class C, int ACT>
hipError_t run_tile(const LinearArgs& a, hipStream_t st) {
    const int tm = (int)((a.M + C::BM - 1) / C::BM), tn = (int)((a.N + C::BN - 1) / C::BN);
    if (res16(a))
        hipLaunchKernelGGL((k_linear_tile<C, ACT, true>), dim3((unsigned)(tm * tn)), dim3(C::THREADS), C::LDS, st, a, tm, tn);
    else
        hipLaunchKernelGGL((k_linear_tile<C, ACT, false>), dim3((unsigned)(tm * tn)), dim3(C::THREADS), C::LDS, st, a, tm, tn);
    return hipGetLastError();
}

// Tiles by how many of them there are.
template <int ACT>
hipError_t run_tiles(const LinearArgs& a, hipStream_t st) {
    const int64_t small = ((a.M + 63) / 64) * ((a.N + 63) / 64), tiles = ((a.M + 127) / 128) * ((a.N + 127) / 128);
    if (small <= 512) return run_tile<Split<64, 64, 2, 2, 3>, ACT>(a, st);
    if (tiles <= 256) return run_tile<Split<128, 128, 2, 4, 3>, ACT>(a, st);
    if (tiles <= 512) return run_tile<Whole<128, 128, 2, 4, 2>, ACT>(a, st);
    return run_tile<Whole<128, 192, 2, 4, 2>, ACT>(a, st);
}

bool vec4(const void* p, int64_t ld, int dt) {
    return ld % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & (dt == 0 ? 15 : 7)) == 0;
}

}  // namespace

hipError_t launch_linear_i8_act(const int8_t* Xq, const float* s_x, int64_t M, int64_t K, const int8_t* Wq,
                                const float* s_w, int64_t N, const float* bias, int act, const void* res, int64_t ldr,
                                void* out, int64_t ldo, int dtype, hipStream_t st) {
    LinearArgs a{};
    a.Xq = Xq; a.s_x = s_x; a.Wq = Wq; a.s_w = s_w; a.bias = bias; a.res = res; a.out = out;
    a.M = M; a.K = K; a.N = N; a.ldr = ldr; a.ldo = ldo; a.dt = dtype;
    a.least = act == QA_ACT_RELU ? 0.0f : -__builtin_inff();
    // 2 sqrt(2 / pi) (x + 0.044715 x^3)
    a.c1 = act == QA_ACT_GELU_TANH ? 1.59576912160573071f : 1.0f;
    a.c3 = act == QA_ACT_GELU_TANH ? 0.0713548162726002527f : 0.0f;
    a.vec = vec4(out, ldo, dtype);
    a.vecr = res && vec4(res, ldr, dtype);
    a.vecn = vec4(s_w, 0, 0) && vec4(bias, 0, 0);
    const int kind = act == QA_ACT_SILU || act == QA_ACT_GELU_TANH ? SIGMA : act == QA_ACT_GELU ? GELU : LINEAR;
    const int64_t groups = (N + 15) / 16;
    if (M <= 64 && groups <= 256) {                          // one round of blocks
        const dim3 g((unsigned)groups);
        if (M <= 16) hipLaunchKernelGGL(k_linear_stream<1>, g, dim3(512), 0, st, a, kind);
        else if (M <= 32) hipLaunchKernelGGL(k_linear_stream<2>, g, dim3(512), 0, st, a, kind);
        else hipLaunchKernelGGL(k_linear_stream<4>, g, dim3(512), 0, st, a, kind);
        return hipGetLastError();
    }
    if (M <= 16) {
        if (res16(a)) hipLaunchKernelGGL(k_linear_few<true>, dim3(256), dim3(512), 0, st, a, kind);
        else hipLaunchKernelGGL(k_linear_few<false>, dim3(256), dim3(512), 0, st, a, kind);
        return hipGetLastError();
    }
    return kind == SIGMA ? run_tiles<SIGMA>(a, st) : kind == GELU ? run_tiles<GELU>(a, st) : run_tiles<LINEAR>(a, st);
}

}  // namespace qa
