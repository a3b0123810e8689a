// k_lora.hip -- a shared int8 projection with the low-rank adapters of many
// requests at once, on gfx950.
//
//   out[m][n] = s_x[m] s_w[n] sum_k Xq[m][k] Wq[n][k]
//             + alpha_a sum_r (sum_k X[m][k] A_a[r][k]) B_a[n][r],
//   a = adapter of the request that token m belongs to (none: first line alone)
//
// Requests are consecutive token ranges; a request without tokens costs a
// comparison.  Two launches: the tokens' r inner products with their adapter
// (k_lora_down_*), and the int8 product whose epilogue adds the second product
// to the dequantized tile in fp32, so the output is rounded once and written
// once.
//
// The inner products h stay in fp32.  Where the second product runs on MFMA they
// enter it as two 16-bit numbers hi + lo = h 2^-e (e from the row's largest |h| of
// 32 ranks), so that the type's range does not limit them.  That keeps h to 2^-23
// of the row's largest in fp16 and to 2^-17 in bf16: next to an output rounded to
// 16 bits (2^-12 or 2^-9) little, but not next to one in fp32, for which bf16 takes
// a third number (all of fp32's digits).  A row with an infinity or NaN among its h
// ends as NaN.
#include "qa_tile.hpp"
#include "qa_launch.hpp"

namespace qa {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

struct LoraArgs {
    const int8_t* Xq;
    const float* s_x;
    const uint16_t* X;
    int64_t M, K, N;
    const int8_t* Wq;
    const float* s_w;
    const uint16_t* A;         // [L][r][K]
    const uint16_t* B;         // [L][N][r]
    const float* alpha;        // [L]
    const int32_t* seg;        // [R + 1] first token of each request
    const int32_t* which;      // [R] adapter or -1
    int32_t r, L, R;
    int32_t* ad;               // [M] adapter of a token or -1, written by the first launch
    float* h;                  // [M][r] (few tokens)
    float* hp;                 // [splits][groups of 32 ranks][M][32] parts of h (many tokens)
    int32_t splits;
    void* out;
    int32_t dt;                // of out
    bool vec;                  // out rows allow 4-element vector stores
};

__device__ __forceinline__ float wide(uint16_t b, bool bf) {
    return bf ? __builtin_bit_cast(float, (uint32_t)b << 16) : h2f(b);
}

// Adapter of request s, or -1.
__device__ __forceinline__ int adapter(const LoraArgs& a, int s) {
    const int w = a.which[s];
    return w >= 0 && w < a.L ? w : -1;
}

// Adapter of token m (wave-uniform m): its request is the last one that starts
// at or before it (starts do not decrease, so an empty request is followed by
// another with the same start).  Up to 256 starts are counted with four loads in
// flight at once; more are searched, a load after the other.
__device__ __forceinline__ int request_of(const LoraArgs& a, int64_t m) {
    const int lane = threadIdx.x & 63;
    if (a.R < 256) {
        int v[4], n = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = q * 64 <= a.R ? a.seg[min(q * 64 + lane, a.R)] : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) n += __popcll(__ballot(q * 64 + lane <= a.R && v[q] <= m));
        return n - 1;
    }
    int lo = 0, hi = a.R + 1;                                // seg[lo - 1] <= m < seg[hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.seg[mid] <= m) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

__device__ __forceinline__ int adapter_of(const LoraArgs& a, int64_t m) {
    if (a.R == 0) return -1;
    const int s = __builtin_amdgcn_readfirstlane(request_of(a, m));
    return s < 0 || s >= a.R ? -1 : adapter(a, s);
}

// Tokens [b, e) and request (-1: none) of block x of the requests' tiles of 16
// tokens, requests in order: every wave counts the tiles of 256 requests at a
// time, four to a lane, and sums them over the lanes.  Whatever the starts hold,
// 0 <= b < e <= M; starts that fall may put a token into two tiles or, past the
// launch's blocks, into none.
__device__ __forceinline__ int tile_of(const LoraArgs& a, int x, int64_t& b, int64_t& e) {
    const int lane = threadIdx.x & 63;
    for (int s0 = 0; s0 < a.R; s0 += 256) {
        int64_t c[5];
#pragma unroll
        for (int q = 0; q < 5; ++q) c[q] = a.seg[min(s0 + lane * 4 + q, a.R)];
        int n[4], sum = 0;
#pragma unroll
        for (int q = 0; q < 5; ++q) c[q] = c[q] < 0 ? 0 : (c[q] > a.M ? a.M : c[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            n[q] = c[q + 1] > c[q] ? (int)((c[q + 1] - c[q] + 15) >> 4) : 0;
            sum += n[q];
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(upto, o, QA_WAVE);
            if (lane >= o) upto += u;
        }
        const uint64_t in = __ballot(x < upto);
        if (in) {
            const int l = (int)__builtin_ctzll(in);          // the lane that holds the request
            int at = upto - sum, s = -1;
            int64_t mb = 0, me = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (s < 0 && x < at + n[q]) {
                    s = s0 + lane * 4 + q;
                    mb = c[q] + (int64_t)(x - at) * 16;
                    me = c[q + 1];
                }
                at += n[q];
            }
            b = __builtin_amdgcn_readlane((int)mb, l);
            e = __builtin_amdgcn_readlane((int)me, l);
            e = e < b + 16 ? e : b + 16;
            return __builtin_amdgcn_readlane(s, l);
        }
        x -= __builtin_amdgcn_readlane(upto, 63);
    }
    return -1;
}

template <bool BF>
__device__ __forceinline__ v4f mfma16(u32x4 x, u32x4 y, v4f c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x), __builtin_bit_cast(v8h, y), c, 0, 0, 0);
}

}  // namespace

// ---------------------------------------------------------------------------
// Few tokens: a block per token and 16 ranks, a wave on each.  The token's row
// is requested before its adapter is looked up (without requests nothing is: X may
// be NULL then).  Bound by latency: 5.0 us at 16 tokens, K = 4096, rank 16.
// ---------------------------------------------------------------------------
template <bool BF>
__global__ __launch_bounds__(1024) void k_lora_down_token(LoraArgs a) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t m = blockIdx.x;
    const rsrc_t rx = make_rsrc(a.X + m * a.K, a.R == 0 ? 0 : a.K * 2);
    const uint32_t KB = (uint32_t)a.K * 2;
    constexpr int U = 8;
    u32x4 x[U], w[U];
#pragma unroll
    for (int q = 0; q < U; ++q) x[q] = bload16(rx, lane * 16 + q * 1024);
    const int ad = adapter_of(a, m);
    if (threadIdx.x == 0 && blockIdx.y == 0) a.ad[m] = ad;
    const int j = blockIdx.y * 16 + wave;
    if (ad < 0 || j >= a.r) return;                          // (without an adapter its h is not read)
    const rsrc_t ra = make_rsrc(a.A + ((int64_t)ad * a.r + j) * a.K, KB);
    float s = 0.0f;
    for (uint32_t k = lane * 16; k - lane * 16 < KB; k += U * 1024) {
#pragma unroll
        for (int q = 0; q < U; ++q) w[q] = bload16(ra, k + q * 1024);
        if (KB > U * 1024) {
#pragma unroll
            for (int q = 0; q < U; ++q) x[q] = bload16(rx, k + q * 1024);
        }
        __builtin_amdgcn_sched_barrier(0);                   // every load in flight before the first use
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
            for (int p = 0; p < 8; ++p)
                s = __builtin_fmaf(wide((uint16_t)(x[q][p >> 1] >> (16 * (p & 1))), BF),
                                   wide((uint16_t)(w[q][p >> 1] >> (16 * (p & 1))), BF), s);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, QA_WAVE);
    if (lane == 0) a.h[m * a.r + j] = s * a.alpha[ad];
}

// The int8 product for few tokens: 16 output columns per block, K split over 8
// waves that bring the weight rows straight into MFMA operands.  The waves also
// share the adapters' part: wave w has the 16 x 16 outputs of tokens 16 (w % MT) ..
// and every (8 / MT)-th chunk of 16 ranks from w / MT.  Its tokens' adapters are
// requested before the weights and its first chunk of B behind them, so that
// neither waits for the other (with the adapter looked up here and B read after
// the weights, 9.3 us instead of 7.4 at 16 x 4096 x 4096, rank 16, where 19 MB of
// weights and adapters make 2.6 TB/s: a launch of one round, bound by latency).
template <int MT, bool BF>
__global__ __launch_bounds__(512) void k_lora_stream(LoraArgs a) {
    __shared__ v4i part[8][MT][64];
    __shared__ v4f dpart[8][64];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const uint32_t K = (uint32_t)a.K;
    const int r16 = lane & 15, c16 = (lane >> 4) * 16;
    const int j0 = wave / MT * 16;                           // the wave's first rank
    const int64_t mo = (wave % MT) * 16 + r16, no = n0 + 4 * (lane >> 4);    // the lane's outputs
    const bool live = mo < a.M && no < a.N;
    const int cols = live ? (int)(a.N - no < 4 ? a.N - no : 4) : 0;
    const int ad = live && j0 < a.r ? a.ad[mo] : -1;
    const bool first = wave < MT && live;                    // this wave also ends its tile
    float sx = 0.0f, sw[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (first) {
        sx = a.s_x[mo];
#pragma unroll
        for (int q = 0; q < 4; ++q) sw[q] = a.s_w[no + min(q, cols - 1)];
    }
    const rsrc_t rh = make_rsrc(a.h, a.M * a.r * 4);         // (rows of tokens without an adapter hold anything)
    auto load_h = [&](int j, v4f* h) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            h[q] = __builtin_bit_cast(v4f, bload16(rh, live && j + q * 4 < a.r ? (uint32_t)(mo * a.r + j + q * 4) * 4 : kOOB));
    };
    v4f h[4];
    load_h(j0, h);
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
    const bool adapt = ad >= 0;
    const uint16_t* bp = a.B + ((int64_t)(adapt ? ad : 0) * a.N + (adapt ? no : 0)) * a.r;
    auto load_b = [&](int j, u32x4 (*b)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                b[q][p] = u32x4{0, 0, 0, 0};
                if (adapt && q < cols && j + p * 8 < a.r)
                    b[q][p] = *reinterpret_cast<const u32x4*>(bp + (int64_t)q * a.r + j + p * 8);
            }
    };
    u32x4 b[4][2];
    load_b(j0, b);
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
    v4f d = v4f{0, 0, 0, 0};
    for (int j = j0; j < a.r; j += 128 / MT) {
        if (j != j0) {
            load_h(j, h);
            load_b(j, b);
        }
        if (adapt)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    if (j + p * 8 < a.r)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            d[q] = __builtin_fmaf(h[2 * p + (e >> 2)][e & 3],
                                                  wide((uint16_t)(b[q][p][e >> 1] >> (16 * (e & 1))), BF), d[q]);
    }
    dpart[wave][lane] = d;
    __syncthreads();
    if (!first) return;
    v4i c = part[0][wave][lane];
#pragma unroll
    for (int p = 1; p < 8; ++p) c += part[p][wave][lane];
#pragma unroll
    for (int p = 1; p < 8 / MT; ++p) d += dpart[p * MT + wave][lane];
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = (float)c[q] * sx * sw[q] + d[q];
    store4(a.out, mo * a.N + no, a.dt, v, cols, a.vec);
}

// ---------------------------------------------------------------------------
// Many tokens: up to 16 tokens of one request x 32 ranks per block on MFMA, K
// split over the blocks z and their 4 waves so that up to 8192 columns are one
// batch of loads.  (Tiles of 16 tokens across requests, their adapters one after
// the other, took 18.7 us for 777 tokens of 48 requests at K = 4096, rank 64.)
// The splits are summed, in order, where h is read.
// 12.6 us at 777 tokens of 48 requests, 32 adapters of rank 64, K = 4096 (23 MB
// that memory has to bring: 1.9 TB/s of the whole, 3 of what is left after a
// launch's own 5 us), 11 at 2048 tokens of 8 requests, rank 16.  Twice the tokens
// or the ranks per block, half the loads ahead at more waves and contiguous tiles
// per XCD all measure 12.3 to 13.4: neither the L1, the L2 nor the waves bound it.
// ---------------------------------------------------------------------------
template <bool BF>
__global__ __launch_bounds__(256) void k_lora_down_tile(LoraArgs a) {
    __shared__ v4f part[4][2][64];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int g = blockIdx.y, z = blockIdx.z;                // group of 32 ranks, part of K
    const int r16 = lane & 15;
    if (g == 0 && z == 0 && threadIdx.x < 16) {              // tokens before the first and after the last request
        const int64_t m = (int64_t)blockIdx.x * 16 + threadIdx.x;
        if (m < a.M && (a.R == 0 || m < a.seg[0] || m >= a.seg[a.R])) a.ad[m] = -1;
    }
    int64_t m0 = 0, m1 = 0;
    const int s = tile_of(a, blockIdx.x, m0, m1);
    if (s < 0) return;
    const int ad = __builtin_amdgcn_readfirstlane(adapter(a, s));
    if (g == 0 && z == 0 && threadIdx.x < m1 - m0) a.ad[m0 + threadIdx.x] = ad;
    if (ad < 0) return;
    const uint32_t c16 = (lane >> 4) * 16;
    const uint32_t KB = (uint32_t)a.K * 2;
    const rsrc_t rx = make_rsrc(a.X + m0 * a.K, (m1 - m0) * KB);
    const rsrc_t ra = make_rsrc(a.A + (int64_t)ad * a.r * a.K, (int64_t)a.r * KB);
    const uint32_t ox = m0 + r16 < m1 ? (uint32_t)r16 * KB : kOOB;
    const int j0 = g * 32 + r16, j1 = j0 + 16;
    const uint32_t o0 = j0 < a.r ? (uint32_t)j0 * KB : kOOB, o1 = j1 < a.r ? (uint32_t)j1 * KB : kOOB;
    const bool wide32 = g * 32 + 16 < a.r;                   // the group's second 16 ranks exist
    const float al = a.alpha[ad];
    constexpr int U = 8;
    const int steps = (int)((KB + 63) / 64), stride = 4 * a.splits, first = z * 4 + wave;
    v4f acc[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
    for (int st = first; st < steps; st += stride * U) {
        u32x4 x[U], p0[U], p1[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const uint32_t kb = (uint32_t)(st + stride * q) * 64 + c16;
            x[q] = bload16(rx, kb < KB ? ox + kb : kOOB);
            p0[q] = bload16(ra, kb < KB ? o0 + kb : kOOB);
        }
        if (wide32) {
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const uint32_t kb = (uint32_t)(st + stride * q) * 64 + c16;
                p1[q] = bload16(ra, kb < KB ? o1 + kb : kOOB);
            }
        }
        __builtin_amdgcn_sched_barrier(0);                   // every load in flight before the first use
#pragma unroll
        for (int q = 0; q < U; ++q) acc[0] = mfma16<BF>(p0[q], x[q], acc[0]);
        if (wide32) {
#pragma unroll
            for (int q = 0; q < U; ++q) acc[1] = mfma16<BF>(p1[q], x[q], acc[1]);
        }
    }
    part[wave][0][lane] = acc[0];
    part[wave][1][lane] = acc[1];
    __syncthreads();
    if (threadIdx.x < 128) {
        const int f = threadIdx.x >> 6, ln = threadIdx.x & 63;
        const int64_t m = m0 + (ln & 15);
        v4f c = part[0][f][ln];
#pragma unroll
        for (int w = 1; w < 4; ++w) c += part[w][f][ln];
        if (m < m1)
            *reinterpret_cast<v4f*>(a.hp + (((int64_t)z * gridDim.y + g) * a.M + m) * 32 + f * 16 + 4 * (ln >> 4)) = c * al;
    }
}

// Many tokens: the int8 product on LDS tiles; the adapters' part joins the fp32
// tile before the one rounding.  2048 x 11008 x 4096, rank 16 (8 requests): 112 to 136
// us with the clock, 125 on average, of which the product alone is 100 at best (1.85
// POPS) and the adapters' part the epilogue's latency; bound as the tile product is.
// 777 x 4096 x 4096, rank 64 (48 requests): 33.4 us, 5 of them the adapters' (28.5
// without any, 29.8 with one for all).  416 tiles, so 160 of the 256 CUs hold two:
// a block alone on its CU takes 0.36 us for each of the 32 stages and 7 besides, and
// two do not overlap wholly; waves spend 51% of their time waiting for data.
//
// THIRD: bf16 with fp32 outputs, h in three numbers: 124 us instead of 122 at 2048 x
// 11008 x 4096, rank 16, and 142 instead of 138 at rank 64 (the largest tile spills
// six registers then; tiles of 128 x 128 instead take 133 and 148).
template <class C, bool BF, bool THIRD>
__global__ __launch_bounds__(C::THREADS, 4) void k_lora_tile(LoraArgs a, int32_t tiles_m, int32_t tiles_n) {
    extern __shared__ uint8_t smem[];
    int tm, tn;
    tile::of_block(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * C::BN;
    const rsrc_t ra = make_rsrc(a.Xq + m0 * a.K, (a.M - m0) * a.K);
    const rsrc_t rw = make_rsrc(a.Wq + n0 * a.K, (a.N - n0) * a.K);
    const uint32_t K = (uint32_t)a.K;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r16 = lane & 15, q16 = lane >> 4;
    int ad[C::FM];
    float sx[C::FM];
    auto rows = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int64_t m = m0 + (wave / C::WN) * C::TM + i * 16 + r16;
            ad[i] = m < a.M ? a.ad[m] : -1;
            if (ad[i] >= a.L) ad[i] = -1;                    // starts that fall may leave what the workspace held
            sx[i] = m < a.M ? a.s_x[m] : 0.0f;
        }
    };
    // Where registers allow, the rows' adapters and scales are requested before the
    // product and the next adapter's rows of B during a multiplication; the largest
    // tile takes both as it comes to them, without spills (4096 x 11008 x 4096, rank
    // 16: 224 us against 235, of the call).
    constexpr bool EARLY = C::FM * C::FN <= 8;
    if (EARLY) rows();
    v4i acc[C::FM][C::FN];
    tile::product<C>(
        ra, rw, K, smem, [&](int r) -> uint32_t { return m0 + r < a.M ? (uint32_t)r * K : kOOB; },
        [&](int r) -> uint32_t { return n0 + r < a.N ? (uint32_t)r * K : kOOB; }, acc);
    const int64_t mw = m0 + (wave / C::WN) * C::TM, nw = n0 + (wave % C::WN) * C::TN;   // the wave's tile
    if (!EARLY) rows();
    // The adapters' part, 32 ranks at a time: the tile's rows of h (hi and lo) into
    // the freed LDS, 16-byte chunk c of row r at c ^ (r & 7), with their scales (and the
    // third number's rows of 64 bytes behind them); then the distinct adapters of
    // the wave's rows in turn (EARLY: the next one's rows of B in flight while one is
    // multiplied).  A row takes the product of its own adapter alone.
    constexpr int HC = C::BM * 8 / C::THREADS;               // quads of ranks of h per thread
    static_assert(HC * C::THREADS == C::BM * 8 && C::BM * (THIRD ? 196 : 132) <= C::LDS, "h of the tile");
    const int groups = (a.r + 31) / 32;
    const rsrc_t none = make_rsrc(a.B, 0);
    v4f hc[HC];
    u32x4 b0[C::FN], b1[EARLY ? C::FN : 1];
    bool left[C::FM];
    auto next = [&]() __attribute__((always_inline)) {       // an adapter that has not had its turn, or -1
        int w = -1;
#pragma unroll
        for (int i = C::FM - 1; i >= 0; --i) {
            const uint64_t b = __ballot(left[i]);
            if (b) w = __builtin_amdgcn_readlane(ad[i], (int)__builtin_ctzll(b));
        }
        return w;
    };
    auto load_b = [&](int w, int g, u32x4* b) __attribute__((always_inline)) {
        const rsrc_t rb = w >= 0 ? make_rsrc(a.B + ((int64_t)w * a.N + nw) * a.r, (a.N - nw) * a.r * 2) : none;
        const int k8 = g * 32 + q16 * 8;                     // the lane's ranks
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            b[j] = bload16(rb, k8 < a.r ? (uint32_t)((j * 16 + r16) * a.r + k8) * 2 : kOOB);
    };
    int cur = -1;
    auto request = [&](int g) __attribute__((always_inline)) {               // what group g needs first
#pragma unroll
        for (int q = 0; q < HC; ++q) hc[q] = v4f{0, 0, 0, 0};
        for (int z = 0; z < a.splits; ++z) {                 // (rows without an adapter hold anything)
            const rsrc_t rh = make_rsrc(a.hp + (((int64_t)z * groups + g) * a.M + m0) * 32, (a.M - m0) * 128);
#pragma unroll
            for (int q = 0; q < HC; ++q)
                hc[q] += __builtin_bit_cast(v4f, bload16(rh, (uint32_t)(q * C::THREADS + threadIdx.x) * 16));
        }
#pragma unroll
        for (int i = 0; i < C::FM; ++i) left[i] = ad[i] >= 0;
        cur = next();
        load_b(cur, g, b0);
    };
    request(0);
    v4f o[C::FM][C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        float sw[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t n = nw + j * 16 + 4 * q16 + q;
            sw[q] = n < a.N ? a.s_w[n] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) o[i][j][q] = (float)acc[i][j][q] * sx[i] * sw[q];
    }
    float* ups = reinterpret_cast<float*>(smem + C::BM * 128);               // 2^e of a row
    auto third_at = [&](int r, int c) -> uint8_t* {          // 16-byte chunk c of row r of the third number
        return smem + C::BM * 132 + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    };
    for (int g = 0; g < groups; ++g) {
        if (g > 0) {
            request(g);
            __syncthreads();                                 // the last group's h has been read
        }
#pragma unroll
        for (int q = 0; q < HC; ++q) {
            // thread: 4 ranks of row r; the row's largest |h| over its 8 threads, 2^e
            // from its exponent bits with hi in [2^7, 2^8), kept within normal
            // numbers (an infinite or NaN row keeps its scale)
            const int P = q * C::THREADS + threadIdx.x, r = P >> 3, c = P & 7;
            float mx = fmaxf(fmaxf(__builtin_fabsf(hc[q][0]), __builtin_fabsf(hc[q][1])),
                             fmaxf(__builtin_fabsf(hc[q][2]), __builtin_fabsf(hc[q][3])));
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, QA_WAVE));
            const uint32_t ex = (__builtin_bit_cast(uint32_t, mx) >> 23) & 0xff;
            const int sh = ex == 0xff || mx == 0.0f ? 0 : clampi((int)ex - 127 - 7, -120, 120);
            const float down = __builtin_bit_cast(float, (uint32_t)(127 - sh) << 23);
            uint16_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float t = hc[q][e] * down;
                hi[e] = BF ? f2bf(t) : f2h(t);
                lo[e] = BF ? f2bf(t - wide(hi[e], true)) : f2h(t - h2f(hi[e]));
            }
            if constexpr (THIRD) {
                uint16_t z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = f2bf(hc[q][e] * down - wide(hi[e], true) - wide(lo[e], true));
                *reinterpret_cast<u32x2*>(third_at(r, c >> 1) + (c & 1) * 8) =
                    u32x2{z[0] | ((uint32_t)z[1] << 16), z[2] | ((uint32_t)z[3] << 16)};
            }
            uint8_t* row = smem + r * 128 + (c & 1) * 8;
            *reinterpret_cast<u32x2*>(row + (((c >> 1) ^ (r & 7)) << 4)) =
                u32x2{hi[0] | ((uint32_t)hi[1] << 16), hi[2] | ((uint32_t)hi[3] << 16)};
            *reinterpret_cast<u32x2*>(row + ((((c >> 1) + 4) ^ (r & 7)) << 4)) =
                u32x2{lo[0] | ((uint32_t)lo[1] << 16), lo[2] | ((uint32_t)lo[3] << 16)};
            if (c == 0) ups[r] = __builtin_bit_cast(float, (uint32_t)(127 + sh) << 23);
        }
        __syncthreads();
        while (cur >= 0) {
            bool mine[C::FM];
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                mine[i] = ad[i] == cur;
                left[i] = left[i] && !mine[i];
            }
            const int nxt = next();
            if constexpr (EARLY) load_b(nxt, g, b1);
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                if (!__any(mine[i])) continue;
                const int r = (wave / C::WN) * C::TM + i * 16 + r16;
                const float up = ups[r];
                const u32x4 hi = *reinterpret_cast<const u32x4*>(smem + r * 128 + ((q16 ^ (r & 7)) << 4));
                const u32x4 lo = *reinterpret_cast<const u32x4*>(smem + r * 128 + (((q16 + 4) ^ (r & 7)) << 4));
                u32x4 z = u32x4{0, 0, 0, 0};
                if constexpr (THIRD) z = *reinterpret_cast<const u32x4*>(third_at(r, q16));
#pragma unroll
                for (int j = 0; j < C::FN; ++j) {
                    v4f d = v4f{0, 0, 0, 0};
                    if constexpr (THIRD) d = mfma16<BF>(b0[j], z, d);
                    d = mfma16<BF>(b0[j], lo, d);
                    d = mfma16<BF>(b0[j], hi, d);
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[i][j][q] = mine[i] ? __builtin_fmaf(d[q], up, o[i][j][q]) : o[i][j][q];
                }
            }
            if constexpr (EARLY) {
#pragma unroll
                for (int j = 0; j < C::FN; ++j) b0[j] = b1[j];
            } else {
                load_b(nxt, g, b0);
            }
            cur = nxt;
        }
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
        const int64_t m = mw + i * 16 + r16;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const int64_t n = nw + j * 16 + 4 * q16;
            if (n >= a.N) continue;
            const float v[4] = {o[i][j][0], o[i][j][1], o[i][j][2], o[i][j][3]};
            store4(a.out, m * a.N + n, a.dt, v, (int)(a.N - n < 4 ? a.N - n : 4), a.vec);
        }
    }
}

namespace {
// The form for few tokens, while its blocks of 16 columns fit the CUs at once, by
// both sides' times at K = 4096, rank 16 (us of the call, stream and tiles of 64 x 64):
//   tokens \ columns    4096          8192          11008         16384
//   16                               17.4  21.2    21.6  21.2    26.5  21.6
//   32                15.1  21.6    20.4  21.9    26.8  21.6    33.5  22.3
//   64                17.4  21.9    27.2  22.2    37.3  22.1
// (48 tokens at 5120 columns: 24.0 and 21.4.)
bool few_tokens(int64_t M, int64_t N) {
    const int64_t blocks = (N + 15) / 16;
    return M <= 16 ? blocks <= 768 : M <= 32 ? blocks <= 512 : M <= 64 && blocks <= 256;
}
constexpr size_t up256(size_t v) { return (v + 255) / 256 * 256; }
}  // namespace

// Parts of K in k_lora_down_tile: 1024 columns to a block, so that its 4 waves
// have all their loads in flight at once; at most 8, since every column tile of
// the second launch sums them.
static int lora_splits(int64_t K) { return (int)(K >= 8192 ? 8 : (K + 1023) / 1024); }

size_t lora_scratch_bytes(int64_t M, int64_t K, int64_t r) {
    const size_t ad = up256((size_t)M * 4);
    // (the form for few tokens needs less: M r floats)
    return ad + up256((size_t)lora_splits(K) * ((size_t)(r + 31) / 32) * (size_t)M * 128);
}

template <class C, bool BF, bool THIRD>
static hipError_t run_lora_tile(const LoraArgs& a, hipStream_t st) {
    const int tm = (int)((a.M + C::BM - 1) / C::BM), tn = (int)((a.N + C::BN - 1) / C::BN);
    hipLaunchKernelGGL((k_lora_tile<C, BF, THIRD>), dim3((unsigned)(tm * tn)), dim3(C::THREADS), C::LDS, st, a, tm, tn);
    return hipGetLastError();
}

template <bool BF, bool THIRD>
static hipError_t run_lora(const LoraArgs& a, hipStream_t st) {
    hipError_t e;
    if (few_tokens(a.M, a.N)) {
        hipLaunchKernelGGL(k_lora_down_token<BF>, dim3((unsigned)a.M, (unsigned)((a.r + 15) / 16)), dim3(1024), 0, st, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        const unsigned nb = (unsigned)((a.N + 15) / 16);
        if (a.M <= 16) hipLaunchKernelGGL((k_lora_stream<1, BF>), dim3(nb), dim3(512), 0, st, a);
        else if (a.M <= 32) hipLaunchKernelGGL((k_lora_stream<2, BF>), dim3(nb), dim3(512), 0, st, a);
        else hipLaunchKernelGGL((k_lora_stream<4, BF>), dim3(nb), dim3(512), 0, st, a);
        return hipGetLastError();
    }
    // upper bound of the requests' tiles: the whole ones and a ragged one each
    const int64_t most = (a.M + 15) / 16 + (a.R < a.M ? a.R : a.M);
    hipLaunchKernelGGL(k_lora_down_tile<BF>,
                       dim3((unsigned)most, (unsigned)((a.r + 31) / 32), (unsigned)a.splits), dim3(256), 0, st, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    // By size, at K = 4096, rank 16 (us of the call; T: tiles of 64 x 64, of 128 x 128):
    //   M x N           T            64 x 64   64 x 128   128 x 128   128 x 192
    //   128 x 4096      128, 32         21.5       24.4        33.8        36.6
    //   320 x 4096      320, 96         23.5       24.8
    //   512 x 4096      512, 128        26.7       27.6        36.4        42.1
    //   777 x 4096      832, 224        56         44          48          55 (rank 64)
    //   1024 x 4096    1024, 256        45.6       36.6        38.9        43.9
    //   1536 x 4096    1536, 384                   52.4        46.3        61.4
    //   2048 x 4096    2048, 512        75.5       63.7        53.3        62.7
    //   1024 x 11008   2752, 688        95.7       83.0        73.9        64.2
    //   2048 x 11008   5504, 1376        178        150         124         119
    // A tile alone on its CU takes as long as two (a stage's chain of barrier, LDS
    // reads and MFMAs), so small tiles as long as 512 of them fit two at a time.
    const int64_t small = ((a.M + 63) / 64) * ((a.N + 63) / 64), tiles = ((a.M + 127) / 128) * ((a.N + 127) / 128);
    if (small <= 512) return run_lora_tile<tile::Cfg<64, 64, 2, 4, 3>, BF, THIRD>(a, st);
    if (tiles <= 256) return run_lora_tile<tile::Cfg<64, 128, 2, 4, 3>, BF, THIRD>(a, st);
    if (tiles <= 512) return run_lora_tile<tile::Cfg<128, 128, 2, 4, 2>, BF, THIRD>(a, st);
    return run_lora_tile<tile::Cfg<128, 192, 2, 4, 2>, BF, THIRD>(a, st);
}

hipError_t launch_lora_i8(const int8_t* Xq, const float* s_x, const void* X, bool bf16, int64_t M, int64_t K,
                          const int8_t* Wq, const float* s_w, int64_t N, const void* A, const void* B,
                          const float* alpha, int r, int L, const int32_t* seg, const int32_t* which, int R, void* out,
                          int out_dtype, void* scratch, hipStream_t st) {
    LoraArgs a{};
    a.Xq = Xq; a.s_x = s_x; a.X = static_cast<const uint16_t*>(X);
    a.M = M; a.K = K; a.N = N; a.Wq = Wq; a.s_w = s_w;
    a.A = static_cast<const uint16_t*>(A); a.B = static_cast<const uint16_t*>(B); a.alpha = alpha;
    a.seg = seg; a.which = which; a.r = r; a.L = L; a.R = R;
    uint8_t* ws = static_cast<uint8_t*>(scratch);
    a.ad = reinterpret_cast<int32_t*>(ws);
    ws += up256((size_t)M * 4);
    a.h = a.hp = reinterpret_cast<float*>(ws);
    a.splits = lora_splits(K);
    a.out = out; a.dt = out_dtype;
    a.vec = N % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (out_dtype == 0 ? 15 : 7)) == 0;
    if (!bf16) return run_lora<false, false>(a, st);
    return out_dtype == 0 ? run_lora<true, true>(a, st) : run_lora<true, false>(a, st);
}

}  // namespace qa
