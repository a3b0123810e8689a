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
// The inner products h stay in fp32, or where the second product runs on MFMA
// as two 16-bit numbers hi + lo = h 2^-e (e from the row's largest |h| of 32
// ranks), so that neither the type's range nor its digits limit them.
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
    float* h;                  // [M][r] (few tokens)
    uint16_t* h16;             // [groups of 32 ranks][M][hi 32, lo 32]
    float* hs;                 // [groups][M] scale 2^e
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

// The last request that starts at or before token m (-1: none).  Starts do not
// decrease, so an empty request is followed by another with the same start.
__device__ __forceinline__ int request_of(const LoraArgs& a, int64_t m) {
    int lo = 0, hi = a.R;                                    // seg[lo - 1] <= m < seg[hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.seg[mid] <= m) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

__device__ __forceinline__ int adapter_of(const LoraArgs& a, int64_t m) {
    const int s = request_of(a, m);
    return s < 0 || m >= a.seg[s + 1] ? -1 : adapter(a, s);
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
// Few tokens: one block per token, its 16 waves on a rank each.
// ---------------------------------------------------------------------------
template <bool BF>
__global__ __launch_bounds__(1024) void k_lora_down_token(LoraArgs a) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t m = blockIdx.x;
    const int ad = adapter_of(a, m);
    if (ad < 0) return;                                      // its h is not read
    const rsrc_t rx = make_rsrc(a.X + m * a.K, a.K * 2);
    for (int j = wave; j < a.r; j += 16) {
        const rsrc_t ra = make_rsrc(a.A + ((int64_t)ad * a.r + j) * a.K, a.K * 2);
        float s = 0.0f;
        for (uint32_t k = lane * 16; k < (uint32_t)a.K * 2; k += 4096) {
            u32x4 x[4], w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                x[q] = bload16(rx, k + q * 1024);
                w[q] = bload16(ra, k + q * 1024);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    s = __builtin_fmaf(wide((uint16_t)(x[q][p >> 1] >> (16 * (p & 1))), BF),
                                       wide((uint16_t)(w[q][p >> 1] >> (16 * (p & 1))), BF), s);
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, QA_WAVE);
        if (lane == 0) a.h[m * a.r + j] = s * a.alpha[ad];
    }
}

// The int8 product for few tokens: 16 output columns per block, K split over
// its 8 waves, the weight rows straight into MFMA operands.
template <int MT, bool BF>
__global__ __launch_bounds__(512) void k_lora_stream(LoraArgs a) {
    __shared__ v4i part[8][MT][64];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16 * MT;
    const uint32_t K = (uint32_t)a.K;
    const int r16 = lane & 15, c16 = (lane >> 4) * 16;
    const rsrc_t rw = make_rsrc(a.Wq + n0 * a.K, (a.N - n0) * a.K);
    const rsrc_t rx = make_rsrc(a.Xq + m0 * a.K, (a.M - m0) * a.K);
    const uint32_t ow = n0 + r16 < a.N ? (uint32_t)r16 * K : kOOB;
    uint32_t ox[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) ox[m] = m0 + m * 16 + r16 < a.M ? (uint32_t)(m * 16 + r16) * K : kOOB;
    v4i acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4i{0, 0, 0, 0};
    const int nk = (int)((K + 63) / 64);
    constexpr int U = 8;
    for (int s = wave; s < nk; s += 8 * U) {
        u32x4 w[U], x[U][MT];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const uint32_t kb = (uint32_t)(s + 8 * q) * 64 + c16;
            const bool in = kb < K;
            w[q] = bload16(rw, in ? ow + kb : kOOB);
#pragma unroll
            for (int m = 0; m < MT; ++m) x[q][m] = bload16(rx, in ? ox[m] + kb : kOOB);
        }
        __builtin_amdgcn_sched_barrier(0);                   // every load in flight before the first use
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, w[q]),
                                                               __builtin_bit_cast(v4i, x[q][m]), acc[m], 0, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][m][lane] = acc[m];
    __syncthreads();
    for (int it = threadIdx.x; it < MT * 64; it += 512) {
        const int t = it >> 6, ln = it & 63;
        const int64_t m = m0 + t * 16 + (ln & 15), n = n0 + 4 * (ln >> 4);
        if (m >= a.M || n >= a.N) continue;
        v4i c = part[0][t][ln];
#pragma unroll
        for (int w = 1; w < 8; ++w) c += part[w][t][ln];
        const int cols = (int)(a.N - n < 4 ? a.N - n : 4);
        const int ad = adapter_of(a, m);
        const float sx = a.s_x[m];
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = q < cols ? (float)c[q] * sx * a.s_w[n + q] : 0.0f;
            if (ad >= 0 && q < cols) {
                const uint16_t* b = a.B + ((int64_t)ad * a.N + n + q) * a.r;
                float d = 0.0f;
                for (int j = 0; j < a.r; j += 8) {
                    const u32x4 bv = *reinterpret_cast<const u32x4*>(b + j);
#pragma unroll
                    for (int p = 0; p < 8; ++p)
                        d = __builtin_fmaf(a.h[m * a.r + j + p], wide((uint16_t)(bv[p >> 1] >> (16 * (p & 1))), BF), d);
                }
                v[q] += d;
            }
        }
        store4(a.out, m * a.N + n, a.dt, v, cols, a.vec);
    }
}

// ---------------------------------------------------------------------------
// Many tokens: 16 tokens x 32 ranks per block on MFMA, K split over 16 waves.
// Block z takes every gridDim.z-th request of the tile that has an adapter;
// rows without one are not written (and not read).
// ---------------------------------------------------------------------------
template <bool BF>
__global__ __launch_bounds__(1024) void k_lora_down_tile(LoraArgs a) {
    __shared__ v4f part[16][2][64];
    __shared__ float hrow[16][33];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t m0 = (int64_t)blockIdx.x * 16, m1 = m0 + 16 < a.M ? m0 + 16 : a.M;
    const int g = blockIdx.y;                                // group of 32 ranks
    const int r16 = lane & 15;
    const uint32_t c16 = (lane >> 4) * 16;
    const uint32_t KB = (uint32_t)a.K * 2;
    const rsrc_t rx = make_rsrc(a.X + m0 * a.K, (a.M - m0) * a.K * 2);
    const uint32_t ox = m0 + r16 < a.M ? (uint32_t)r16 * KB : kOOB;
    const int steps = (int)((KB + 63) / 64);
    const bool wide32 = g * 32 + 16 < a.r;                   // the group's second 16 ranks exist
    int s = request_of(a, m0), nth = 0;
    for (s = s < 0 ? 0 : s; s < a.R; ++s) {
        if (a.seg[s] >= m1) break;
        const int64_t b = a.seg[s] > m0 ? a.seg[s] : m0, e = a.seg[s + 1] < m1 ? a.seg[s + 1] : m1;
        const int ad = adapter(a, s);
        if (e <= b || ad < 0) continue;
        if (nth++ % (int)gridDim.z != (int)blockIdx.z) continue;
        const rsrc_t ra = make_rsrc(a.A + (int64_t)ad * a.r * a.K, (int64_t)a.r * KB);
        const int j0 = g * 32 + r16, j1 = j0 + 16;
        const uint32_t o0 = j0 < a.r ? (uint32_t)j0 * KB : kOOB, o1 = j1 < a.r ? (uint32_t)j1 * KB : kOOB;
        v4f acc[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
        constexpr int U = 8;
        for (int st = wave; st < steps; st += 16 * U) {
            u32x4 x[U], p0[U], p1[U];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const uint32_t kb = (uint32_t)(st + 16 * q) * 64 + c16;
                const bool in = kb < KB;
                x[q] = bload16(rx, in ? ox + kb : kOOB);
                p0[q] = bload16(ra, in ? o0 + kb : kOOB);
            }
            if (wide32) {
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const uint32_t kb = (uint32_t)(st + 16 * q) * 64 + c16;
                    p1[q] = bload16(ra, kb < KB ? o1 + kb : kOOB);
                }
            }
            __builtin_amdgcn_sched_barrier(0);               // every load in flight before the first use
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
            const int f = threadIdx.x >> 6, ln = threadIdx.x & 63, row = ln & 15;
            v4f c = part[0][f][ln];
#pragma unroll
            for (int w = 1; w < 16; ++w) c += part[w][f][ln];
            const float al = a.alpha[ad];
#pragma unroll
            for (int q = 0; q < 4; ++q) hrow[row][f * 16 + 4 * (ln >> 4) + q] = c[q] * al;
        }
        __syncthreads();
        // hi + lo = h 2^-e with the row's largest |h| in [2^7, 2^8)
        if (threadIdx.x < 512) {
            const int row = threadIdx.x >> 5, j = threadIdx.x & 31;
            const int64_t m = m0 + row;
            const float v = hrow[row][j];
            float mx = __builtin_fabsf(v);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 32));
            // 2^e from the exponent bits, kept within normal numbers; an
            // infinite or NaN row keeps its values
            const uint32_t ex = (__builtin_bit_cast(uint32_t, mx) >> 23) & 0xff;
            const int sh = ex == 0xff || mx == 0.0f ? 0 : clampi((int)ex - 127 - 7, -120, 120);
            const float up = __builtin_bit_cast(float, (uint32_t)(127 + sh) << 23);
            const float t = v * __builtin_bit_cast(float, (uint32_t)(127 - sh) << 23);
            if (m >= b && m < e) {
                const uint16_t hi = BF ? f2bf(t) : f2h(t);
                const uint16_t lo = BF ? f2bf(t - wide(hi, true)) : f2h(t - h2f(hi));
                uint16_t* o = a.h16 + ((int64_t)g * a.M + m) * 64 + j;
                o[0] = hi;
                o[32] = lo;
                if (j == 0) a.hs[(int64_t)g * a.M + m] = up;
            }
        }
        __syncthreads();
    }
}

template <class C, bool BF>
__global__ __launch_bounds__(C::THREADS, 4) void k_lora_tile(LoraArgs a, int32_t tiles_m, int32_t tiles_n) {
    extern __shared__ uint8_t smem[];
    int tm, tn;
    tile::of_block(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * C::BN;
    const rsrc_t ra = make_rsrc(a.Xq + m0 * a.K, (a.M - m0) * a.K);
    const rsrc_t rw = make_rsrc(a.Wq + n0 * a.K, (a.N - n0) * a.K);
    const uint32_t K = (uint32_t)a.K;
    v4i acc[C::FM][C::FN];
    tile::product<C>(
        ra, rw, K, smem, [&](int r) -> uint32_t { return m0 + r < a.M ? (uint32_t)r * K : kOOB; },
        [&](int r) -> uint32_t { return n0 + r < a.N ? (uint32_t)r * K : kOOB; }, acc);
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r16 = lane & 15, q16 = lane >> 4;
    const int64_t mw = m0 + (wave / C::WN) * C::TM, nw = n0 + (wave % C::WN) * C::TN;   // the wave's tile
    v4f o[C::FM][C::FN];
    {
        float sx[C::FM];
#pragma unroll
        for (int i = 0; i < C::FM; ++i) sx[i] = mw + i * 16 + r16 < a.M ? a.s_x[mw + i * 16 + r16] : 0.0f;
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
    }
    // the adapters of the requests in the wave's rows
    const int64_t me = mw + C::TM < a.M ? mw + C::TM : a.M;
    const int groups = (a.r + 31) / 32;
    if (mw < me) {
        int s = request_of(a, mw);
        for (s = s < 0 ? 0 : s; s < a.R; ++s) {
            const int64_t sb = a.seg[s], se = a.seg[s + 1];
            if (sb >= me) break;
            const int ad = __builtin_amdgcn_readfirstlane(adapter(a, s));
            if (se <= mw || se <= sb || ad < 0) continue;
            for (int g = 0; g < groups; ++g) {
                const rsrc_t rb = make_rsrc(a.B + ((int64_t)ad * a.N + nw) * a.r, (a.N - nw) * a.r * 2);
                u32x4 bf[C::FN];
                const int k8 = g * 32 + q16 * 8;             // the lane's ranks
#pragma unroll
                for (int j = 0; j < C::FN; ++j) {
                    const int64_t n = nw + j * 16 + r16;
                    bf[j] = bload16(rb, n < a.N && k8 < a.r ? (uint32_t)((j * 16 + r16) * a.r + k8) * 2 : kOOB);
                }
#pragma unroll
                for (int i = 0; i < C::FM; ++i) {
                    if (mw + i * 16 + 16 <= sb || mw + i * 16 >= se) continue;
                    const int64_t m = mw + i * 16 + r16;
                    const bool mine = m >= sb && m < se && m < a.M;
                    const uint16_t* hp = a.h16 + ((int64_t)g * a.M + (mine ? m : 0)) * 64 + q16 * 8;
                    u32x4 hi{0, 0, 0, 0}, lo{0, 0, 0, 0};
                    float up = 0.0f;
                    if (mine) {
                        hi = *reinterpret_cast<const u32x4*>(hp);
                        lo = *reinterpret_cast<const u32x4*>(hp + 32);
                        up = a.hs[(int64_t)g * a.M + m];
                    }
#pragma unroll
                    for (int j = 0; j < C::FN; ++j) {
                        v4f d = mfma16<BF>(bf[j], lo, v4f{0, 0, 0, 0});
                        d = mfma16<BF>(bf[j], hi, d);
                        // a row of another request has zeros here, unless its
                        // neighbour's adapter is infinite: it is left as it is
#pragma unroll
                        for (int q = 0; q < 4; ++q) o[i][j][q] = mine ? __builtin_fmaf(d[q], up, o[i][j][q]) : o[i][j][q];
                    }
                }
            }
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
constexpr int64_t FEW = 64;                                  // tokens of the one-block-per-token form
constexpr size_t up256(size_t v) { return (v + 255) / 256 * 256; }
}  // namespace

size_t lora_scratch_bytes(int64_t M, int64_t r) {
    if (M <= FEW) return up256((size_t)M * (size_t)r * 4);
    const size_t groups = (size_t)(r + 31) / 32;
    return up256(groups * (size_t)M * 128) + up256(groups * (size_t)M * 4);
}

template <class C, bool BF>
static hipError_t run_lora_tile(const LoraArgs& a, hipStream_t st) {
    static const hipError_t once = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_lora_tile<C, BF>),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (once != hipSuccess) return once;
    const int tm = (int)((a.M + C::BM - 1) / C::BM), tn = (int)((a.N + C::BN - 1) / C::BN);
    hipLaunchKernelGGL((k_lora_tile<C, BF>), dim3((unsigned)(tm * tn)), dim3(C::THREADS), C::LDS, st, a, tm, tn);
    return hipGetLastError();
}

template <bool BF>
static hipError_t run_lora(const LoraArgs& a, hipStream_t st) {
    hipError_t e;
    if (a.M <= FEW) {
        hipLaunchKernelGGL(k_lora_down_token<BF>, dim3((unsigned)a.M), dim3(1024), 0, st, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        const unsigned nb = (unsigned)((a.N + 15) / 16);
        if (a.M <= 16) hipLaunchKernelGGL((k_lora_stream<1, BF>), dim3(nb, 1), dim3(512), 0, st, a);
        else if (a.M <= 32) hipLaunchKernelGGL((k_lora_stream<2, BF>), dim3(nb, 1), dim3(512), 0, st, a);
        else hipLaunchKernelGGL((k_lora_stream<4, BF>), dim3(nb, 1), dim3(512), 0, st, a);
        return hipGetLastError();
    }
    const unsigned z = a.R > 4 ? 4 : (a.R > 0 ? a.R : 1);
    hipLaunchKernelGGL(k_lora_down_tile<BF>, dim3((unsigned)((a.M + 15) / 16), (unsigned)((a.r + 31) / 32), z),
                       dim3(1024), 0, st, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t big = ((a.M + 127) / 128) * ((a.N + 255) / 256);
    if (big >= 192) return run_lora_tile<tile::Cfg<128, 256, 2, 4, 3>, BF>(a, st);
    return run_lora_tile<tile::Cfg<64, 128, 2, 2, 3>, BF>(a, st);
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
    a.h = static_cast<float*>(scratch);
    a.h16 = static_cast<uint16_t*>(scratch);
    a.hs = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + up256((size_t)((r + 31) / 32) * (size_t)M * 128));
    a.out = out; a.dt = out_dtype;
    a.vec = N % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (out_dtype == 0 ? 15 : 7)) == 0;
    return bf16 ? run_lora<true>(a, st) : run_lora<false>(a, st);
}

}  // namespace qa
