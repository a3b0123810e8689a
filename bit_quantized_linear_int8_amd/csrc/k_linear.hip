// k_linear.hip -- the int8 linear on codes with bias, activation and residual in
// its epilogue, on gfx950.
//
//   out[m][n] = act(s_x[m] s_w[n] sum_k Xq[m][k] Wq[n][k] + bias[n]) + res[m][n]
//
// The product is exact (int32); the rest is fp32 and rounded once.  Two forms, of
// the products that the adapters' linear has: weights streamed straight into MFMA
// operands for few tokens, the tile product of qa_tile.hpp for many.
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
    bool vec, vecr;            // rows of out, of res allow 4-element vectors
};

enum Act { LINEAR = 0, SIGMA = 1, GELU = 2 };

template <int ACT>
__device__ __forceinline__ float activate(const LinearArgs& a, float x) {
    if constexpr (ACT == SIGMA) return x * sigmoid(x * __builtin_fmaf(a.c3 * x, x, a.c1));
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
        return (x < 0.0f ? 0.0f : x) - z * (0.5f * t * p * e);
    }
    return x < a.least ? a.least : x;                        // (a NaN stays)
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

// Few tokens (16 MT): 16 output columns per block, K split over its 8 waves.
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

// Many tokens: one tile of the product per block.
template <class C, int ACT>
__global__ __launch_bounds__(C::THREADS, 4) void k_linear_tile(LinearArgs a, int32_t tiles_m, int32_t tiles_n) {
    extern __shared__ uint8_t smem[];
    int tm, tn;
    tile::of_block(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * C::BN;
    const rsrc_t ra = make_rsrc(a.Xq + m0 * a.K, (a.M - m0) * a.K);
    const rsrc_t rw = make_rsrc(a.Wq + n0 * a.K, (a.N - n0) * a.K);
    const uint32_t K = (uint32_t)a.K;
    const int lane = threadIdx.x & 63, wave = wave_id();
    v4i acc[C::FM][C::FN];
    tile::product<C>(
        ra, rw, K, smem, [&](int r) -> uint32_t { return m0 + r < a.M ? (uint32_t)r * K : kOOB; },
        [&](int r) -> uint32_t { return n0 + r < a.N ? (uint32_t)r * K : kOOB; }, acc);
    const int64_t mw = m0 + (wave / C::WN) * C::TM + (lane & 15), nw = n0 + (wave % C::WN) * C::TN + 4 * (lane >> 4);
    float sx[C::FM];
#pragma unroll
    for (int i = 0; i < C::FM; ++i) sx[i] = mw + i * 16 < a.M ? a.s_x[mw + i * 16] : 0.0f;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        const int64_t n = nw + j * 16;
        if (n >= a.N) continue;
        const int cols = (int)(a.N - n < 4 ? a.N - n : 4);
        float sw[4], bi[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            sw[q] = a.s_w[n + min(q, cols - 1)];
            if (a.bias) bi[q] = a.bias[n + min(q, cols - 1)];
        }
        v4f res[C::FM];
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            res[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            if (a.res && mw + i * 16 < a.M) res[i] = load4(a.res, (mw + i * 16) * a.ldr + n, a.dt, cols, a.vecr);
        }
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            if (mw + i * 16 >= a.M) continue;
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = activate<ACT>(a, (float)acc[i][j][q] * sx[i] * sw[q] + bi[q]) + res[i][q];
            store4(a.out, (mw + i * 16) * a.ldo + n, a.dt, v, cols, a.vec);
        }
    }
}

namespace {

// The streaming form while its blocks of 16 columns fit the CUs at once (the rule of
// the adapters' linear, whose products these are).
bool few_rows(int64_t M, int64_t N) {
    const int64_t blocks = (N + 15) / 16;
    return M <= 16 ? blocks <= 768 : M <= 32 ? blocks <= 512 : M <= 64 && blocks <= 256;
}

template <class C, int ACT>
hipError_t run_tile(const LinearArgs& a, hipStream_t st) {
    const int tm = (int)((a.M + C::BM - 1) / C::BM), tn = (int)((a.N + C::BN - 1) / C::BN);
    hipLaunchKernelGGL((k_linear_tile<C, ACT>), dim3((unsigned)(tm * tn)), dim3(C::THREADS), C::LDS, st, a, tm, tn);
    return hipGetLastError();
}

// Tiles by how many of them there are, as in the adapters' linear.
template <int ACT>
hipError_t run_tiles(const LinearArgs& a, hipStream_t st) {
    const int64_t small = ((a.M + 63) / 64) * ((a.N + 63) / 64), tiles = ((a.M + 127) / 128) * ((a.N + 127) / 128);
    if (small <= 512) return run_tile<tile::Cfg<64, 64, 2, 4, 3>, ACT>(a, st);
    if (tiles <= 256) return run_tile<tile::Cfg<64, 128, 2, 4, 3>, ACT>(a, st);
    if (tiles <= 512) return run_tile<tile::Cfg<128, 128, 2, 4, 2>, ACT>(a, st);
    return run_tile<tile::Cfg<128, 192, 2, 4, 2>, ACT>(a, st);
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
    const int kind = act == QA_ACT_SILU || act == QA_ACT_GELU_TANH ? SIGMA : act == QA_ACT_GELU ? GELU : LINEAR;
    if (few_rows(M, N)) {
        const unsigned nb = (unsigned)((N + 15) / 16);
        if (M <= 16) hipLaunchKernelGGL(k_linear_stream<1>, dim3(nb), dim3(512), 0, st, a, kind);
        else if (M <= 32) hipLaunchKernelGGL(k_linear_stream<2>, dim3(nb), dim3(512), 0, st, a, kind);
        else hipLaunchKernelGGL(k_linear_stream<4>, dim3(nb), dim3(512), 0, st, a, kind);
        return hipGetLastError();
    }
    return kind == SIGMA ? run_tiles<SIGMA>(a, st) : kind == GELU ? run_tiles<GELU>(a, st) : run_tiles<LINEAR>(a, st);
}

}  // namespace qa
