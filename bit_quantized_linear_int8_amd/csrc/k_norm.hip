// k_norm.hip -- residual addition, root-mean-square norm and int8 codes in one
// pass on gfx950.
//
//   h = x + r          (fp32; rounded to the type only where it is stored)
//   y = h * g / sqrt(mean_j h_j^2 + eps)
//   s = max_j |y_j| / 127 (1 where that is 0),  q = rint(y / s)
//
// Two reductions hang on each other (the mean, then the maximum of what it
// scales), so the row has to be at hand twice.  It stays in registers: a row
// is split over WPR waves of one block, each lane holding NC chunks of eight
// values in fp32, and each reduction is DPP within a wave and one LDS exchange
// between the row's waves.  Memory is touched once: x, r and g in, the codes,
// the scale and (where wanted) the sum and the norm out.  Rows too long for
// that take k_rmsnorm_i8_long, which reads the row three times.
//
// Bound by memory from a few hundred rows on (residual added, fp16 or bf16, 7
// bytes a value): 16384 x 8192 in 157 us, 6.0 TB/s; 2048 x 4096 in 12.3 to 13.3,
// 4.4 to 4.8 (13.0 with y kept too, 5.8; in fp32 with y 26.7, 5.3); rows that are not
// multiples of eight values 16384 x 8191 in 194, 4.8; the long form, which reads x
// and r three times, 256 x 32768 in 20, 2.9.  One row of 4096 is a launch and two
// exchanges, 3.2 us.
#include "qa_device.hpp"
#include "qa_launch.hpp"

namespace qa {

namespace {

template <int DT> struct Elem { static constexpr int BYTES = DT == 0 ? 4 : 2; };

__device__ __forceinline__ float bf2f(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }

// One element of type DT at p[j].
template <int DT>
__device__ __forceinline__ float ld1(const void* p, int64_t j) {
    if constexpr (DT == 0) return static_cast<const float*>(p)[j];
    const uint16_t b = static_cast<const uint16_t*>(p)[j];
    return DT == 1 ? h2f(b) : bf2f(b);
}
template <int DT>
__device__ __forceinline__ void st1(void* p, int64_t j, float v) {
    if constexpr (DT == 0) static_cast<float*>(p)[j] = v;
    else static_cast<uint16_t*>(p)[j] = DT == 1 ? f2h(v) : f2bf(v);
}

// The raw bytes of eight elements.
template <int DT> struct Raw8 { u32x4 v[DT == 0 ? 2 : 1]; };

template <int DT>
__device__ __forceinline__ Raw8<DT> bld8(rsrc_t r, uint32_t j0, bool in) {
    Raw8<DT> o;
    o.v[0] = bload16(r, in ? j0 * Elem<DT>::BYTES : kOOB);
    if constexpr (DT == 0) o.v[1] = bload16(r, in ? j0 * 4 + 16 : kOOB);
    return o;
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& w, float* x) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (DT == 0) {
            const uint32_t u = w.v[j >> 2][j & 3];
            x[j] = __builtin_bit_cast(float, u);
        } else {
            const uint16_t u = (uint16_t)(w.v[0][j >> 1] >> (16 * (j & 1)));
            x[j] = DT == 1 ? h2f(u) : bf2f(u);
        }
    }
}
template <int DT>
__device__ __forceinline__ void st8(void* p, int64_t j0, const float* x) {
    if constexpr (DT == 0) {
        v4f* o = reinterpret_cast<v4f*>(static_cast<float*>(p) + j0);
        o[0] = v4f{x[0], x[1], x[2], x[3]};
        o[1] = v4f{x[4], x[5], x[6], x[7]};
    } else {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = DT == 1 ? f2h(x[2 * j]) : f2bf(x[2 * j]);
            const uint32_t hi = DT == 1 ? f2h(x[2 * j + 1]) : f2bf(x[2 * j + 1]);
            w[j] = lo | (hi << 16);
        }
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + j0) = w;
    }
}

// Rows that start anywhere: eight elements from `at`, at their own alignment
// (the hardware splits accesses that cross a line), moved back to the row's last
// eight where the row ends before them; shifted() then brings the wanted ones to
// the front and zeros behind them.  K >= 8.
template <int DT>
__device__ __forceinline__ Raw8<DT> ldu8(const uint8_t* row, int64_t at, int64_t K) {
    Raw8<DT> o;
    __builtin_memcpy(&o, row + (at < K - 8 ? at : K - 8) * Elem<DT>::BYTES, sizeof(o));
    return o;
}
__device__ __forceinline__ int past(int64_t at, int64_t K) {
    const int64_t s = at - (K - 8);
    return s < 0 ? 0 : (s > 8 ? 8 : (int)s);
}
__device__ __forceinline__ void shifted(float* x, int s) {
    if (!__any(s > 0)) return;
#pragma unroll
    for (int b = 4; b >= 1; b >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s & b ? (j + b < 8 ? x[j + b] : 0.0f) : x[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = s >= 8 ? 0.0f : x[j];
}
// Store of the elements of eight from `at` that the row has.
template <int DT>
__device__ __forceinline__ void stu8(uint8_t* row, int64_t at, int64_t K, const float* x) {
    if (at + 8 <= K) {
        if constexpr (DT == 0) {
            __builtin_memcpy(row + at * 4, x, 32);
        } else {
            uint16_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = DT == 1 ? f2h(x[j]) : f2bf(x[j]);
            __builtin_memcpy(row + at * 2, h, 16);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (at + j < K) st1<DT>(row, at + j, x[j]);
}
__device__ __forceinline__ void stu_codes(int8_t* row, int64_t at, int64_t K, u32x2 c) {
    if (at + 8 <= K) {
        __builtin_memcpy(row + at, &c, 8);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (at + j < K) row[at + j] = (int8_t)(c[j >> 2] >> (8 * (j & 3)));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, QA_WAVE);
    return v;
}

// Scale of a row from its absmax and mean square; false where the row holds no
// finite norm (an infinity or NaN in it, or a square sum past fp32): then the
// scale is NaN and the codes are 0.
__device__ __forceinline__ bool row_scale(float ms, float amax, float& s, float& r) {
    const bool fine = ms < __builtin_inff() && amax < __builtin_inff();
    s = amax / 127.0f;
    if (s == 0.0f) s = 1.0f;
    if (!fine) s = __builtin_nanf("");
    r = 1.0f / s;
    return fine;
}

// Eight codes; a scale so small that its reciprocal overflows or loses digits
// takes the division for every value.
__device__ __forceinline__ u32x2 codes8_any(const float* x, float s, float r, bool fine) {
    if (!fine) return u32x2{0u, 0u};
    if (s >= 0x1p-120f) return codes8_dyn(x, s, r);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j >> 2] |= ((uint32_t)(int)__builtin_rintf(x[j] / s) & 0xffu) << (8 * (j & 3));
    return u32x2{w[0], w[1]};
}

}  // namespace

struct NormArgs {
    const void* X;
    const void* R;       // residual or nullptr
    const void* g;
    void* sum;           // or nullptr
    void* y;             // or nullptr
    int8_t* q;
    float* s;
    int64_t rows, K, ldx, ldr, lds;
    float eps;
};

// EVEN: K % 8 == 0 and every row of every array starts at a 16-byte boundary:
// range-checked 16-byte loads.  Otherwise the same chunks of eight at any
// alignment (ldu8).  Lane l of the row owns the chunks l, l + LANES, ...
template <int DT, int WPR, int NC, bool EVEN>
__global__ __launch_bounds__(WPR < 4 ? 256 : 64 * WPR) void k_rmsnorm_i8(NormArgs a) {
    constexpr int WPB = WPR < 4 ? 4 : WPR;                   // waves per block
    __shared__ float part_sum[WPB], part_max[WPB];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t row = (int64_t)blockIdx.x * (WPB / WPR) + wave / WPR;
    const int part = wave % WPR;
    const bool live = row < a.rows;
    const int64_t rw = live ? row : 0;
    const uint8_t* xp = static_cast<const uint8_t*>(a.X) + rw * a.ldx * Elem<DT>::BYTES;
    const uint8_t* rp = static_cast<const uint8_t*>(a.R) + rw * a.ldr * Elem<DT>::BYTES;
    const int lp = part * 64 + lane;                         // lane of the row
    constexpr int LANES = 64 * WPR;
    auto el = [&](int i) -> int64_t { return ((int64_t)i * LANES + lp) * 8; };
    float h[NC][8], g[NC][8];
    if constexpr (EVEN) {
        const rsrc_t rx = make_rsrc(xp, live ? a.K * Elem<DT>::BYTES : 0);
        const rsrc_t rr = make_rsrc(rp, live && a.R ? a.K * Elem<DT>::BYTES : 0);
        const rsrc_t rg = make_rsrc(a.g, a.K * Elem<DT>::BYTES);
        Raw8<DT> vx[NC], vr[NC], vg[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            vx[i] = bld8<DT>(rx, (uint32_t)el(i), true);
            vr[i] = bld8<DT>(rr, (uint32_t)el(i), true);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) vg[i] = bld8<DT>(rg, (uint32_t)el(i), true);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float t[8];
            widen8<DT>(vx[i], h[i]);
            widen8<DT>(vr[i], t);                            // zeros without a residual
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += t[j];
            widen8<DT>(vg[i], g[i]);
        }
    } else {
        Raw8<DT> vx[NC], vr[NC], vg[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            vx[i] = ldu8<DT>(xp, el(i), a.K);
            if (a.R) vr[i] = ldu8<DT>(rp, el(i), a.K);
            vg[i] = ldu8<DT>(static_cast<const uint8_t*>(a.g), el(i), a.K);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int s = past(el(i), a.K);
            widen8<DT>(vx[i], h[i]);
            if (a.R) {
                float t[8];
                widen8<DT>(vr[i], t);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] += t[j];
            }
            shifted(h[i], s);
            widen8<DT>(vg[i], g[i]);
            shifted(g[i], s);
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(h[i][j], h[i][j], ss);
    ss = wave_sum(ss);
    if constexpr (WPR > 1) {
        if (lane == 0) part_sum[wave] = ss;
        lds_only_barrier();
        ss = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) ss += part_sum[wave - part + w];
    }
    const float ms = ss / (float)a.K;
    const float rstd = 1.0f / __builtin_sqrtf(ms + a.eps);
    if (live && a.sum) {
        uint8_t* o = static_cast<uint8_t*>(a.sum) + rw * a.lds * Elem<DT>::BYTES;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if constexpr (EVEN) {
                if (el(i) < a.K) st8<DT>(o, el(i), h[i]);
            } else {
                stu8<DT>(o, el(i), a.K, h[i]);
            }
        }
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[i][j] = h[i][j] * rstd * g[i][j];
            amax = fmaxf(amax, __builtin_fabsf(h[i][j]));
        }
    amax = wave_max(amax);
    if constexpr (WPR > 1) {
        if (lane == 0) part_max[wave] = amax;
        lds_only_barrier();
        amax = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) amax = fmaxf(amax, part_max[wave - part + w]);
    }
    if (!live) return;
    float s, r;
    const bool fine = row_scale(ms, amax, s, r);
    if (lp == 0) a.s[row] = s;
    int8_t* q = a.q + row * a.K;
    uint8_t* yo = static_cast<uint8_t*>(a.y) + row * a.K * Elem<DT>::BYTES;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if constexpr (EVEN) {
            if (el(i) < a.K) {
                st_codes8(q + el(i), codes8_any(h[i], s, r, fine));
                if (a.y) st8<DT>(yo, el(i), h[i]);
            }
        } else {
            stu_codes(q, el(i), a.K, codes8_any(h[i], s, r, fine));
            if (a.y) stu8<DT>(yo, el(i), a.K, h[i]);
        }
    }
}

// Rows past 16384 values (and under 8): one block of 16 waves per row, the row
// read once for each reduction and once for the codes.  The sum is stored in the
// last pass, by the thread that has just read the elements, so it may replace x
// or r; a row's last chunk is read element by element, not moved back, so that no
// other thread's elements are read then.
template <int DT>
__global__ __launch_bounds__(1024) void k_rmsnorm_i8_long(NormArgs a) {
    __shared__ float red[16];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int64_t row = blockIdx.x;
    const uint8_t* xp = static_cast<const uint8_t*>(a.X) + row * a.ldx * Elem<DT>::BYTES;
    const uint8_t* rp = static_cast<const uint8_t*>(a.R) + row * a.ldr * Elem<DT>::BYTES;
    auto load = [&](const void* p, int64_t at, float* x) {
        if (at + 8 <= a.K) {
            widen8<DT>(ldu8<DT>(static_cast<const uint8_t*>(p), at, a.K), x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = at + j < a.K ? ld1<DT>(p, at + j) : 0.0f;
        }
    };
    auto sum8 = [&](int64_t at, float* h) {
        load(xp, at, h);
        if (a.R) {
            float t[8];
            load(rp, at, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] += t[j];
        }
    };
    float ss = 0.0f;
    for (int64_t at = threadIdx.x * 8; at < a.K; at += 8192) {
        float h[8];
        sum8(at, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(h[j], h[j], ss);
    }
    ss = wave_sum(ss);
    if (lane == 0) red[wave] = ss;
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) ss += red[w];
    __syncthreads();
    const float ms = ss / (float)a.K;
    const float rstd = 1.0f / __builtin_sqrtf(ms + a.eps);
    float amax = 0.0f;
    for (int64_t at = threadIdx.x * 8; at < a.K; at += 8192) {
        float h[8], g[8];
        sum8(at, h);
        load(a.g, at, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, __builtin_fabsf(h[j] * rstd * g[j]));
    }
    amax = wave_max(amax);
    if (lane == 0) red[wave] = amax;
    __syncthreads();
    amax = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) amax = fmaxf(amax, red[w]);
    float s, r;
    const bool fine = row_scale(ms, amax, s, r);
    if (threadIdx.x == 0) a.s[row] = s;
    for (int64_t at = threadIdx.x * 8; at < a.K; at += 8192) {
        float h[8], g[8], y[8];
        sum8(at, h);
        load(a.g, at, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = h[j] * rstd * g[j];
        if (a.sum) stu8<DT>(static_cast<uint8_t*>(a.sum) + row * a.lds * Elem<DT>::BYTES, at, a.K, h);
        if (a.y) stu8<DT>(static_cast<uint8_t*>(a.y) + row * a.K * Elem<DT>::BYTES, at, a.K, y);
        stu_codes(a.q + row * a.K, at, a.K, codes8_any(y, s, r, fine));
    }
}

// Two chunks to a lane and as many waves as that takes (fp16 with a residual, us):
//   rows x K        4 chunks   2 chunks   1 chunk
//   64 x 4096           4.7        3.9        3.8
//   2048 x 2048         8.7        8.4        9.8
//   2048 x 4096        12.4       12.3       15.9
//   16384 x 4096       82.3       80.4       99.5
//   16384 x 8192        158        162        215
// One chunk has each wave wait twice for so little; with four the registers leave
// fewer rows in flight, which costs only where there are few.
template <int DT, bool EVEN>
static void norm_dispatch(const NormArgs& a, hipStream_t st) {
    const int64_t nch = (a.K + 7) / 8;
#define QA_NORM(WPR, NC)                                                                                         \
    hipLaunchKernelGGL((k_rmsnorm_i8<DT, WPR, NC, EVEN>),                                                          \
                       dim3((unsigned)((a.rows + (WPR < 4 ? 4 / WPR : 1) - 1) / (WPR < 4 ? 4 / WPR : 1))),        \
                       dim3(WPR < 4 ? 256 : 64 * WPR), 0, st, a)
    if (a.K < 8) hipLaunchKernelGGL((k_rmsnorm_i8_long<DT>), dim3((unsigned)a.rows), dim3(1024), 0, st, a);
    else if (nch <= 64) QA_NORM(1, 1);
    else if (nch <= 128) QA_NORM(1, 2);
    else if (nch <= 256) QA_NORM(2, 2);
    else if (nch <= 512) QA_NORM(4, 2);
    else if (nch <= 1024) QA_NORM(8, 2);
    else if (nch <= 2048) QA_NORM(16, 2);
    else hipLaunchKernelGGL((k_rmsnorm_i8_long<DT>), dim3((unsigned)a.rows), dim3(1024), 0, st, a);
#undef QA_NORM
}

hipError_t launch_rmsnorm_i8(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* g, int dtype,
                             int64_t rows, int64_t K, float eps, int8_t* q, float* s, void* sum, int64_t lds, void* y,
                             hipStream_t st) {
    const int64_t step = dtype == 0 ? 4 : 8;                 // elements in 16 bytes
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const bool even = K % 8 == 0 && al(X) && al(R) && al(g) && al(q) && al(sum) && al(y) && ldx % step == 0 &&
                      (!R || ldr % step == 0) && (!sum || lds % step == 0);
    // a launch counts its threads in 32 bits: 2^21 rows of 1024 threads at a time
    const int64_t el = dtype == 0 ? 4 : 2;
    auto at = [](const void* p, int64_t bytes) -> void* {
        return p ? const_cast<uint8_t*>(static_cast<const uint8_t*>(p)) + bytes : nullptr;
    };
    for (int64_t r = 0; r < rows; r += (int64_t)1 << 21) {
        const NormArgs a{at(X, r * ldx * el), at(R, r * ldr * el), g, at(sum, r * lds * el), at(y, r * K * el),
                         q + r * K, s + r, rows - r < ((int64_t)1 << 21) ? rows - r : (int64_t)1 << 21, K, ldx, ldr, lds, eps};
        if (dtype == 0) { if (even) norm_dispatch<0, true>(a, st); else norm_dispatch<0, false>(a, st); }
        else if (dtype == 1) { if (even) norm_dispatch<1, true>(a, st); else norm_dispatch<1, false>(a, st); }
        else { if (even) norm_dispatch<2, true>(a, st); else norm_dispatch<2, false>(a, st); }
    }
    return hipGetLastError();
}

}  // namespace qa
