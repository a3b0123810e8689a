// k_route.hip -- routing of tokens to experts on gfx950: scores, the choice of
// k experts per token, their weights, and the chosen (token, slot) pairs
// grouped by expert for the experts' products.
//
//   s_e  = softmax(x)_e or 1 / (1 + exp(-x_e));   c_e = s_e + b_e
//   with groups: only the top_groups groups with the largest value keep their
//   experts, a group's value being its largest c_e or the sum of its two
//   largest; then the k largest c_e, ties to the lower index
//   w_j  = s_{e_j} (/ sum_j s_{e_j}) * scale
//
// Softmax keeps the order of the logits, so without a bias (and with groups
// valued by their largest member) the choice is made on the logits themselves
// and the exponentials are taken for the k chosen and the row's sum alone.
//
// A logit of -inf or NaN masks its expert; where fewer than k are left, the
// last slots hold expert -1 with weight 0 and are in no group.
//
// LPT lanes work on one token (16 for up to 256 experts, so that a wave takes
// four tokens and every reduction is four DPP steps in a row of 16 lanes; 64
// above that), lane l holding the EPL experts l EPL .. in registers.
//
// The grouping is stable (ascending pair index within an expert) and uses no
// order-dependent atomics: a token chooses an expert at most once, so a block of
// 64 tokens keeps one 64-bit token mask per expert in LDS (atomic or, any
// order), the expert's count is its popcount and a pair's rank the popcount
// below its token.
#include "qa_device.hpp"
#include "qa_launch.hpp"

namespace qa {

namespace {

constexpr int TB = 64;                       // tokens per block
constexpr int RT = 512;                      // threads per block
constexpr float NEG = -__builtin_inff();

// LDS accesses of a wave's lanes before this are seen by its lanes after it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int CTRL>
__device__ __forceinline__ int dpp(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false); }

// f(a, b) reduced over the LPT lanes of a token; every lane gets the result.
template <int LPT, class T, class F>
__device__ __forceinline__ T reduce(T v, F f) {
    auto i = [](T x) { return __builtin_bit_cast(int, x); };
    auto t = [](int x) { return __builtin_bit_cast(T, x); };
    v = f(v, t(dpp<0xB1>(i(v))));
    v = f(v, t(dpp<0x4E>(i(v))));
    v = f(v, t(dpp<0x141>(i(v))));
    v = f(v, t(dpp<0x140>(i(v))));
    if constexpr (LPT == 64) {
        v = f(v, t(__shfl_xor(i(v), 16, QA_WAVE)));
        v = f(v, t(__shfl_xor(i(v), 32, QA_WAVE)));
    }
    return v;
}

template <int LPT> __device__ __forceinline__ float rmax(float v) { return reduce<LPT>(v, [](float a, float b) { return fmaxf(a, b); }); }
template <int LPT> __device__ __forceinline__ float rsum(float v) { return reduce<LPT>(v, [](float a, float b) { return a + b; }); }
template <int LPT> __device__ __forceinline__ int rmin(int v) { return reduce<LPT>(v, [](int a, int b) { return min(a, b); }); }

template <int DT>
__device__ __forceinline__ float ldx(const void* p, int64_t j) {
    if constexpr (DT == 0) return static_cast<const float*>(p)[j];
    const uint16_t b = static_cast<const uint16_t*>(p)[j];
    return DT == 1 ? h2f(b) : __builtin_bit_cast(float, (uint32_t)b << 16);
}

}  // namespace

struct RouteArgs {
    const void* x;
    const float* bias;       // or nullptr
    int32_t* ids;
    float* w;
    int32_t* hist;           // [E][nb] counts per block of TB tokens
    int64_t T, ld;
    int32_t E, k, groups, gsize, top_groups, nb;
    float scale;
    bool sigmoid, top2, renorm;
};

// LDS words a token needs: the choice values when groups are valued, the scores
// when the bias hides them.
template <int DT, int LPT, int EPL>
__global__ __launch_bounds__(RT) void k_route(RouteArgs a) {
    constexpr int TPW = 64 / LPT;                            // tokens per wave
    constexpr int TPP = RT / LPT;                            // tokens per pass of the block
    constexpr int NS = 32 / LPT > 0 ? (32 + LPT - 1) / LPT : 1;   // slots per lane (k <= 32)
    extern __shared__ uint8_t smem[];
    uint64_t* mask = reinterpret_cast<uint64_t*>(smem);      // [E]
    float* lc = reinterpret_cast<float*>(smem + (size_t)a.E * 8);     // [TPP][E + 1] scores or choice values
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int l = lane % LPT;
    const int slot = wave * TPW + lane / LPT;                // token of the pass
    float* row = lc + (size_t)slot * (a.E + 1);
    for (int e = threadIdx.x; e < a.E; e += RT) mask[e] = 0;
    __syncthreads();
    // the choice goes by the logits themselves
    const bool by_logit = !a.sigmoid && !a.bias && (a.groups == 1 || !a.top2);
#pragma unroll 1
    for (int t0 = 0; t0 < TB; t0 += TPP) {
        const int tb = t0 + slot;
        const int64_t t = (int64_t)blockIdx.x * TB + tb;
        const bool live = t < a.T && tb < TB;
        const uint8_t* xp = static_cast<const uint8_t*>(a.x) + (live ? t : 0) * a.ld * (DT == 0 ? 4 : 2);
        float c[EPL];                                        // what is chosen by; -inf: not to be chosen
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = l * EPL + i;
            float v = NEG;
            if (live && e < a.E) v = ldx<DT>(xp, e);
            // NaN masks; +inf counts as the largest finite value
            c[i] = v != v ? NEG : fminf(v, 3.4028234663852886e38f);
        }
        float mx = c[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, c[i]);
        mx = rmax<LPT>(mx);
        float den = 1.0f;
        if (!a.sigmoid) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) s += c[i] == NEG ? 0.0f : expf(c[i] - mx);
            den = rsum<LPT>(s);
        }
        if (!by_logit) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = l * EPL + i;
                const bool in = c[i] != NEG;
                const float s = a.sigmoid ? 1.0f / (1.0f + expf(-c[i])) : expf(c[i] - mx) / den;
                if (a.bias && e < a.E) row[e] = s;
                c[i] = in ? s + (a.bias ? a.bias[min(e, a.E - 1)] : 0.0f) : NEG;
            }
        }
        if (a.groups > 1) {
            // the groups' values, over the choice values in LDS (the scores are
            // put back there afterwards when the bias needs them)
            float keep_s[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = l * EPL + i;
                keep_s[i] = a.bias && e < a.E ? row[e] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (l * EPL + i < a.E) row[l * EPL + i] = c[i];
            wave_sync();
            float val[NS];
            uint32_t kept = 0;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int g = n * LPT + l;
                float m1 = NEG, m2 = NEG;
                if (g < a.groups)
                    for (int j = 0; j < a.gsize; ++j) {
                        const float v = row[g * a.gsize + j];
                        m2 = fmaxf(m2, fminf(m1, v));
                        m1 = fmaxf(m1, v);
                    }
                val[n] = a.top2 && m2 != NEG ? m1 + m2 : m1;
            }
            wave_sync();
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (n * LPT + l < a.groups) row[n * LPT + l] = val[n];       // groups <= E
            wave_sync();
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int g = n * LPT + l;
                int before = 0;
                for (int o = 0; o < a.groups; ++o) {
                    const float v = row[o];
                    before += v > val[n] || (v == val[n] && o < g) ? 1 : 0;
                }
                if (g < a.groups && before < a.top_groups) kept |= 1u << g;
            }
            kept = reduce<LPT>((int)kept, [](int p, int q) { return p | q; });
            wave_sync();
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = l * EPL + i;
                if (!((kept >> (min(e, a.E - 1) / a.gsize)) & 1)) c[i] = NEG;
                if (a.bias && e < a.E) row[e] = keep_s[i];
            }
        }
        wave_sync();
        // k rounds: the largest value left, the lowest index among equals
        int id[NS];
        float wt[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) { id[n] = -1; wt[n] = 0.0f; }
        for (int j = 0; j < a.k; ++j) {
            float b = c[0];
            int bi = 0;
#pragma unroll
            for (int i = 1; i < EPL; ++i)
                if (c[i] > b) { b = c[i]; bi = i; }
            const float m = rmax<LPT>(b);
            int e = rmin<LPT>(b == m ? l * EPL + bi : 0x7fffffff);
            if (m == NEG) e = -1;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (l * EPL + i == e) c[i] = NEG;
#pragma unroll
            for (int n = 0; n < NS; ++n)
                if (j == n * LPT + l) { id[n] = e; wt[n] = m; }
        }
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            if (id[n] < 0) wt[n] = 0.0f;
            else if (by_logit) wt[n] = expf(wt[n] - mx) / den;
            else if (a.bias) wt[n] = row[id[n]];
            sum += wt[n];
        }
        sum = rsum<LPT>(sum);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int j = n * LPT + l;
            if (live && j < a.k) {
                const float w = a.renorm && sum > 0.0f ? wt[n] / sum : wt[n];
                a.ids[t * a.k + j] = id[n];
                a.w[t * a.k + j] = w * a.scale;
                if (id[n] >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mask[id[n]]), 1ull << tb);
            }
        }
        wave_sync();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += RT) a.hist[(int64_t)e * a.nb + blockIdx.x] = __popcll(mask[e]);
}

// Exclusive prefix of an expert's counts over the blocks, in place, and its
// total: one wave per expert.
__global__ __launch_bounds__(256) void k_route_scan(int32_t* __restrict__ hist, int32_t* __restrict__ total, int32_t E,
                                                    int32_t nb) {
    const int lane = threadIdx.x & 63;
    const int e = blockIdx.x * 4 + wave_id();
    if (e >= E) return;
    int32_t* h = hist + (int64_t)e * nb;
    int base = 0;
    for (int b0 = 0; b0 < nb; b0 += 64) {
        const int b = b0 + lane;
        const int v = b < nb ? h[b] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(s, o, QA_WAVE);
            if (lane >= o) s += u;
        }
        if (b < nb) h[b] = base + s - v;
        base += __shfl(s, 63, QA_WAVE);
    }
    if (lane == 0) total[e] = base;
}

// Every pair of the block's tokens to its place: expert start + the expert's
// pairs in earlier blocks + its tokens before this one in the block.
__global__ __launch_bounds__(RT) void k_route_scatter(const int32_t* __restrict__ ids, const int32_t* __restrict__ pre,
                                                      const int32_t* __restrict__ total, int64_t T, int32_t E,
                                                      int32_t k, int32_t nb, int32_t* __restrict__ order,
                                                      int32_t* __restrict__ offsets) {
    extern __shared__ uint8_t smem[];
    uint64_t* mask = reinterpret_cast<uint64_t*>(smem);      // [E]
    int32_t* base = reinterpret_cast<int32_t*>(smem + (size_t)E * 8);   // [E]
    __shared__ int32_t wsum[RT / 64];
    const int lane = threadIdx.x & 63, wave = wave_id();
    // exclusive prefix of the totals: thread t takes experts 2t, 2t + 1
    const int e0 = threadIdx.x * 2;
    const int v0 = e0 < E ? total[e0] : 0, v1 = e0 + 1 < E ? total[e0 + 1] : 0;
    int s = v0 + v1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o, QA_WAVE);
        if (lane >= o) s += u;
    }
    if (lane == 63) wsum[wave] = s;
    for (int e = threadIdx.x; e < E; e += RT) mask[e] = 0;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < RT / 64; ++w) {
        before += w < wave ? wsum[w] : 0;
        all += wsum[w];
    }
    const int st = before + s - v0 - v1;
    if (e0 < E) base[e0] = st + pre[(int64_t)e0 * nb + blockIdx.x];
    if (e0 + 1 < E) base[e0 + 1] = st + v0 + pre[(int64_t)(e0 + 1) * nb + blockIdx.x];
    if (blockIdx.x == 0) {
        if (e0 < E) offsets[e0] = st;
        if (e0 + 1 < E) offsets[e0 + 1] = st + v0;
        if (threadIdx.x == 0) offsets[E] = all;
    }
    const int64_t p0 = (int64_t)blockIdx.x * TB * k, p1 = min(p0 + (int64_t)TB * k, T * k);
    for (int64_t p = p0 + threadIdx.x; p < p1; p += RT) {
        const int e = ids[p];
        if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mask[e]), 1ull << ((int)(p - p0) / k));
        if (p >= all) order[p] = -1;                         // places after the last pair
    }
    __syncthreads();
    for (int64_t p = p0 + threadIdx.x; p < p1; p += RT) {
        const int e = ids[p];
        if (e >= 0) {
            const int tb = (int)(p - p0) / k;
            order[base[e] + __popcll(mask[e] & ((1ull << tb) - 1))] = (int32_t)p;
        }
    }
}

__global__ void k_route_none(int32_t* offsets, int32_t E) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

size_t route_scratch_bytes(int64_t T, int64_t E) {
    const int64_t nb = (T + TB - 1) / TB;
    return (size_t)(E * nb + E) * 4;
}

hipError_t launch_route(const void* x, int dtype, int64_t T, int64_t E, int64_t ld, const float* bias, bool sigmoid,
                        int groups, int top_groups, bool top2, int k, bool renorm, float scale, int32_t* ids, float* w,
                        int32_t* order, int32_t* offsets, void* scratch, hipStream_t st) {
    if (T == 0) {
        hipLaunchKernelGGL(k_route_none, dim3(1), dim3(256), 0, st, offsets, (int32_t)E);
        return hipGetLastError();
    }
    const int nb = (int)((T + TB - 1) / TB);
    int32_t* hist = static_cast<int32_t*>(scratch);
    int32_t* total = hist + E * nb;
    const RouteArgs a{x, bias, ids, w, hist, T, ld, (int32_t)E, k, groups, (int32_t)(E / groups), top_groups, nb, scale,
                      sigmoid, top2, renorm};
    const int lpt = E <= 256 ? 16 : 64;
    const bool rows_in_lds = bias || groups > 1;
    const size_t lds = (size_t)E * 8 + (rows_in_lds ? (size_t)(RT / lpt) * (E + 1) * 4 : 0);
#define QA_ROUTE(DT, LPT, EPL) hipLaunchKernelGGL((k_route<DT, LPT, EPL>), dim3(nb), dim3(RT), lds, st, a)
#define QA_ROUTE_E(DT)                                                                          \
    do {                                                                                        \
        if (E <= 32) QA_ROUTE(DT, 16, 2);                                                       \
        else if (E <= 64) QA_ROUTE(DT, 16, 4);                                                  \
        else if (E <= 128) QA_ROUTE(DT, 16, 8);                                                 \
        else if (E <= 256) QA_ROUTE(DT, 16, 16);                                                \
        else if (E <= 512) QA_ROUTE(DT, 64, 8);                                                 \
        else QA_ROUTE(DT, 64, 16);                                                              \
    } while (0)
    if (dtype == 0) QA_ROUTE_E(0);
    else if (dtype == 1) QA_ROUTE_E(1);
    else QA_ROUTE_E(2);
#undef QA_ROUTE_E
#undef QA_ROUTE
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_route_scan, dim3((unsigned)((E + 3) / 4)), dim3(256), 0, st, hist, total, (int32_t)E, nb);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(k_route_scatter, dim3(nb), dim3(RT), (size_t)E * 12, st, ids, hist, total, T, (int32_t)E, k, nb,
                       order, offsets);
    return hipGetLastError();
}

}  // namespace qa
