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
// Both scores keep the order of the logits, so without a bias (and with groups
// valued by their largest member) the choice is made on the logits themselves,
// which also differ where their scores round to the same number (sigmoid(17) is 1
// in fp32), and the exponentials are taken for the k chosen and softmax's sum alone.
//
// A logit of -inf or NaN masks its expert; where fewer than k are left, the
// last slots hold expert -1 with weight 0 and are in no group.
//
// LPT lanes work on one token (16 for up to 256 experts, so that a wave takes
// four tokens and every reduction is four DPP steps in a row of 16 lanes; 64
// above that), lane l holding the EPL experts l EPL .. in registers.
//
// The choice: k rounds of "largest left" cost each lane its EPL registers in
// every round.  Instead the k-th largest of the lanes' own maxima is a bound
// that the k chosen reach (k lanes hold a value as large), and few others do:
// the values that reach it go to LDS, one or two to a lane, and a value's rank
// among them is its slot.  For more than 8, or with groups, the bound is taken from
// the lanes' two largest.  Only where more than 32 reach it (many ties), for k > 16
// and above 256 experts the rounds are run.  First launch at 50001 x 128 (bf16,
// k = 8): 28.8 us with the rounds, 18.4 with the bound (17.6 at best); at 4096 x 256
// in 8 groups 34 and 9.6.  With the rounds in this form 4096 x 256 at k = 24 takes
// 15.3, 4096 x 384 at k = 8 10.8, 4096 x 512 at k = 10 12.2.  At 50001 tokens it
// issues 415 vector instructions per wave of four tokens, 9 us of the SIMDs' time;
// reading the logits is 2.5 us.  The rest is waiting (56% of the waves' time): 1024
// threads of 72 registers leave one block to a CU, with nothing to run at its
// barriers.  32 tokens to a block run it in 14.8 us, but the counts of twice the
// blocks cost that again in the two launches after (k_route_scan 5.6 us,
// k_route_scatter 3.0 to 5.4: little more than launches).
//
// The grouping is stable (ascending pair index within an expert) and uses no
// order-dependent atomics: a token chooses an expert at most once, so a block of
// up to 64 tokens keeps one 64-bit token mask per expert in LDS (atomic or, any
// order), the expert's count is its popcount and a pair's rank the popcount
// below its token.
#include "qa_device.hpp"
#include "qa_launch.hpp"

namespace qa {

namespace {

constexpr float NEG = -__builtin_inff(), FMAX = 3.4028234663852886e38f;
constexpr int CAP = 32;                      // values that may reach the bound
constexpr int MAXK = 32;

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

// The order of floats as unsigned numbers (no NaN; -0 counts as 0).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

template <int DT>
__device__ __forceinline__ float ldx(const void* p, int64_t j) {
    if constexpr (DT == 0) return static_cast<const float*>(p)[j];
    const uint16_t b = static_cast<const uint16_t*>(p)[j];
    return DT == 1 ? h2f(b) : __builtin_bit_cast(float, (uint32_t)b << 16);
}

// N consecutive elements at p, aligned to their whole size (16 bytes at most).
template <int DT, int N>
__device__ __forceinline__ void ldv(const uint8_t* p, float* x) {
    constexpr int B = N * (DT == 0 ? 4 : 2);
    uint32_t w[(B + 3) / 4];
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) {
            const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
        }
    } else if constexpr (B == 8) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
        w[0] = v[0];
        w[1] = v[1];
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (DT == 0) {
            x[i] = __builtin_bit_cast(float, w[i]);
        } else {
            const uint16_t b = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            x[i] = DT == 1 ? h2f(b) : __builtin_bit_cast(float, (uint32_t)b << 16);
        }
    }
}

// Rotation within a row of 16 lanes, and an inclusive prefix sum over it.
template <int N> __device__ __forceinline__ int ror16(int v) { return dpp<0x120 + N>(v); }
__device__ __forceinline__ int prefix16(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    return v;
}

// For each lane of a row of 16: how many of the other 15 f(theirs, mine, other lane) counts.
template <int N, class F>
__device__ __forceinline__ int count15(float v, int l, F f) {
    if constexpr (N == 16) return 0;
    else {
        // row_ror:N hands lane l the value of lane (l - N) mod 16
        const float o = __builtin_bit_cast(float, ror16<N>(__builtin_bit_cast(int, v)));
        return (f(o, v, (l + 16 - N) & 15) ? 1 : 0) + count15<N + 1>(v, l, f);
    }
}

// How many of the other 15 lanes' m1 and m2 are larger than v.
template <int N>
__device__ __forceinline__ int count15x2(float m1, float m2, float v) {
    if constexpr (N == 16) return 0;
    else {
        const float a = __builtin_bit_cast(float, ror16<N>(__builtin_bit_cast(int, m1)));
        const float b = __builtin_bit_cast(float, ror16<N>(__builtin_bit_cast(int, m2)));
        return (a > v ? 1 : 0) + (b > v ? 1 : 0) + count15x2<N + 1>(m1, m2, v);
    }
}

}  // namespace

struct RouteArgs {
    const void* x;
    const float* bias;       // or nullptr
    int32_t* ids;
    float* w;
    int32_t* hist;           // [nb][E] counts per block of tokens
    int32_t* order;          // written here when one block holds every token
    int32_t* offsets;
    int64_t T, ld;
    int32_t E, k, groups, gsize, top_groups, nb;
    float scale;
    bool sigmoid, top2, renorm;
    bool vec;                // rows allow whole-vector loads of EPL elements
};

// Exclusive prefix of v over the block's threads; *all gets the total.
template <int THREADS>
__device__ __forceinline__ int block_prefix(int v, int32_t* wsum, int* all) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    int s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o, QA_WAVE);
        if (lane >= o) s += u;
    }
    if (lane == 63) wsum[wave] = s;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        before += w < wave ? wsum[w] : 0;
        sum += wsum[w];
    }
    *all = sum;
    return before + s - v;
}

// Values of the groups and the experts of the kept ones, out of c in registers
// when a group is m whole lanes (m a power of two), else over `row` in LDS.
template <int LPT, int EPL>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, float (&c)[EPL], float* row, int l) {
    const int m = a.gsize / EPL;
    if (LPT == 16 && a.gsize % EPL == 0 && (m & (m - 1)) == 0) {
        float m1 = NEG, m2 = NEG;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            m2 = fmaxf(m2, fminf(m1, c[i]));
            m1 = fmaxf(m1, c[i]);
        }
        auto join = [&](float o1, float o2) {
            m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
            m1 = fmaxf(m1, o1);
        };
        auto f = [](int v) { return __builtin_bit_cast(float, v); };
        auto i = [](float v) { return __builtin_bit_cast(int, v); };
        if (m >= 2) join(f(dpp<0xB1>(i(m1))), f(dpp<0xB1>(i(m2))));
        if (m >= 4) join(f(dpp<0x4E>(i(m1))), f(dpp<0x4E>(i(m2))));
        if (m >= 8) join(f(dpp<0x141>(i(m1))), f(dpp<0x141>(i(m2))));
        if (m >= 16) join(f(dpp<0x140>(i(m1))), f(dpp<0x140>(i(m2))));
        const float val = a.top2 && m2 != NEG ? m1 + m2 : m1;
        const int sh = 31 - __builtin_clz(m);
        // every group is seen through each of its m lanes
        const int before = count15<1>(val, l, [&](float o, float v, int ol) {
            return o > v || (o == v && (ol >> sh) < (l >> sh));
        });
        if (before >= a.top_groups << sh)
#pragma unroll
            for (int q = 0; q < EPL; ++q) c[q] = NEG;
        return;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (l * EPL + i < a.E) row[l * EPL + i] = c[i];
    wave_sync();
    constexpr int NS = (32 + LPT - 1) / LPT;
    float val[NS];
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
        if (n * LPT + l < a.groups) row[n * LPT + l] = val[n];               // groups <= E
    wave_sync();
    uint32_t kept = 0;
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
    for (int i = 0; i < EPL; ++i)
        if (!((kept >> (min(l * EPL + i, a.E - 1) / a.gsize)) & 1)) c[i] = NEG;
}

// One token per LPT lanes, TB tokens per block (TB LPT threads).
template <int DT, int LPT, int EPL, int TB>
__global__ __launch_bounds__(TB * LPT) void k_route(RouteArgs a) {
    constexpr int THREADS = TB * LPT;
    constexpr int NS = (MAXK + LPT - 1) / LPT;               // slots per lane
    extern __shared__ uint8_t smem[];
    uint64_t* mask = reinterpret_cast<uint64_t*>(smem);      // [E] tokens of the block that chose the expert
    float* rows = reinterpret_cast<float*>(smem + (size_t)a.E * 8);           // [TB][E + 1], for keep_groups
    __shared__ uint64_t ckey[TB][CAP];
    __shared__ float cscore[TB][CAP];
    __shared__ int sid[TB][MAXK];
    __shared__ float swt[TB][MAXK];
    const int l = threadIdx.x % LPT, tb = threadIdx.x / LPT;
    for (int e = threadIdx.x; e < a.E; e += THREADS) mask[e] = 0;
    __syncthreads();
    const int64_t t = (int64_t)blockIdx.x * TB + tb;
    const bool live = t < a.T;
    const uint8_t* xp = static_cast<const uint8_t*>(a.x) + (live ? t : 0) * a.ld * (DT == 0 ? 4 : 2);
    // the choice goes by the logits themselves
    const bool by_logit = !a.bias && (a.groups == 1 || !a.top2);
    float c[EPL], s[EPL];                                    // chosen by (-inf: not to be chosen), score
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = NEG;
    if (live) {
        if (a.vec) {
            if (l * EPL < a.E) ldv<DT, EPL>(xp + (size_t)l * EPL * (DT == 0 ? 4 : 2), c);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (l * EPL + i < a.E) c[i] = ldx<DT>(xp, l * EPL + i);
        }
    }
    // NaN masks (the maximum of NaN and a number is the number); +inf counts as
    // the largest finite value
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = fminf(fmaxf(c[i], NEG), FMAX);
    float mx = c[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, c[i]);
    const float lane_top = mx;
    mx = rmax<LPT>(mx);
    float den = 1.0f;
    if (a.sigmoid) {
        if (!by_logit) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] = sigmoid(c[i]);
        }
    } else {
        den = 0.0f;
        const float m0 = mx == NEG ? 0.0f : mx;
        if (by_logit) {
            // only the sum is wanted: 2^((x - max) log2 e), whose relative error
            // grows with max - x, where the term itself vanishes
            constexpr float L2E = 1.44269502162933349609375f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) den += __builtin_amdgcn_exp2f((c[i] - m0) * L2E);
            den = rsum<LPT>(den);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = fexp(c[i] - m0);
                den += s[i];
            }
            den = rsum<LPT>(den);
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] = s[i] / den;
        }
    }
    float top = lane_top;
    if (!by_logit) {
        top = NEG;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool in = c[i] != NEG;
            // (a NaN bias masks its expert, as a NaN logit does)
            c[i] = in ? fmaxf(s[i] + (a.bias ? a.bias[min(l * EPL + i, a.E - 1)] : 0.0f), NEG) : NEG;
            top = fmaxf(top, c[i]);
        }
    }
    if (a.groups > 1) {
        keep_groups<LPT, EPL>(a, c, rows + (size_t)tb * (a.E + 1), l);
        top = c[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = fmaxf(top, c[i]);
    }
    // the bound: the k-th largest of the lanes' maxima
    bool few = false;
    if (LPT == 16 && a.k <= 16) {
        // (a lane whose maximum fewer than k lanes exceed has one as large as the
        // k-th largest; the least of those is the bound)
        auto more = [](float o, float v, int) { return o > v; };
        float least = FMAX;
        if (a.groups == 1 && a.k <= 8) {
            if (count15<1>(top, l, more) < a.k) least = top;
        } else {
            // more than 8, or the kept groups' experts in few lanes: the lanes' two largest
            float m1 = NEG, m2 = NEG;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                m2 = fmaxf(m2, fminf(m1, c[i]));
                m1 = fmaxf(m1, c[i]);
            }
            if (count15x2<1>(m1, m2, m1) < a.k) least = m1;
            if (count15x2<1>(m1, m2, m2) + (m1 > m2 ? 1 : 0) < a.k) least = m2;
        }
        float bound = reduce<16>(least, [](float p, float q) { return fminf(p, q); });
        bound = fmaxf(bound, -FMAX);                         // masked experts never reach it
        int n = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) n += c[i] >= bound ? 1 : 0;
        const int upto = prefix16(n);
        const int total = reduce<16>(upto, [](int p, int q) { return max(p, q); });
        few = !__any(total > CAP);
        if (few) {
            int at = upto - n;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (c[i] >= bound) {
                    ckey[tb][at] = ((uint64_t)__builtin_bit_cast(uint32_t, c[i]) << 32) | (uint32_t)(l * EPL + i);
                    if (!by_logit) cscore[tb][at] = s[i];
                    ++at;
                }
            sid[tb][l] = -1;
            const bool wide = __any(total > 16);
            wave_sync();
            // one value (or two) to a lane, as a number that orders by value and
            // then by lower index; 0 in the places without one
            uint64_t key[2];
            uint32_t e[2], bits[2];
            int rank[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint64_t mine = ckey[tb][h * 16 + l];
                e[h] = (uint32_t)mine;
                bits[h] = (uint32_t)(mine >> 32);
                key[h] = h * 16 + l < total ? ((uint64_t)ordered(__builtin_bit_cast(float, bits[h])) << 32) | (0xffffu - e[h]) : 0;
            }
            wave_sync();
            ckey[tb][l] = key[0];
            ckey[tb][16 + l] = key[1];
            wave_sync();
#pragma unroll
            for (int o = 0; o < 16; ++o) rank[0] += ckey[tb][o] > key[0] ? 1 : 0;
            if (wide) {
#pragma unroll
                for (int o = 0; o < 16; ++o) {
                    const uint64_t u = ckey[tb][16 + o];
                    rank[0] += u > key[0] ? 1 : 0;
                    rank[1] += (ckey[tb][o] > key[1] ? 1 : 0) + (u > key[1] ? 1 : 0);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (h * 16 + l < total && rank[h] < a.k) {
                    sid[tb][rank[h]] = (int)e[h];
                    swt[tb][rank[h]] = by_logit ? __builtin_bit_cast(float, bits[h]) : cscore[tb][h * 16 + l];
                }
        }
    }
    if (!few) {
        // k rounds: the largest value left, the lowest index among equals
        for (int j = 0; j < a.k; ++j) {
            float b = c[0];
            int bi = 0;
#pragma unroll
            for (int i = 1; i < EPL; ++i)
                if (c[i] > b) { b = c[i]; bi = i; }
            const float m = rmax<LPT>(b);
            int e = rmin<LPT>(b == m ? l * EPL + bi : 0x7fffffff);
            if (m == NEG) e = -1;
            float sc = m;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (l * EPL + i == e) {
                    c[i] = NEG;
                    sc = s[i];
                }
            if (e < 0 ? l == 0 : e / EPL == l) {             // the expert's lane, or lane 0 for none
                sid[tb][j] = e;
                swt[tb][j] = by_logit ? m : sc;
            }
        }
    }
    wave_sync();
    int id[NS];
    float wt[NS], sum = 0.0f;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        const int j = n * LPT + l;
        id[n] = j < a.k ? sid[tb][j] : -1;
        wt[n] = 0.0f;
        if (id[n] >= 0) {
            wt[n] = swt[tb][j];
            if (by_logit) wt[n] = a.sigmoid ? sigmoid(wt[n]) : expf(wt[n] - mx) / den;
        }
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
    __syncthreads();
    if (a.nb > 1) {
        for (int e = threadIdx.x; e < a.E; e += THREADS) a.hist[(int64_t)blockIdx.x * a.E + e] = __popcll(mask[e]);
        return;
    }
    // one block holds every token: the experts' starts and the pairs' places here
    __shared__ int32_t wsum[THREADS / 64];
    int32_t* base = reinterpret_cast<int32_t*>(rows);        // [E]: the token rows are no longer read
    constexpr int PER = (1024 + THREADS - 1) / THREADS;
    int v[PER], mysum = 0, all;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x * PER + i;
        v[i] = e < a.E ? __popcll(mask[e]) : 0;
        mysum += v[i];
    }
    int st = block_prefix<THREADS>(mysum, wsum, &all);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x * PER + i;
        if (e < a.E) {
            base[e] = st;
            a.offsets[e] = st;
        }
        st += v[i];
    }
    if (threadIdx.x == 0) a.offsets[a.E] = all;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        const int j = n * LPT + l;
        if (live && j < a.k && id[n] >= 0)
            a.order[base[id[n]] + __popcll(mask[id[n]] & ((1ull << tb) - 1))] = (int32_t)(t * a.k + j);
    }
    for (int p = all + threadIdx.x; p < a.T * a.k; p += THREADS) a.order[p] = -1;
}

// Exclusive prefix of an expert's counts over the blocks, in place, and its
// total.  A block takes 16 experts (a row's 64 bytes side by side), its threads
// 64 ranges of `per` rows each.
__global__ __launch_bounds__(1024) void k_route_scan(int32_t* __restrict__ hist, int32_t* __restrict__ total, int32_t E,
                                                     int32_t nb, int32_t per) {
    __shared__ int32_t sums[16][65];
    const int e = blockIdx.x * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4;
    const int64_t b0 = (int64_t)part * per, b1 = min(b0 + per, (int64_t)nb);
    constexpr int V = 16;                                    // counts kept: up to 1024 blocks are read once
    int v[V], s = 0;
    for (int64_t b = b0; b < b1; b += V) {
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] = e < E && b + q < b1 ? hist[(b + q) * E + e] : 0;
#pragma unroll
        for (int q = 0; q < V; ++q) s += v[q];
    }
    sums[threadIdx.x & 15][part] = s;
    __syncthreads();
    {
        const int lane = threadIdx.x & 63, w = wave_id();    // wave w scans expert w's 64 sums
        const int v = sums[w][lane];
        int t = v;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(t, o, QA_WAVE);
            if (lane >= o) t += u;
        }
        sums[w][lane] = t - v;
        if (lane == 63 && blockIdx.x * 16 + w < E) total[blockIdx.x * 16 + w] = t;
    }
    __syncthreads();
    if (e >= E) return;
    int at = sums[threadIdx.x & 15][part];
    for (int64_t b = b0; b < b1; b += V) {
        if (per > V) {
#pragma unroll
            for (int q = 0; q < V; ++q) v[q] = b + q < b1 ? hist[(b + q) * E + e] : 0;
        }
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (b + q < b1) {
                hist[(b + q) * E + e] = at;
                at += v[q];
            }
    }
}

// Every pair of the block's tokens to its place: expert start + the expert's
// pairs in earlier blocks + its tokens before this one in the block.
template <int TB>
__global__ __launch_bounds__(512) void k_route_scatter(const int32_t* __restrict__ ids, const int32_t* __restrict__ pre,
                                                       const int32_t* __restrict__ total, int64_t T, int32_t E,
                                                       int32_t k, int32_t* __restrict__ order,
                                                       int32_t* __restrict__ offsets) {
    constexpr int RT = 512, PP = (TB * MAXK + RT - 1) / RT;  // pairs per thread
    extern __shared__ uint8_t smem[];
    uint64_t* mask = reinterpret_cast<uint64_t*>(smem);      // [E]
    int32_t* base = reinterpret_cast<int32_t*>(smem + (size_t)E * 8);   // [E]
    __shared__ int32_t wsum[RT / 64];
    const int64_t p0 = (int64_t)blockIdx.x * TB * k;
    const int np = (int)min((int64_t)TB * k, T * k - p0);
    int id[PP];
#pragma unroll
    for (int i = 0; i < PP; ++i) {
        const int p = threadIdx.x + i * RT;
        id[i] = p < np ? ids[p0 + p] : -1;
    }
    const int e0 = threadIdx.x * 2;                          // thread t takes experts 2t, 2t + 1
    const int v0 = e0 < E ? total[e0] : 0, v1 = e0 + 1 < E ? total[e0 + 1] : 0;
    const int q0 = e0 < E ? pre[(int64_t)blockIdx.x * E + e0] : 0;
    const int q1 = e0 + 1 < E ? pre[(int64_t)blockIdx.x * E + e0 + 1] : 0;
    for (int e = threadIdx.x; e < E; e += RT) mask[e] = 0;
    int all;
    const int st = block_prefix<RT>(v0 + v1, wsum, &all);    // its barrier also ends the clearing
    if (e0 < E) base[e0] = st + q0;
    if (e0 + 1 < E) base[e0 + 1] = st + v0 + q1;
    if (blockIdx.x == 0) {
        if (e0 < E) offsets[e0] = st;
        if (e0 + 1 < E) offsets[e0 + 1] = st + v0;
        if (threadIdx.x == 0) offsets[E] = all;
    }
#pragma unroll
    for (int i = 0; i < PP; ++i) {
        const int p = threadIdx.x + i * RT;
        if (id[i] >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mask[id[i]]), 1ull << (p / k));
        if (p < np && p0 + p >= all) order[p0 + p] = -1;     // places after the last pair
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PP; ++i) {
        const int p = threadIdx.x + i * RT;
        if (id[i] >= 0)
            order[base[id[i]] + __popcll(mask[id[i]] & ((1ull << (p / k)) - 1))] = (int32_t)(p0 + p);
    }
}

__global__ void k_route_none(int32_t* offsets, int32_t E) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

// Tokens per block.  A block is one pass over its tokens, so few tokens want
// small blocks (4096 x 256: 16 tokens fill 256 blocks, 64 tokens only 64: 12.3
// against 19.8 us of the first launch); many want few counts to scan (50001 x 128:
// 32.7 against 33.5 us for the call, both measured before the bound's last form).
// Up to 64 tokens one block of 64 does the grouping as well, without the other two
// launches (32 x 64: 4.4 us in all).  Above 256 experts a token takes a whole wave,
// 16 to a block.
static int route_tb(int64_t T, int64_t E) { return E <= 256 && (T <= 64 || T > 16384) ? 64 : 16; }

size_t route_scratch_bytes(int64_t T, int64_t E) {
    const int64_t tb = route_tb(T, E), nb = (T + tb - 1) / tb;
    return (size_t)(E * nb + E) * 4;
}

template <int DT, int LPT, int EPL, int TB>
static hipError_t run_route(RouteArgs a, hipStream_t st) {
    constexpr int SZ = DT == 0 ? 4 : 2;
    const int bytes = EPL * SZ < 16 ? EPL * SZ : 16;
    a.vec = a.E % EPL == 0 && a.ld * SZ % bytes == 0 && reinterpret_cast<uintptr_t>(a.x) % bytes == 0;
    const int m = a.gsize / EPL;
    const bool in_lanes = LPT == 16 && a.gsize % EPL == 0 && (m & (m - 1)) == 0;
    const size_t rows = a.groups > 1 && !in_lanes ? (size_t)TB * (a.E + 1) * 4 : (size_t)a.E * 4;
    hipLaunchKernelGGL((k_route<DT, LPT, EPL, TB>), dim3(a.nb), dim3(TB * LPT), (size_t)a.E * 8 + rows, st, a);
    return hipGetLastError();
}

template <int DT>
static hipError_t route_by_experts(const RouteArgs& a, int tb, hipStream_t st) {
#define QA_ROUTE(EPL) (tb == 64 ? run_route<DT, 16, EPL, 64>(a, st) : run_route<DT, 16, EPL, 16>(a, st))
    if (a.E <= 32) return QA_ROUTE(2);
    if (a.E <= 64) return QA_ROUTE(4);
    if (a.E <= 128) return QA_ROUTE(8);
    if (a.E <= 256) return QA_ROUTE(16);
#undef QA_ROUTE
    if (a.E <= 512) return run_route<DT, 64, 8, 16>(a, st);
    return run_route<DT, 64, 16, 16>(a, st);
}

hipError_t launch_route(const void* x, int dtype, int64_t T, int64_t E, int64_t ld, const float* bias, bool sigmoid,
                        int groups, int top_groups, bool top2, int k, bool renorm, float scale, int32_t* ids, float* w,
                        int32_t* order, int32_t* offsets, void* scratch, hipStream_t st) {
    if (T == 0) {
        hipLaunchKernelGGL(k_route_none, dim3(1), dim3(256), 0, st, offsets, (int32_t)E);
        return hipGetLastError();
    }
    const int tb = route_tb(T, E);
    const int nb = (int)((T + tb - 1) / tb);
    int32_t* hist = static_cast<int32_t*>(scratch);
    int32_t* total = hist + E * nb;
    const RouteArgs a{x, bias, ids, w, hist, order, offsets, T, ld, (int32_t)E, k, groups, (int32_t)(E / groups),
                      top_groups, nb, scale, sigmoid, top2, renorm, false};
    hipError_t e = dtype == 0 ? route_by_experts<0>(a, tb, st)
                              : (dtype == 1 ? route_by_experts<1>(a, tb, st) : route_by_experts<2>(a, tb, st));
    if (e != hipSuccess || nb == 1) return e;
    hipLaunchKernelGGL(k_route_scan, dim3((unsigned)((E + 15) / 16)), dim3(1024), 0, st, hist, total, (int32_t)E, nb,
                       (nb + 63) / 64);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (tb == 64)
        hipLaunchKernelGGL(k_route_scatter<64>, dim3(nb), dim3(512), (size_t)E * 12, st, ids, hist, total, T, (int32_t)E,
                           k, order, offsets);
    else
        hipLaunchKernelGGL(k_route_scatter<16>, dim3(nb), dim3(512), (size_t)E * 12, st, ids, hist, total, T, (int32_t)E,
                           k, order, offsets);
    return hipGetLastError();
}

}  // namespace qa
