// k_kv.hip -- a paged cache of keys and values in int8 or int4 codes: written
// from new tokens and read back, on gfx950.
//
//   s = max_d |x_d| / q_max (1 where that is 0),  q = rint(x / s)      (write)
//   x = fl32(q s), rounded to the type                                  (read)
//
// per token and head, q_max 127 or 7.  A page holds `page` tokens of every head,
// head by head: codes [pages][heads][page][D], scales [pages][heads][page]; four-bit
// codes are packed eight to a word like every int4 row of this library.
//
// A row of D values is eight values to a lane and 8, 16 or 32 lanes; the maximum
// over them is the only exchange (moves between lanes).  The lanes of a token do its key and its
// value, so a place is looked up once and two rows are in flight.  Consecutive
// rows of a block are consecutive tokens of one head: prompts then write whole
// pieces of a page, codes and scales.
#include "qa_device.hpp"
#include "qa_launch.hpp"

namespace qa {

namespace {

struct KvArgs {
    const void* x[2];          // write: keys and values, rows of heads x D
    int64_t ld[2];             // their token strides in elements
    void* y[2];                // read: outputs [T][heads][D]
    uint8_t* codes[2];
    float* scales[2];
    const int64_t* slots;      // [T] page * page_size + place in the page
    int64_t T, places;         // places: pages * page_size
    int32_t heads, D, shift;   // shift: log2 of the page's tokens
};

__device__ __forceinline__ float bf2f(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }

// Eight values of a row as they stand in memory.
template <int DT>
struct Raw {
    u32x4 w[DT == 0 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw<DT> load8(const void* p, int64_t at) {
    Raw<DT> r;
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p) + at * (DT == 0 ? 4 : 2));
    r.w[0] = q[0];
    if constexpr (DT == 0) r.w[1] = q[1];
    return r;
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw<DT>& r, float* x) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (DT == 0) {
            const uint32_t u = r.w[j >> 2][j & 3];
            x[j] = __builtin_bit_cast(float, u);
        } else {
            const uint16_t u = (uint16_t)(r.w[0][j >> 1] >> (16 * (j & 1)));
            x[j] = DT == 1 ? h2f(u) : bf2f(u);
        }
    }
}
// The bits of the largest magnitude of the eight, as a number of the type: patterns order like the values,
// infinities and NaNs above all.
template <int DT>
__device__ __forceinline__ uint32_t largest8(const Raw<DT>& r) {
    uint32_t m = 0;
    if constexpr (DT == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, r.w[j >> 2][j & 3] & 0x7fffffffu);
        return m;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) m = pk_max_u16(m, r.w[0][j] & 0x7fff7fffu);
    return max(m & 0xffffu, m >> 16);
}
// The largest over N = 8, 16 or 32 lanes side by side: moves within rows of 16 lanes, and between two of them.
template <int N>
__device__ __forceinline__ uint32_t largest_of(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));     // lane ^ 1
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));     // lane ^ 2
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));    // the other four of eight
    if constexpr (N >= 16) m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
    if constexpr (N == 32) m = max(m, (uint32_t)__builtin_amdgcn_ds_swizzle((int)m, 0x401F));    // lane ^ 16
    return m;
}
// m / Q for a whole number Q, rounded to nearest, for m of at least 2^-107: the product with the rounded reciprocal is
// within one step of the quotient, and its exact remainder times the reciprocal rounds it (all 2^23 significands
// of m agree with the division for 127 and for 7).
template <int Q>
__device__ __forceinline__ float divide_by(float m) {
    constexpr float r = 1.0f / Q;
    const float q = m * r;
    return __builtin_fmaf(__builtin_fmaf(-q, (float)Q, m), r, q);
}

template <bool NT, class T>
__device__ __forceinline__ void store(T v, T* p) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <bool NT, class T>
__device__ __forceinline__ T load(const T* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    return *p;
}

template <int DT, bool NT>
__device__ __forceinline__ void store8(void* p, int64_t at, const float* x) {
    if constexpr (DT == 0) {
        v4f* o = reinterpret_cast<v4f*>(static_cast<float*>(p) + at);
        store<NT>(v4f{x[0], x[1], x[2], x[3]}, o);
        store<NT>(v4f{x[4], x[5], x[6], x[7]}, o + 1);
    } else {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = DT == 1 ? f2h(x[2 * j]) : f2bf(x[2 * j]);
            const uint32_t hi = DT == 1 ? f2h(x[2 * j + 1]) : f2bf(x[2 * j + 1]);
            w[j] = lo | (hi << 16);
        }
        store<NT>(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at));
    }
}

// Row of a place in codes and scales.
__device__ __forceinline__ int64_t row_of(const KvArgs& a, int64_t slot, int h) {
    return (((slot >> a.shift) * a.heads + h) << a.shift) + (slot & ((1 << a.shift) - 1));
}

// LPR lanes to a row, 256 / LPR tokens of head blockIdx.y to a block.  16411 tokens of 8
// heads of 128, bf16 to 8 bits: 23.4 us, 4.4 TB/s (a large copy reaches 4.9); 8192 of 32
// heads of 64, fp16 to 4 bits: 22.4.  With divisions for the scale and its reciprocal, maxima
// exchanged through LDS and codes packed byte by byte instructions bound it: 26.1 and 24.9.
template <int DT, int BITS, int LPR>
__global__ __launch_bounds__(256) void k_kv_write(KvArgs a) {
    const int j = threadIdx.x % LPR;
    const int64_t t = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int h = blockIdx.y;
    const int64_t slot = t < a.T ? a.slots[t] : -1;
    const bool row = slot >= 0 && slot < a.places;           // the same for a row's lanes
    const bool live = row && j * 8 < a.D;
    Raw<DT> raw[2] = {};
    if (live)
#pragma unroll
        for (int w = 0; w < 2; ++w) raw[w] = load8<DT>(a.x[w], t * a.ld[w] + (int64_t)h * a.D + j * 8);
    const int64_t at = row ? row_of(a, slot, h) : 0;
    constexpr int QM = BITS == 8 ? 127 : 7;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint32_t bits = largest_of<LPR>(largest8<DT>(raw[w]));
        const float m = DT == 0 ? __builtin_bit_cast(float, bits) : DT == 1 ? h2f((uint16_t)bits) : bf2f((uint16_t)bits);
        float x[8];
        widen8<DT>(raw[w], x);
        float y[8];                                          // 4 bits: even values, then odd ones
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[BITS == 8 ? e : 2 * (e & 3) + (e >> 2)];
        float s = divide_by<QM>(m);
        u32x2 c = u32x2{0u, 0u};
        if (m >= 0x1p-107f && m < __builtin_inff()) {
            // (the reciprocal's own step more than codes8_dyn counts with is 2^-17 of the sum, far inside its margin)
            c = codes8_dyn(y, s, __builtin_amdgcn_rcpf(s));
        } else if (m < 0x1p-107f) {                          // the reciprocal overflows or loses digits, and
            s = m / (float)QM;                               // a scale of few digits lets quotients pass q_max
            if (s == 0.0f) s = 1.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                c[e >> 2] |= ((uint32_t)(int)__builtin_amdgcn_fmed3f(__builtin_rintf(y[e] / s), -(float)QM, (float)QM) & 0xffu)
                             << (8 * (e & 3));
        } else {
            s = __builtin_nanf("");
        }
        if (live) {
            if constexpr (BITS == 8) *reinterpret_cast<u32x2*>(a.codes[w] + at * a.D + j * 8) = c;
            else *reinterpret_cast<uint32_t*>(a.codes[w] + at * (a.D / 2) + j * 4) =
                (c[0] & 0x0f0f0f0fu) | ((c[1] & 0x0f0f0f0fu) << 4);
        }
        if (row && j == 0) a.scales[w][at] = s;
    }
}

// 16411 tokens of 8 heads of 128 out of 8 bits, which the write before left in the cache:
// 17 us, 6 TB/s; 24 contexts of up to 8192 out of 4 bits: 132 us, 4.9 TB/s.
// NT: codes and outputs with the non-temporal hint, for outputs that pass the 256 MB
// cache (8 heads of 128, 8 bits, fp16: 65536 tokens and a kernel that reads them 137
// us against 142; 16384 tokens, whose outputs that kernel finds in the cache, 39
// against 33).
template <int DT, int BITS, int LPR, bool NT>
__global__ __launch_bounds__(256) void k_kv_read(KvArgs a) {
    const int j = threadIdx.x % LPR;
    const int64_t t = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int h = blockIdx.y;
    if (t >= a.T || j * 8 >= a.D) return;
    const int64_t slot = a.slots[t];
    const bool row = slot >= 0 && slot < a.places;
    const int64_t at = row ? row_of(a, slot, h) : 0;
    u32x2 c[2] = {u32x2{0u, 0u}, u32x2{0u, 0u}};
    float s[2] = {0.0f, 0.0f};
    if (row) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if constexpr (BITS == 8) c[w] = load<NT>(reinterpret_cast<const u32x2*>(a.codes[w] + at * a.D + j * 8));
            else c[w][0] = load<NT>(reinterpret_cast<const uint32_t*>(a.codes[w] + at * (a.D / 2) + j * 4));
            s[w] = a.scales[w][at];
        }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int q = BITS == 8 ? (int)(int8_t)(c[w][e >> 2] >> (8 * (e & 3))) : (int)(c[w][0] << (28 - 4 * e)) >> 28;
            x[e] = (float)q * s[w];
            asm("" : "+v"(x[e]));                            // (or product and rounding fuse for fp16, and for it alone)
        }
        store8<DT, NT>(a.y[w], (t * a.heads + h) * a.D + j * 8, x);
    }
}

template <bool WRITE, int DT, int BITS>
hipError_t run_kv(const KvArgs& a, hipStream_t st) {
    const int lpr = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
    const dim3 g((unsigned)((a.T + 256 / lpr - 1) / (256 / lpr)), (unsigned)a.heads);
    const bool large = 2 * a.T * a.heads * a.D * (DT == 0 ? 4 : 2) >= ((int64_t)256 << 20);
#define QA_KV(L)                                                                             \
    if constexpr (WRITE) hipLaunchKernelGGL((k_kv_write<DT, BITS, L>), g, dim3(256), 0, st, a); \
    else if (large) hipLaunchKernelGGL((k_kv_read<DT, BITS, L, true>), g, dim3(256), 0, st, a); \
    else hipLaunchKernelGGL((k_kv_read<DT, BITS, L, false>), g, dim3(256), 0, st, a);
    if (lpr == 8) { QA_KV(8) }
    else if (lpr == 16) { QA_KV(16) }
    else { QA_KV(32) }
#undef QA_KV
    return hipGetLastError();
}

template <bool WRITE>
hipError_t run_kv(const KvArgs& a, int dtype, int bits, hipStream_t st) {
    if (bits == 8) {
        if (dtype == 0) return run_kv<WRITE, 0, 8>(a, st);
        return dtype == 1 ? run_kv<WRITE, 1, 8>(a, st) : run_kv<WRITE, 2, 8>(a, st);
    }
    if (dtype == 0) return run_kv<WRITE, 0, 4>(a, st);
    return dtype == 1 ? run_kv<WRITE, 1, 4>(a, st) : run_kv<WRITE, 2, 4>(a, st);
}

KvArgs kv_args(const int64_t* slots, int64_t T, const KvCache& c) {
    KvArgs a{};
    a.slots = slots; a.T = T;
    a.codes[0] = static_cast<uint8_t*>(c.k_codes); a.codes[1] = static_cast<uint8_t*>(c.v_codes);
    a.scales[0] = c.k_scales; a.scales[1] = c.v_scales;
    a.places = c.pages << c.shift; a.heads = c.heads; a.D = c.D; a.shift = c.shift;
    return a;
}

}  // namespace

hipError_t launch_kv_write(const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype, int64_t T,
                           const int64_t* slots, const KvCache& c, hipStream_t st) {
    KvArgs a = kv_args(slots, T, c);
    a.x[0] = k; a.x[1] = v; a.ld[0] = ldk; a.ld[1] = ldv;
    return run_kv<true>(a, dtype, c.bits, st);
}

hipError_t launch_kv_read(const int64_t* slots, int64_t T, const KvCache& c, void* k, void* v, int dtype,
                          hipStream_t st) {
    KvArgs a = kv_args(slots, T, c);
    a.y[0] = k; a.y[1] = v;
    return run_kv<false>(a, dtype, c.bits, st);
}

}  // namespace qa
