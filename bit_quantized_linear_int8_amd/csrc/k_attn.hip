// k_attn.hip -- attention of one new token per sequence over a paged cache of
// int8 or int4 keys and values, on gfx950.
//
//   x_t = scale s_k[t] sum_d q_d k[t][d],   p_t = exp(x_t - m)
//   o_d = sum_t p_t s_v[t] v[t][d] / sum_t p_t,   lse = m + log sum_t p_t
//
// over the tokens t of a sequence (inside its window, on a page that the cache
// has).  The heads that share a key head are the 16 columns of one MFMA tile.
//
// A wave takes 32 tokens at a time through a stage of LDS of its own (no barrier in
// the loop), filled by direct global -> LDS loads of whole lines while the tile before
// is worked on in registers:
//   - keys are the rows of A of an int8 product: lane (m, c) takes 16-byte pieces
//     c, c + 4, ... of token m (and 16 + m), as they are (int4: the nibbles in the
//     upper halves of bytes, 16 times the codes);
//   - x comes out with four consecutive tokens of column g = lane % 16 in each
//     lane, which is where p has to be as the operand B of the second product;
//   - values are A of the second product, transposed: lane (m, c) takes the
//     16th part m of the D values of tokens 4 c + j and 16 + 4 c + j, and
//     the codes of two tokens are put side by side in registers.
// Lanes exchange nothing inside the loop.  (Keys straight into the operand's
// registers have every lane of a load in a line of its own: 460 accesses of the L1
// for a tile's 68 lines, which bounded the kernel at 4.4 TB/s.)
//
// Queries enter as whole numbers next to the head's largest, in balanced digits of
// base 256, so that the scores of integers are exact: an int8 product for each digit
// costs less than to convert every key's codes to fp16.  fp32 queries have 30 bits and a
// sign, four digits: what is left out, 2^-30 of the largest times sum |k|, is below the
// roundings of fp32 sums of their products.  fp16 and bf16 ones have 22 and a sign, three
// digits: values down to 2^-11 and 2^-14 of the largest are as they were, smaller
// ones within 2^-22 of it, 2^10 times less than the half step that the largest itself
// came with.  (A fourth digit for them: 64 ragged sequences of up to 8192 105.1 -> 106.5 us,
// with heads of 256 114 -> 124, windows of 1000 over 32 heads of 64 25.5 -> 28.2.)  Values'
// codes become fp16 (times 2^-10) exactly: the byte or nibble with its sign bit
// flipped is an fp16 number below the normal ones, and a fused multiply-add
// scales it and takes the flip away.  p s_v enters as two fp16 numbers with a power
// of two per head: 2^-22 of the value, and 2^-37 of the wave's largest, below which
// fp16 has no numbers; one fp16 number would add an error as large as the rounding
// of an fp16 output.  Sums are fp32.
//
// The reference m of the exponentials and the power of two of p s_v follow their
// running maxima lazily: only when a tile passes one by 2^16 (or fp16's largest
// number) are they taken anew, with the lanes' exchange that this needs; 2^16 leaves
// the sums far inside fp32's range.
//
// The four waves of a block take tiles in turn and are joined through LDS.  Where
// there are few sequences and heads for their length, the work of all of them, in units of 128 tokens
// of a head, is one line that the blocks that fit the card share evenly, whatever the
// lengths are (a block finds its place by a sum over them); a head that reaches over
// several blocks is joined by k_attn_join.  (Equal chunks of each sequence leave
// blocks of unequal size: half the card's waves were idle with ragged lengths.)
//
// What bounds it: 64 ragged sequences of up to 8192 (8 key heads of 128, 4 queries each,
// 8 bits, 580 MB) take 98 to 103 us, 5.6 to 5.9 TB/s, and 7 the join: the memory (the loads alone take
// no less).  4 of up to 131072 in 4 bits with 8 queries each take 86 to 92, 4.9 to 5.3 TB/s:
// the loads alone and the arithmetic alone (vector instructions busy for 62% of
// the time, most of them values' codes made fp16) are about 85 each.  A single sequence of 4096 is
// latency: 8.2 to 9.2 and 4.3 to 4.8 for the join.  Many short ones, where no block shares, are their
// bytes and 7 us of dependent loads (length, table, codes) at the beginning and the joint of
// the waves at the end.
#include "qa_device.hpp"
#include "qa_launch.hpp"

namespace qa {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

struct AttnArgs {
    const void* q;             // [B][H][D], token stride ldq
    int64_t ldq;
    const uint8_t* kc;
    const float* ks;
    const uint8_t* vc;
    const float* vs;
    const int32_t* table;      // [B][width], row stride ldt: pages of a sequence
    int64_t ldt;
    const int32_t* lengths;    // [B]
    int32_t H, heads, group, gtiles, D, shift, pages, qdt;
    int32_t max_len;           // lengths past it (or past the table) count as it
    int32_t window;            // 0: none
    int32_t B, share;          // parts that the work of a tile of heads is shared in; 0: a block to each sequence and tile
    float scale2;              // scale log2(e)
    void* out;                 // [B][H][D]
    int32_t dt;
    float* lse;                // [B][H] or nullptr
    float* part;               // parts of sequences, [(share + B) heads gtiles][16][D]
    float* plse;               // and their log-sum-exp, base 2, [..][16]
    int32_t* before;           // [B + 1] units of all the sequences before one
};

constexpr float kLow = -3.0e38f;           // the reference before any token
constexpr float kLn2 = 0.693147180559945309f;

// Weights p s_v times 2^-ex: taken anew, the largest lies in [2^12, 2^13); up to kMostWeight, fp16's largest number,
// they may grow before that.  Half a step of fp16's smallest numbers is then at most 2^-37 of the largest weight.  (With
// a largest below 1 the weights of 32768 tokens 17.5 nats below one were lost, 2^-24 being the smallest number.  A
// largest of 2^13 or more has to be taken anew more often: 64 ragged sequences of up to 8192 in 8 bits take 106.4 us
// against 105.3, 4 of up to 131072 in 4 bits with fp32 queries 96.3 against 95.0; of 2^11 or more, 105.4 and 94.9.)
constexpr int kWeightBits = 13;
constexpr float kMostWeight = 65504.0f;
constexpr float kLeastExp = -126.0f;       // of 2^-ex in fp32

__device__ __forceinline__ v2h pk(uint32_t u) { return __builtin_bit_cast(v2h, u); }
__device__ __forceinline__ uint32_t up(v2h h) { return __builtin_bit_cast(uint32_t, h); }

// Pairs of codes as fp16 times 2^-10, from their bytes plus 128 in the low bytes of
// each half: u 2^-24 as it stands, times 2^14, less 128 2^-10.
__device__ __forceinline__ uint32_t byte_pair(uint32_t u) {
    return up(__builtin_elementwise_fma(pk(u), v2h{(_Float16)16384, (_Float16)16384},
                                        v2h{(_Float16)-0.125, (_Float16)-0.125}));
}
// The same from nibbles plus 8 in bits 0..3, or 4..7, of each half of y.
__device__ __forceinline__ uint32_t nib_pair0(uint32_t y) {
    return up(__builtin_elementwise_fma(pk(y & 0x000f000fu), v2h{(_Float16)16384, (_Float16)16384},
                                        v2h{(_Float16)-0.0078125, (_Float16)-0.0078125}));
}
__device__ __forceinline__ uint32_t nib_pair1(uint32_t y) {
    return up(__builtin_elementwise_fma(pk(y & 0x00f000f0u), v2h{(_Float16)1024, (_Float16)1024},
                                        v2h{(_Float16)-0.0078125, (_Float16)-0.0078125}));
}

// w less the fp16 number in the low (high) half of h, in one instruction (the compiler makes two).
__device__ __forceinline__ float less_low(float w, uint32_t h) {
    float r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r) : "v"(h), "v"(w));
    return r;
}
__device__ __forceinline__ float less_high(float w, uint32_t h) {
    float r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r) : "v"(h), "v"(w));
    return r;
}

// Byte K of four words, side by side.
template <int K>
__device__ __forceinline__ uint32_t bytes4(const uint32_t (&n)[4]) {
    constexpr uint32_t two = 0x0c0c0000u | (uint32_t)K | ((uint32_t)(4 + K) << 8);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(n[3], n[2], two), __builtin_amdgcn_perm(n[1], n[0], two), 0x05040100u);
}

// Query j of a 16-byte piece: fp32, fp16 or bf16.
template <bool F32, bool F16>
__device__ __forceinline__ float query(const u32x4& u, int j) {
    if constexpr (F32) return __builtin_bit_cast(v4f, u)[j];
    const uint32_t v = u[j >> 1] >> (16 * (j & 1));
    return F16 ? h2f((uint16_t)v) : __builtin_bit_cast(float, v << 16);
}

// Four consecutive outputs of type dt at p[at].
__device__ __forceinline__ void store_quad(void* p, int64_t at, int dt, v4f v) {
    if (dt == 0) {
        *reinterpret_cast<v4f*>(static_cast<float*>(p) + at) = v;
        return;
    }
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t lo = dt == 1 ? f2h(v[2 * j]) : f2bf(v[2 * j]), hi = dt == 1 ? f2h(v[2 * j + 1]) : f2bf(v[2 * j + 1]);
        w[j] = lo | (hi << 16);
    }
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + at) = u32x2{w[0], w[1]};
}

// First and last tokens that a sequence's query sees, and the place that its
// chunks are counted from.
__device__ __forceinline__ void span_of(const AttnArgs& a, int b, int& first, int& end, int& from) {
    int n = a.lengths[b];
    end = n < 0 ? 0 : (n > a.max_len ? a.max_len : n);
    first = a.window > 0 && end > a.window ? end - a.window : 0;
    from = first & ~31;
}
constexpr int kUnit = 128;
// Units of a sequence per head.
__device__ __forceinline__ int units_of(int end, int from) { return (end - from + kUnit - 1) / kUnit; }

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void glb_void;

// Sixteen bytes from each lane's offset, and four from each lane's address, to LDS, lane
// after lane.  Codes come with the non-temporal hint: between two steps of a layer the
// other layers pass through the caches, so nothing is there to be found again (64 ragged
// sequences up to 8192: 107 us of the call against 121; where all of it fits the 256 MB
// cache and is read again at once, 27.5 against 26.6).
__device__ __forceinline__ void load_lds16(rsrc_t r, uint32_t off, void* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, 0, 0, 2);
}
__device__ __forceinline__ void load_lds4(const void* p, void* lds) {
    __builtin_amdgcn_global_load_lds((glb_void*)p, (lds_void*)lds, 4, 0, 0);
}

// s_waitcnt immediate waiting for vmcnt <= n only (gfx9 encoding)
constexpr int vmcnt_only(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// Blocks on a CU, by D rounded up: as many as the registers hold in the loop over tiles (what they do not hold beside it,
// for heads of 256 in int8 and with fp32 queries, and of 128 in int4 with them, is put aside before
// the loop and taken up after it), but for 64 with fp32 queries (33 windows of 1000 over 32 heads: 29.3 us of the call
// with three, 29.8 with four) and for 128 in int8, where two bring long sequences in faster than three (64
// ragged ones up to 8192: 105.6 us against 113; 200 of up to 200 tokens 27.3 against 23.6; 4 of up to
// 131072 in int4: 89.6 with three, 93.3 with two).  At 256 one block of two stages took 48.3
// us for 78 sequences of 21 tokens and 19 heads, two of one stage 30.6.  A second stage of
// LDS for each wave was no faster in the others either (107.4 and 94.2): a stage is read into
// registers at once and filled again, so that two tiles of each wave are under way as it is.
constexpr int blocks_on_cu(int DP, int BITS, bool F32) { return DP == 64 ? (F32 ? 3 : 4) : DP == 128 && BITS == 4 ? 3 : 2; }

__device__ __forceinline__ float max4(v4f v) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); }
// Of magnitudes: weights have the sign of their value scale.
__device__ __forceinline__ float most4(v4f v) {
    return fmaxf(fmaxf(__builtin_fabsf(v[0]), __builtin_fabsf(v[1])), fmaxf(__builtin_fabsf(v[2]), __builtin_fabsf(v[3])));
}

}  // namespace

// DP: D rounded up to 64, 128 or 256 (what lies behind D meets queries of 0, or is
// not stored).  F32: fp32 queries.
template <int BITS, int DP, bool F32>
__global__ __launch_bounds__(256, blocks_on_cu(DP, BITS, F32)) void k_attn_decode(AttnArgs a) {
    constexpr int CC = BITS == 8 || DP == 64 ? 16 : 32;      // codes of a lane's piece of a key
    constexpr int NS = DP / (4 * CC);                        // pieces of a lane
    constexpr int PB = CC * BITS / 8;                        // bytes of a piece
    constexpr int NM = DP / 64;                              // MFMA steps of a key
    constexpr int ND = F32 ? 4 : 3, QB = F32 ? 30 : 22;      // a query's digits, and its bits
    constexpr int VN = DP / 16;                              // values of a lane per token
    constexpr int VB = VN * BITS / 8;                        // their bytes
    constexpr int VW = VB < 4 ? 1 : VB / 4;                  // their words
    constexpr int DPB = DP * BITS / 8, NCH = DPB / 16;       // a row in LDS, its chunks
    constexpr int INS = 16 * DPB < 1024 ? 1 : 16 * DPB / 1024;    // loads of 16 rows
    constexpr int HALF = INS * 1024;
    constexpr int SB = 4 * HALF + 256;                       // a stage
    constexpr int RED = 4 * 16 * (DP / 4 + 1) * 16;
    __shared__ __attribute__((aligned(16))) uint8_t smem[4 * SB > RED ? 4 * SB : RED];
    auto swz = [](int r) { return (NCH <= 8 ? r / (8 / (NCH <= 8 ? NCH : 8)) : r) & (NCH - 1); };
    __shared__ float st_m[4][16], st_l[4][16], st_e[4][16];
    __shared__ int power[16];
    __shared__ int plan[6];

    const int lane = threadIdx.x & 63, wave = wave_id();
    const int m16 = lane & 15, c4 = lane >> 4;
    const int HG = a.heads * a.gtiles;                       // tiles of heads of a sequence
    int b = 0, hg = 0, k0 = 0, left = 0;                     // the next unit's sequence, tile, place; units to do
    if (a.share) {
        // sums of the units over the sequences, four to a thread, and where the block's share begins
        int n[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = 4 * threadIdx.x + j;
            int first, end, from;
            n[j] = 0;
            if (i < a.B) {
                span_of(a, i, first, end, from);
                n[j] = units_of(end, from);
            }
            sum += n[j];
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o, QA_WAVE);
            if (lane >= o) upto += v;
        }
        if (lane == 63) plan[wave] = upto;
        __syncthreads();
        int total = 0, pre = upto - sum;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) pre += plan[w];
            total += plan[w];
        }
        const int share = total < a.share ? total : a.share;
        const int part = blockIdx.x / (uint32_t)HG;
        hg = blockIdx.x - (uint32_t)part * HG;
        if (blockIdx.x == 0)
#pragma unroll
            for (int j = 0, at = pre; j < 4; ++j) {
                const int i = 4 * threadIdx.x + j;
                if (i < a.B) a.before[i] = at;
                at += n[j];
                if (i == a.B - 1) a.before[a.B] = at;
            }
        if (part >= share) return;
        const int each = total / share, more = total - each * share;    // the first `more` shares have one unit more
        const int u0 = part * each + min(part, more), u1 = u0 + each + (part < more ? 1 : 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (pre <= u0 && u0 < pre + n[j]) plan[4] = 4 * threadIdx.x + j, plan[5] = u0 - pre;
            pre += n[j];
        }
        __syncthreads();
        b = __builtin_amdgcn_readfirstlane(plan[4]);
        k0 = __builtin_amdgcn_readfirstlane(plan[5]);
        left = u1 - u0;
    } else {
        b = blockIdx.x / (uint32_t)HG;
        hg = blockIdx.x - (uint32_t)b * HG;
        int first, end, from;
        span_of(a, b, first, end, from);
        left = units_of(end, from);
        if (left == 0) {                                     // no token to see
            const int h = hg / a.gtiles, gt = hg - h * a.gtiles;
            const int heads_here = a.group - gt * 16 < 16 ? a.group - gt * 16 : 16;
            const int64_t row0 = (int64_t)b * a.H + h * a.group + gt * 16;
            if ((int)threadIdx.x < heads_here && a.lse) a.lse[row0 + threadIdx.x] = -__builtin_inff();
            for (int i = threadIdx.x; i < heads_here * a.D / 4; i += 256)
                store_quad(a.out, row0 * a.D + 4 * i, a.dt, v4f{0.0f, 0.0f, 0.0f, 0.0f});
            return;
        }
    }

    while (left > 0) {
    int first, end, from;
    span_of(a, b, first, end, from);
    const int n1 = units_of(end, from);
    if (n1 == 0) {                                           // (its rows are written by the join)
        ++b;
        continue;
    }
    const int k1 = n1 - k0 < left ? n1 : k0 + left;
    const bool whole = k0 == 0 && k1 == n1;
    const int64_t slot = (int64_t)b * HG + blockIdx.x;       // of a part: grows with the sequence and with the block's share
    const int h = hg / a.gtiles, gt = hg - h * a.gtiles;
    const int g = gt * 16 + m16;                             // the lane's head within the group
    const int heads_here = a.group - gt * 16 < 16 ? a.group - gt * 16 : 16;
    const int64_t row0 = (int64_t)b * a.H + h * a.group + gt * 16;    // the first row of the output
    const int lo = from + k0 * kUnit;
    const int hi = end - from <= k1 * kUnit ? end : from + k1 * kUnit;

    const int32_t* tab = a.table + (int64_t)b * a.ldt;
    const int page = 1 << a.shift;
    const uint32_t RB = (uint32_t)a.D * BITS / 8;            // bytes of a row
    // Pages of the wave's tiles: lane 2 i + u of `ent` holds the table's entry for 16 tokens u of tile i of 32.
    auto entries = [&](int t) __attribute__((always_inline)) {
        const int64_t at = (int64_t)t + 128 * (lane >> 1) + 16 * (lane & 1);
        return tab[(int)(at < a.max_len ? at : a.max_len - 1) >> a.shift];
    };
    // the page of the 16 tokens from t, or -1 (past the end, or not one of the cache's)
    auto page_of = [&](int t, int p) __attribute__((always_inline)) {
        return t < hi && (uint32_t)p < (uint32_t)a.pages ? p : -1;
    };
    // the rows of this head from token t on in page p: a descriptor that ends with the page (p < 0: of nothing)
    auto rows_of = [&](const uint8_t* x, int t, int p) __attribute__((always_inline)) {
        const uint32_t at = (uint32_t)t & (uint32_t)(page - 1);
        const int64_t row = (((int64_t)(p < 0 ? 0 : p) * a.heads + h) << a.shift) + at;
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(x + row * RB), (short)0,
                                                 p < 0 ? 0 : (int)(((uint32_t)page - at) * RB), 0x00020000);
    };

    // The stage: keys and values of two times 16 tokens, rows of DPB bytes whose 16-byte chunk c is at c ^ swz(row), so
    // that reads of 16 rows meet all banks; behind them 32 scales of keys and 32 of values.
    uint8_t* const mine = smem + wave * SB;
    uint32_t src[INS];                                       // a lane's part of a load of 16 rows
#pragma unroll
    for (int n = 0; n < INS; ++n) {
        const int P = n * 64 + lane, rr = P / NCH, c = (P % NCH) ^ swz(rr);
        src[n] = rr < 16 && (uint32_t)(16 * c) < RB ? (uint32_t)rr * RB + 16 * c : kOOB;
    }
    const float* const scales_at = (lane < 32 ? a.ks : a.vs) + (((int64_t)h << a.shift) + m16);
    auto fill = [&](int t, int q0, int q1) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const rsrc_t rk = rows_of(a.kc, t + 16 * u, u ? q1 : q0), rv = rows_of(a.vc, t + 16 * u, u ? q1 : q0);
#pragma unroll
            for (int n = 0; n < INS; ++n) {
                load_lds16(rk, src[n], mine + u * HALF + n * 1024);
                load_lds16(rv, src[n], mine + (2 + u) * HALF + n * 1024);
            }
        }
        // scales: 16 tokens of u to 16 lanes, keys' and then values' (of page 0 where there is none: not looked at)
        const int64_t r0 = (((int64_t)(q0 < 0 ? 0 : q0) * a.heads) << a.shift) + ((uint32_t)t & (uint32_t)(page - 1));
        const int64_t r1 = (((int64_t)(q1 < 0 ? 0 : q1) * a.heads) << a.shift) + ((uint32_t)(t + 16) & (uint32_t)(page - 1));
        load_lds4(scales_at + (lane & 16 ? r1 : r0), mine + 4 * HALF);
    };

    // the wave's first tile, and the queries while it comes
    int t0 = lo + 32 * wave, it = 0;
    int ent = entries(t0), ent2 = entries(t0 + 32 * 128);
    int p0 = page_of(t0, __builtin_amdgcn_readlane(ent, 0)), p1 = page_of(t0 + 16, __builtin_amdgcn_readlane(ent, 1));
    fill(t0, p0, p1);
    v4i qd[ND][NM];                                          // digits of 1, 256, 65536, 2^24
    float qscale;
    {
        constexpr uint32_t EL = F32 ? 4 : 2;                 // bytes of a query value
        const rsrc_t rq = make_rsrc(static_cast<const uint8_t*>(a.q) + ((int64_t)b * a.ldq + (int64_t)h * a.group * a.D) * EL,
                                    (int64_t)a.group * a.D * EL);
        // 16 values to an MFMA step: int8 piece s is step s; an int4 piece of 32 codes is two,
        // its even and its odd codes, one of 16 is its even and then its odd codes
        float x[NS][CC];
        uint32_t bits = 0;                                   // of magnitudes: they order like them, infinities and NaNs above all
        constexpr int V = 16 / EL;                           // values of a load
        u32x4 raw[NS][CC / V];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int f = 0; f < CC / V; ++f) {
                const int d = (c4 + 4 * s) * CC + V * f;
                raw[s][f] = bload16(rq, d < a.D ? (uint32_t)(g * a.D + d) * EL : kOOB);    // (heads past the group: zeros)
            }
        if (a.qdt == 1) {
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int k = 0; k < CC; ++k) x[s][k] = query<F32, true>(raw[s][k / V], k % V);
        } else {
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int k = 0; k < CC; ++k) x[s][k] = query<F32, false>(raw[s][k / V], k % V);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int k = 0; k < CC; ++k) bits = max(bits, __builtin_bit_cast(uint32_t, x[s][k]) & 0x7fffffffu);
        bits = max(bits, (uint32_t)__shfl_xor((int)bits, 16, QA_WAVE));
        bits = max(bits, (uint32_t)__shfl_xor((int)bits, 32, QA_WAVE));
        // times 2^e the head's largest is in [2^(QB - 1), 2^QB)
        const bool fine = bits < 0x7f800000u;
        const int e = bits != 0 && fine ? QB - __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, bits)) : 0;
        // (of queries below 2^-89 in all qscale is subnormal and loses digits; scores show them beside key scales above 2^60)
        qscale = fine ? __builtin_ldexpf(a.scale2, -e - (BITS == 8 ? 0 : 4)) : __builtin_nanf("");
        const float f1 = __builtin_ldexpf(1.0f, e / 2), f2 = __builtin_ldexpf(1.0f, e - e / 2);
#pragma unroll
        for (int i = 0; i < NM; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                // A digit is a byte of the whole number, or of it with what carries into the next digit: n,
                // n + 128, n + 128 + 2^15, n + 128 + 2^15 + 2^23.  (22 bits: beside 3 2^22 the number is in the
                // low bits of the sum.)
                uint32_t n[4], n1[4], n2[4], n3[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // value at byte k of step i
                    const int k = 4 * w + j;
                    float y;
                    if constexpr (BITS == 8) y = x[i][k];
                    else if constexpr (CC == 32) y = x[i / 2][2 * k + (i & 1)];
                    else y = x[i][k < 8 ? 2 * k : 2 * (k - 8) + 1];
                    if constexpr (ND == 4) n[j] = (uint32_t)(int)__builtin_rintf(y * f1 * f2);
                    else n[j] = __builtin_bit_cast(uint32_t, __builtin_fmaf(y * f1, f2, 12582912.0f));
                    n1[j] = n[j] + (ND == 4 ? 128u : 128u - 0x4b400000u);
                    n2[j] = n1[j] + 0x8000u;
                    n3[j] = n2[j] + 0x800000u;
                }
                qd[0][i][w] = (int)bytes4<0>(n);
                qd[1][i][w] = (int)bytes4<1>(n1);
                qd[2][i][w] = (int)bytes4<2>(n2);
                if constexpr (ND == 4) qd[3][i][w] = (int)bytes4<3>(n3);
            }
    }

    v4f acc[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    float m = kLow, l = 0.0f, ex = kLeastExp, r = 0.0f;       // r = 2^-ex, the factor of p s_v

    // a lane's places in a stage
    uint32_t ak[NS], av[4];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int byte = (c4 + 4 * i) * PB;
        ak[i] = m16 * DPB + (((byte >> 4) ^ swz(m16)) << 4) + (byte & 15);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int rr = 4 * c4 + j, byte = m16 * VB;
        av[j] = 2 * HALF + rr * DPB + (((byte >> 4) ^ swz(rr)) << 4) + (byte & 15);
    }
    while (t0 < hi) {
        // the stage into registers
        __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
        asm volatile("" ::: "memory");
        u32x4 kq[2][NS];
        uint32_t vq[8][VW];
        v4f ks[2], vs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const uint8_t* q = mine + u * HALF + ak[i];
                if constexpr (PB == 16) kq[u][i] = *reinterpret_cast<const u32x4*>(q);
                else {
                    const u32x2 w = *reinterpret_cast<const u32x2*>(q);
                    kq[u][i] = u32x4{w[0], w[1], 0u, 0u};
                }
            }
            ks[u] = *reinterpret_cast<const v4f*>(mine + 4 * HALF + 64 * u + 16 * c4);
            vs[u] = *reinterpret_cast<const v4f*>(mine + 4 * HALF + 128 + 64 * u + 16 * c4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint8_t* q = mine + u * HALF + av[j];
                uint32_t* o = vq[4 * u + j];
                if constexpr (VB == 2) o[0] = *reinterpret_cast<const uint16_t*>(q);
                else if constexpr (VB == 4) o[0] = *reinterpret_cast<const uint32_t*>(q);
                else if constexpr (VB == 8) {
                    const u32x2 w = *reinterpret_cast<const u32x2*>(q);
                    o[0] = w[0], o[1] = w[1];
                } else {
                    const u32x4 w = *reinterpret_cast<const u32x4*>(q);
                    o[0] = w[0], o[1] = w[1], o[2] = w[2], o[3] = w[3];
                }
            }
        }
        // and the next tile into it, once it is read
        __builtin_amdgcn_s_waitcnt(0xC07F);                  // lgkmcnt(0)
        asm volatile("" ::: "memory");
        const int q0 = p0, q1 = p1;                          // this tile's pages
        {
            const int at = it + 1, tn = t0 + 128;
            if ((at & 31) == 0) {                            // the next 32 tiles' entries
                ent = ent2;
                ent2 = entries(tn + 32 * 128);
            }
            p0 = page_of(tn, __builtin_amdgcn_readlane(ent, 2 * (at & 31)));
            p1 = page_of(tn + 16, __builtin_amdgcn_readlane(ent, 2 * (at & 31) + 1));
            fill(tn, p0, p1);
        }

        // scores as exact integers / 2^k, with their factors
        v4f f[2], fs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            v4i kf[NM];
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                if constexpr (BITS == 8) kf[i] = __builtin_bit_cast(v4i, kq[u][i]);
                else if constexpr (CC == 32) {
                    const u32x4 w = kq[u][i / 2];
                    kf[i] = __builtin_bit_cast(v4i, (i & 1 ? w : w << 4) & 0xf0f0f0f0u);
                } else {
                    const u32x4 w = kq[u][i];
                    kf[i] = __builtin_bit_cast(v4i, u32x4{w[0] << 4, w[1] << 4, w[0], w[1]} & 0xf0f0f0f0u);
                }
            }
            // Two digits to a sum, the upper one's products times 256 under the lower one's: |s| <= 256 * 128 * 128 of a
            // digit, and the uppermost is at most 65: both sums fit.  (Sums of their own for each digit take
            // registers: heads of 64 with fp32 queries, windows of 1000, 33.0 us against 29.3.)
            v4i low = v4i{0, 0, 0, 0}, high = low;
            auto add = [&](int d, v4i s) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < NM; ++i) s = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[i], qd[d][i], s, 0, 0, 0);
                return s;
            };
            low = add(1, low);
            high = add(ND - 1, high);
            low = add(0, low << 8);
            if constexpr (ND == 4) high = add(2, high << 8);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[u][e] = __builtin_fmaf((float)high[e], 65536.0f, (float)low[e]);
                fs[u][e] = ks[u][e] * qscale;
            }
        }

        v4f sv[2] = {vs[0], vs[1]};
        if (t0 < first || t0 + 32 > hi || q0 < 0 || q1 < 0) {    // tokens that are not seen
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = t0 + 16 * u + 4 * c4 + e;
                    const bool live = t >= first && t < hi && (u ? q1 : q0) >= 0;
                    f[u][e] = live ? f[u][e] : -__builtin_inff();
                    fs[u][e] = live ? fs[u][e] : 1.0f;
                    sv[u][e] = live ? sv[u][e] : 0.0f;
                }
        }
        v4f p[2], w[2];
        auto weigh = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[u][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(f[u][e], fs[u][e], -m));
                    w[u][e] = p[u][e] * sv[u][e] * r;
                }
        };
        weigh();
        if (__any(fmaxf(max4(p[0]), max4(p[1])) > 65536.0f || fmaxf(most4(w[0]), most4(w[1])) > kMostWeight)) {
            // New references from this tile's maxima and the old ones, whole: the factors are powers of two, and the
            // exponent of the weights falls by as much as m grows.
            float tm = -__builtin_inff(), wm = 0.0f;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) tm = fmaxf(tm, f[u][e] * fs[u][e]);
            tm = fmaxf(tm, __shfl_xor(tm, 16, QA_WAVE));
            tm = fmaxf(tm, __shfl_xor(tm, 32, QA_WAVE));
            const float mn = fmaxf(m, __builtin_ceilf(tm));
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    wm = fmaxf(wm, __builtin_fabsf(__builtin_amdgcn_exp2f(__builtin_fmaf(f[u][e], fs[u][e], -mn)) * sv[u][e]));
            wm = fmaxf(wm, __shfl_xor(wm, 16, QA_WAVE));
            wm = fmaxf(wm, __shfl_xor(wm, 32, QA_WAVE));
            const float down = m - mn;
            // (a tile without weight, whose frexp exponent is 0, raises nothing)
            const float ew = wm > 0.0f ? (float)(__builtin_amdgcn_frexp_expf(wm) - kWeightBits) : kLeastExp;
            const float en = fmaxf(kLeastExp, fmaxf(ex + down, ew));
            l *= __builtin_amdgcn_exp2f(down);
            const float z = __builtin_ldexpf(__builtin_amdgcn_exp2f(down), (int)fmaxf(ex - en, -300.0f));
#pragma unroll
            for (int i = 0; i < VN; ++i) acc[i] *= z;
            m = mn;
            ex = en;
            r = __builtin_amdgcn_exp2f(-en);
            weigh();
        }
        u32x4 hi4, lo4;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float w0 = w[u][2 * e], w1 = w[u][2 * e + 1];
                l += p[u][2 * e] + p[u][2 * e + 1];
                const uint32_t both = up(v2h{(_Float16)w0, (_Float16)w1});
                hi4[2 * u + e] = both;
                lo4[2 * u + e] = up(v2h{(_Float16)less_low(w0, both), (_Float16)less_high(w1, both)});
            }
        const v8h ph = __builtin_bit_cast(v8h, hi4), pl = __builtin_bit_cast(v8h, lo4);
        auto pv = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) __attribute__((always_inline)) {
            const v8h vf = __builtin_bit_cast(v8h, u32x4{a0, a1, a2, a3});
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, ph, acc[i], 0, 0, 0);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pl, acc[i], 0, 0, 0);
        };
        if constexpr (BITS == 8) {
#pragma unroll
            for (int q = 0; q < VW; ++q) {
                uint32_t y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = vq[j][q] ^ 0x80808080u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t sel = 0x0c000c00u | (uint32_t)i | ((uint32_t)(4 + i) << 16);
                    pv(4 * q + i, byte_pair(__builtin_amdgcn_perm(y[1], y[0], sel)),
                       byte_pair(__builtin_amdgcn_perm(y[3], y[2], sel)), byte_pair(__builtin_amdgcn_perm(y[5], y[4], sel)),
                       byte_pair(__builtin_amdgcn_perm(y[7], y[6], sel)));
                }
            }
        } else {
#pragma unroll
            for (int q = 0; q < VN / 4; ++q) {               // halves of words: four nibbles of two tokens
                const uint32_t sel = q & 1 ? 0x07060302u : 0x05040100u;
                uint32_t y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y[j] = __builtin_amdgcn_perm(vq[2 * j + 1][q / 2], vq[2 * j][q / 2], sel) ^ 0x88888888u;
                pv(4 * q, nib_pair0(y[0]), nib_pair0(y[1]), nib_pair0(y[2]), nib_pair0(y[3]));
                pv(4 * q + 1, nib_pair1(y[0]), nib_pair1(y[1]), nib_pair1(y[2]), nib_pair1(y[3]));
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] >>= 8;
                pv(4 * q + 2, nib_pair0(y[0]), nib_pair0(y[1]), nib_pair0(y[2]), nib_pair0(y[3]));
                pv(4 * q + 3, nib_pair1(y[0]), nib_pair1(y[1]), nib_pair1(y[2]), nib_pair1(y[3]));
            }
        }
        t0 += 128;
        ++it;
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_only(0));               // no load may land in what the waves share below
    __syncthreads();

    // the block's waves: common references, then the sums of the accumulators
    l += __shfl_xor(l, 16, QA_WAVE);
    l += __shfl_xor(l, 32, QA_WAVE);
    if (c4 == 0) {
        st_m[wave][m16] = m;
        st_l[wave][m16] = l;
        st_e[wave][m16] = ex;
    }
    // head m16, values VN (4 c4 + e) + i; rows one piece longer, so that 16 of them start at different banks
    v4f* const red = reinterpret_cast<v4f*>(smem);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < VN / 4; ++i)
            red[(wave * 16 + m16) * (DP / 4 + 1) + VN / 4 * (4 * c4 + e) + i] = v4f{acc[4 * i][e], acc[4 * i + 1][e], acc[4 * i + 2][e], acc[4 * i + 3][e]};
    __syncthreads();
    if (threadIdx.x < 16) {
        float mg = kLow, lg = 0.0f, e[4], top = -1000.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) mg = fmaxf(mg, st_m[w][threadIdx.x]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float down = st_m[w][threadIdx.x] - mg;
            lg += st_l[w][threadIdx.x] * __builtin_amdgcn_exp2f(down);
            e[w] = st_e[w][threadIdx.x] + down;              // of the wave's sums, 2^e
            top = fmaxf(top, e[w]);
        }
        // Factors next to the largest, divided; its power of two comes last: together they, or sums that are divided
        // afterwards, may pass fp32 although the output does not.
        const float inv = lg == 0.0f ? 0.0f : 1.0f / lg;
#pragma unroll
        for (int w = 0; w < 4; ++w) st_e[w][threadIdx.x] = __builtin_amdgcn_exp2f(e[w] - top) * inv;
        power[threadIdx.x] = (int)top + 10;                  // (values' codes came times 2^-10)
        if ((int)threadIdx.x < heads_here) {
            const float lse = lg == 0.0f ? -__builtin_inff() : mg + __builtin_log2f(lg);
            if (!whole) a.plse[slot * 16 + threadIdx.x] = lse;
            else if (a.lse) a.lse[row0 + threadIdx.x] = lse * kLn2;
        }
    }
    __syncthreads();
    const int L = a.D / 4;
    for (int i = threadIdx.x; i < heads_here * L; i += 256) {
        const int r = i / L, d = i - r * L;
        v4f o = red[r * (DP / 4 + 1) + d] * st_e[0][r];
#pragma unroll
        for (int w = 1; w < 4; ++w) o += red[(w * 16 + r) * (DP / 4 + 1) + d] * st_e[w][r];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __builtin_ldexpf(o[j], power[r]);
        if (!whole) *reinterpret_cast<v4f*>(a.part + (slot * 16 + r) * a.D + 4 * d) = o;
        else store_quad(a.out, (row0 + r) * a.D + 4 * d, a.dt, o);
    }
    left -= k1 - k0;
    k0 = 0;
    ++b;
    if (left > 0) __syncthreads();                           // the stages are free again
    }
}

// The parts of one row (sequence and head): weights 2^(lse_i - max), four values to
// a lane, the parts over groups of D / 4 lanes.  Two dependent loads (the places, the parts)
// and two barriers: 3.9 us for 32 rows of 64 parts, 6.6 for 2048 rows of 2 on average.
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
    __shared__ float wt[1024];
    __shared__ v4f sum[256];
    __shared__ float red[8];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
    const int64_t row = blockIdx.x;
    const int b = (int)(row / a.H), hq = (int)(row - (int64_t)b * a.H), h = hq / a.group, g = hq - h * a.group;
    const int HG = a.heads * a.gtiles, hg = h * a.gtiles + (g >> 4);
    const int u0 = a.before[b], all = a.before[a.B], share = all < a.share ? all : a.share;
    const int n1 = a.before[b + 1] - u0, L = a.D / 4;
    if (n1 == 0) {                                           // no token to see
        if (tid < L) store_quad(a.out, row * a.D + 4 * tid, a.dt, v4f{0.0f, 0.0f, 0.0f, 0.0f});
        if (tid == 0 && a.lse) a.lse[row] = -__builtin_inff();
        return;
    }
    // the shares of the sequence's first and last unit (the first `more` shares have one unit more)
    const int each = all / share, more = all - each * share;
    auto share_of = [&](int u) __attribute__((always_inline)) {
        return u < more * (each + 1) ? u / (each + 1) : more + (u - more * (each + 1)) / each;
    };
    const int i0 = share_of(u0), n = share_of(u0 + n1 - 1) - i0 + 1;
    if (n == 1) return;                                      // a single block has written it
    const int64_t slot = (int64_t)(b + i0) * HG + hg;        // of the first part; the next ones HG further on each
    const float* plse = a.plse + slot * 16 + (g & 15);
    const float* part = a.part + (slot * 16 + (g & 15)) * a.D;
    const int groups = 256 / L, grp = tid / L, j = tid - grp * L;
    const bool mine = grp < groups && grp < n;
    auto part_at = [&](int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const v4f*>(part + (int64_t)i * HG * 16 * a.D + 4 * j);
    };
    v4f s = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (mine) s = part_at(grp);                              // requested before the weights are known
    float top = -__builtin_inff();
    for (int i = tid; i < n; i += 256) top = fmaxf(top, plse[(int64_t)i * HG * 16]);
    top = wave_max(top);
    if (lane == 0) red[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    float total = 0.0f;
    for (int i = tid; i < n; i += 256) {
        const float v = plse[(int64_t)i * HG * 16];
        // a part without a token weighs nothing, and a NaN stays one
        const float w = v == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(v - top);
        wt[i] = w;
        total += w;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o, QA_WAVE);
    if (lane == 0) red[4 + wave] = total;
    __syncthreads();
    total = red[4] + red[5] + red[6] + red[7];
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    if (mine) {
        // Divided weights, at most 1 together: a sum that is divided afterwards may pass fp32 although the parts do not.
        // (a part without a token holds zeros; four requests at a time: 512 parts of one head of 128 in 11 us less, and
        // eight at a time, or four times the threads, no faster or slower where rows are many)
        s *= wt[grp] * inv;
#pragma unroll 4
        for (int i = grp + groups; i < n; i += groups) s += wt[i] * inv * part_at(i);
    }
    sum[tid] = s;
    __syncthreads();
    if (tid >= L) return;
    for (int i = 1; i < groups; ++i) s += sum[i * L + tid];
    store_quad(a.out, row * a.D + 4 * tid, a.dt, s);
    if (tid == 0 && a.lse) a.lse[row] = total == 0.0f ? -__builtin_inff() : (top + __builtin_log2f(total)) * kLn2;
}

namespace {

constexpr int64_t kMaxShare = 1024;        // blocks that share the work: at most four on each CU

// Whether the blocks share the work, as far as the sums over sequences fit a block and
// 31 bits.  Shares balance the card, but a block that takes up several sequences
// begins and ends each, and the join is a launch.  By sequences of 8 key heads and
// their longest length (us; a block to each sequence and head, and shared; lengths
// evenly spread below it; heads of 128, 32 queries, 8 bits):
//       1000          2000          4000          8000
//    1  13.1  11.1    20.5  11.6    35.9  12.9    65.1  16.0
//    8  13.9  14.3    21.6  17.0    36.2  22.9    65.6  30.3
//   32  14.5  20.9    22.7  27.8    38.8  39.5    69.8  60.5
//   64  19.5  32.7    32.7  47.3    57.9  66.9     108   108
//   90  27.2  44.2    41.4  56.4    72.7  85.6     138   140
// The lengths are not known here, and where one is much longer than the others only the
// first column grows with it, by 7.5 us for 1000 tokens: the border lies below the
// point where evenly spread ones are equal.  From 768 pairs of a sequence and a key head on
// nothing is shared.  Evenly long sequences take the same there either way (96 of 8000 tokens
// 263 us and 263), but one of 100000 tokens beside 95 of 1000 takes 742 us by itself, 74 if
// the blocks shared it (beside 94, where they do, 76).  The table is for heads of 128 in
// 8 bits; head size, bits and blocks on a CU do not enter the rule.
bool shared_work(int64_t B, int32_t H, int32_t heads, int64_t max_len, int32_t window) {
    const int64_t group = H / heads, pairs = B * heads * ((group + 15) / 16);
    const int64_t span = window > 0 && (int64_t)window + 31 < max_len ? (int64_t)window + 31 : max_len;
    return B <= 1024 && pairs < 768 && span > 512 + 7 * pairs && pairs * ((span + kUnit - 1) / kUnit) < ((int64_t)1 << 30);
}

template <int BITS, int DP>
hipError_t run_attn(const AttnArgs& a, int64_t blocks, hipStream_t st) {
    if (a.qdt == 0) hipLaunchKernelGGL((k_attn_decode<BITS, DP, true>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_attn_decode<BITS, DP, false>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}
template <int BITS>
hipError_t run_attn(const AttnArgs& a, int64_t blocks, hipStream_t st) {
    if (a.D <= 64) return run_attn<BITS, 64>(a, blocks, st);
    return a.D <= 128 ? run_attn<BITS, 128>(a, blocks, st) : run_attn<BITS, 256>(a, blocks, st);
}

}  // namespace

size_t attn_scratch_bytes(int64_t B, int32_t H, int32_t heads, int32_t D, int64_t max_len, int32_t window) {
    if (!shared_work(B, H, heads, max_len, window)) return 0;
    const int64_t HG = (int64_t)heads * ((H / heads + 15) / 16);
    const size_t slots = (size_t)((kMaxShare > HG ? kMaxShare / HG : 1) + B) * HG;
    return slots * 16 * (D + 1) * 4 + (size_t)(B + 1) * 4;
}

hipError_t launch_attn_decode(const void* q, int64_t ldq, int q_dtype, int64_t B, int32_t H, const KvCache& c,
                              const int32_t* table, int64_t ldt, int64_t width, const int32_t* lengths, int64_t max_len,
                              int32_t window, float scale, void* out, int out_dtype, float* lse, void* scratch,
                              hipStream_t st) {
    AttnArgs a{};
    a.q = q; a.ldq = ldq; a.qdt = q_dtype;
    a.kc = static_cast<const uint8_t*>(c.k_codes); a.ks = c.k_scales;
    a.vc = static_cast<const uint8_t*>(c.v_codes); a.vs = c.v_scales;
    a.table = table; a.ldt = ldt; a.lengths = lengths;
    a.B = (int32_t)B; a.H = H; a.heads = c.heads; a.group = H / c.heads; a.gtiles = (a.group + 15) / 16;
    a.D = c.D; a.shift = c.shift; a.pages = (int32_t)c.pages;
    const int64_t most = width << c.shift, pairs = B * c.heads * a.gtiles;
    a.max_len = (int32_t)(c.pages == 0 ? 0 : max_len < most ? max_len : most);
    a.window = window;
    a.scale2 = scale * 1.44269504088896340736f;
    a.out = out; a.dt = out_dtype; a.lse = lse;
    const bool shared = shared_work(B, H, c.heads, max_len, window);
    if (shared) {
        const int64_t fit = 256 * blocks_on_cu(c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256, c.bits, q_dtype == 0), HG = (int64_t)c.heads * a.gtiles;
        a.share = (int32_t)(fit > HG ? fit / HG : 1);
        const int64_t slots = (a.share + B) * HG;
        a.part = static_cast<float*>(scratch);
        a.plse = a.part + slots * 16 * c.D;
        a.before = reinterpret_cast<int32_t*>(a.plse + slots * 16);
    }
    const int64_t blocks = shared ? (int64_t)a.share * c.heads * a.gtiles : pairs;
    hipError_t e = c.bits == 8 ? run_attn<8>(a, blocks, st) : run_attn<4>(a, blocks, st);
    if (e != hipSuccess || !shared) return e;
    hipLaunchKernelGGL(k_attn_join, dim3((unsigned)(B * H)), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace qa
