// qa_tile.hpp -- the int8 tile product shared by the grouped, the adapter and the
// epilogue linears: acc[FM][FN] = A rows x B rows^T with rows picked by the caller.
//
// Both operands are K-contiguous int8 rows.  A stage holds BK = 128 bytes of K
// of the tile's BM rows of A followed by its BN rows of B; it is filled by
// direct global -> LDS loads (one instruction: 64 lanes x 16 bytes = 8 rows),
// and since every lane names its own address, the rows may come from anywhere:
// gathered tokens, or gate and up rows in turn.  STAGES stages, all but one in
// flight.  The 16-byte chunk c of row r is stored at chunk c ^ (r & 7), which
// makes the fragment reads of 8 consecutive rows hit 8 different bank groups;
// the permutation is produced by the chunk that each lane fetches.
//
// What bounds it: the chain of a stage (its loads into LDS, barrier, fragment
// reads, MFMAs), of which two blocks on a CU overlap a part.  The MFMAs are busy
// for 35 to 42% of the time at 16396 rows of 4096 x 4096 and 2048, waves spend 45%
// of theirs waiting for data and 36 to 41% for an instruction to issue, and LDS has no
// bank conflicts.  A wave with nothing but fragment reads and MFMAs reaches 3.4
// POPS; in this library's loop of 256-row tiles, half the fragment reads changed
// nothing, so the stages' traffic is the larger part.  64-byte stages fetch every
// 128-byte line twice from L2, in two stages: at 8192 x 8192 x 4096 a 128 x 128 tile
// went from 1.61 to 1.97 POPS with 128-byte stages.  Two blocks on a CU overlap one's reads with the other's MFMAs and
// hide its prologue and epilogue, so the tile is as large as two blocks' LDS
// allow: 128 x 192 with two stages (80 KB) 2.04 POPS, against 1.81 for 128 x 256
// (96 KB, one block), and 102 against 118 us at 2048 x 11008 x 4096.  The
// library's int8 product reaches 2.13 POPS on this card at 8192^3.
//
// The MFMA takes B first, so it makes the transposed 16 x 16 tile: lane l,
// element e of acc[i][j] is row 16 i + l % 16, column 16 j + 4 (l / 16) + e of
// the wave's tile.
#pragma once

#include "qa_device.hpp"

namespace qa {
namespace tile {

typedef __attribute__((address_space(3))) void lds_void;

template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct Cfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN;
    static constexpr int BK = 128, STAGES = STAGES_, THREADS = 64 * NW;
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    static constexpr int INS = (BM + BN) / 8 / NW;           // load instructions of a wave per stage
    static constexpr int STAGE = (BM + BN) * BK, LDS = STAGES * STAGE;
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0, "wave tiles are whole fragments");
    static_assert((BM + BN) % (8 * NW) == 0 && BM % 8 == 0, "a stage's rows split evenly over the waves");
    static_assert(STAGES == 2 || STAGES == 3, "the waits know one or two stages ahead");
};

__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// s_waitcnt immediate waiting for vmcnt <= n only (gfx9 encoding)
constexpr int vmcnt(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

__device__ __forceinline__ void block_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Block -> output tile: block b runs on XCD b % 8; every XCD takes a contiguous
// range of tiles, walked eight tile rows at a time, so that neighbours in time
// share rows of A and of B in that XCD's L2.
__device__ __forceinline__ void of_block(int bid, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int ntiles = tiles_m * tiles_n, per = ntiles >> 3, rem = ntiles & 7;
    const int xcd = bid & 7, slot = bid >> 3;
    const int t = xcd < rem ? xcd * (per + 1) + slot : rem * (per + 1) + (xcd - rem) * per + slot;
    const int g = t / (8 * tiles_n), first = g * 8;
    const int gm = tiles_m - first < 8 ? tiles_m - first : 8;
    const int r = t - g * 8 * tiles_n;
    tm = first + r % gm;
    tn = r / gm;
}

// row_a(r), row_b(r): byte offset of tile row r in its descriptor, or kOOB for
// a row of zeros.  K is a multiple of 16.  On return no load is in flight and
// every wave has passed its last fragment read, so smem is free.
template <class C, class RA, class RB>
__device__ __forceinline__ void product(rsrc_t rsa, rsrc_t rsb, uint32_t K, uint8_t* smem, RA&& row_a, RB&& row_b,
                                        v4i (&acc)[C::FM][C::FN]) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int wm = wave / C::WN, wn = wave % C::WN;
    uint32_t off[C::INS], ck[C::INS];
#pragma unroll
    for (int q = 0; q < C::INS; ++q) {
        const int P = (q * C::NW + wave) * 64 + lane;        // 16-byte chunk of the stage
        const int r = P >> 3, c = (P & 7) ^ (r & 7);
        const uint32_t base = r < C::BM ? row_a(r) : row_b(r - C::BM);
        off[q] = base == kOOB ? kOOB : base + c * 16;
        ck[q] = c * 16;
    }
    const int nk = (int)((K + C::BK - 1) / C::BK);
    auto issue = [&](int kt) __attribute__((always_inline)) {
        uint8_t* st = smem + (kt % C::STAGES) * C::STAGE;
        const uint32_t k0 = (uint32_t)kt * C::BK;
#pragma unroll
        for (int q = 0; q < C::INS; ++q) {
            const bool a = (q * C::NW + wave) * 8 < C::BM;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(a ? rsa : rsb, (lds_void*)(st + (q * C::NW + wave) * 1024), 16,
                                                     k0 + ck[q] < K ? off[q] + k0 : kOOB, 0, 0, 0);
        }
    };
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    constexpr int AHEAD = C::STAGES - 1;
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
        if (q < nk) issue(q);
    const int c = lane >> 4;
    for (int kt = 0; kt < nk; ++kt) {
        if (AHEAD == 2 && kt + 1 < nk) __builtin_amdgcn_s_waitcnt(vmcnt(C::INS));    // stage kt + 1 may be in flight
        else __builtin_amdgcn_s_waitcnt(vmcnt(0));
        block_barrier();
        // stage kt + AHEAD takes the buffer of stage kt - 1, whose reads every
        // wave finished before its MFMAs of iteration kt - 1, before this barrier
        if (kt + AHEAD < nk) issue(kt + AHEAD);
        const uint8_t* sa = smem + (kt % C::STAGES) * C::STAGE;
        const uint8_t* sb = sa + C::BM * C::BK;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            v4i fa[C::FM], fb[C::FN];
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
                fa[i] = *reinterpret_cast<const v4i*>(sa + swz(wm * C::TM + i * 16 + (lane & 15), c + 4 * ks));
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                fb[j] = *reinterpret_cast<const v4i*>(sb + swz(wn * C::TN + j * 16 + (lane & 15), c + 4 * ks));
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
    }
    __syncthreads();
}

}  // namespace tile

// Four outputs at p (element type dt: 0 fp32, 1 fp16, 2 bf16), of which the
// first n exist; whole vectors where `vec` says that rows allow them.
__device__ __forceinline__ void store4(void* p, int64_t at, int dt, const float* v, int n, bool vec) {
    if (dt == 0) {
        float* o = static_cast<float*>(p) + at;
        if (vec && n >= 4) {
            *reinterpret_cast<v4f*>(o) = v4f{v[0], v[1], v[2], v[3]};
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) o[e] = v[e];
        return;
    }
    uint16_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = dt == 1 ? f2h(v[e]) : f2bf(v[e]);
    uint16_t* o = static_cast<uint16_t*>(p) + at;
    if (vec && n >= 4) {
        *reinterpret_cast<u32x2*>(o) = u32x2{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n) o[e] = h[e];
}

}  // namespace qa
