// bf16 matrix products of the vocabulary loss, for gfx950: C = A B^T over
// tiles, fp32 sums, with an epilogue of the caller's.
//
// An operand is K-contiguous (its rows are C's rows or columns, 16-byte reads
// of 8 K each) or K-strided (its rows are K; ds_read_b64_tr_b16 hands a lane
// 4 K of one column).  So the loss' three products need no transposed copy:
//   logits  [v, t] = w [v, h] x [t, h]        both K-contiguous
//   dx      [h, t] = w [v, h] dl [t, v]       A K-strided, B K-contiguous
//   dw      [h, v] = x [t, h] dl [t, v]       both K-strided
// C's rows are the contiguous dimension of what is stored: a fragment's 32
// rows are dealt out so that a lane ends up with 16 adjacent ones, half a wave
// each with one half of the fragment.
#pragma once

#include <stdint.h>

#include "gemm_common.h"

namespace fp8mi {
namespace ce {

using gemm::v4f;
using gemm::v4u;
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kStageK = 32;             // K of a stage: 64 bytes of a K-contiguous row
constexpr int kRing = 4;                // stages in LDS

struct Operand {
    const uint8_t* p;
    int64_t ld;                         // bytes between rows
};

struct GemmShape {
    Operand a, b;
    int m, n, k;                        // a row of a K-contiguous operand holds zeros from k to the next multiple of 8
    int tiles_m, tiles_n, group_m;
    int splits;                         // of K
};

// One unit of work: a tile and its range of stages.
struct Item {
    int id;                             // past the last: none
    int tm, tn, split;
    int first, end;                     // stages
};

// Linear item number to tile and split: numbers go to the XCDs in turn, so XCD
// x takes a contiguous range of the order, which walks group_m tile rows at a
// time through all tiles of one split, then of the next.
__device__ inline Item item_of(const GemmShape& s, int id)
{
    Item it{id, 0, 0, 0, 0, 0};
    const int tiles = s.tiles_m * s.tiles_n, total = tiles * s.splits;
    if (id >= total) return it;
    const int xcd = id & 7, local = id >> 3;
    int t = xcd * (total >> 3) + min(xcd, total & 7) + local;
    it.split = t / tiles;
    t -= it.split * tiles;
    const int in_group = s.group_m * s.tiles_n;
    const int g = t / in_group;
    const int first_m = g * s.group_m;
    const int gsize = min(s.tiles_m - first_m, s.group_m);
    const int r = t - g * in_group;
    it.tm = first_m + r % gsize;
    it.tn = r / gsize;
    // the first (stages % splits) splits are one stage longer
    const int stages = (s.k + kStageK - 1) / kStageK;
    const int each = stages / s.splits, more = stages - each * s.splits;
    it.first = __builtin_amdgcn_readfirstlane(each * it.split + min(it.split, more));
    it.end = it.first + __builtin_amdgcn_readfirstlane(each + (it.split < more));
    return it;
}

// Position of 16-byte chunk c (0..3) in the 64-byte LDS row r of a
// K-contiguous operand (an involution in c).  Fragment reads of 32 rows, in
// order or dealt out, run at the rate of adjacent addresses (measured: 195 to
// 203 bytes a clock and CU, adjacent ones 192).
__device__ inline int swz64(int r, int c) { return c ^ (((r >> 2) & 1) | (((r >> 1) ^ (r >> 2) ^ (r >> 3)) & 1) << 1); }

// A K-strided operand's stage holds 32 rows of 2 T bytes; its 32-byte granules
// are permuted by the row, so that the 4 rows and 64 bytes of each (granules 2 j
// and 2 j + 1) which half a wave reads lie in different banks (172 bytes a clock
// and CU; unpermuted 64).
template <int T>
__device__ inline int swz_strided(int row)
{
    return (row & 3) << 1;
}

// The tile C[TM, TN] of one item: WR x WC waves of MF x NF fragments of 32 x
// 32.  The stages of all of a workgroup's items are one stream in a ring of
// four, filled by DMA four ahead, so an item's first stages arrive during the
// epilogue of the one before.  Fragments are read half a stage ahead of their
// products; one barrier a stage, in its middle, past which every wave has read
// all of it.
template <bool ATR, bool BTR, int WR, int WC, int MF, int NF>
struct Tile {
    static constexpr int W = WR * WC, TM = 32 * MF * WR, TN = 32 * NF * WC;
    static constexpr int kStage = (TM + TN) * 64;
    // what an epilogue wants of its tile's columns: 16 bytes each, in runs of 64
    // columns of a wave, of the items whose stages are on their way and the one at work
    static constexpr int kRuns = (NF + 1) / 2, kNotes = 1024 * kRuns * WC;
    template <typename Epi>
    static constexpr int lds_bytes()
    {
        return kRing * kStage + (Epi::kNotes ? (kRing + 1) * kNotes : 0);
    }
    // DMA instructions of a wave and stage; where an operand has fewer than
    // waves, some repeat another's (the same bytes to the same place)
    static constexpr int kA = TM / 16 >= W ? TM / 16 / W : 1;
    static constexpr int kB = TN / 16 >= W ? TN / 16 / W : 1;
    static constexpr int kPer = kA + kB;
    static_assert((!ATR || TM >= 128) && (!BTR || TN >= 128), "K-strided rows of 8 granules or more");
    static_assert((TM / 16 % W == 0 || TM / 16 < W) && (TN / 16 % W == 0 || TN / 16 < W), "whole DMA instructions");

    typedef v16f Acc[NF][MF];

    // Epi: operator()(item, acc, row, column, notes): a lane holds rows row + 32 i
    // + r in acc[j][i][r], column + 32 j.  It returns whether it has issued
    // at least kStores vector memory operations.  With kNotes
    // set, note(lds, column) brings 1 KB for each run of 64 columns, which a call finds at notes.
    template <typename Epi>
    __device__ static void run(const GemmShape& s, uint8_t* lds, Epi& epi)
    {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int lane = threadIdx.x & 63;
        const uint32_t base = gemm::lds_addr(lds);

        // ---- the stream of fills
        Item f = item_of(s, blockIdx.x);
        int ft = f.first, fslot = 0, fnote = 0;
        // K-contiguous: lane l brings chunk l % 4 of row l / 4 of 16; K-strided:
        // 16 bytes of a row of 2 T.
        const int kc_chunk = 16 * swz64(lane >> 2, lane & 3);
        const auto first_dma = [&](int per, int t) { return t / 16 >= W ? wave * per : wave % (t / 16); };
        const int ua = first_dma(kA, TM), ub = first_dma(kB, TN);
        uint32_t va[kA], vb[kB];
#pragma unroll
        for (int j = 0; j < kA; ++j) {
            const int byte = 1024 * (ua + j) + 16 * lane, row = byte / (2 * TM), in = byte % (2 * TM);
            va[j] = ATR ? (uint32_t)(row * s.a.ld + (((in >> 5) ^ swz_strided<TM>(row)) << 5) + (in & 31))
                        : (uint32_t)((16 * (ua + j) + (lane >> 2)) * s.a.ld + kc_chunk);
        }
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const int byte = 1024 * (ub + j) + 16 * lane, row = byte / (2 * TN), in = byte % (2 * TN);
            vb[j] = BTR ? (uint32_t)(row * s.b.ld + (((in >> 5) ^ swz_strided<TN>(row)) << 5) + (in & 31))
                        : (uint32_t)((16 * (ub + j) + (lane >> 2)) * s.b.ld + kc_chunk);
        }
        // Where an operand's stage lies and what of it may be read.  K-contiguous:
        // the tile's rows, the same for all stages of an item.  K-strided: the
        // rows from K k0 on, 32 or what is left.  Past the last item: nothing.
        const uint8_t *pa, *pb;
        uint32_t bytes_a, bytes_b;
        int k_left;
        const uint32_t row_bytes = 2u * (uint32_t)((s.k + 7) & ~7);
        const int total = s.tiles_m * s.tiles_n * s.splits;
        const auto describe = [&]() {
            const bool live = f.id < total;
            const int m0 = f.tm * TM, n0 = f.tn * TN;
            const int k0 = ft * kStageK;
            if constexpr (ATR) {
                pa = s.a.p + k0 * s.a.ld + 2 * (int64_t)m0;
                bytes_a = 2u * (uint32_t)(s.m - m0);
            } else {
                pa = s.a.p + m0 * s.a.ld;
                bytes_a = live ? (uint32_t)((min(s.m - m0, TM) - 1) * s.a.ld) + row_bytes : 0u;
            }
            if constexpr (BTR) {
                pb = s.b.p + k0 * s.b.ld + 2 * (int64_t)n0;
                bytes_b = 2u * (uint32_t)(s.n - n0);
            } else {
                pb = s.b.p + n0 * s.b.ld;
                bytes_b = live ? (uint32_t)((min(s.n - n0, TN) - 1) * s.b.ld) + row_bytes : 0u;
            }
            k_left = live ? s.k - k0 : 0;
            if (!live) f.end = 0x7FFFFFFF;      // no item after it
            if constexpr (Epi::kNotes) {
                if (wave < WC && live) {
#pragma unroll
                    for (int h = 0; h < kRuns; ++h)
                        epi.note(base + kRing * kStage + fnote * kNotes + 1024 * (kRuns * wave + h), n0 + 32 * NF * wave + 64 * h);
                }
                fnote = fnote == kRing ? 0 : fnote + 1;
            }
        };
        describe();
        // The next stage: what its instructions share, the j-th of them, the step on.
        uint32_t to;
        v4u ra, rb;
        bool past;
        const auto fill_begin = [&]() {
            to = base + fslot * kStage;
            past = (uint32_t)ft * (2 * kStageK) + kc_chunk >= row_bytes;     // K-contiguous: behind the row's end
            const int rows = min(k_left, kStageK);
            ra = gemm::make_rsrc(ATR ? pa : pa + ft * (2 * kStageK),
                                 !ATR ? bytes_a - min(bytes_a, (uint32_t)ft * (2 * kStageK))
                                      : rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)s.a.ld + bytes_a : 0u);
            rb = gemm::make_rsrc(BTR ? pb : pb + ft * (2 * kStageK),
                                 !BTR ? bytes_b - min(bytes_b, (uint32_t)ft * (2 * kStageK))
                                      : rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)s.b.ld + bytes_b : 0u);
        };
        const auto fill_one = [&](int j) {
            if (j < kA)
                gemm::dma16(to + 1024 * (ua + j), !ATR && past ? gemm::kOutOfRange : va[j], ra);
            else
                gemm::dma16(to + TM * 64 + 1024 * (ub + j - kA), !BTR && past ? gemm::kOutOfRange : vb[j - kA], rb);
        };
        const auto fill_end = [&]() {
            fslot = (fslot + 1) & (kRing - 1);
            if constexpr (ATR) pa += kStageK * s.a.ld;
            if constexpr (BTR) pb += kStageK * s.b.ld;
            k_left -= kStageK;
            if (++ft >= f.end) {
                f = item_of(s, f.id + gridDim.x);
                ft = f.first;
                describe();
            }
        };

        // ---- the fragments
        const int wm = (wave % WR) * 32 * MF, wn = (wave / WR) * 32 * NF;
        const int c = lane & 31, half = lane >> 5;
        // K 16 kk + 8 half .. + 7 of both operands.  K-contiguous: chunk half + 2 kk.
        // A's row of instruction row c: 16 (c / 4 % 2) + 4 (c / 8) + c % 4
        const int ar = 16 * ((c >> 2) & 1) + 4 * (c >> 3) + (c & 3);
        const int tk = 8 * half + ((lane & 15) >> 2);           // K-strided: this lane's row of a read
        const int tc = (lane >> 4 & 1) * 4 + (lane & 3);        // and its 4 columns' place among the fragment's 32
        // K-strided: a row's address for each fragment, the second half stage 16 rows
        // on.  K-contiguous: fragments lie 32 rows apart, the second half stage
        // across bit 5 (chunk half + 2).
        constexpr int kAt = ATR ? MF : 2, kBt = BTR ? NF : 2;
        uint32_t at[kAt], bt[kBt];
#pragma unroll
        for (int i = 0; i < kAt; ++i)
            at[i] = ATR ? tk * 2 * TM + (((((wm + 32 * i) >> 4) + (tc & 1)) ^ swz_strided<TM>(tk)) << 5) + (tc >> 1) * 8
                        : ((wm + ar) * 64 + 16 * swz64(ar, half)) ^ (32 * i);
#pragma unroll
        for (int j = 0; j < kBt; ++j)
            bt[j] = TM * 64 + (BTR ? tk * 2 * TN + (((((wn + 32 * j) >> 4) + (tc >> 2)) ^ swz_strided<TN>(tk)) << 5) + (tc & 3) * 8
                                   : ((wn + c) * 64 + 16 * swz64(c, half)) ^ (32 * j));
        v8bf fa[2][MF], fb[2][NF];
        int slot = 0;
        const auto strided = [&](uint32_t from, int kk, int row_bytes) -> v8bf {
            struct {
                v4s lo, hi;
            } v;
            v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + from + 16 * kk * row_bytes));
            v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + from + (16 * kk + 4) * row_bytes));
            return __builtin_bit_cast(v8bf, v);
        };
        // The j-th of a half stage's fragments, B's first.
        const auto read_one = [&](auto KK, int j) {
            constexpr int kk = decltype(KK)::value;
            const uint32_t ring = slot * kStage;
            if (j < NF)
                fb[kk][j] = BTR ? strided(bt[j % kBt] + ring, kk, 2 * TN)
                                : *reinterpret_cast<const v8bf*>(lds + (bt[kk] + ring) + 2048 * j);
            else
                fa[kk][j - NF] = ATR ? strided(at[(j - NF) % kAt] + ring, kk, 2 * TM)
                                     : *reinterpret_cast<const v8bf*>(lds + (at[kk] + ring) + 2048 * (j - NF));
        };
        Acc acc;
        // A half stage's matrix instructions, and after the m-th what `between` does.
        // Nothing moves from its place: the reads and DMA of other stages are
        // issued under the matrix instructions' time.
        const auto products = [&](auto KK, auto between) {
            constexpr int kk = decltype(KK)::value;
#pragma unroll
            for (int m = 0; m < MF * NF; ++m) {
                acc[m % NF][m / NF] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[kk][m / NF], fb[kk][m % NF],
                                                                              acc[m % NF][m / NF], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                between(m);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        const auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;
        };
        constexpr int kAll = MF * NF, kReads = MF + NF;
        constexpr std::integral_constant<int, 0> k0{};
        constexpr std::integral_constant<int, 1> k1{};
        clear();
#pragma unroll 1
        for (int i = 0; i < kRing; ++i) {
            fill_begin();
#pragma unroll
            for (int j = 0; j < kPer; ++j) fill_one(j);
            fill_end();
        }
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * kPer) : "memory");     // the first stage
        gemm::barrier_lds();
#pragma unroll
        for (int j = 0; j < kReads; ++j) read_one(k0, j);
        int stored = 3;         // stages since the last epilogue's stores, up to 3
        int note = 0;
        for (Item it = item_of(s, blockIdx.x); it.id < total; it = item_of(s, it.id + gridDim.x)) {
            for (int t = it.first; t < it.end; ++t) {
                products(k0, [&](int m) {
#pragma unroll
                    for (int j = 0; j < kReads; ++j)
                        if (j * kAll / kReads == m) read_one(k1, j);
                });
                // The next stage has landed: the two after it are younger, and an
                // epilogue's stores are to the three stages filled before them.
                constexpr int kLoose = 2 * kPer + Epi::kStores < 63 ? 2 * kPer + Epi::kStores : 63;
                if (stored < 3) {
                    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoose) : "memory");
                    ++stored;
                } else {
                    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kPer) : "memory");
                }
                // past this every wave has read the whole stage: its slot is free
                gemm::barrier_lds();
                fill_begin();
                slot = (slot + 1) & (kRing - 1);
                products(k1, [&](int m) {
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        if (j * kAll / kPer == m) fill_one(j);
#pragma unroll
                    for (int j = 0; j < kReads; ++j)
                        if (j * kAll / kReads == m) read_one(k0, j);
                });
                fill_end();
            }
            const uint8_t* notes = lds + kRing * kStage + note * kNotes + 1024 * kRuns * (wave / WR);
            stored = epi(it, acc, it.tm * TM + wm + 16 * half, it.tn * TN + wn + c, notes) ? 0 : 3;
            note = note == kRing ? 0 : note + 1;
            clear();
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");        // the fills past the end
    }
};

}  // namespace ce
}  // namespace fp8mi
