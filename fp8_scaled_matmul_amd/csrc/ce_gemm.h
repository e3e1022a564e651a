// bf16 matrix products of the vocabulary loss, for gfx950: C = A B^T over
// tiles, fp32 sums, with an epilogue of the caller's.
//
// An operand is K-contiguous (its rows are C's rows or columns, 16-byte reads
// of 8 K each) or K-strided (its rows are K; ds_read_b64_tr_b16 hands a lane
// 4 K of one column).  So the loss' three products need no transposed copy:
//   logits  [v, t] = w [v, h] x [t, h]        both K-contiguous
//   dx      [h, t] = w [v, h] dl [t, v]       A K-strided, B K-contiguous
//   dw      [h, v] = x [t, h] dl [t, v]       both K-strided
// C's rows are the contiguous dimension of what is stored.
//
// The matrix instruction is v_mfma_f32_16x16x32_bf16 (32x32x16, of the same rate,
// was 6 % slower: its reads come in larger steps).  A workgroup walks tiles; stages
// of 32 K come by DMA into a ring of four in LDS, so that the next tile's first
// stages arrive under this one's epilogue.  A stage has one barrier, in its middle:
// a wave reads its second half's fragments and the next stage's first ones under
// the matrix instructions, into registers as they fall free.  256 x 256 and eight
// waves, two a SIMD: 128 accumulators and all fragments in 205 of 256 registers.  It
// is bound by power: 1.19 to 1.25 PFLOP/s at 8192 x 32768 x 4096, whichever operands
// are strided; the same work on zeros takes a sixth less.  Tiles of 128 x 256 or
// four waves of 128 x 128 were slower (twice the LDS reads; spills).
#pragma once

#include <stdint.h>

#include "gemm_common.h"

namespace fp8mi {
namespace ce {

using gemm::v4f;
using gemm::v4u;
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kStageK = 32;             // K of a stage: 64 bytes of a K-contiguous row
constexpr int kRing = 4;                // stages in LDS

// Notes (what an epilogue wants of its tile's columns) come when an item is
// described, at the end of the stage whose fill, kRing ahead, was the last of the
// item before; they are read in the item's epilogue.  Items described whose
// epilogue is still to come, with `stages` each:
constexpr int notes_held(int stages)
{
    int most = 0;
    for (int s = 0; s < 2 * kRing * stages; ++s) {
        const int filled = s + kRing;       // at the end of stage s
        const int described = filled / stages + (filled % stages == stages - 1);
        most = most > described - s / stages + 1 ? most : described - s / stages + 1;
    }
    return most;
}
// One stage an item would need two slots more, and 64 tokens' tiles a workgroup of
// three a CU less: where K has one, a second of zeros follows.
constexpr int kNoteSlots = kRing, kNoteStages = 2;
static_assert(notes_held(kNoteStages) <= kNoteSlots && notes_held(kNoteStages + 1) <= kNoteSlots, "a slot an item");

struct Operand {
    const uint8_t* p;
    int64_t ld;                         // bytes between rows
};

struct GemmShape {
    Operand a, b;
    int m, n, k;                        // a row of a K-contiguous operand holds zeros from k to the next multiple of 8
    int tiles_m, tiles_n, group_m;
    int splits;                         // of K
    int least_stages;                   // of an item: kNoteStages where it has notes, else 1
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
    const int stages = max((s.k + kStageK - 1) / kStageK, s.least_stages);
    const int each = stages / s.splits, more = stages - each * s.splits;
    it.first = __builtin_amdgcn_readfirstlane(each * it.split + min(it.split, more));
    it.end = it.first + __builtin_amdgcn_readfirstlane(each + (it.split < more));
    return it;
}

// Position of 16-byte chunk c (0..3) in the 64-byte LDS row r of a
// K-contiguous operand (an involution in c): 16 rows at one chunk fill the 16
// slots of a 256-byte line.
__device__ inline int swz64(int r, int c) { return c ^ (((r >> 2) & 1) | (((r >> 1) ^ (r >> 2) ^ (r >> 3)) & 1) << 1); }

// A K-strided operand's stage holds 32 rows of 2 T bytes; its 32-byte granules
// (16 columns) are permuted by the row, so that the 8 rows (K 0 .. 3 and 8 .. 11,
// say) whose granules half a wave reads lie in different banks.
__device__ inline int swz_strided(int row) { return (row & 3) | (row >> 1 & 4); }

// The tile C[TM, TN] of one item: WR x WC waves of MF x NF fragments of 16 x
// 16.  The stages of all of a workgroup's items are one stream in a ring of
// four, filled by DMA four ahead, so an item's first stages arrive during the
// epilogue of the one before.  A stage is one matrix instruction deep; its
// products go by halves of A's fragments, column by column in each, and a
// fragment's registers take the next stage's as soon as they are done with.  One
// barrier a stage, in its middle, past which every wave has read all of it.
template <bool ATR, bool BTR, int WR, int WC, int MF, int NF>
struct Tile {
    static constexpr int W = WR * WC, TM = 16 * MF * WR, TN = 16 * NF * WC;
    static constexpr int kStage = (TM + TN) * 64;
    // notes: 16 bytes a column, in runs of 64 columns of a wave
    static constexpr int kRuns = (NF + 3) / 4, kNotes = 1024 * kRuns * WC;
    template <typename Epi>
    static constexpr int lds_bytes()
    {
        return kRing * kStage + (Epi::kNotes ? kNoteSlots * kNotes : 0);
    }
    // DMA instructions of a wave and stage; where an operand has fewer than
    // waves, some repeat another's (the same bytes to the same place)
    static constexpr int kA = TM / 16 >= W ? TM / 16 / W : 1;
    static constexpr int kB = TN / 16 >= W ? TN / 16 / W : 1;
    static constexpr int kPer = kA + kB;
    static_assert((!ATR || TM >= 128) && (!BTR || TN >= 128), "K-strided rows of 8 granules or more");
    static_assert(MF % 2 == 0, "halves");
    static_assert((TM / 16 % W == 0 || TM / 16 < W) && (TN / 16 % W == 0 || TN / 16 < W), "whole DMA instructions");

    typedef v4f Acc[NF][MF];

    // Epi: operator()(item, acc, row, column, notes): a lane holds rows row + 16 i
    // + r in acc[j][i][r], column + 16 j.  It returns whether it has issued
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
            va[j] = ATR ? (uint32_t)(row * s.a.ld + (((in >> 5) ^ swz_strided(row)) << 5) + (in & 31))
                        : (uint32_t)((16 * (ua + j) + (lane >> 2)) * s.a.ld + kc_chunk);
        }
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const int byte = 1024 * (ub + j) + 16 * lane, row = byte / (2 * TN), in = byte % (2 * TN);
            vb[j] = BTR ? (uint32_t)(row * s.b.ld + (((in >> 5) ^ swz_strided(row)) << 5) + (in & 31))
                        : (uint32_t)((16 * (ub + j) + (lane >> 2)) * s.b.ld + kc_chunk);
        }
        // Where an operand's stage lies and what of it may be read.  K-contiguous:
        // the tile's rows, the same for all stages of an item.  K-strided: the
        // rows from K k0 on, 32 or what is left.  Past the last item: nothing.
        const uint8_t *pa, *pb;
        int bytes_a, bytes_b;       // below 2^31: a tile's rows, or 32
        int k_left;
        const int row_bytes = 2 * ((s.k + 7) & ~7);
        const int total = s.tiles_m * s.tiles_n * s.splits;
        const auto describe = [&]() {
            const bool live = f.id < total;
            const int m0 = f.tm * TM, n0 = f.tn * TN;
            const int k0 = ft * kStageK;
            if constexpr (ATR) {
                pa = s.a.p + k0 * s.a.ld + 2 * (int64_t)m0;
                bytes_a = 2 * min(s.m - m0, TM);
            } else {
                pa = s.a.p + m0 * s.a.ld;
                bytes_a = live ? (int)((min(s.m - m0, TM) - 1) * s.a.ld) + row_bytes : 0;
            }
            if constexpr (BTR) {
                pb = s.b.p + k0 * s.b.ld + 2 * (int64_t)n0;
                bytes_b = 2 * min(s.n - n0, TN);
            } else {
                pb = s.b.p + n0 * s.b.ld;
                bytes_b = live ? (int)((min(s.n - n0, TN) - 1) * s.b.ld) + row_bytes : 0;
            }
            k_left = live ? s.k - k0 : 0;
            if (!live) f.end = 0x7FFFFFFF;      // no item after it
            if constexpr (Epi::kNotes) {
                if (wave < WC && live) {
#pragma unroll
                    for (int h = 0; h < kRuns; ++h)
                        epi.note(base + kRing * kStage + fnote * kNotes + 1024 * (kRuns * wave + h), n0 + 16 * NF * wave + 64 * h);
                }
                fnote = (fnote + 1) % kNoteSlots;
            }
        };
        describe();
        // The next stage: what its instructions share, the j-th of them, the step on.
        uint32_t to;
        v4u ra, rb;
        bool past;
        const auto fill_begin = [&]() {
            to = base + fslot * kStage;
            const int kb = ft * (2 * kStageK);
            past = kb + kc_chunk >= row_bytes;      // K-contiguous: behind the row's end
            const int rows = min(k_left, kStageK) - 1;
            ra = gemm::make_rsrc(ATR ? pa : pa + kb, ATR ? (rows < 0 ? 0 : rows * (int)s.a.ld + bytes_a) : max(bytes_a - kb, 0));
            rb = gemm::make_rsrc(BTR ? pb : pb + kb, BTR ? (rows < 0 ? 0 : rows * (int)s.b.ld + bytes_b) : max(bytes_b - kb, 0));
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
        const int wm = (wave % WR) * 16 * MF, wn = (wave / WR) * 16 * NF;
        const int c = lane & 15, quarter = lane >> 4;
        // K 8 quarter .. + 7 of both operands.  K-contiguous: chunk `quarter` of row c,
        // fragments 16 rows apart.  K-strided: two reads of 4 rows, of which this
        // lane brings 4 columns; fragment i a granule on, across the permutation.
        const int tk = 8 * quarter + (c >> 2), tc = (c & 3) * 8;
        const auto strided_at = [&](int first, int row_bytes) {
            return (uint32_t)(tk * row_bytes + (((first >> 4) ^ swz_strided(tk)) << 5) + tc);
        };
        const uint32_t contiguous = c * 64 + 16 * swz64(c, quarter);
        const uint32_t at = ATR ? strided_at(wm, 2 * TM) : wm * 64 + contiguous;
        const uint32_t bt = TM * 64 + (BTR ? strided_at(wn, 2 * TN) : wn * 64 + contiguous);
        v8bf fa[MF], fb[NF], last_b;
        int slot = 0;
        const auto strided = [&](uint32_t from, int row_bytes) -> v8bf {
            struct {
                v4s lo, hi;
            } v;
            v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + from));
            v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + from + 4 * row_bytes));
            return __builtin_bit_cast(v8bf, v);
        };
        // rows 4 .. 7 of 8 have the permutation of rows 0 .. 3
        const auto read_a = [&](v8bf& f, int i) {
            f = ATR ? strided((at + slot * kStage) ^ (32 * i), 2 * TM)
                        : *reinterpret_cast<const v8bf*>(lds + (at + slot * kStage) + 1024 * i);
        };
        const auto read_b = [&](v8bf& f, int j) {
            f = BTR ? strided((bt + slot * kStage) ^ (32 * j), 2 * TN)
                        : *reinterpret_cast<const v8bf*>(lds + (bt + slot * kStage) + 1024 * j);
        };
        Acc acc;
        constexpr int kHalf = MF / 2 * NF;      // matrix instructions of half a stage
        // Half h of a stage's products, and after the m-th what `between` does.
        // Nothing moves from its place: reads and DMA are issued under the
        // matrix instructions' time.
        const auto products = [&](int h, auto between) {
#pragma unroll
            for (int m = 0; m < kHalf; ++m) {
                const int j = m / (MF / 2), i = m % (MF / 2) + h * (MF / 2);
                acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[j][i], 0, 0, 0);
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
                    for (int r = 0; r < 4; ++r) acc[j][i][r] = 0.0f;
        };
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
        for (int i = 0; i < MF / 2; ++i) read_a(fa[i], i);
#pragma unroll
        for (int j = 0; j < NF; ++j) read_b(fb[j], j);
        int stored = 3;         // stages since the last epilogue's stores, up to 3
        int note = 0;
        for (Item it = item_of(s, blockIdx.x); it.id < total; it = item_of(s, it.id + gridDim.x)) {
            for (int t = it.first; t < it.end; ++t) {
                products(0, [&](int m) {
#pragma unroll
                    for (int i = 0; i < MF / 2; ++i)
                        if (i * (kHalf / 2) / (MF / 2) == m) read_a(fa[MF / 2 + i], MF / 2 + i);
                    if (m == kHalf / 2) fill_begin();
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
                slot = (slot + 1) & (kRing - 1);
                products(1, [&](int m) {
#pragma unroll
                    for (int i = 0; i < MF / 2; ++i)
                        if (i * (kHalf / 4) / (MF / 2) == m) read_a(fa[i], i);
                    // a column's fragment follows its products, the last one's waits
                    // beside it for a move: it would come too late
                    const int j = m / (MF / 2);
                    if (m % (MF / 2) == MF / 2 - 1 && j < NF - 1) read_b(fb[j], j);
                    if (m == kHalf / 2) read_b(last_b, NF - 1);
#pragma unroll
                    for (int u = 0; u < kPer; ++u)
                        if (kHalf / 4 + u * (kHalf - kHalf / 4) / kPer == m) fill_one(u);
                });
                fb[NF - 1] = last_b;
                fill_end();
            }
            const uint8_t* notes = lds + kRing * kStage + note * kNotes + 1024 * kRuns * (wave / WR);
            stored = epi(it, acc, it.tm * TM + wm + 4 * quarter, it.tn * TN + wn + c, notes) ? 0 : 3;
            note = (note + 1) % kNoteSlots;
            clear();
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");        // the fills past the end
    }
};

}  // namespace ce
}  // namespace fp8mi
