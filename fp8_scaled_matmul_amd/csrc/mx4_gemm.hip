// 4-bit (OCP MXFP4) GEMM for gfx950: y = A B^T, A [m, k] and B [n, k] rows of
// E2M1 codes with one E8M0 scale byte per 32 elements, fp32 accumulation,
// bf16 output.
//
// y[i, j] = sum_b 2^(ea[i,b]-127) 2^(eb[j,b]-127) sum_{e in block b} A[i,e] B[j,e].
// v_mfma_scale_f32_32x32x64_f8f6f4 computes exactly that sum for a 32 x 32
// tile and 64 K: lane l holds 32 consecutive elements (16 bytes) of row l % 32
// of each operand and the byte of its own block's scale, so the scales cost no
// arithmetic and the products are exact before the fp32 sum (off by 2^-22.9 of
// the summed sizes at most, measured).  At the nominal clock the instruction
// does about 10 PFLOP/s on the chip; on random codes power holds the clock near
// 1.6 GHz: 6.6 with operands in registers, 6.0 with a tile's reads from LDS.
//
// Three kernels: 256 x 256 tiles where the output has enough of them, 128 x
// 128 tiles, and small tiles straight from memory where outputs are few.  The
// first two are bound by what L2 delivers to a CU, about 20 bytes a clock
// (41 to 45 GB/s at the nominal one), which falls with the clock.
#include <algorithm>

#include "device_common.h"
#include "fp8mi_internal.h"
#include "gemm_common.h"
#include "mx4_common.h"

namespace fp8mi {

namespace {

using gemm::v4f;
using gemm::v4u;
using gemm::v8i;
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kRowBytes = 128;      // one K step: 256 elements of a row
constexpr int kScaleBytes = 16;     // a row's scale bytes of one panel (two K steps)

struct MxArgs {
    const uint8_t* a;
    const uint8_t* b;
    int64_t lda, ldb;               // bytes
    const uint8_t* sa;
    const uint8_t* sb;
    int64_t psa, psb;               // bytes between scale panels
    int m, n;
    int steps;                      // K steps: ceil(k / 256)
    uint16_t* c;
    int64_t ldc;
    int tiles_m, tiles_n, group_m;
    int pair_store;                 // two adjacent outputs can be stored as one word
    fp8_counters* ctr;
};

// Position of 16-byte chunk c (0..7) in the 128-byte LDS row r.  A fragment
// read takes chunk c of 32 rows for the lower half wave and chunk c + 4 for
// the upper: 16 lanes fill the 16 slots of a 256-byte line, 32 lanes the 32
// slots of 512 bytes.  An involution in c.
__device__ inline int swz32(int r, int c)
{
    return c ^ (((r >> 2) & 1) | ((r & 2) ^ ((r >> 3) & 2)) | ((r >> 1) & 4));
}

// Lane l's 16 bytes of K quarter q (64 elements: 32 for each half wave) of
// row row0 + l % 32.
__device__ inline v8i frag(const uint8_t* lds, int row0, int q)
{
    const int l = threadIdx.x & 63;
    const int r = row0 + (l & 31);
    const uint4 v = *reinterpret_cast<const uint4*>(lds + r * kRowBytes + swz32(r, 4 * (l >> 5) + q) * 16);
    return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

template <int Q>
__device__ inline v16f mfma(const v8i& a, const v8i& b, const v16f& c, uint32_t ea, uint32_t eb)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, Q, (int)ea, Q, (int)eb);
}

// Linear workgroup id to (tile row, tile column): ids go to the XCDs in turn,
// so XCD x takes a contiguous range of the tile order, which walks group_m
// tile rows at a time.
__device__ inline void item_of(const MxArgs& p, int bid, int& tm, int& tn)
{
    const int total = p.tiles_m * p.tiles_n;
    const int xcd = bid & 7, local = bid >> 3;
    const int t = xcd * (total >> 3) + min(xcd, total & 7) + local;
    const int in_group = p.group_m * p.tiles_n;
    const int g = t / in_group;
    const int first_m = g * p.group_m;
    const int gsize = min(p.tiles_m - first_m, p.group_m);
    const int r = t - g * in_group;
    tm = first_m + r % gsize;
    tn = r / gsize;
}

// Stores one wave's MF x 2 accumulators: rows row0 + 32 i + 8 (r / 4) +
// 4 (lane / 32) + r % 4, columns col and col + 1 (col already the lane's).
template <int MF>
__device__ inline uint32_t store_out(const MxArgs& p, const v16f (&acc)[MF][2], int row0, int col)
{
    const int lane = threadIdx.x & 63;
    uint32_t nonfinite = 0;
    if (col >= p.n) return 0;
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = row0 + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
            if (row >= p.m) continue;
            const float lo = acc[i][0][r], hi = acc[i][1][r];
            const uint32_t h = gemm::pack_bf16(lo, hi);
            uint16_t* c = p.c + row * p.ldc + col;
            nonfinite += (h & 0x7F80u) == 0x7F80u;
            if (p.pair_store && col + 1 < p.n) {
                __builtin_nontemporal_store(h, reinterpret_cast<uint32_t*>(c));
                nonfinite += (h & 0x7F800000u) == 0x7F800000u;
            } else {
                c[0] = (uint16_t)h;
                if (col + 1 < p.n) {
                    c[1] = (uint16_t)(h >> 16);
                    nonfinite += (h & 0x7F800000u) == 0x7F800000u;
                }
            }
        }
    return nonfinite;
}

// ------------------------------------------------------------------ one tile per workgroup
// WR x WC waves of MF x 2 fragments (32 MF x 64 outputs) each.  A ring of
// STAGES K steps in LDS, filled by DMA STAGES - 1 steps ahead; one barrier a
// step: past it every wave has read the step before, whose slot the next DMA
// refills.  1024 x 4096 x 4096, one tile a CU: 15.7 us; its operands alone,
// 576 KB a CU, take 12.8 at what L2 delivers.  Rows of B lie permuted in each 64-row group (LDS row R holds row
// 2 (R % 32) + R / 32), so that a lane ends up with two adjacent outputs of a
// row and a half wave with 128 adjacent bytes.
template <int WR, int WC, int MF, int STAGES>
__global__ void __launch_bounds__(64 * WR * WC) k_mx4_tile_gemm(MxArgs p)
{
    constexpr int W = WR * WC;
    constexpr int TM = 32 * MF * WR, TN = 64 * WC;
    constexpr int kA = TM * kRowBytes, kB = TN * kRowBytes;
    constexpr int kStage = kA + kB + (TM + TN) * kScaleBytes;
    constexpr int kData = (TM + TN) / 8 / W;        // DMA instructions of a wave and step
    constexpr int kScale = (TM + TN) / 64;          // over all waves
    static_assert((TM + TN) / 8 % W == 0 && TM / 8 % W == 0, "whole DMA instructions");
    static_assert(kScale <= W || kScale % W == 0, "scale DMA");
    constexpr int kScalePer = (kScale + W - 1) / W;
    constexpr int kPer = kData + kScalePer;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    int tm, tn;
    item_of(p, blockIdx.x, tm, tn);
    const int m0 = tm * TM, n0 = tn * TN;
    const int nt = p.steps;
    const int64_t rows_a = min(p.m - m0, TM), rows_b = min(p.n - n0, TN);
    const v4u ra = gemm::make_rsrc(p.a + (int64_t)m0 * p.lda, (uint32_t)(rows_a * p.lda));
    const v4u rb = gemm::make_rsrc(p.b + (int64_t)n0 * p.ldb, (uint32_t)(rows_b * p.ldb));
    const uint32_t base = gemm::lds_addr(lds);

    // K step t into its ring slot: kPer instructions per wave
    const auto fill = [&](int t) {
        const bool live = t < nt;
        const int slot = t % STAGES;
        const uint32_t to = base + slot * kStage;
        const int q = lane >> 3, pos = lane & 7;
#pragma unroll
        for (int j = 0; j < kData; ++j) {
            const int R = 8 * (j * W + wave) + q;       // LDS row: A's, then B's
            uint32_t off;
            v4u rs;
            if (8 * (j * W) < TM) {                     // uniform in j: TM is a multiple of 8 W
                off = (uint32_t)(R * p.lda + 16 * swz32(R, pos));
                rs = ra;
            } else {
                const int Rb = R - TM;
                const int g = (Rb & ~63) + 2 * (Rb & 31) + ((Rb >> 5) & 1);
                off = (uint32_t)(g * p.ldb + 16 * swz32(Rb, pos));
                rs = rb;
            }
            rs.z = live ? rs.z : 0u;
            gemm::dma16(to + 1024 * (j * W + wave), off + (uint32_t)t * kRowBytes, rs);
        }
#pragma unroll
        for (int j = 0; j < kScalePer; ++j) {
            const int u = j * W + wave;                 // 64 rows of scales; past the last: a repeat of it
            const int uu = min(u, kScale - 1);
            const int64_t panel = t >> 1;
            const uint8_t* src;
            uint32_t off, bytes;
            if (uu < TM / 64) {
                src = p.sa + panel * p.psa + (int64_t)m0 * kScaleBytes;
                bytes = (uint32_t)rows_a * kScaleBytes;
                off = (uint32_t)(64 * uu + lane) * kScaleBytes;
            } else {
                src = p.sb + panel * p.psb + (int64_t)n0 * kScaleBytes;
                bytes = (uint32_t)rows_b * kScaleBytes;
                off = (uint32_t)(64 * (uu - TM / 64) + 2 * (lane & 31) + (lane >> 5)) * kScaleBytes;
            }
            gemm::dma16(to + kA + kB + 1024 * uu, off, gemm::make_rsrc(src, live ? bytes : 0u));
        }
    };

    v16f acc[MF][2];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    const int wm = (wave % WR) * 32 * MF, wn = (wave / WR) * 64;
#pragma unroll
    for (int t = 0; t < STAGES - 1; ++t) fill(t);
    for (int t = 0; t < nt; ++t) {
        // all but the newest STAGES - 2 steps have landed
        if constexpr (kPer * (STAGES - 2) == 0)
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        else
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kPer * (STAGES - 2)) : "memory");
        gemm::barrier_lds();
        fill(t + STAGES - 1);
        const uint8_t* st = lds + (t % STAGES) * kStage;
        const uint8_t* la = st;
        const uint8_t* lb = st + kA;
        const uint8_t* ls = st + kA + kB + (t & 1) * 8 + 4 * (lane >> 5);
        uint32_t ea[MF], eb[2];
#pragma unroll
        for (int i = 0; i < MF; ++i)
            ea[i] = *reinterpret_cast<const uint32_t*>(ls + (wm + 32 * i + (lane & 31)) * kScaleBytes);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            eb[j] = *reinterpret_cast<const uint32_t*>(ls + (TM + wn + 32 * j + (lane & 31)) * kScaleBytes);
        const auto quarter = [&](auto Q) {
            constexpr int q = decltype(Q)::value;
            v8i fa[MF], fb[2];
#pragma unroll
            for (int i = 0; i < MF; ++i) fa[i] = frag(la, wm + 32 * i, q);
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[j] = frag(lb, wn + 32 * j, q);
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mfma<q>(fa[i], fb[j], acc[i][j], ea[i], eb[j]);
        };
        quarter(std::integral_constant<int, 0>{});
        quarter(std::integral_constant<int, 1>{});
        quarter(std::integral_constant<int, 2>{});
        quarter(std::integral_constant<int, 3>{});
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t nonfinite = store_out<MF>(p, acc, m0 + wm, n0 + wn + 2 * (lane & 31));
    flush_counters(p.ctr, 0, 0, 0, nonfinite);
}

int tiles_of(int64_t size, int64_t tile) { return (int)((size + tile - 1) / tile); }

template <int WR, int WC, int MF, int STAGES>
hipError_t launch_tile(MxArgs p, hipStream_t stream)
{
    constexpr int TM = 32 * MF * WR, TN = 64 * WC;
    constexpr int kLds = STAGES * ((TM + TN) * (kRowBytes + kScaleBytes));
    p.tiles_m = tiles_of(p.m, TM);
    p.tiles_n = tiles_of(p.n, TN);
    p.group_m = 4;
    const auto kernel = k_mx4_tile_gemm<WR, WC, MF, STAGES>;
    static mx4::LdsLimit limit;
    const hipError_t e = limit.raise(reinterpret_cast<const void*>(kernel), kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(p.tiles_m * p.tiles_n), dim3(64 * WR * WC), kLds, stream, p);
    return hipGetLastError();
}

// ------------------------------------------------------------------ 256 x 256 tiles
// 8 waves of 4 x 2 fragments (128 x 64 outputs, 128 accumulator registers), one
// workgroup per CU, which walks its tiles.  A stage is 128 K (64 bytes of a
// row, two matrix instructions deep); a ring of four in LDS, and three panels
// of scales (512 K: four stages, or the two that end a K range) beside it.
// The stages of all of a workgroup's tiles are one stream, filled by DMA four
// ahead, so that a tile's first stages arrive while the one before is stored.
// Fragments are read half a stage ahead of their products, which leaves one
// barrier a stage: in its middle, once the whole of it has been read.
// 16384 x 8192 x 7168: 460 to 480 us, 4.0 to 4.2 PFLOP/s, matrix units busy 53 %
// of the time at 1.8 GHz; zeros for operands, which take little power, 358 us: the
// 34 KB of a stage at 43.5 GB/s a CU.  (One tile a workgroup: 522 us; reads and
// products of a stage not overlapped: 587 us on random operands.)
constexpr int kBig = 256, kBigThreads = 512;
constexpr int kStageBytes = 2 * kBig * 64;      // A's 256 rows, then B's
constexpr int kPanelBytes = 2 * kBig * kScaleBytes;
constexpr int kBigPanels = 3;
constexpr int kBigLds = 4 * kStageBytes + kBigPanels * kPanelBytes;
constexpr int kBigStores = 64;                  // of a tile, by a wave

// Position of 16-byte chunk c (0..3) in the 64-byte LDS row r: as for swz32,
// 16 rows at one chunk fill the 16 slots of a 256-byte line and 32 rows with
// two chunks the 32 of 512 bytes (timed alone, as fast as adjacent addresses;
// the scale words, 16 bytes apart, take 1.3 times as long as adjacent ones).  An
// involution in c.
__device__ inline int swz64(int r, int c) { return c ^ (((r >> 2) & 1) | (((r >> 1) ^ (r >> 2) ^ (r >> 3)) & 1) << 1); }

struct BigTile {
    int id;             // past the last: no tile
    int m0, n0;
};
__device__ inline BigTile big_tile(const MxArgs& p, int id)
{
    BigTile it{id, 0, 0};
    if (id < p.tiles_m * p.tiles_n) {
        int tm, tn;
        item_of(p, id, tm, tn);
        it.m0 = tm * kBig;
        it.n0 = tn * kBig;
    }
    return it;
}

// Tracks the largest |bf16| stored, two packed maxima.
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
__device__ inline void track_max(us2& mx, uint32_t w)
{
    mx = __builtin_elementwise_max(mx, __builtin_bit_cast(us2, w & 0x7FFF7FFFu));
}

__global__ void __launch_bounds__(kBigThreads, 2) k_mx4_big_gemm(MxArgs p)
{
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int total = p.tiles_m * p.tiles_n;
    const int nt = 2 * p.steps;         // stages of a tile
    const uint32_t base = gemm::lds_addr(lds);
    const uint32_t scales = base + 4 * kStageBytes;

    // ---- the stream of fills
    // This wave's DMA of a stage: 2 x 16 rows of A and of B, 1 KB each.  Rows
    // of B lie permuted as in the kernel above.  Waves 0-3 bring the scales
    // of 64 rows of A, 4-7 of B.
    uint32_t va[2], vb[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int R = 32 * wave + 16 * j + (lane >> 2);
        const int g = (R & ~63) + 2 * (R & 31) + ((R >> 5) & 1);
        va[j] = (uint32_t)(R * p.lda + 16 * swz64(R, lane & 3));
        vb[j] = (uint32_t)(g * p.ldb + 16 * swz64(R, lane & 3));
    }
    const int scale_row = wave < 4 ? 64 * wave + lane : 64 * (wave - 4) + 2 * (lane & 31) + (lane >> 5);
    const uint32_t vs = (uint32_t)scale_row * kScaleBytes;
    const int64_t ps = wave < 4 ? p.psa : p.psb;
    BigTile f = big_tile(p, blockIdx.x);        // the tile being filled, its next stage
    int ft = 0, fslot = 0, fpanel = 0;          // ring positions of the next stage and panel
    v4u ra, rb, rs;
    const uint8_t* sp;
    const auto describe = [&]() {
        const bool live = f.id < total;
        const int64_t rows_a = min(p.m - f.m0, kBig), rows_b = min(p.n - f.n0, kBig);
        ra = gemm::make_rsrc(p.a + (int64_t)f.m0 * p.lda, live ? (uint32_t)(rows_a * p.lda) : 0u);
        rb = gemm::make_rsrc(p.b + (int64_t)f.n0 * p.ldb, live ? (uint32_t)(rows_b * p.ldb) : 0u);
        sp = (wave < 4 ? p.sa + (int64_t)f.m0 * kScaleBytes : p.sb + (int64_t)f.n0 * kScaleBytes);
        rs = gemm::make_rsrc(sp, live ? (uint32_t)(wave < 4 ? rows_a : rows_b) * kScaleBytes : 0u);
    };
    describe();
    // The next stage (4 instructions a wave; one more where it begins a panel).
    const auto fill = [&]() {
        if ((ft & 3) == 0) {
            gemm::dma16(scales + fpanel * kPanelBytes + 1024 * wave, vs,
                        gemm::make_rsrc(sp + (int64_t)(ft >> 2) * ps, rs.z));
            fpanel = fpanel == kBigPanels - 1 ? 0 : fpanel + 1;
        }
        const uint32_t to = base + fslot * kStageBytes + 2048 * wave;
        const uint32_t kb = (uint32_t)ft * 64;
#pragma unroll
        for (int j = 0; j < 2; ++j) gemm::dma16(to + 1024 * j, va[j] + kb, ra);
#pragma unroll
        for (int j = 0; j < 2; ++j) gemm::dma16(to + kBig * 64 + 1024 * j, vb[j] + kb, rb);
        fslot = (fslot + 1) & 3;
        if (++ft == nt && f.id < total) {
            f = big_tile(p, f.id + gridDim.x);
            ft = 0;
            describe();
        }
    };

    // ---- the fragments
    // This lane's row of a fragment and its chunk of the first matrix
    // instruction (the second's lies 32 bytes across); the swizzle is the
    // same in every fragment.
    const int wm = (wave & 1) * 128, wn = (wave >> 1) * 64;
    const int fr = lane & 31, half = lane >> 5;
    const uint32_t at0 = (uint32_t)(fr * 64 + 16 * swz64(fr, half)), at1 = at0 ^ 32u;
    const uint8_t* fa_at[2] = {lds + wm * 64 + at0, lds + wm * 64 + at1};
    const uint8_t* fb_at[2] = {lds + (kBig + wn) * 64 + at0, lds + (kBig + wn) * 64 + at1};
    const uint8_t* sa_at = lds + 4 * kStageBytes + (wm + fr) * kScaleBytes;
    const uint8_t* sb_at = lds + 4 * kStageBytes + (kBig + wn + fr) * kScaleBytes;
    v8i fa[2][4], fb[2][2];
    uint32_t ea[4], eb[2], na[4], nb[2];        // scale words of this stage, of the next
    int slot = 0, panel = 0;                    // the ring position and panel of the next fragments
    const auto read = [&](auto KK) {
        constexpr int kk = decltype(KK)::value;
        const auto get = [](const uint8_t* from) {
            const uint4 v = *reinterpret_cast<const uint4*>(from);
            return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
        };
        const int ring = slot * kStageBytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) fb[kk][i] = get(fb_at[kk] + ring + 2048 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) fa[kk][i] = get(fa_at[kk] + ring + 2048 * i);
    };
    // block 2 kk + lane / 32 of stage t: that byte of the panel's word t % 4
    const auto read_scales = [&](int t) {
        const int at = panel * kPanelBytes + 4 * (t & 3);
#pragma unroll
        for (int i = 0; i < 2; ++i) nb[i] = *reinterpret_cast<const uint32_t*>(sb_at + at + 512 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) na[i] = *reinterpret_cast<const uint32_t*>(sa_at + at + 512 * i);
    };
    const auto take_scales = [&]() {
#pragma unroll
        for (int i = 0; i < 2; ++i) eb[i] = nb[i] >> (8 * half);
#pragma unroll
        for (int i = 0; i < 4; ++i) ea[i] = na[i] >> (8 * half);
    };

    v16f acc[4][2];
    // Matrix instructions lo .. hi - 1 of the 8 of a half stage.  What is
    // written around a call stays on its side.
    const auto products = [&](auto KK, int lo, int hi) {
        constexpr int kk = decltype(KK)::value;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 8; ++m)
            if (m >= lo && m < hi)
                acc[m >> 1][m & 1] =
                    mfma<2 * kk>(fa[kk][m >> 1], fb[kk][m & 1], acc[m >> 1][m & 1], ea[m >> 1], eb[m & 1]);
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    };
    clear();

#pragma unroll 1
    for (int i = 0; i < 4; ++i) fill();
    // the first stage and its scales (three stages and at most one panel are younger)
    asm volatile("s_waitcnt vmcnt(12)" ::: "memory");
    gemm::barrier_lds();
    read(std::integral_constant<int, 0>{});
    read_scales(0);
    uint32_t nonfinite = 0;
    int stored = 3;                             // stages since the last tile's stores, up to 3
    for (BigTile it = big_tile(p, blockIdx.x); it.id < total; it = big_tile(p, it.id + gridDim.x)) {
        for (int t = 0; t < nt; ++t) {
            // the stage's second half is read under the first's products
            take_scales();
            products(std::integral_constant<int, 0>{}, 0, 2);
            read(std::integral_constant<int, 1>{});
            products(std::integral_constant<int, 0>{}, 2, 8);
            // The next stage has landed: the two after it are younger.  So are
            // a tile's stores to the three stages that were filled before them.
            if (stored < 3) {
                static_assert(kBigStores + 8 >= 63, "stores and fills younger than the stage");
                asm volatile("s_waitcnt vmcnt(63)" ::: "memory");
                ++stored;
            } else {
                asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
            }
            // past this every wave has read the whole stage: its slot is free
            gemm::barrier_lds();
            products(std::integral_constant<int, 1>{}, 0, 4);
            fill();
            slot = (slot + 1) & 3;
            const int next = t + 1 == nt ? 0 : t + 1;
            if ((next & 3) == 0) panel = panel == kBigPanels - 1 ? 0 : panel + 1;
            read(std::integral_constant<int, 0>{});
            read_scales(next);
            products(std::integral_constant<int, 1>{}, 4, 8);
        }
        if (p.pair_store) {
            // 64 stores of two adjacent outputs, those out of range dropped
            const int64_t rows_c = min(p.m - it.m0, kBig);
            const __amdgpu_buffer_rsrc_t rc = gemm::make_store_rsrc(
                p.c + (int64_t)it.m0 * p.ldc, (uint32_t)(((rows_c - 1) * p.ldc + p.n) * 2));
            const int col = it.n0 + wn + 2 * fr;
            const uint32_t at = col < p.n ? (uint32_t)((wm + 4 * half) * p.ldc + col) * 2 : gemm::kOutOfRange;
            us2 mx = us2{0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const uint32_t h = gemm::pack_bf16(acc[i][0][r], acc[i][1][r]);
                    track_max(mx, h);
                    const uint32_t down = (uint32_t)(32 * i + 8 * (r >> 2) + (r & 3)) * (uint32_t)p.ldc * 2;
                    __builtin_amdgcn_raw_buffer_store_b32(h, rc, (int)(at + down), 0, 0);
                }
            stored = 0;
            if (p.ctr && (mx.x >= 0x7F80u || mx.y >= 0x7F80u)) {
                // past the edges a NaN scale of the other operand makes NaN, too
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        if (col >= p.n || wm + 4 * half + 32 * i + 8 * (r >> 2) + (r & 3) >= rows_c) continue;
                        const uint32_t h = gemm::pack_bf16(acc[i][0][r], acc[i][1][r]);
                        nonfinite += ((h & 0x7F80u) == 0x7F80u) + ((h & 0x7F800000u) == 0x7F800000u);
                    }
            }
        } else {
            nonfinite += store_out<4>(p, acc, it.m0 + wm, it.n0 + wn + 2 * fr);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        clear();
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");    // the fills past the end
    flush_counters(p.ctr, 0, 0, 0, nonfinite);
}

hipError_t launch_big(MxArgs p, hipStream_t stream)
{
    p.tiles_m = tiles_of(p.m, kBig);
    p.tiles_n = tiles_of(p.n, kBig);
    p.group_m = 4;
    p.pair_store = p.pair_store && p.n % 2 == 0;
    static mx4::LdsLimit limit;
    const hipError_t e = limit.raise(reinterpret_cast<const void*>(k_mx4_big_gemm), kBigLds);
    if (e != hipSuccess) return e;
    const int grid = std::min(p.tiles_m * p.tiles_n, gemm_num_cus());
    hipLaunchKernelGGL(k_mx4_big_gemm, dim3(grid), dim3(kBigThreads), kBigLds, stream, p);
    return hipGetLastError();
}

// ------------------------------------------------------------------ straight from memory
// Few outputs, where the read of B (a weight) or the mere latency counts: a
// workgroup takes 16 CT rows of A by 16 RT rows of B, its KW waves share K,
// and the operands go from memory to the registers of
// v_mfma_scale_f32_16x16x128 (B's rows as the instruction's rows, A's as its
// columns): no LDS but for the waves' sums at the end, which are added in
// order.  A step is U units of 256 K; the next one is read under this one's
// products.  1 x 8192 x 8192: 8.5 us, 4.2 TB/s; 333 x 1000 x 1568: 7 us, which
// is latency (a launch alone takes 2.2).
struct Unit {
    uint4 q[2];         // K 32 (l / 16) on of either 128
};

template <int RT, int CT, int KW, int U>
__global__ void __launch_bounds__(64 * KW) k_mx4_direct_gemm(MxArgs p)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    v4f* red = reinterpret_cast<v4f*>(lds);     // [KW, RT CT, 64]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, q = lane >> 4;
    int tm, tn;
    item_of(p, blockIdx.x, tm, tn);
    const int m0 = tm * 16 * CT, n0 = tn * 16 * RT;

    // operands 0 .. RT - 1: B's rows, then A's
    constexpr int F = RT + CT;
    uint32_t at[F], sat[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const int row = f < RT ? min(16 * f + c16, p.n - 1 - n0) : min(16 * (f - RT) + c16, p.m - 1 - m0);
        at[f] = (uint32_t)(row * (f < RT ? p.ldb : p.lda) + 16 * q);
        sat[f] = (uint32_t)(row * kScaleBytes);
    }
    const uint8_t* b = p.b + (int64_t)n0 * p.ldb;
    const uint8_t* a = p.a + (int64_t)m0 * p.lda;
    const uint8_t* sb = p.sb + (int64_t)n0 * kScaleBytes;
    const uint8_t* sa = p.sa + (int64_t)m0 * kScaleBytes;
    struct Step {
        Unit u[U][F];
        uint2 s[U][F];
    };
    const int steps = (p.steps + U - 1) / U;
    const int first = steps * wave / KW, end = steps * (wave + 1) / KW;
    const auto get = [&](Step& x, int i) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            // past the end the last unit again, not used
            const int u = min(min(i, end - 1) * U + k, p.steps - 1);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const uint8_t* from = (f < RT ? b : a) + 128 * u;
                const uint8_t* sfrom = (f < RT ? sb + (u >> 1) * p.psb : sa + (u >> 1) * p.psa) + 8 * (u & 1);
                x.s[k][f] = *reinterpret_cast<const uint2*>(sfrom + sat[f]);
                x.u[k][f].q[0] = *reinterpret_cast<const uint4*>(from + at[f]);
                x.u[k][f].q[1] = *reinterpret_cast<const uint4*>(from + 64 + at[f]);
            }
        }
    };
    v4f acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = v4f{0, 0, 0, 0};
    const auto products = [&](const Step& x, int i) {
        const int sh = 8 * q;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i >= end || i * U + k >= p.steps) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v8i v[F];
                uint32_t e[F];
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    const uint4 w = x.u[k][f].q[h];
                    v[f] = v8i{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
                    e[f] = (h ? x.s[k][f].y : x.s[k][f].x) >> sh;
                }
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v[r], v[RT + c], acc[r][c], 4, 4, 0,
                                                                                     (int)e[r], 0, (int)e[RT + c]);
            }
        }
    };
    Step x0, x1;
    if (first < end) {
        get(x0, first);
        for (int i = first; i < end; i += 2) {
            get(x1, i + 1);
            products(x0, i);
            get(x0, i + 2);
            products(x1, i + 1);
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) red[(wave * RT * CT + r * CT + c) * 64 + lane] = acc[r][c];
    __syncthreads();
    uint32_t nonfinite = 0;
    for (int i = threadIdx.x; i < RT * CT * 64; i += 64 * KW) {
        v4f s = red[i];
#pragma unroll
        for (int w = 1; w < KW; ++w) s += red[w * RT * CT * 64 + i];
        const int l = i & 63, c = (i >> 6) % CT, r = (i >> 6) / CT;
        const int row = m0 + 16 * c + (l & 15), col = n0 + 16 * r + 4 * (l >> 4);
        if (row >= p.m || col >= p.n) continue;
        const uint32_t lo = gemm::pack_bf16(s[0], s[1]), hi = gemm::pack_bf16(s[2], s[3]);
        uint16_t* to = p.c + row * p.ldc + col;
        if (p.pair_store && col + 3 < p.n) {
            reinterpret_cast<uint32_t*>(to)[0] = lo;
            reinterpret_cast<uint32_t*>(to)[1] = hi;
            nonfinite += ((lo & 0x7F80u) == 0x7F80u) + ((lo & 0x7F800000u) == 0x7F800000u) +
                         ((hi & 0x7F80u) == 0x7F80u) + ((hi & 0x7F800000u) == 0x7F800000u);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < p.n) {
                    const uint16_t h = (uint16_t)((j < 2 ? lo : hi) >> (16 * (j & 1)));
                    to[j] = h;
                    nonfinite += (h & 0x7F80u) == 0x7F80u;
                }
        }
    }
    flush_counters(p.ctr, 0, 0, 0, nonfinite);
}

template <int RT, int CT, int KW, int U>
hipError_t launch_direct(MxArgs p, hipStream_t stream)
{
    p.tiles_m = tiles_of(p.m, 16 * CT);
    p.tiles_n = tiles_of(p.n, 16 * RT);
    p.group_m = 4;
    const int lds = KW * RT * CT * 1024;
    hipLaunchKernelGGL((k_mx4_direct_gemm<RT, CT, KW, U>), dim3(p.tiles_m * p.tiles_n), dim3(64 * KW), lds, stream, p);
    return hipGetLastError();
}

}  // namespace

bool mx4_gemm_fits(int64_t m, int64_t n)
{
    return ((m + kBig - 1) / kBig) * ((n + kBig - 1) / kBig) < (int64_t)1 << 31;
}

hipError_t launch_mx4_gemm(const Mx4GemmArgs& g, hipStream_t stream)
{
    if (g.m == 0 || g.n == 0) return hipSuccess;
    if (g.k == 0) return launch_zero_bf16(static_cast<uint16_t*>(g.c), (int)g.m, (int)g.n, g.ldc, stream);
    MxArgs p;
    p.a = g.a;
    p.b = g.b;
    p.lda = g.lda;
    p.ldb = g.ldb;
    p.sa = g.sa;
    p.sb = g.sb;
    p.psa = g.psa;
    p.psb = g.psb;
    p.m = (int)g.m;
    p.n = (int)g.n;
    p.steps = (int)((g.k + mx4::kRowAlign - 1) / mx4::kRowAlign);
    p.c = static_cast<uint16_t*>(g.c);
    p.ldc = g.ldc;
    p.pair_store = g.ldc % 2 == 0 && (reinterpret_cast<uintptr_t>(g.c) & 3u) == 0;
    p.ctr = g.ctr;
    // The tile with the least to bring to the busiest CU: its rows of A and B
    // times the tiles that fall to one CU, where a row costs the tiles that
    // share it through LDS about 0.55 (128 x 128) and 0.65 (256 x 256) of what
    // it costs those that read it straight.  Measured, us (weights from memory,
    // kernels back to back), the chosen one first:
    //   1 x 8192 x 8192      16 x 32: 10.1    16 x 16: 10.7    32 x 32: 10.8
    //   12 x 16000 x 3000    16 x 64: 10.0    16 x 32: 12.4    64 x 64: 9.8
    //   128 x 512 x 512      16 x 16: 2.9     16 x 32: 3.2     32 x 32: 3.6
    //   100 x 700 x 16384    16 x 32: 15.8    16 x 16: 20.4    32 x 32: 20.3
    //   500 x 300 x 4096     32 x 32: 7.9     16 x 32: 10.8    64 x 32: 9.9
    //   333 x 1000 x 1568    64 x 32: 7.2     32 x 32: 8.9     64 x 64: 8.6
    //   2000 x 300 x 1000    64 x 64: 6.7     64 x 32: 11.5    128 x 128: 7.7
    //   1500 x 1500 x 8192   128 x 128: 26.0  64 x 64: 69.5
    //   4096 x 2048 x 7168   128 x 128: 38.5  256 x 256: 50.0
    //   3000 x 3000 x 512    256 x 256: 11.7  128 x 128: 13.6
    const int64_t cus = gemm_num_cus();
    static constexpr struct {
        int tm, tn;
        double row;
        int threads;        // of a tile; 0: workgroups walk the tiles
    } kTiles[] = {{16, 16, 1.0, 256}, {16, 32, 1.0, 256}, {16, 64, 1.0, 256},    {32, 32, 1.0, 256},
                  {64, 32, 1.0, 256}, {64, 64, 1.0, 128}, {128, 128, 0.55, 512}, {256, 256, 0.65, 0}};
    int best = -1;
    double least = 0.0;
    for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
        const int64_t tiles = ((g.m + kTiles[i].tm - 1) / kTiles[i].tm) * ((g.n + kTiles[i].tn - 1) / kTiles[i].tn);
        if (tiles * kTiles[i].threads >= kMaxLaunch) continue;
        const double cost = (double)((tiles + cus - 1) / cus) * (kTiles[i].tm + kTiles[i].tn) * kTiles[i].row;
        if (best < 0 || cost < least) {
            best = i;
            least = cost;
        }
    }
    switch (best) {
    case 0: return launch_direct<1, 1, 4, 2>(p, stream);
    case 1: return launch_direct<2, 1, 4, 2>(p, stream);
    case 2: return launch_direct<4, 1, 4, 1>(p, stream);
    case 3: return launch_direct<2, 2, 4, 2>(p, stream);
    case 4: return launch_direct<2, 4, 4, 1>(p, stream);
    case 5: return launch_direct<4, 4, 2, 1>(p, stream);
    case 6: {
        // One tile a CU: three stages (108 KB of LDS); more: two, and two
        // workgroups a CU.  512 x 8192 x 4096 (256 tiles): 16.6 and 19.8 us;
        // 1100 x 4096 x 4096 (288): 28.5 and 20.3 us.
        const int64_t tiles = ((g.m + 127) / 128) * ((g.n + 127) / 128);
        return tiles <= cus ? launch_tile<4, 2, 1, 3>(p, stream) : launch_tile<4, 2, 1, 2>(p, stream);
    }
    default: return launch_big(p, stream);
    }
}

}  // namespace fp8mi
