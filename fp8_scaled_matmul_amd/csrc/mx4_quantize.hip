// 4-bit (OCP MXFP4) quantizer and dequantizer for gfx950.
//
// Per block of 32 consecutive elements: amax over the finite ones, the
// smallest power of two s with amax / s <= 6, then E2M1(x / s), to nearest
// even or stochastically.  The optional transposed copy is the quantization
// of x^T (blocks of 32 rows of one column, with scales of their own), not a
// transposition of the codes.
//
// Both directions come from one read of x.  A lane holds 8 columns of one or
// several rows, so a row block is a quad of lanes and its amax two
// quad-permutes away; in the tile kernel a lane holds 8 x 8 elements, so a
// column block is the 4 lanes 16 apart.  The casts are one conversion
// instruction per two elements, which leaves the kernels bound by memory:
// per element 2 (4) bytes read and 17/32 written, twice with the transposed
// copy.
#include <algorithm>

#include "device_common.h"
#include "fp8mi_internal.h"
#include "mx4_common.h"

namespace fp8mi {

namespace {

typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
// The same 16 bytes wherever an element may lie: one access of any alignment.
typedef uint32_t u4x2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u4x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f4x4 __attribute__((ext_vector_type(4), aligned(4)));

constexpr uint32_t kNonFinite = 0x7F800000u;
constexpr uint32_t kNanKey = 0xFFFFFFFFu;   // the key of a block that holds a NaN

struct Mx4Args {
    const void* x;
    int64_t rows, cols, ld;
    uint8_t* q;
    int64_t ldq;
    uint8_t* s;
    int64_t sps;        // bytes between the scale panels
    uint8_t* qt;
    int64_t ldqt;
    uint8_t* st;
    int64_t stps;
    const uint64_t* seed;
    fp8_counters* ctr;
    int tiles_c;
};

// ------------------------------------------------------------------ lanes
template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128;

__device__ inline uint32_t quad_max(uint32_t v)
{
    v = max(v, dpp<kXor1>(v));
    return max(v, dpp<kXor2>(v));
}
// Over the 4 lanes that are 16 apart.
__device__ inline uint32_t stride16_max(uint32_t v)
{
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max((uint32_t)b[0], (uint32_t)b[1]);
}
__device__ inline us2 pkmax(us2 a, us2 b) { return __builtin_elementwise_max(a, b); }
__device__ inline us2 stride16_pkmax(us2 v)
{
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    const uint32_t m = __builtin_bit_cast(uint32_t, pkmax(__builtin_bit_cast(us2, (uint32_t)a[0]),
                                                          __builtin_bit_cast(us2, (uint32_t)a[1])));
    const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return pkmax(__builtin_bit_cast(us2, (uint32_t)b[0]), __builtin_bit_cast(us2, (uint32_t)b[1]));
}

// ------------------------------------------------------------------ eight elements of a row
template <int DT>
struct Row8 {
    static constexpr int kWords = DT == 0 ? 4 : 8;
    uint32_t w[kWords];

    __device__ float get(int c) const
    {
        if constexpr (DT == 0)
            return (c & 1) ? bf16_hi(w[c >> 1]) : bf16_lo(w[c >> 1]);
        else
            return __builtin_bit_cast(float, w[c]);
    }
    // |x| as fp32 bits; Inf counts as 0, NaN as kNanKey
    __device__ uint32_t key(int c) const
    {
        const uint32_t a = __builtin_bit_cast(uint32_t, get(c)) & 0x7FFFFFFFu;
        return a < kNonFinite ? a : a == kNonFinite ? 0u : kNanKey;
    }
    // max |x| bits with nothing left out
    __device__ uint32_t raw_max() const
    {
        if constexpr (DT == 0) {
            us2 m = us2{0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) m = pkmax(m, __builtin_bit_cast(us2, w[i] & 0x7FFF7FFFu));
            return (uint32_t)(m.x > m.y ? m.x : m.y) << 16;
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
            return m;
        }
    }
};

// Elements col .. col + 7 of a row, zeros past the matrix.
template <int DT>
__device__ inline Row8<DT> load8(const Mx4Args& p, int64_t row, int64_t col)
{
    Row8<DT> r;
#pragma unroll
    for (int i = 0; i < Row8<DT>::kWords; ++i) r.w[i] = 0;
    if (row >= p.rows) return r;
    if constexpr (DT == 0) {
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.ld + col;
        if (col + 8 <= p.cols) {
            const u4 v = __builtin_nontemporal_load(reinterpret_cast<const u4x2*>(x));
            r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (col + c < p.cols) r.w[c >> 1] |= (uint32_t)x[c] << (16 * (c & 1));
        }
    } else {
        const uint32_t* x = static_cast<const uint32_t*>(p.x) + row * p.ld + col;
        if (col + 8 <= p.cols) {
            const u4 v = __builtin_nontemporal_load(reinterpret_cast<const u4x4*>(x));
            const u4 u = __builtin_nontemporal_load(reinterpret_cast<const u4x4*>(x + 4));
            r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
            r.w[4] = u.x; r.w[5] = u.y; r.w[6] = u.z; r.w[7] = u.w;
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (col + c < p.cols) r.w[c] = x[c];
        }
    }
    return r;
}

__device__ inline uint32_t byte_of_key(uint32_t key) { return key == kNanKey ? 255u : mx4::scale_byte(key); }

// One row's eight codes.  h: the random bits of its four column pairs.
template <int DT, bool SR>
__device__ inline uint32_t cast_row(const Row8<DT>& r, float s, const uint32_t h[4])
{
    if constexpr (SR) {
        float x[8];
        uint32_t se[4], so[4];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = r.get(c);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            se[p] = h[p] << 16;
            so[p] = (h[p] >> 1) & 0x7FFF8000u;
        }
        return mx4::cast8_sr(x, se, so, s);
    } else if constexpr (DT == 0) {
        return mx4::cast8_rne(r.w, s);
    } else {
        float x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = r.get(c);
        return mx4::cast8_rne(x, s);
    }
}

// Events among the eight elements of a row and their codes.
template <int DT>
__device__ inline void count_row(const Row8<DT>& r, uint32_t codes, uint32_t byte, uint32_t& sat, uint32_t& und,
                                 uint32_t& nan)
{
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t a = __builtin_bit_cast(uint32_t, r.get(c)) & 0x7FFFFFFFu;
        nan += a > kNonFinite;
        sat += a == kNonFinite;
        und += a != 0 && byte != 255u && ((codes >> (4 * c)) & 7u) == 0;
    }
}

// ------------------------------------------------------------------ along the rows only
constexpr int kRowThreads = 256;
constexpr int kRowsPerWave = 4;

// A wave takes 512 columns of kRowsPerWave rows, 8 columns a lane, every load
// first: 16 blocks a row, whose codes are 256 and whose scales 16 adjacent
// bytes.  8192 x 8192 fp32: 55 us, 5.5 TB/s (a device copy of 2 GiB: 5.0);
// one row: 2.4 us.
template <int DT, bool SR, bool COUNT>
__global__ void __launch_bounds__(kRowThreads) k_mx4_rows(Mx4Args p)
{
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t group = item / p.tiles_c;
    const int panel = (int)(item - group * p.tiles_c);
    const int64_t row0 = group * kRowsPerWave;
    const int64_t col = (int64_t)panel * mx4::kPanel + 8 * lane;
    uint32_t sat = 0, und = 0, nan = 0;
    if (row0 < p.rows) {
        Row8<DT> r[kRowsPerWave];
#pragma unroll
        for (int j = 0; j < kRowsPerWave; ++j) r[j] = load8<DT>(p, row0 + j, col);
        uint32_t seed_lo = 0, pk[4];
        if constexpr (SR) {
            const uint64_t seed = *p.seed;
            seed_lo = (uint32_t)seed;
#pragma unroll
            for (int c = 0; c < 4; ++c) pk[c] = mx4::pair_key((uint32_t)(col >> 1) + c, (uint32_t)(seed >> 32));
        }
        const int64_t padded = (p.cols + mx4::kRowAlign - 1) & ~(int64_t)(mx4::kRowAlign - 1);
#pragma unroll
        for (int j = 0; j < kRowsPerWave; ++j) {
            const int64_t row = row0 + j;
            uint32_t key = quad_max(r[j].raw_max());
            if (key >= kNonFinite) {
                uint32_t k = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) k = max(k, r[j].key(c));
                key = quad_max(k);
            }
            const uint32_t byte = byte_of_key(key);
            uint32_t h[4] = {0, 0, 0, 0};
            if constexpr (SR) {
                const uint32_t rk = mx4::row_key((uint32_t)row, seed_lo);
#pragma unroll
                for (int c = 0; c < 4; ++c) h[c] = mx4::mix(rk ^ pk[c]);
            }
            uint32_t w = cast_row<DT, SR>(r[j], mx4::scale_float(byte), h);
            w = byte == 255u ? 0u : w;
            // the four blocks of 16 lanes: their bytes to one word
            uint32_t sw = byte << (8 * ((lane >> 2) & 3));
            sw |= dpp<kRor4>(sw);
            sw |= dpp<kRor8>(sw);
            if (row < p.rows) {
                if (col < padded)
                    __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(p.q + row * p.ldq + (col >> 1)));
                if ((lane & 15) == 0)
                    *reinterpret_cast<uint32_t*>(p.s + panel * p.sps + row * 16 + (lane >> 4) * 4) = sw;
                if constexpr (COUNT) count_row<DT>(r[j], w, byte, sat, und, nan);
            }
        }
    }
    if constexpr (COUNT) flush_counters_block(p.ctr, sat, und, nan);
}

// ------------------------------------------------------------------ both directions
constexpr int kTileThreads = 256;
constexpr int kTileRows = 128, kTileCols = 128;

// A workgroup of 4 waves takes 128 x 128 elements, a wave 32 rows: lane
// (c8, rq) holds rows 8 rq .. + 7 of columns 8 c8 .. + 7.  Row codes go
// straight out, 64 adjacent bytes a row; transposed ones (4 bytes a lane and
// column) meet in LDS, so that a column's 128 codes leave as 64 adjacent
// bytes.  In LDS column 8 c8 + c is the 64 bytes from 64 (16 c + c8) on, and
// wave w's 16 bytes of it lie at chunk w ^ (c8 / 4): the lanes of a wave then
// write to all 64 banks.  Of the 16 columns that a wave reads at once eight start
// at the same bank: such reads, two a lane against eight writes, take 1.35 times
// as long as adjacent ones, and LDS is busy 7 % of the time at most.  16384 x 7168
// bf16: 71 us, 5.1 TB/s; 16384 x 2048: 25 us, 4.1.  (256 rows and 8 waves left
// one workgroup a CU: 96 and 30 us; forcing more waves onto a CU spills: 89 and
// 31 us.)  Rounding stochastically, 8191 x 5000 takes 47 us, 2.7 TB/s: two
// random words and four conversions a pair of elements, about 1300 VALU
// instructions for a lane's 64 elements, are then half of the time, and a lane
// that loads, computes and ends overlaps them with its reads only as far as
// other waves do.
template <int DT, bool SR, bool COUNT>
__global__ void __launch_bounds__(kTileThreads) k_mx4_tile(Mx4Args p)
{
    __shared__ __attribute__((aligned(16))) uint8_t codes[kTileCols * 64];
    __shared__ __attribute__((aligned(16))) uint8_t scales[kTileCols * 4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c8 = lane & 15, rq = lane >> 4;
    // neighbouring tiles on one XCD, two rows of tiles abreast, whose L2 then
    // joins their lines
    const int total = (int)gridDim.x;
    const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
    const int tile = xcd * (total >> 3) + min(xcd, total & 7) + at;
    const int64_t pair = tile / (2 * p.tiles_c), in = tile - pair * 2 * p.tiles_c;
    const int64_t tr = 2 * pair + (in & 1), tc = in >> 1;
    const int64_t row0 = tr * kTileRows + wave * 32 + rq * 8;
    const int64_t col0 = tc * kTileCols, col = col0 + c8 * 8;

    Row8<DT> r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = load8<DT>(p, row0 + j, col);
    uint32_t h[8][4];
    if constexpr (SR) {
        const uint64_t seed = *p.seed;
        uint32_t pk[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) pk[c] = mx4::pair_key((uint32_t)(col >> 1) + c, (uint32_t)(seed >> 32));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t rk = mx4::row_key((uint32_t)(row0 + j), (uint32_t)seed);
#pragma unroll
            for (int c = 0; c < 4; ++c) h[j][c] = mx4::mix(rk ^ pk[c]);
        }
    }

    // amax of the 8 row blocks and the 8 column blocks this lane is part of
    uint32_t rkey[8], ckey[8], all = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        rkey[j] = quad_max(r[j].raw_max());
        all = max(all, rkey[j]);
    }
    const bool special = __any(all >= kNonFinite);
    if (special) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t k = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) k = max(k, r[j].key(c));
            rkey[j] = quad_max(k);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t k = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) k = max(k, r[j].key(c));
            ckey[c] = stride16_max(k);
        }
    } else if constexpr (DT == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            us2 m = us2{0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) m = pkmax(m, __builtin_bit_cast(us2, r[j].w[i] & 0x7FFF7FFFu));
            m = stride16_pkmax(m);
            ckey[2 * i] = (uint32_t)m.x << 16;
            ckey[2 * i + 1] = (uint32_t)m.y << 16;
        }
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t k = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) k = max(k, r[j].w[c] & 0x7FFFFFFFu);
            ckey[c] = stride16_max(k);
        }
    }

    uint32_t sat = 0, und = 0, nan = 0;
    // along the rows
    const int64_t padded = (p.cols + mx4::kRowAlign - 1) & ~(int64_t)(mx4::kRowAlign - 1);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t row = row0 + j;
        const uint32_t byte = byte_of_key(rkey[j]);
        uint32_t w = cast_row<DT, SR>(r[j], mx4::scale_float(byte), SR ? h[j] : nullptr);
        w = byte == 255u ? 0u : w;
        uint32_t sw = byte << (8 * ((lane >> 2) & 3));
        sw |= dpp<kRor4>(sw);
        sw |= dpp<kRor8>(sw);
        if (row < p.rows) {
            if (col < padded) *reinterpret_cast<uint32_t*>(p.q + row * p.ldq + (col >> 1)) = w;
            if (c8 == 0)
                *reinterpret_cast<uint32_t*>(p.s + (col0 >> 9) * p.sps + row * 16 + ((col0 >> 5) & 12)) = sw;
            if constexpr (COUNT) count_row<DT>(r[j], w, byte, sat, und, nan);
        }
    }
    // along the columns
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t byte = byte_of_key(ckey[c]);
        const float s = mx4::scale_float(byte);
        uint32_t w;
        if constexpr (SR) {
            float x[8];
            uint32_t se[4], so[4];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = r[j].get(c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t he = h[2 * i][c >> 1], ho = h[2 * i + 1][c >> 1];
                se[i] = (c & 1) ? he & 0xFFFF0000u : he << 16;
                so[i] = (c & 1) ? (ho >> 1) & 0x7FFF8000u : (ho & 0xFFFFu) << 15;
            }
            w = mx4::cast8_sr(x, se, so, s);
        } else if constexpr (DT == 0) {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __builtin_amdgcn_perm(r[2 * i + 1].w[c >> 1], r[2 * i].w[c >> 1],
                                             (c & 1) ? 0x07060302u : 0x05040100u);
            w = mx4::cast8_rne(v, s);
        } else {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = r[j].get(c);
            w = mx4::cast8_rne(x, s);
        }
        w = byte == 255u ? 0u : w;
        const int lc = c8 * 8 + c;
        *reinterpret_cast<uint32_t*>(codes + (16 * c + c8) * 64 + ((wave ^ (c8 >> 2)) * 16) + rq * 4) = w;
        if (rq == 0) scales[lc * 4 + wave] = (uint8_t)byte;
    }
    __syncthreads();
    const int64_t padded_t = (p.rows + mx4::kRowAlign - 1) & ~(int64_t)(mx4::kRowAlign - 1);
    if (tr * kTileRows < padded_t) {
#pragma unroll
        for (int i = 0; i < kTileCols * 4 / kTileThreads; ++i) {
            const int t = i * kTileThreads + threadIdx.x;
            const int lc = t >> 2, ch = t & 3;
            if (col0 + lc < p.cols) {
                const int at = 16 * (lc & 7) + (lc >> 3);
                const u4 v = *reinterpret_cast<const u4*>(codes + at * 64 + ((ch ^ (lc >> 5)) * 16));
                __builtin_nontemporal_store(
                    v, reinterpret_cast<u4*>(p.qt + (col0 + lc) * p.ldqt + tr * (kTileRows / 2) + ch * 16));
            }
        }
    }
    if (threadIdx.x < kTileCols && col0 + (int)threadIdx.x < p.cols)
        *reinterpret_cast<uint32_t*>(p.st + (tr >> 2) * p.stps + (col0 + threadIdx.x) * 16 + (tr & 3) * 4) =
            *reinterpret_cast<const uint32_t*>(scales + threadIdx.x * 4);
    if constexpr (COUNT) flush_counters_block(p.ctr, sat, und, nan);
}

// ------------------------------------------------------------------ dequantize
struct Mx4DeqArgs {
    const uint8_t* q;
    int64_t ldq;
    const uint8_t* s;
    int64_t sps;
    int64_t rows, cols;
    void* y;
    int64_t ldy;
    int panels;
};

// A wave writes 512 columns of kRowsPerWave rows.  bf16: 8 columns a lane;
// fp32: 4 columns a lane of either half, so that the lanes' 16 bytes are
// adjacent in both (8192 x 8192: 54 us, 5.6 TB/s; with 8 columns a lane as two
// stores 108 us).  bf16, 16384 x 2048: 14 us, 6.1 TB/s.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) k_mx4_dequantize(Mx4DeqArgs p)
{
    constexpr int kParts = DT == 0 ? 1 : 2;
    constexpr int kCols = 8 / kParts;           // of a lane and part
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t group = item / p.panels;
    const int panel = (int)(item - group * p.panels);
    const int64_t row0 = group * kRowsPerWave;
    if (row0 >= p.rows) return;
    uint32_t w[kRowsPerWave][kParts], b[kRowsPerWave][kParts];
#pragma unroll
    for (int j = 0; j < kRowsPerWave; ++j) {
        const int64_t row = min(row0 + j, p.rows - 1);
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
            // rows of codes end on 128 bytes, panels of scales on 16
            const int64_t in = 64 * kCols * h + kCols * lane;
            const int64_t col = min((int64_t)panel * mx4::kPanel + in, (p.cols - 1) & ~(int64_t)(kCols - 1));
            const uint8_t* q = p.q + row * p.ldq + (col >> 1);
            if constexpr (DT == 0)
                w[j][h] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q));
            else
                w[j][h] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(q));
            b[j][h] = p.s[panel * p.sps + row * 16 + (in >> 5)];
        }
    }
#pragma unroll
    for (int j = 0; j < kRowsPerWave; ++j) {
        const int64_t row = row0 + j;
        if (row >= p.rows) break;
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
            const int64_t col = (int64_t)panel * mx4::kPanel + 64 * kCols * h + kCols * lane;
            const float s = mx4::scale_float(b[j][h]);
            if constexpr (DT == 0) {
                uint32_t v[4];
                v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j][h], s, 0));
                v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j][h], s, 1));
                v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j][h], s, 2));
                v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j][h], s, 3));
                uint16_t* y = static_cast<uint16_t*>(p.y) + row * p.ldy + col;
                if (col + 8 <= p.cols) {
                    __builtin_nontemporal_store((u4x2{v[0], v[1], v[2], v[3]}), reinterpret_cast<u4x2*>(y));
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (col + c < p.cols) y[c] = (uint16_t)(v[c >> 1] >> (16 * (c & 1)));
                }
            } else {
                const mx4::v2f lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j][h], s, 0);
                const mx4::v2f hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j][h], s, 1);
                const float v[4] = {lo[0], lo[1], hi[0], hi[1]};
                float* y = static_cast<float*>(p.y) + row * p.ldy + col;
                if (col + 4 <= p.cols) {
                    __builtin_nontemporal_store((f4x4{v[0], v[1], v[2], v[3]}), reinterpret_cast<f4x4*>(y));
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (col + c < p.cols) y[c] = v[c];
                }
            }
        }
    }
}

int64_t panels_of(int64_t cols) { return (cols + mx4::kPanel - 1) / mx4::kPanel; }
// Workgroups: of four waves that take kRowsPerWave rows of a panel each; of a
// tile each, in column tiles to the end of the last scale panel and row tiles
// to the end of the transposed copy's.
int64_t row_groups(int64_t rows, int64_t cols)
{
    return ((rows + kRowsPerWave - 1) / kRowsPerWave * panels_of(cols) + kRowThreads / 64 - 1) / (kRowThreads / 64);
}
int64_t tile_groups(int64_t rows, int64_t cols)
{
    return panels_of(cols) * (mx4::kPanel / kTileCols) * panels_of(rows) * (mx4::kPanel / kTileRows);
}

template <int DT, bool SR, bool COUNT>
hipError_t launch_dir(const Mx4Args& p, hipStream_t stream)
{
    Mx4Args a = p;
    if (p.qt) {
        a.tiles_c = (int)panels_of(p.cols) * (mx4::kPanel / kTileCols);
        const dim3 grid((unsigned)tile_groups(p.rows, p.cols));
        hipLaunchKernelGGL((k_mx4_tile<DT, SR, COUNT>), grid, dim3(kTileThreads), 0, stream, a);
        return hipGetLastError();
    }
    a.tiles_c = (int)panels_of(p.cols);
    const dim3 grid((unsigned)row_groups(p.rows, p.cols));
    hipLaunchKernelGGL((k_mx4_rows<DT, SR, COUNT>), grid, dim3(kRowThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

int64_t mx4_quantize_items(int64_t rows, int64_t cols, bool transposed)
{
    return transposed ? tile_groups(rows, cols) * kTileThreads : row_groups(rows, cols) * kRowThreads;
}
int64_t mx4_dequantize_items(int64_t rows, int64_t cols) { return row_groups(rows, cols) * kRowThreads; }

hipError_t launch_mx4_quantize(const Mx4QuantArgs& g, hipStream_t stream)
{
    if (g.rows == 0 || g.cols == 0) return hipSuccess;
    Mx4Args p;
    p.x = g.x;
    p.rows = g.rows;
    p.cols = g.cols;
    p.ld = g.ld;
    p.q = g.q;
    p.ldq = g.ldq;
    p.s = g.s;
    p.sps = g.sps;
    p.qt = g.qt;
    p.ldqt = g.ldqt;
    p.st = g.st;
    p.stps = g.stps;
    p.seed = g.seed;
    p.ctr = g.ctr;
    p.tiles_c = 0;
    if (g.dtype == FP8_IN_BF16) {
        if (g.seed) return g.ctr ? launch_dir<0, true, true>(p, stream) : launch_dir<0, true, false>(p, stream);
        return g.ctr ? launch_dir<0, false, true>(p, stream) : launch_dir<0, false, false>(p, stream);
    }
    if (g.seed) return g.ctr ? launch_dir<1, true, true>(p, stream) : launch_dir<1, true, false>(p, stream);
    return g.ctr ? launch_dir<1, false, true>(p, stream) : launch_dir<1, false, false>(p, stream);
}

hipError_t launch_mx4_dequantize(const uint8_t* q, int64_t ldq, const uint8_t* s, int64_t sps, int64_t rows,
                                 int64_t cols, void* y, int dtype, int64_t ldy, hipStream_t stream)
{
    if (rows == 0 || cols == 0) return hipSuccess;
    Mx4DeqArgs p{q, ldq, s, sps, rows, cols, y, ldy, (int)panels_of(cols)};
    const dim3 grid((unsigned)row_groups(rows, cols));
    if (dtype == FP8_IN_BF16)
        hipLaunchKernelGGL((k_mx4_dequantize<0>), grid, dim3(kRowThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((k_mx4_dequantize<1>), grid, dim3(kRowThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace fp8mi
