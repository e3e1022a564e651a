// Softmax cross entropy of a projection onto a vocabulary, for gfx950:
//   l = x w^T,  z = cap tanh(l / cap) or l,  lse = log sum_v exp z_v,
//   loss = lse - z_target,
// and its gradients
//   dl = g (exp(z - lse) - [v = target]) (1 - (z / cap)^2),  dx = dl w,  dw = dl^T x.
// The logits exist only as fp32 accumulators of a tile: the forward keeps of a
// tile each token's maximum and sum of exponentials, the backward recomputes
// them for a piece of the vocabulary at a time and writes dl, rounded to bf16,
// for the two products that follow: 8 T V H operations in all, 2 T V H of them
// the logits' second time (to keep them would take 2 T V bytes).
//
// Measured: 8192 x 131072 x 4096, four pieces of 32768: forward 7.0 to 7.7 ms (1.14
// to 1.25 PFLOP/s), of a piece the logits' gradient 1.78 to 1.84 ms, dx and dw 1.77
// to 1.85 each (1.19 to 1.24).  The matrix pipes are busy 63 to 66 % of the cycles at
// the 1.5 to 1.8 GHz that power leaves (a library product of this shape: 1.12 to
// 1.34 PFLOP/s, 80 to 85 % busy at a lower clock).  One token, 32768 x 2048: 33 us for
// W's 134 MB from HBM (4.0 TB/s; 20 to 22 where the last-level cache holds it) and
// 4.6 us for the sum over the blocks.  Rows of w that are not at 16-byte places cost a copy
// of w a pass and dw in 2-byte stores: 64 x 50304 x 769 takes 266 us, x 768 101.
#include <algorithm>

#include "ce_gemm.h"
#include "device_common.h"
#include "fp8mi_internal.h"
#include "mx4_common.h"

namespace fp8mi {

namespace {

using ce::GemmShape;
using ce::Item;
using gemm::v4f;
using gemm::v4u;
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ inline float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// cap tanh(l / cap).  For |u| <= 1, u = l / cap: tanh u = u + u t Q(t), t = u^2, Q
// the polynomial through (tanh u / u - 1) / t at the 7 Chebyshev points of 0 <= t
// <= 1 (off by 3e-8 of tanh u with its coefficients in fp32, which also rounds
// them; all in all 2.1 steps of 2^-24).  Past that 1 - 2 / (exp(2 |u|) + 1), which
// loses nothing there.
__device__ inline float softcap_near(float l, float inv_cap)
{
    constexpr float kQ[7] = {-0.3333333f, 0.13333128f, -0.05393479f, 0.02166012f, -0.00821892f, 0.00251046f, -0.0004207f};
    const float u = l * inv_cap, t = u * u;
    float q = kQ[6];
#pragma unroll
    for (int i = 5; i >= 0; --i) q = __builtin_fmaf(q, t, kQ[i]);
    return __builtin_fmaf(l * t, q, l);
}
__device__ inline float softcap_any(float l, float cap, float inv_cap)
{
    const float u = __builtin_fabsf(l * inv_cap);
    const float far = cap - 2.0f * cap * __builtin_amdgcn_rcpf(exp2_fast(2.0f * kLog2e * u) + 1.0f);
    return u <= 1.0f ? softcap_near(l, inv_cap) : l != l ? l : __builtin_copysignf(far, l);
}
// Of a fragment's column, the far form only where one of the wave's needs it.
template <int MF>
__device__ inline void softcap_column(v4f (&acc)[MF], float cap, float inv_cap)
{
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) most = fmaxf(most, __builtin_fabsf(acc[i][r]));      // NaN: either form gives NaN
    const bool far = __any(most * inv_cap > 1.0f);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        __builtin_amdgcn_sched_barrier(0);      // one fragment after another: registers
        if (far) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][r] = softcap_any(acc[i][r], cap, inv_cap);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][r] = softcap_near(acc[i][r], inv_cap);
        }
    }
}

// ------------------------------------------------------------------ epilogues
// A lane holds, for tokens (columns) col + 16 j, the rows row + 16 i + r:
// acc[j][i][r].

// Two fragments below each other (16 i and 16 (i + 1)) to bf16, for a store of
// 16 bytes a lane.  As they lie a lane has 4 rows of either; odd groups of 16
// lanes of the first and even ones of the second change places, and a lane has 8
// rows from chunk_row() on, the four lanes of a column 32: 64 bytes.
__device__ inline v4u to_bf16_chunk(const v4f& first, const v4f& second)
{
    v4u out;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const auto r = __builtin_amdgcn_permlane16_swap(gemm::pack_bf16(first[2 * q], first[2 * q + 1]),
                                                        gemm::pack_bf16(second[2 * q], second[2 * q + 1]), false, false);
        out[q] = r[0];
        out[2 + q] = r[1];
    }
    return out;
}
__device__ inline int chunk_row() { return 16 * (threadIdx.x >> 4 & 1) + 8 * (threadIdx.x >> 5 & 1); }

// The forward's: of each token and block of 16 MF vocabulary rows the maximum
// and the sum of exp(z - maximum); the target's z, by the one lane that has it.
template <int WR, int MF, int NF>
struct StatsEpilogue {
    static constexpr int kStores = NF;
    static constexpr bool kNotes = true;
    int m, n;                   // vocabulary rows of this launch, tokens
    int v0;                     // its first row
    int block0;                 // its first block
    float cap, inv_cap;
    const int64_t* targets;
    float2* part;               // [blocks, n]
    float* zt;

    // the targets' low halves: a match by mistake is of a target that is not used
    __device__ void note(uint32_t lds, int col) const
    {
        gemm::dma4(lds, (uint32_t)(col + (threadIdx.x & 63)) * 8u, gemm::make_rsrc(targets, (uint32_t)n * 8u));
    }

    __device__ bool operator()(const Item& it, v4f (&acc)[NF][MF], int row, int col, const uint8_t* notes) const
    {
        const int lane = threadIdx.x & 63;
        const int wave_row = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % WR;
        float2* to = part + (int64_t)(block0 + it.tm * WR + wave_row) * n;
        const __amdgpu_buffer_rsrc_t rp = gemm::make_store_rsrc(to, (uint32_t)n * 8u);
        const bool edge = (it.tm + 1) * (16 * MF * WR) > m;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int t = col + 16 * j;
            __builtin_amdgcn_sched_barrier(0);
            if (cap != 0.0f) softcap_column<MF>(acc[j], cap, inv_cap);
            if (edge) {
                int left = m - row;
                asm("" : "+v"(left));       // one column's comparisons are not kept for the next: registers
#pragma unroll
                for (int i = 0; i < MF; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * i + r >= left) acc[j][i][r] = -__builtin_inff();
            }
            const int at = reinterpret_cast<const int*>(notes + 1024 * (j / 4))[16 * (j % 4) + (lane & 15)] - v0 - row;
            if (__any((uint32_t)at < 16u * MF)) {
                float z = 0.0f;
#pragma unroll
                for (int i = 0; i < MF; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) z = at == 16 * i + r ? acc[j][i][r] : z;
                const bool here = (uint32_t)at < 16u * MF && (at & 12) == 0;
                if (here && t < n && row + at < m) zt[t] = z;
            }
            float mx = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, acc[j][i][r]);
            mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            // (the difference first: the product alone may overflow, and its
            // rounding grows with the logits)
            const float base = mx == -__builtin_inff() ? 0.0f : mx;
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] += exp2_fast((acc[j][i][r] - base) * kLog2e);
            float sum = (s[0] + s[1]) + (s[2] + s[3]);
            sum += __shfl_xor(sum, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            const uint32_t where = lane < 16 && t < n ? (uint32_t)t * 8u : gemm::kOutOfRange;
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u, float2{mx, sum}), rp, (int)where, 0, 0);
        }
        return true;
    }
};

// What the backward's logits need of a token: a token that does not count has
// an lse of +Inf, so exponentials of 0, and the gradient 0 (and x all zeros).
struct TokenNote {
    float lse;                  // +Inf: the token does not count
    float grad;                 // of its loss, over the largest of all tokens'
    int target;                 // -1: none
    int unused;
};

// The backward's: dl over the largest gradient of the losses, rounded to bf16 (by
// 2^-8 of each value at most, what the operands' own type has; the matrix
// instruction takes one type), rows past the vocabulary's end as zeros.  Losses
// have one gradient as a rule, the mean's, and most targets one near -1: divided by
// it they round to -1 with almost no error, where the gradient's own mantissa
// would put the same error into all of them (0.0031 of the gradients' size).  Errors of
// dx and dw, of their norm: 0.0018 to 0.0020 with one gradient for all, 0.0021 with a
// cap of 15 too, which takes the targets' entries away from -1, 0.0023 to 0.0024 with
// gradients that differ; their own rounding alone 0.0017.
template <int WR, int MF, int NF>
struct GradEpilogue {
    static constexpr int kStores = MF / 2 * NF;
    static constexpr bool kNotes = true;
    int m, n;
    int v0;
    float cap, inv_cap;
    const TokenNote* tokens;
    uint16_t* dl;               // [n, ld]
    int64_t ld;

    __device__ void note(uint32_t lds, int col) const
    {
        const int64_t left = (int64_t)(n - col) * 16;
        gemm::dma16(lds, (uint32_t)(threadIdx.x & 63) * 16u,
                    gemm::make_rsrc(tokens + col, (uint32_t)min(max(left, (int64_t)0), (int64_t)1024)));
    }

    __device__ bool operator()(const Item& it, v4f (&acc)[NF][MF], int row, int col, const uint8_t* notes) const
    {
        const int lane = threadIdx.x & 63;
        const int n0 = __builtin_amdgcn_readfirstlane(col & ~15);       // this wave's first token
        const __amdgpu_buffer_rsrc_t rd =
            gemm::make_store_rsrc(dl + n0 * ld, (uint32_t)(max(min(n - n0, 16 * NF), 0) * ld * 2));
        const uint32_t to = (uint32_t)((lane & 15) * ld + (row & ~15) + chunk_row()) * 2u;
        const bool edge = (it.tm + 1) * (16 * MF * WR) > m;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const TokenNote k = reinterpret_cast<const TokenNote*>(notes)[16 * j + (lane & 15)];
            const int at = k.target < 0 ? -1 : k.target - v0 - row;
            // of tokens that do not count: an infinite w times their zeros is NaN
            if (__any(k.target < 0)) {
#pragma unroll
                for (int i = 0; i < MF; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[j][i][r] = k.target < 0 ? 0.0f : acc[j][i][r];
            }
            if (cap != 0.0f) softcap_column<MF>(acc[j], cap, inv_cap);
            const bool target_here = __any((uint32_t)at < 16u * MF);
#pragma unroll
            for (int i = 0; i < MF; i += 2) {
                __builtin_amdgcn_sched_barrier(0);      // one pair after another: registers
                v4f d[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) d[h][r] = exp2_fast((acc[j][i + h][r] - k.lse) * kLog2e);
                if (target_here) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) d[h][r] = at == 16 * (i + h) + r ? d[h][r] - 1.0f : d[h][r];
                }
                if (cap != 0.0f) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float u = acc[j][i + h][r] * inv_cap;
                            d[h][r] *= __builtin_fmaf(-u, u, 1.0f);
                        }
                }
                d[0] *= k.grad;
                d[1] *= k.grad;
                if (edge) {
                    int left = m - row;
                    asm("" : "+v"(left));   // as above
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) d[h][r] = 16 * (i + h) + r < left ? d[h][r] : 0.0f;
                }
                gemm::store16(to_bf16_chunk(d[0], d[1]), to + (uint32_t)(16 * j * ld + 16 * i) * 2u, rd);
            }
        }
        return true;
    }
};

// A gradient in bf16.  TOKENS: dx, whose rows of tokens that do not count are zeros
// also where w is infinite (0 times that is NaN); by a mask on the packed words, a
// lane's being of one token (a choice of sums spilled).
template <int MF, int NF, bool FAR, bool TOKENS>
struct Bf16Out {
    static constexpr int kStores = MF / 2 * NF;
    static constexpr bool kNotes = false;
    int m, n;                   // the gradient's columns and rows
    uint16_t* out;              // bf16 [n, ld]
    int64_t ld;
    int wide;                   // 16-byte stores are in place
    const float* scale;
    const TokenNote* tokens;

    __device__ void note(uint32_t, int) const {}

    __device__ bool operator()(const Item&, v4f (&acc)[NF][MF], int row, int col, const uint8_t*) const
    {
        const int lane = threadIdx.x & 63;
        const int n0 = __builtin_amdgcn_readfirstlane(col & ~15);
        const int rows = max(min(n - n0, 16 * NF), 0);
        const float by = *scale;
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int i = 0; i < MF; ++i) acc[j][i] *= by;
        uint32_t keep[NF];
#pragma unroll
        for (int j = 0; j < NF; ++j)
            keep[j] = !TOKENS || (col + 16 * j < n && tokens[col + 16 * j].target >= 0) ? ~0u : 0u;
        if (wide) {
            const __amdgpu_buffer_rsrc_t ro =
                gemm::make_store_rsrc(out + n0 * ld, rows ? (uint32_t)(((rows - 1) * ld + m) * 2) : 0u);
            const int first = (row & ~15) + chunk_row();
            const uint32_t to = (uint32_t)((lane & 15) * ld + first) * 2u;
#pragma unroll
            for (int j = 0; j < NF; ++j)
#pragma unroll
                for (int i = 0; i < MF; i += 2)
                    __builtin_amdgcn_raw_buffer_store_b128(
                        to_bf16_chunk(acc[j][i], acc[j][i + 1]) & keep[j], ro,
                        (int)(first + 16 * i < m ? to + (uint32_t)(16 * j * ld + 16 * i) * 2u : gemm::kOutOfRange), 0,
                        FAR ? 18 : 0);              // sc1 nt
            return true;
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int t = col + 16 * j;
            if (t >= n) continue;
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                uint16_t* to = out + t * ld + row + 16 * i;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (row + 16 * i + r < m) to[r] = gemm::to_bf16(acc[j][i][r]) & keep[j];
            }
        }
        return false;
    }
};

template <int WR, int MF, int NF>
struct NearEpilogue : Bf16Out<MF, NF, false, false> {};
template <int WR, int MF, int NF>
struct FarEpilogue : Bf16Out<MF, NF, true, false> {};
template <int WR, int MF, int NF>
struct TokensEpilogue : Bf16Out<MF, NF, false, true> {};

// A gradient in parts: fp32 planes, one for each split of K, added to what an
// earlier piece of the vocabulary left.
template <int WR, int MF, int NF>
struct PlanesEpilogue {
    static constexpr int kStores = MF * NF;
    static constexpr bool kNotes = false;
    int m, n;                   // the gradient's columns and rows
    float* plane;               // [splits, n, ld]
    int64_t ld;                 // a multiple of 16
    int add;

    __device__ void note(uint32_t, int) const {}

    __device__ bool operator()(const Item& it, v4f (&acc)[NF][MF], int row, int col, const uint8_t*) const
    {
        const int lane = threadIdx.x & 63;
        const int n0 = __builtin_amdgcn_readfirstlane(col & ~15);
        const int rows = max(min(n - n0, 16 * NF), 0);
        const __amdgpu_buffer_rsrc_t rp =
            gemm::make_store_rsrc(plane + ((int64_t)it.split * n + n0) * ld, (uint32_t)(rows * ld * 4));
        const uint32_t at = (uint32_t)((lane & 15) * ld + row) * 4u;
        const auto place = [&](int i, int j) {
            return row + 16 * i < m ? at + (uint32_t)(16 * j * ld + 16 * i) * 4u : gemm::kOutOfRange;
        };
        // a column after another: more loads in flight would spill
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            if (add) {
#pragma unroll
                for (int i = 0; i < MF; ++i)
                    acc[j][i] += __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rp, (int)place(i, j), 0, 0));
            }
#pragma unroll
            for (int i = 0; i < MF; ++i) gemm::store16(__builtin_bit_cast(v4u, acc[j][i]), place(i, j), rp);
            __builtin_amdgcn_sched_barrier(0);
        }
        return true;
    }
};

template <bool ATR, bool BTR, int WR, int WC, int MF, int NF, template <int, int, int> class Epi>
__global__ void __launch_bounds__(64 * WR * WC, 2) k_ce_gemm(GemmShape s, Epi<WR, MF, NF> epi)
{
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    ce::Tile<ATR, BTR, WR, WC, MF, NF>::run(s, lds, epi);
}

int tiles_of(int64_t size, int64_t tile) { return (int)((size + tile - 1) / tile); }

template <bool ATR, bool BTR, int WR, int WC, int MF, int NF, template <int, int, int> class Epi, typename Init>
hipError_t launch_tile(GemmShape s, Init init, hipStream_t stream)
{
    using T = ce::Tile<ATR, BTR, WR, WC, MF, NF>;
    using E = Epi<WR, MF, NF>;
    constexpr int kLds = T::template lds_bytes<E>();
    s.tiles_m = tiles_of(s.m, T::TM);
    s.tiles_n = tiles_of(s.n, T::TN);
    s.group_m = 4;
    s.least_stages = E::kNotes ? ce::kNoteStages : 1;
    E epi;
    init(epi);
    const auto kernel = k_ce_gemm<ATR, BTR, WR, WC, MF, NF, Epi>;
    static mx4::LdsLimit limit;
    const hipError_t e = limit.raise(reinterpret_cast<const void*>(kernel), kLds);
    if (e != hipSuccess) return e;
    const int64_t items = (int64_t)s.tiles_m * s.tiles_n * s.splits;
    const int per_cu = std::min(160 * 1024 / kLds, 3);
    const int grid = (int)std::min<int64_t>(items, (int64_t)gemm_num_cus() * per_cu);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * WR * WC), kLds, stream, s, epi);
    return hipGetLastError();
}

// Tokens of a tile: the least of 32, 64, 128, 256 that holds them all.  This one and
// the next larger one, x 50304 x 1024, forward and backward to dx, us:
//    32 tokens   25.7 and 46.3 with 32, 26.8 and 47.6 with 64
//    64 tokens   27.8 and 51.3 with 64, 27.5 and 54.9 with 128
//   128 tokens   29.2 and 70.7 with 128, 34.7 and 76.9 with 256
// Hidden 512 and 2048 the same way; of 64 tokens' forward, 64 and 128 are within 4 %.
int token_tile(int64_t tokens) { return tokens <= 32 ? 32 : tokens <= 64 ? 64 : tokens <= 128 ? 128 : 256; }

template <bool ATR, template <int, int, int> class Epi, typename Init>
hipError_t launch_tokens(int tile, const GemmShape& s, Init init, hipStream_t stream)
{
    switch (tile) {
    case 32: return launch_tile<ATR, false, 4, 1, 2, 2, Epi>(s, init, stream);
    case 64: return launch_tile<ATR, false, 4, 1, 2, 4, Epi>(s, init, stream);
    case 128: return launch_tile<ATR, false, 4, 2, 4, 4, Epi>(s, init, stream);
    default: return launch_tile<ATR, false, 2, 4, 8, 4, Epi>(s, init, stream);
    }
}
// Rows of such a tile, and the vocabulary rows of a block of statistics (a wave's).
int row_tile(int tile) { return tile <= 64 ? 128 : 256; }
int stat_rows(int tile) { return tile <= 64 ? 32 : tile <= 128 ? 64 : 128; }

// The tile of the logits of `rows` of the vocabulary: where that leaves CUs without
// one, the next smaller one, 128 tokens (of 256 rows) if there is one a CU at most,
// 64 (of 128 rows) if there are three for two CUs at most.  Forward, us, by this rule,
// with token_tile(), and by twice the rule's numbers of tiles:
//                hidden 512         1856            4096
//    100 x 8600   12.9 16.5 12.9   22.6 32.1 22.4   36.9 57.8 37.0
//    250 x 8600   15.7 22.9 15.7   29.3 47.8 29.4   52.1 89.3 52.2
//    500 x 8600   17.8 23.5 21.1   34.8 48.3 44.4   63.8 90.8 88.2
//   1000 x 8600   24.6 24.2 26.8   51.2 49.6 64.8   97.9 97.8 125.9
//   1000 x 2000   12.6 23.7 12.7   21.8 48.3 22.4   39.4 90.4 39.1
//   2000 x 2000   17.1 24.2 16.5   33.1 49.0 34.6   58.4 90.4 63.4
// The backward's logits gain and lose as much.
int logit_tile(int64_t rows, int64_t tokens)
{
    const int64_t cus = gemm_num_cus();
    int tile = token_tile(tokens);
    if (tile == 256 && (int64_t)tiles_of(rows, 256) * tiles_of(tokens, 128) <= cus) tile = 128;
    if (tile == 128 && (int64_t)tiles_of(rows, 128) * tiles_of(tokens, 64) <= cus + cus / 2) tile = 64;
    return tile;
}

// Tiles of 256 x 256 come in rounds of one a CU.  Where the last round would be a
// small part of one, the rows behind the whole rounds go in tiles of 128 x 128
// instead, one a CU at most, in a launch of their own: returns the rows before
// them.  2001 x 50001 x 1000, 6.1 rounds: backward 698 us against 733; 1023 tokens,
// 3.1 rounds: forward 134 against 144.  (Up to two small tiles a CU: the same.)
int64_t whole_rounds(int64_t rows, int64_t others)
{
    const int64_t cus = gemm_num_cus(), across = tiles_of(others, 256), tiles = tiles_of(rows, 256);
    const int64_t main = tiles * across / cus * cus / across;
    if (main == 0 || main >= tiles) return rows;
    return (int64_t)tiles_of(rows - 256 * main, 128) * tiles_of(others, 128) <= cus ? 256 * main : rows;
}
constexpr int kTailRows = 128, kTailStatRows = 64;

// Blocks of statistics of `rows` of the vocabulary.
int64_t stat_blocks(int64_t rows, int64_t tokens)
{
    const int tile = logit_tile(rows, tokens);
    if (tile < 256) return (int64_t)tiles_of(rows, row_tile(tile)) * (row_tile(tile) / stat_rows(tile));
    const int64_t big = whole_rounds(rows, tokens);
    return (int64_t)tiles_of(big, 256) * 2 + (int64_t)tiles_of(rows - big, kTailRows) * (kTailRows / kTailStatRows);
}

// ------------------------------------------------------------------ around the products
// Rows of bf16 at 16-byte places with zeros behind them.  For tokens of a
// backward pass, rows of those that do not count as zeros (their x may hold
// anything), and the notes.
struct PackTokens {
    const int64_t* targets;
    int64_t vocab;
    const float* lse;
    const float* grad;
    int64_t grad_step;
    float* scale;
    TokenNote* notes;
};
// The largest |gradient| of the losses that count (1 where all are 0 or one is no
// number: the quotients then say so), by a whole workgroup.
template <int THREADS>
__device__ inline float largest_grad(const PackTokens& k, int64_t n)
{
    __shared__ float sh[THREADS / 64];
    float most = 0.0f;
    bool bad = false;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < n; t += THREADS) {
        const int64_t at = k.targets[t];
        const float g = __builtin_fabsf(k.grad[t * k.grad_step]);
        const bool on = at >= 0 && at < k.vocab;
        most = on ? fmaxf(most, g) : most;
        bad |= on && !(g <= 3.0e38f);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = most;
    const bool any_bad = __syncthreads_or(bad);
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) most = fmaxf(most, sh[w]);
    // (below the smallest normal number a quotient could overflow)
    return any_bad || most < 0x1p-126f ? 1.0f : most;
}
__global__ void __launch_bounds__(1024) k_ce_scale(PackTokens k, int64_t n)
{
    const float by = largest_grad<1024>(k, n);
    if (threadIdx.x == 0) *k.scale = by;
}
constexpr int64_t kFewTokens = 1024;        // each workgroup of the copy looks through them itself

template <bool TOKENS>
__global__ void __launch_bounds__(256) k_ce_pack(const uint16_t* x, int64_t ld, int64_t rows, int cols, uint4* out,
                                                 int chunks, int aligned, PackTokens k)
{
    const int64_t total = rows * chunks;
    float by = 1.0f;
    if constexpr (TOKENS) {
        if (rows <= kFewTokens) {
            by = largest_grad<256>(k, rows);
            if (blockIdx.x == 0 && threadIdx.x == 0) *k.scale = by;
        } else {
            by = *k.scale;
        }
    }
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
        const int64_t r = u / chunks;
        const int c = (int)(u - r * chunks) * 8;
        uint4 v = {0, 0, 0, 0};
        bool on = true;
        if constexpr (TOKENS) {
            const int64_t t = k.targets[r];
            on = t >= 0 && t < k.vocab;
            if (c == 0) {
                TokenNote note = {__builtin_inff(), 0.0f, -1, 0};
                if (on) note = TokenNote{k.lse[r], k.grad[r * k.grad_step] / by, (int)t, 0};
                k.notes[r] = note;
            }
        }
        if (on) {
            const uint16_t* from = x + r * ld + c;
            if (aligned && c + 8 <= cols) {
                v = *reinterpret_cast<const uint4*>(from);
            } else {
                uint16_t e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = c + i < cols ? from[i] : 0;
                v = uint4{e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                          e[6] | (uint32_t)e[7] << 16};
            }
        }
        out[u] = v;
    }
}

// Of each token the blocks' maxima and sums to lse, and the loss.  TX tokens a
// workgroup, 256 / TX threads each over the blocks: one token, of few, that many
// CUs read at once; 8, whose 64 bytes lie side by side (32: no faster at 512 to 8192).
template <int TX>
__global__ void __launch_bounds__(256) k_ce_loss(const float2* part, int blocks, int n, const float* zt,
                                                 const int64_t* targets, int64_t vocab, float* loss, float* lse)
{
    __shared__ float2 sh[256];
    const int x = threadIdx.x % TX, y = threadIdx.x / TX;
    const int t = blockIdx.x * TX + x;
    constexpr int TY = 256 / TX;
    const auto join = [](float2 a, float2 b) {
        const float m = fmaxf(a.x, b.x);
        if (m == -__builtin_inff()) return float2{m, a.y + b.y};
        return float2{m, a.y * exp2_fast((a.x - m) * kLog2e) + b.y * exp2_fast((b.x - m) * kLog2e)};
    };
    float2 a = {-__builtin_inff(), 0.0f};
    if (t < n) {
        int b = y;
        for (; b + 3 * TY < blocks; b += 4 * TY) {
            float2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = part[(int64_t)(b + i * TY) * n + t];
            a = join(a, join(join(v[0], v[1]), join(v[2], v[3])));
        }
        for (; b < blocks; b += TY) a = join(a, part[(int64_t)b * n + t]);
    }
    sh[threadIdx.x] = a;
    __syncthreads();
    for (int h = TY / 2; h >= 1; h >>= 1) {
        if (y < h) sh[threadIdx.x] = join(sh[threadIdx.x], sh[threadIdx.x + h * TX]);
        __syncthreads();
    }
    if (y == 0 && t < n) {
        const float2 s = sh[x];
        // the loss without lse's rounding: where the target is the largest, it is the
        // logarithm alone
        const float log_sum = logf(s.y);
        const int64_t at = targets[t];
        lse[t] = s.x + log_sum;
        loss[t] = at < 0 ? 0.0f : at < vocab ? (s.x - zt[t]) + log_sum : __builtin_nanf("");
    }
}

// The planes' sum to bf16: S threads share a chunk of 8 columns, each adds up
// every S-th plane, and their sums are added in order.  16 where there are 8 planes
// or more: 64 x 50304 x 1024, backward to dx 56.6 us against 60.4 with one.
template <int S>
__global__ void __launch_bounds__(256) k_ce_reduce(const float* plane, int splits, int64_t rows, int cols, int64_t ld_plane,
                                                   uint16_t* out, int64_t ld, int wide, const float* scale,
                                                   const TokenNote* tokens)
{
    __shared__ v4f sh[S > 1 ? 512 : 1];
    const float by = *scale;
    constexpr int C = 256 / S;          // chunks of a workgroup
    const int x = threadIdx.x % C, y = threadIdx.x / C;
    const int chunks = (int)(ld_plane / 8);
    const int64_t total = rows * chunks;
    for (int64_t u0 = (int64_t)blockIdx.x * C; u0 < total; u0 += (int64_t)gridDim.x * C) {
        const int64_t u = u0 + x;
        const int64_t r = u / chunks;
        const int c = (int)(u - r * chunks) * 8;
        v4f a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (u < total) {
            const float* from = plane + r * ld_plane + c;
#pragma unroll 4
            for (int s = y; s < splits; s += S) {
                a += *reinterpret_cast<const v4f*>(from + s * rows * ld_plane);
                b += *reinterpret_cast<const v4f*>(from + s * rows * ld_plane + 4);
            }
        }
        if constexpr (S > 1) {
            sh[threadIdx.x] = a;
            sh[256 + threadIdx.x] = b;
            __syncthreads();
            if (y == 0) {
#pragma unroll
                for (int s = 1; s < S; ++s) {
                    a += sh[s * C + x];
                    b += sh[256 + s * C + x];
                }
            }
            __syncthreads();
        }
        if (y != 0 || u >= total) continue;
        const bool on = tokens[r].target >= 0;      // else the planes may hold NaN: zeros times an infinite w
        a = on ? a * by : v4f{0, 0, 0, 0};
        b = on ? b * by : v4f{0, 0, 0, 0};
        uint16_t* to = out + r * ld + c;
        if (wide && c + 8 <= cols) {
            *reinterpret_cast<v4u*>(to) = v4u{gemm::pack_bf16(a[0], a[1]), gemm::pack_bf16(a[2], a[3]),
                                              gemm::pack_bf16(b[0], b[1]), gemm::pack_bf16(b[2], b[3])};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < cols) to[i] = gemm::to_bf16(i < 4 ? a[i] : b[i - 4]);
        }
    }
}

int grid_of(int64_t units) { return (int)std::min<int64_t>((units + 255) / 256, 8 * gemm_num_cus()); }

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

bool aligned16(const void* p, int64_t ld) { return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * 2)) & 15u) == 0; }

hipError_t pack(const void* x, int64_t ld, int64_t rows, int64_t cols, void* out, const PackTokens* tokens, hipStream_t stream)
{
    const int chunks = (int)(up(cols, 8) / 8);
    const auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid_of(rows * chunks)), dim3(256), 0, stream, static_cast<const uint16_t*>(x), ld, rows,
                           (int)cols, static_cast<uint4*>(out), chunks, (int)aligned16(x, ld), tokens ? *tokens : PackTokens{});
        return hipGetLastError();
    };
    return tokens ? launch(k_ce_pack<true>) : launch(k_ce_pack<false>);
}

// ------------------------------------------------------------------ plans
// Tokens of a forward pass, which bounds its statistics (8 bytes a token and
// block), and the bytes of a piece of dl or of w's packed rows.  256 MiB, 1 and 2 GiB
// a piece: within 1 % for 8192 tokens.
constexpr int64_t kTokenChunk = 32768;
constexpr int64_t kPieceBytes = (int64_t)1 << 29;
// A dw of more than this is written past the caches: 64 x 65536 x 2048 61 us against
// 116, x 1536 52 against 75, x 1024 (128 MiB) 35 against 38, x 768 30 against 28.
constexpr int64_t kFarBytes = (int64_t)1 << 27;

struct Layout {
    int64_t piece, pieces;      // vocabulary rows (a multiple of 256) and number
    int64_t splits;             // of dx
    size_t x, w, stats, zt, scale, notes, dl, planes, total;      // offsets in the workspace
};
size_t take(size_t& at, int64_t bytes)
{
    const size_t here = at;
    at += (size_t)up(bytes, 256);
    return here;
}
void pieces_of(Layout& l, int64_t vocab, int64_t most)
{
    most = std::max<int64_t>(most / 256 * 256, 256);
    l.pieces = (vocab + most - 1) / most;
    l.piece = up((vocab + l.pieces - 1) / l.pieces, 256);
    l.pieces = (vocab + l.piece - 1) / l.piece;
}
Layout forward_layout(int64_t tokens, int64_t vocab, int64_t hidden)
{
    Layout l = {};
    const int64_t row = up(hidden, 8) * 2, chunk = std::min(tokens, kTokenChunk);
    pieces_of(l, vocab, std::max<int64_t>(kPieceBytes / row, 4096));
    size_t at = 0;
    l.x = take(at, chunk * row);
    l.w = take(at, std::min(l.piece, vocab) * row);
    int64_t stats = 0;          // of a full chunk and of the last one, w copied or not
    for (const int64_t n : {chunk, tokens % kTokenChunk ? tokens % kTokenChunk : chunk}) {
        const int64_t last = vocab - (l.pieces - 1) * l.piece;
        const int64_t copied = (l.pieces - 1) * stat_blocks(l.piece, n) + stat_blocks(last, n);
        stats = std::max(stats, std::max(stat_blocks(vocab, n), copied) * n * 8);
    }
    l.stats = take(at, stats);
    l.zt = take(at, chunk * 4);
    l.total = at;
    return l;
}
Layout backward_layout(int64_t tokens, int64_t vocab, int64_t hidden)
{
    Layout l = {};
    const int64_t row = up(hidden, 8) * 2;
    pieces_of(l, vocab, std::max<int64_t>(kPieceBytes / (2 * tokens), 4096));
    // too few tiles of dx for the chip: its K, the vocabulary, is split.  Unsplit
    // 64 x 50304 x 1024 takes 407 us against 57, 2048 tokens 1290 against 473.
    const int tile = token_tile(tokens);
    const int64_t tiles = (int64_t)tiles_of(hidden, row_tile(tile)) * tiles_of(tokens, tile);
    const int64_t want = (int64_t)gemm_num_cus() * (tile <= 64 ? 2 : 1);
    l.splits = std::max<int64_t>(std::min<int64_t>(want / tiles, std::min(l.piece, vocab) / 512), 1);
    size_t at = 0;
    l.x = take(at, tokens * row);
    l.w = take(at, std::min(l.piece, vocab) * row);
    l.scale = take(at, 4);
    l.notes = take(at, tokens * (int64_t)sizeof(TokenNote));
    l.dl = take(at, tokens * l.piece * 2);
    l.planes = take(at, l.splits > 1 || l.pieces > 1 ? l.splits * tokens * up(hidden, 16) * 4 : 0);
    l.total = at;
    return l;
}

}  // namespace

size_t ce_forward_workspace(int64_t tokens, int64_t vocab, int64_t hidden)
{
    return forward_layout(tokens, vocab, hidden).total;
}
size_t ce_backward_workspace(int64_t tokens, int64_t vocab, int64_t hidden)
{
    return backward_layout(tokens, vocab, hidden).total;
}

hipError_t launch_ce_forward(const CeArgs& g, hipStream_t stream)
{
    const Layout l = forward_layout(g.tokens, g.vocab, g.hidden);
    uint8_t* ws = static_cast<uint8_t*>(g.ws);
    const bool pack_w = !aligned16(g.w, g.ldw) || g.hidden % 8 != 0, pack_x = !aligned16(g.x, g.ldx) || g.hidden % 8 != 0;
    hipError_t e;
    for (int64_t t0 = 0; t0 < g.tokens; t0 += kTokenChunk) {
        const int64_t n = std::min(g.tokens - t0, kTokenChunk);
        const uint16_t* x = static_cast<const uint16_t*>(g.x) + t0 * g.ldx;
        GemmShape s = {};
        s.b = {reinterpret_cast<const uint8_t*>(x), g.ldx * 2};
        if (pack_x) {
            if ((e = pack(x, g.ldx, n, g.hidden, ws + l.x, nullptr, stream)) != hipSuccess) return e;
            s.b = {ws + l.x, up(g.hidden, 8) * 2};
        }
        s.n = (int)n;
        s.k = (int)g.hidden;
        s.splits = 1;
        int blocks = 0;
        for (int64_t p = 0; p < (pack_w ? l.pieces : 1); ++p) {
            const int64_t v0 = p * l.piece, m = pack_w ? std::min(l.piece, g.vocab - v0) : g.vocab;
            const uint16_t* w = static_cast<const uint16_t*>(g.w) + v0 * g.ldw;
            s.a = {reinterpret_cast<const uint8_t*>(w), g.ldw * 2};
            if (pack_w) {
                if ((e = pack(w, g.ldw, m, g.hidden, ws + l.w, nullptr, stream)) != hipSuccess) return e;
                s.a = {ws + l.w, up(g.hidden, 8) * 2};
            }
            const int tile = logit_tile(m, n);
            const int64_t big = tile == 256 ? whole_rounds(m, n) : m;
            const auto rows = [&](int64_t from, int64_t count, int block) {
                return [=, &g](auto& epi) {
                    epi.m = (int)count;
                    epi.n = (int)n;
                    epi.v0 = (int)(v0 + from);
                    epi.block0 = block;
                    epi.cap = g.softcap;
                    epi.inv_cap = g.softcap != 0.0f ? 1.0f / g.softcap : 0.0f;
                    epi.targets = g.targets + t0;
                    epi.part = reinterpret_cast<float2*>(ws + l.stats);
                    epi.zt = reinterpret_cast<float*>(ws + l.zt);
                };
            };
            s.m = (int)big;
            if ((e = launch_tokens<false, StatsEpilogue>(tile, s, rows(0, big, blocks), stream)) != hipSuccess) return e;
            if (big < m) {
                s.a.p += big * s.a.ld;
                s.m = (int)(m - big);
                e = launch_tile<false, false, 2, 2, 4, 4, StatsEpilogue>(s, rows(big, m - big, blocks + (int)(big / 128)), stream);
                if (e != hipSuccess) return e;
            }
            blocks += (int)stat_blocks(m, n);
        }
        const auto finish = [&](auto kernel, int tx) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)((n + tx - 1) / tx)), dim3(256), 0, stream,
                               reinterpret_cast<const float2*>(ws + l.stats), blocks, (int)n,
                               reinterpret_cast<const float*>(ws + l.zt), g.targets + t0, g.vocab, g.loss + t0, g.lse + t0);
            return hipGetLastError();
        };
        e = n <= 512 ? finish(k_ce_loss<1>, 1) : finish(k_ce_loss<8>, 8);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_ce_backward(const CeArgs& g, hipStream_t stream)
{
    hipError_t e;
    if (g.tokens == 0) {
        if (!g.dw) return hipSuccess;
        return launch_zero_bf16(static_cast<uint16_t*>(g.dw), (int)g.vocab, (int)g.hidden, g.lddw, stream);
    }
    const Layout l = backward_layout(g.tokens, g.vocab, g.hidden);
    uint8_t* ws = static_cast<uint8_t*>(g.ws);
    const bool pack_w = !aligned16(g.w, g.ldw) || g.hidden % 8 != 0;
    const int64_t packed = up(g.hidden, 8) * 2;
    const int T = (int)g.tokens, H = (int)g.hidden, H8 = (int)up(g.hidden, 8);
    // x always as a copy, in which the tokens that do not count are zeros:
    // their products with dl's zeros have to be zeros in dw
    TokenNote* notes = reinterpret_cast<TokenNote*>(ws + l.notes);
    float* scale = reinterpret_cast<float*>(ws + l.scale);
    const PackTokens tokens = {g.targets, g.vocab, g.lse, g.grad, g.grad_step, scale, notes};
    if (g.tokens > kFewTokens) {
        hipLaunchKernelGGL(k_ce_scale, dim3(1), dim3(1024), 0, stream, tokens, g.tokens);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if ((e = pack(g.x, g.ldx, g.tokens, g.hidden, ws + l.x, &tokens, stream)) != hipSuccess) return e;
    const ce::Operand x = {ws + l.x, packed};
    float* planes = reinterpret_cast<float*>(ws + l.planes);
    uint16_t* dl = reinterpret_cast<uint16_t*>(ws + l.dl);
    const ce::Operand d = {ws + l.dl, l.piece * 2};
    for (int64_t p = 0; p < l.pieces; ++p) {
        const int64_t v0 = p * l.piece, m = std::min(l.piece, g.vocab - v0);
        const uint16_t* wp = static_cast<const uint16_t*>(g.w) + v0 * g.ldw;
        ce::Operand w = {reinterpret_cast<const uint8_t*>(wp), g.ldw * 2};
        if (pack_w) {
            if ((e = pack(wp, g.ldw, m, g.hidden, ws + l.w, nullptr, stream)) != hipSuccess) return e;
            w = {ws + l.w, packed};
        }
        GemmShape s = {};
        s.a = w;
        s.b = x;
        s.n = T;
        s.k = H;
        s.splits = 1;
        const int tile = logit_tile(m, T);
        const int64_t big = tile == 256 ? whole_rounds(m, T) : m;
        const auto rows = [&](int64_t from, int64_t count) {
            return [=, &g](auto& epi) {
                epi.m = (int)count;
                epi.n = T;
                epi.v0 = (int)(v0 + from);
                epi.cap = g.softcap;
                epi.inv_cap = g.softcap != 0.0f ? 1.0f / g.softcap : 0.0f;
                epi.tokens = notes;
                epi.dl = dl + from;
                epi.ld = l.piece;
            };
        };
        s.m = (int)big;
        if ((e = launch_tokens<false, GradEpilogue>(tile, s, rows(0, big), stream)) != hipSuccess) return e;
        if (big < m) {
            s.a.p += big * s.a.ld;
            s.m = (int)(m - big);
            e = launch_tile<false, false, 2, 2, 4, 4, GradEpilogue>(s, rows(big, m - big), stream);
            if (e != hipSuccess) return e;
        }
        if (g.dx) {
            s.a = w;
            s.b = d;
            s.m = H8;
            s.n = T;
            s.k = (int)m;
            s.splits = (int)std::min<int64_t>(l.splits, (m + ce::kStageK - 1) / ce::kStageK);
            if (l.splits == 1 && l.pieces == 1)
                e = launch_tokens<true, TokensEpilogue>(token_tile(T), s, [&](auto& epi) {
                    epi.m = H;
                    epi.n = T;
                    epi.out = static_cast<uint16_t*>(g.dx);
                    epi.ld = g.lddx;
                    epi.wide = aligned16(g.dx, g.lddx) && H % 8 == 0;
                    epi.scale = scale;
                    epi.tokens = notes;
                }, stream);
            else
                e = launch_tokens<true, PlanesEpilogue>(token_tile(T), s, [&](auto& epi) {
                    epi.m = H;
                    epi.n = T;
                    epi.plane = planes;
                    epi.ld = up(g.hidden, 16);
                    epi.add = p > 0;
                }, stream);
            if (e != hipSuccess) return e;
            if (p == l.pieces - 1 && (l.splits > 1 || l.pieces > 1)) {
                const int64_t ld = up(g.hidden, 16);
                // a short last piece may have had fewer splits; the first has written all planes
                const auto reduce = [&](auto kernel, int share) {
                    const int64_t groups = (g.tokens * ld / 8 + 256 / share - 1) / (256 / share);
                    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(groups, 8 * gemm_num_cus())), dim3(256), 0, stream,
                                       planes, (int)l.splits, g.tokens, H, ld, static_cast<uint16_t*>(g.dx), g.lddx,
                                       (int)aligned16(g.dx, g.lddx), scale, notes);
                };
                l.splits >= 8 ? reduce(k_ce_reduce<16>, 16) : reduce(k_ce_reduce<1>, 1);
                if ((e = hipGetLastError()) != hipSuccess) return e;
            }
        }
        if (g.dw) {
            s.a = x;
            s.m = H8;
            s.k = T;
            s.splits = 1;
            const auto rows = [&](int64_t from, int64_t count) {
                uint16_t* dw = static_cast<uint16_t*>(g.dw) + (v0 + from) * g.lddw;
                return [=, &g](auto& epi) {
                    epi.m = H;
                    epi.n = (int)count;
                    epi.out = dw;
                    epi.ld = g.lddw;
                    epi.wide = aligned16(dw, g.lddw) && H % 8 == 0;
                    epi.scale = scale;
                    epi.tokens = nullptr;
                };
            };
            const int64_t big = whole_rounds(m, H);
            s.b = d;
            s.n = (int)up(big, 8);          // dl's rows go on with zeros
            if (g.vocab * g.hidden * 2 > kFarBytes)
                e = launch_tile<true, true, 2, 4, 8, 4, FarEpilogue>(s, rows(0, big), stream);
            else
                e = launch_tile<true, true, 2, 4, 8, 4, NearEpilogue>(s, rows(0, big), stream);
            if (e != hipSuccess) return e;
            if (big < m) {
                s.b.p = d.p + 2 * big;
                s.n = (int)up(m - big, 8);
                e = launch_tile<true, true, 2, 2, 4, 4, NearEpilogue>(s, rows(big, m - big), stream);
                if (e != hipSuccess) return e;
            }
        }
    }
    return hipSuccess;
}

}  // namespace fp8mi
