// Dropout for gfx950 with the random bits of the stochastic quantizer's
// generator, on a stream of their own: an element's 16 bits come from (seed,
// row, column pair) alone, so the backward pass draws the forward's mask anew
// and nothing is stored.
//   y = (r >= cut ? x 65536 / (65536 - cut) : 0) + residual
// Bound by memory: 2 reads and a write of 16 bytes a lane (bf16), about 12
// VALU operations an element.
#include <algorithm>

#include "device_common.h"
#include "fp8mi_internal.h"
#include "gemm_common.h"
#include "mx4_common.h"

namespace fp8mi {

namespace {

// Keeps dropout's bits apart from those that round under the same seed.
constexpr uint32_t kStream = 0xA54FF53Au;

struct DropArgs {
    const void* x;
    int64_t rows, cols, ld;
    const void* residual;       // nullable
    int64_t ldr;
    uint32_t cut;               // of 65536
    float scale;
    const uint64_t* seed;
    void* y;
    int64_t ldy;
    int lanes_log2;             // lanes of a row: 8 columns each
    int64_t chunks;             // of 8 << lanes_log2 columns
    int64_t units;              // of 64 lanes
};

// 8 elements at any alignment of theirs.
struct __attribute__((packed, aligned(2))) Bf16x8 {
    uint32_t w[4];
};
struct __attribute__((packed, aligned(4))) F32x8 {
    float v[8];
};

__device__ inline void load8(const uint16_t* from, float v[8])
{
    const Bf16x8 b = *reinterpret_cast<const Bf16x8*>(from);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(b.w[i]);
        v[2 * i + 1] = bf16_hi(b.w[i]);
    }
}
__device__ inline void load8(const float* from, float v[8])
{
    const F32x8 b = *reinterpret_cast<const F32x8*>(from);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = b.v[i];
}
__device__ inline void store8(uint16_t* to, const float v[8])
{
    Bf16x8 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.w[i] = gemm::pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<Bf16x8*>(to) = b;
}
__device__ inline void store8(float* to, const float v[8])
{
    F32x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b.v[i] = v[i];
    *reinterpret_cast<F32x8*>(to) = b;
}
__device__ inline float load1(const uint16_t* from) { return __builtin_bit_cast(float, (uint32_t)*from << 16); }
__device__ inline float load1(const float* from) { return *from; }
__device__ inline void store1(uint16_t* to, float v) { *to = gemm::to_bf16(v); }
__device__ inline void store1(float* to, float v) { *to = v; }

template <typename T, bool RES>
__global__ void __launch_bounds__(256) k_dropout(DropArgs p)
{
    const int lane = threadIdx.x & 63;
    const uint64_t seed = *p.seed;
    const uint32_t hi = (uint32_t)(seed >> 32) ^ kStream;
    const int per_row = 1 << p.lanes_log2, sub = lane & (per_row - 1);
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < p.units; u += step) {
        const int64_t block = u / p.chunks;
        const int64_t row = (block << (6 - p.lanes_log2)) + (lane >> p.lanes_log2);
        const int64_t col = ((u - block * p.chunks) << (3 + p.lanes_log2)) + 8 * sub;
        if (row >= p.rows || col >= p.cols) continue;
        const T* x = static_cast<const T*>(p.x) + row * p.ld + col;
        const T* res = static_cast<const T*>(p.residual) + row * p.ldr + col;
        T* y = static_cast<T*>(p.y) + row * p.ldy + col;
        const int n = (int)min(p.cols - col, (int64_t)8);
        float v[8], r[8];
        if (n == 8) {
            load8(x, v);
            if (RES) load8(res, r);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = i < n ? load1(x + i) : 0.0f;
                if (RES) r[i] = i < n ? load1(res + i) : 0.0f;
            }
        }
        const uint32_t rk = mx4::row_key((uint32_t)row, (uint32_t)seed);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t h = mx4::mix(rk ^ ((uint32_t)((col >> 1) + c) * 0x3C6EF373u + hi));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool keep = (e ? h >> 16 : h & 0xFFFFu) >= p.cut;
                const int i = 2 * c + e;
                if (RES)
                    v[i] = keep ? __builtin_fmaf(v[i], p.scale, r[i]) : r[i];
                else
                    v[i] = keep ? v[i] * p.scale : 0.0f;
            }
        }
        if (n == 8) {
            store8(y, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) store1(y + i, v[i]);
        }
    }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& g, hipStream_t stream)
{
    if (g.rows == 0 || g.cols == 0) return hipSuccess;
    DropArgs p;
    p.x = g.x;
    p.rows = g.rows;
    p.cols = g.cols;
    p.ld = g.ld;
    p.residual = g.residual;
    p.ldr = g.ldr;
    p.cut = g.cut;
    p.scale = g.cut < 65536u ? (float)(65536.0 / (65536 - g.cut)) : 0.0f;
    p.seed = g.seed;
    p.y = g.y;
    p.ldy = g.ldy;
    const int64_t groups = (g.cols + 7) / 8;
    p.lanes_log2 = 0;
    while (p.lanes_log2 < 6 && ((int64_t)1 << p.lanes_log2) < groups) ++p.lanes_log2;
    p.chunks = (groups + (1 << p.lanes_log2) - 1) >> p.lanes_log2;
    const int64_t per = 64 >> p.lanes_log2;
    p.units = (g.rows + per - 1) / per * p.chunks;
    const unsigned grid = (unsigned)std::min<int64_t>((p.units + 3) / 4, (int64_t)gemm_num_cus() * 64);
    const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, p); };
    if (g.dtype == FP8_IN_BF16)
        g.residual ? launch(k_dropout<uint16_t, true>) : launch(k_dropout<uint16_t, false>);
    else
        g.residual ? launch(k_dropout<float, true>) : launch(k_dropout<float, false>);
    return hipGetLastError();
}

}  // namespace fp8mi
