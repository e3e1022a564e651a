// Dropout for gfx950 with the random bits of the stochastic quantizer's
// generator, on a stream of their own: an element's 16 bits come from (seed,
// row, column pair) alone, so the backward pass draws the forward's mask anew
// and nothing is stored.
//   y = (r >= cut ? x 65536 / (65536 - cut) : 0) + residual
// Bound by memory; about 13 VALU operations an element, two 32-bit products among
// them.  16384 x 2048 bf16: 26 us (5.1 TB/s), onto a residual 37.5 us (5.3);
// 8191 x 5000 fp32: 54 us (6.0).  Two or four pieces of a wave read before the
// first is written: 30 to 65 us for the first of these.
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
    int lanes_log2;             // lanes of a row: 16 bytes each
    int64_t chunks;             // of 16 << lanes_log2 bytes
    int64_t units;              // of 64 lanes
};

// A lane's 16 bytes as words, at any alignment of its elements.
template <typename T>
using Lane = uint32_t __attribute__((ext_vector_type(4), aligned(sizeof(T))));
template <typename T, bool FAR>
__device__ inline Lane<T> load16(const T* from)
{
    const Lane<T>* p = reinterpret_cast<const Lane<T>*>(from);
    return FAR ? __builtin_nontemporal_load(p) : *p;
}
template <typename T, bool FAR>
__device__ inline void store16(T* to, Lane<T> v)
{
    Lane<T>* p = reinterpret_cast<Lane<T>*>(to);
    if (FAR)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}
__device__ inline void unpack(const gemm::v4u& w, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ inline void unpack(const gemm::v4u& w, float (&v)[4])
{
    // (Cast as a whole: the compiler takes element 0 four times for four casts.)
    const gemm::v4f f = __builtin_bit_cast(gemm::v4f, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f[i];
}
__device__ inline gemm::v4u pack(const float (&v)[8])
{
    return {gemm::pack_bf16(v[0], v[1]), gemm::pack_bf16(v[2], v[3]), gemm::pack_bf16(v[4], v[5]), gemm::pack_bf16(v[6], v[7])};
}
__device__ inline gemm::v4u pack(const float (&v)[4])
{
    return __builtin_bit_cast(gemm::v4u, gemm::v4f{v[0], v[1], v[2], v[3]});
}
__device__ inline float load1(const uint16_t* from) { return __builtin_bit_cast(float, (uint32_t)*from << 16); }
__device__ inline float load1(const float* from) { return *from; }
__device__ inline void store1(uint16_t* to, float v) { *to = gemm::to_bf16(v); }
__device__ inline void store1(float* to, float v) { *to = v; }

template <typename T, bool RES, bool FAR>
__global__ void __launch_bounds__(256) k_dropout(DropArgs p)
{
    constexpr int E = 16 / sizeof(T);
    const int lane = threadIdx.x & 63;
    const uint64_t seed = *p.seed;
    const uint32_t hi = (uint32_t)(seed >> 32) ^ kStream;
    const int sub = lane & ((1 << p.lanes_log2) - 1);
    const int64_t waves = (int64_t)gridDim.x * 4;
    for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < p.units; u += waves) {
        const int64_t block = u / p.chunks;
        const int64_t row = (block << (6 - p.lanes_log2)) + (lane >> p.lanes_log2);
        const int64_t col = ((u - block * p.chunks) << p.lanes_log2) * E + E * sub;
        if (row >= p.rows || col >= p.cols) continue;
        const T* x = static_cast<const T*>(p.x) + row * p.ld + col;
        const T* res = static_cast<const T*>(p.residual) + row * p.ldr + col;
        T* y = static_cast<T*>(p.y) + row * p.ldy + col;
        const int n = (int)min(p.cols - col, (int64_t)E);
        float v[E], r[E];
        if (n == E) {
            unpack(load16<T, FAR>(x), v);
            if (RES) unpack(load16<T, FAR>(res), r);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                v[i] = i < n ? load1(x + i) : 0.0f;
                if (RES) r[i] = i < n ? load1(res + i) : 0.0f;
            }
        }
        const uint32_t rk = mx4::row_key((uint32_t)row, (uint32_t)seed);
        const uint32_t pk = mx4::pair_key((uint32_t)(col >> 1), hi);
#pragma unroll
        for (int c = 0; c < E / 2; ++c) {
            const uint32_t h = mx4::mix(rk ^ (pk + (uint32_t)c * 0x3C6EF373u));
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
        if (n == E) {
            store16<T, FAR>(y, pack(v));
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
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
    const int64_t each = g.dtype == FP8_IN_BF16 ? 8 : 4, groups = (g.cols + each - 1) / each;
    p.lanes_log2 = 0;
    while (p.lanes_log2 < 6 && ((int64_t)1 << p.lanes_log2) < groups) ++p.lanes_log2;
    p.chunks = (groups + (1 << p.lanes_log2) - 1) >> p.lanes_log2;
    const int64_t per = 64 >> p.lanes_log2;
    p.units = (g.rows + per - 1) / per * p.chunks;
    const unsigned grid = (unsigned)std::min<int64_t>((p.units + 3) / 4, (int64_t)gemm_num_cus() * 64);
    // More than the last-level cache holds (256 MB): reads and writes that leave
    // it alone, 8191 x 5000 fp32 54 us against 63 (16384 x 2048 bf16 onto a
    // residual 34 against 37.5).  Below that the plain forms: what reads y next
    // may find it there.
    const int64_t moved = g.rows * g.cols * (16 / each) * (g.residual ? 3 : 2);
    const bool far = moved > (int64_t)256 << 20;
    const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, p); };
    const auto with = [&](auto t) {
        using T = decltype(t);
        if (g.residual)
            far ? launch(k_dropout<T, true, true>) : launch(k_dropout<T, true, false>);
        else
            far ? launch(k_dropout<T, false, true>) : launch(k_dropout<T, false, false>);
    };
    g.dtype == FP8_IN_BF16 ? with(uint16_t{}) : with(float{});
    return hipGetLastError();
}

}  // namespace fp8mi
