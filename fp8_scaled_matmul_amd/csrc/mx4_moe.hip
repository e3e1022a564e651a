// A mixture-of-experts layer with 4-bit (OCP MXFP4) weights for at most 64
// tokens, gfx950.
//
//   l[t, e]  = sum_c x[t, c] R[e, c]                          (router, float64 sums)
//   E(t)     = the top_k experts by l, equal logits to the lower expert
//   p[t, e]  = exp(l - max) / sum exp(l - max), over E(t) or over all experts
//   g, u     = W1[e] x[t]  (gate rows, then up rows)
//   a[t, e]  = p g / (1 + exp(-g)) u
//   y[t]     = sum over e in E(t) of W2[e] a[t, e]
//
// What bounds it is the read of the chosen experts' codes, half a byte a
// weight, each read once; so the weights go from memory to the registers of
// v_mfma_scale_f32_16x16x128_f8f6f4 as they lie (16 rows of weights by up to
// 16 tokens), with no decoding.  The activations are the instruction's E4M3
// operand: a block of 32 values is the sum of pieces, each E4M3 (4 bits) with
// a power of two scale of its own, every next piece's 2^-4 of the one before
// and holding what the last left.  Two pieces hold a bf16 x exactly, but for
// elements under 2^-13 of their block's largest, which are off by at most
// 2^-21 of that; three hold the fp32 intermediate a to 2^-12 of itself (or
// 2^-25 of the block's largest), a sixteenth of the output's own rounding.
// Sums are fp32, in an order that only the sizes and the chosen experts set:
// no atomics on values.
#include <algorithm>

#include "device_common.h"
#include "fp8mi_internal.h"
#include "gemm_common.h"
#include "mx4_common.h"

namespace fp8mi {

namespace {

using gemm::v4f;
using gemm::v8i;
typedef double v4d __attribute__((ext_vector_type(4)));

constexpr int kUnit = 256;          // K elements of a row read at a time: two matrix instructions
constexpr int kXPieces = 2, kAPieces = 3;
constexpr int kRouteThreads = 512;
constexpr int kUpThreads = 256;
constexpr int kDownThreads = 1024;

struct MoeArgs {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* router;
    int64_t ldr;
    int tokens, experts, top_k, hidden, inner, renormalize;
    int hp, ip;                     // hidden, inner in whole units
    const uint8_t* q1;
    const uint8_t* s1;
    int64_t ldq1, eq1, ps1, es1;    // bytes between rows, experts, scale panels, experts' scales
    const uint8_t* q2;
    const uint8_t* s2;
    int64_t ldq2, eq2, ps2, es2;
    uint16_t* y;
    int64_t ldy;
    int32_t* ids;
    float* weights;
    // workspace
    uint32_t* arrived;              // [4]: router tiles done, of 16 tokens each; zero between calls
    double* logits;                 // [tokens, experts]
    uint8_t* xq;                    // [tokens, 2, hp]
    uint8_t* xs;                    // [tokens, hp / 32]
    uint8_t* aq;                    // [tokens top_k, 3, ip]
    uint8_t* as;                    // [tokens top_k, ip / 32]
    fp8_counters* ctr;
    int tiles_e, tiles_t;           // router tiles
    int by_pair;                    // a slot is a (token, rank) pair, else an expert
};

// ------------------------------------------------------------------ pieces
// E8M0 byte of the first piece's scale of a block with that amax: v / s in
// [128, 256).  At least 2^-119, so that the third piece's byte is a number.
__device__ inline uint32_t piece_byte(uint32_t amax_bits)
{
    return (uint32_t)max((int)(amax_bits >> 23) - 7, 8);
}

// Four values to a word of E4M3 codes for each piece; inv = 1 / s.
template <int P>
__device__ inline void to_pieces(const float x[4], float inv, uint32_t out[P])
{
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i] * inv;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
        out[p] = (uint32_t)w;
        if (p + 1 < P) {
            // what is left is exact: both terms are multiples of the code's last place
            v[0] = 16.0f * (v[0] - __builtin_amdgcn_cvt_f32_fp8(w, 0));
            v[1] = 16.0f * (v[1] - __builtin_amdgcn_cvt_f32_fp8(w, 1));
            v[2] = 16.0f * (v[2] - __builtin_amdgcn_cvt_f32_fp8(w, 2));
            v[3] = 16.0f * (v[3] - __builtin_amdgcn_cvt_f32_fp8(w, 3));
        }
    }
}

// The reciprocal of the scale of byte b, 8 <= b <= 247.
__device__ inline float inv_scale(uint32_t b) { return __builtin_bit_cast(float, (254u - b) << 23); }

// ------------------------------------------------------------------ matrix instruction
__device__ inline v8i weights_of(const uint4& v) { return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0}; }
__device__ inline v8i codes_of(const uint4& a, const uint4& b)
{
    return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}
// 16 rows of weights x 16 tokens x 128 K.  Lane l holds 32 weights of row
// l % 16, K 32 (l / 16) on; of token l % 16 the codes of K 16 (l / 16) on and
// of K 64 + 16 (l / 16) on; the scale bytes of both for K block l / 16.
__device__ inline v4f mma(const v8i& w, const v8i& x, const v4f& c, uint32_t sw, uint32_t sx)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, 0, 0, (int)sw, 0, (int)sx);
}

// ------------------------------------------------------------------ router
// Eight elements of a row from column c on, zeros past the end.
template <bool VEC>
__device__ inline uint4 row8(const uint16_t* row, int c, int cols)
{
    uint4 v = uint4{0, 0, 0, 0};
    if constexpr (VEC) {
        if (c < cols) v = *reinterpret_cast<const uint4*>(row + c);
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < cols) w[j >> 1] |= (uint32_t)row[c + j] << (16 * (j & 1));
        v = uint4{w[0], w[1], w[2], w[3]};
    }
    return v;
}

// fp64 as an unsigned key of the same order; NaN lowest, +0 and -0 alike
__device__ inline uint64_t key_of(double v)
{
    if (v != v) return 0;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

__device__ inline double logit_at(const MoeArgs& p, int t, int e)
{
    return __builtin_bit_cast(double, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p.logits) + (int64_t)t * p.experts + e,
                                                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// One wave: the top_k experts of token t and their weights.
constexpr int kMaxExperts = 512;
__device__ inline void select(const MoeArgs& p, int t)
{
    const int lane = threadIdx.x & 63;
    constexpr int kPer = kMaxExperts / 64;
    uint64_t key[kPer];
    double l[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = 64 * j + lane;
        key[j] = 0;
        l[j] = 0;
        if (64 * j < p.experts && e < p.experts) {
            l[j] = logit_at(p, t, e);
            key[j] = key_of(l[j]);
        }
    }
    uint32_t taken = 0;
    double top = 0, mine = 0;           // lane r keeps rank r's
    int id = 0;
    for (int r = 0; r < p.top_k; ++r) {
        uint64_t best = 0;
        int at = -1;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (64 * j + lane < p.experts && !(taken >> j & 1) && (at < 0 || key[j] > best)) {
                best = key[j];
                at = j;
            }
        int e = at < 0 ? 0x7FFFFFFF : 64 * at + lane;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const uint64_t ob = __shfl_xor(best, off, 64);
            const int oe = __shfl_xor(e, off, 64);
            const bool take = oe != 0x7FFFFFFF && (e == 0x7FFFFFFF || ob > best || (ob == best && oe < e));
            best = take ? ob : best;
            e = take ? oe : e;
        }
        const int owner = e & 63, slot = e >> 6;
        double v = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) v = j == slot ? l[j] : v;
        v = __shfl(v, owner, 64);
        if (lane == owner) taken |= 1u << slot;
        if (r == 0) top = v;
        if (lane == r) {
            mine = v;
            id = e;
        }
    }
    const float z = lane < p.top_k ? expf((float)(mine - top)) : 0.0f;
    float sum = z;
    if (!p.renormalize) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (64 * j + lane < p.experts) sum += expf((float)(l[j] - top));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane < p.top_k) {
        p.ids[t * p.top_k + lane] = id;
        p.weights[t * p.top_k + lane] = z / sum;
    }
}

// Workgroups below tiles_e tiles_t take 16 tokens x 16 experts of the logits,
// K over their waves; the last of a token tile's to arrive selects.  The
// others cut x into pieces, 512 columns of a token a wave.
template <bool VEC>
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(MoeArgs p)
{
    constexpr int kWaves = kRouteThreads / 64;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nroute = p.tiles_e * p.tiles_t;
    if ((int)blockIdx.x >= nroute) {
        const int panels = (p.hp + mx4::kPanel - 1) / mx4::kPanel;
        const int item = ((int)blockIdx.x - nroute) * kWaves + wave;
        const int t = item / panels, c = (item - t * panels) * mx4::kPanel + 8 * lane;
        if (t >= p.tokens || c >= p.hp) return;
        const uint4 v = row8<VEC>(p.x + t * p.ldx, c, p.hidden);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7FFF0000u, (w[j] << 16) & 0x7FFF0000u));
        amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1, 64));
        amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2, 64));
        const bool finite = amax < 0x7F800000u;
        const uint32_t b = finite ? piece_byte(amax) : 255u;
        uint8_t* q = p.xq + (int64_t)t * kXPieces * p.hp + c;
        uint32_t o[2][kXPieces];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float f[4] = {bf16_lo(w[2 * h]), bf16_hi(w[2 * h]), bf16_lo(w[2 * h + 1]), bf16_hi(w[2 * h + 1])};
            to_pieces<kXPieces>(f, inv_scale(finite ? b : 127u), o[h]);
        }
#pragma unroll
        for (int i = 0; i < kXPieces; ++i)
            *reinterpret_cast<uint2*>(q + (int64_t)i * p.hp) = finite ? uint2{o[0][i], o[1][i]} : uint2{0, 0};
        if ((lane & 3) == 0) p.xs[(int64_t)t * (p.hp / 32) + c / 32] = (uint8_t)b;
        return;
    }

    __shared__ double red[kWaves][256];
    __shared__ int s_last;
    const int tt = blockIdx.x / p.tiles_e, te = blockIdx.x - tt * p.tiles_e;
    const int t = min(16 * tt + (lane & 15), p.tokens - 1), e = min(16 * te + (lane & 15), p.experts - 1);
    const uint16_t* xr = p.x + t * p.ldx;
    const uint16_t* rr = p.router + e * p.ldr;
    v4d acc = {0, 0, 0, 0};
    const int chunks = (p.hidden + 31) / 32;
    for (int c = wave; c < chunks; c += kWaves) {
        const uint4 a = row8<VEC>(rr, 32 * c + 8 * (lane >> 4), p.hidden);
        const uint4 b = row8<VEC>(xr, 32 * c + 8 * (lane >> 4), p.hidden);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)bf16_lo(aw[j]), (double)bf16_lo(bw[j]), acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)bf16_hi(aw[j]), (double)bf16_hi(bw[j]), acc, 0, 0, 0);
        }
    }
    // register i of lane l: expert 4 i + l / 16, token l % 16
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][(4 * i + (lane >> 4)) * 16 + (lane & 15)] = acc[i];
    __syncthreads();
    if (threadIdx.x < 256) {
        double s = red[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += red[w][threadIdx.x];
        const int oe = 16 * te + (threadIdx.x >> 4), ot = 16 * tt + (threadIdx.x & 15);
        // agent-scope stores and loads need no write-back of the L2s between them
        if (oe < p.experts && ot < p.tokens)
            __hip_atomic_store(reinterpret_cast<uint64_t*>(p.logits) + (int64_t)ot * p.experts + oe,
                               __builtin_bit_cast(uint64_t, s), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");    // the stores have completed
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t n = __hip_atomic_fetch_add(p.arrived + tt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = n + 1 == (uint32_t)p.tiles_e;
        if (s_last) __hip_atomic_store(p.arrived + tt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_last) return;
    for (int i = wave; i < 16; i += kWaves)
        if (16 * tt + i < p.tokens) select(p, 16 * tt + i);
}

// ------------------------------------------------------------------ up
// One unit (256 K) of R tiles of 16 weight rows against 16 tokens.
struct RowPtr {
    const uint8_t* q;       // this lane's row of codes, 16 (l / 16) bytes in
    const uint8_t* s;       // its first panel's scale bytes
};

template <int P>
struct UnitX {
    uint4 q[2][P][2];
    uint2 s;
};
// x: this lane's token, 16 (l / 16) bytes in; piece bytes apart.
template <int P>
__device__ inline void load_x(UnitX<P>& o, const uint8_t* q, int64_t piece, const uint8_t* s, int u)
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const uint8_t* a = q + i * piece + u * kUnit + 128 * k;
            o.q[k][i][0] = *reinterpret_cast<const uint4*>(a);
            o.q[k][i][1] = *reinterpret_cast<const uint4*>(a + 64);
        }
    o.s = *reinterpret_cast<const uint2*>(s + 8 * u);
}
struct UnitW {
    uint4 q[2];
    uint2 s;
};
__device__ inline void load_w(UnitW& o, const RowPtr& r, int64_t ps, int u)
{
    o.q[0] = *reinterpret_cast<const uint4*>(r.q + u * 128);
    o.q[1] = *reinterpret_cast<const uint4*>(r.q + u * 128 + 64);
    o.s = *reinterpret_cast<const uint2*>(r.s + (u >> 1) * ps + 8 * (u & 1));
}
template <int P>
__device__ inline void unit_mma(v4f& acc, const UnitW& w, const UnitX<P>& x)
{
    const int sh = 8 * ((threadIdx.x & 63) >> 4);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t sw = (k ? w.s.y : w.s.x) >> sh, sx = (k ? x.s.y : x.s.x) >> sh;
#pragma unroll
        for (int i = 0; i < P; ++i)
            acc = mma(weights_of(w.q[k]), codes_of(x.q[k][i][0], x.q[k][i][1]), acc, sw, sx - 4 * i);
    }
}

__device__ inline uint64_t tokens_of(const MoeArgs& p, int e, int& rank)
{
    const int lane = threadIdx.x & 63;
    bool has = false;
    rank = 0;
    if (lane < p.tokens)
        for (int j = 0; j < p.top_k; ++j)
            if (p.ids[lane * p.top_k + j] == e) {
                has = true;
                rank = j;
            }
    return __ballot(has);
}

// A workgroup takes an expert's 32 gate rows and the 32 up rows of the same
// outputs, K over its waves.
__global__ void __launch_bounds__(kUpThreads) k_moe_up(MoeArgs p)
{
    constexpr int kWaves = kUpThreads / 64;
    __shared__ v4f red[kWaves][4][64];
    __shared__ int s_pair[64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = (p.inner + 31) / 32;
    const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
    const int e = p.by_pair ? __builtin_amdgcn_readfirstlane(p.ids[slot]) : slot;
    if ((uint32_t)e >= (uint32_t)p.experts) return;     // no selection: the workspace was not zeroed
    int rank;
    const uint64_t mask = tokens_of(p, e, rank);
    // an expert's first pair stands for all of its tokens
    if (mask == 0 || (p.by_pair && __builtin_ctzll(mask) != slot / p.top_k)) return;
    if (wave == 0 && (mask >> lane & 1))
        s_pair[__builtin_popcountll(mask & ((1ull << lane) - 1))] = lane * p.top_k + rank;
    __syncthreads();
    const int n = __builtin_popcountll(mask);
    const int c16 = lane & 15, q = lane >> 4;

    RowPtr w[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = min(32 * tile + 16 * (r & 1) + c16, p.inner - 1) + (r >> 1) * p.inner;
        w[r].q = p.q1 + e * p.eq1 + row * p.ldq1 + 16 * q;
        w[r].s = p.s1 + e * p.es1 + row * 16;
    }
    const int units = p.hp / kUnit;
    for (int c0 = 0; c0 < n; c0 += 16) {
        const int pair = s_pair[min(c0 + c16, n - 1)];
        const int t = pair / p.top_k;
        const uint8_t* xq = p.xq + (int64_t)t * kXPieces * p.hp + 16 * q;
        const uint8_t* xs = p.xs + (int64_t)t * (p.hp / 32);
        v4f acc[4] = {};
        for (int u = wave; u < units; u += kWaves) {
            UnitW uw[4];
            UnitX<kXPieces> ux;
#pragma unroll
            for (int r = 0; r < 4; ++r) load_w(uw[r], w[r], p.ps1, u);
            load_x(ux, xq, p.hp, xs, u);
#pragma unroll
            for (int r = 0; r < 4; ++r) unit_mma(acc[r], uw[r], ux);
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][r][lane] = acc[r];
        __syncthreads();
        if (wave != 0) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int o = 1; o < kWaves; ++o) acc[r] += red[o][r][lane];
        // lane: token c16, outputs 32 tile + 16 r + 4 q + i
        const float prob = p.weights[pair];
        float a[2][4];
        uint32_t amax = 0;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g = acc[r][i], u = acc[r + 2][i];
                const float v = prob * (g / (1.0f + expf(-g)) * u);
                a[r][i] = 32 * tile + 16 * r + 4 * q + i < p.inner ? v : 0.0f;
                amax = max(amax, __builtin_bit_cast(uint32_t, a[r][i]) & 0x7FFFFFFFu);
            }
        amax = max(amax, (uint32_t)__shfl_xor((int)amax, 16, 64));
        amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32, 64));
        const bool finite = amax < 0x7F800000u;
        const uint32_t b = finite ? piece_byte(amax) : 255u;
        if (c0 + c16 >= n) continue;
        uint8_t* out = p.aq + (int64_t)pair * kAPieces * p.ip + 32 * tile + 4 * q;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint32_t o[kAPieces];
            to_pieces<kAPieces>(a[r], inv_scale(finite ? b : 127u), o);
#pragma unroll
            for (int i = 0; i < kAPieces; ++i)
                *reinterpret_cast<uint32_t*>(out + (int64_t)i * p.ip + 16 * r) = finite ? o[i] : 0u;
        }
        uint8_t* os = p.as + (int64_t)pair * (p.ip / 32);
        if (q == 0) os[tile] = (uint8_t)b;
        // zeros to the end of the last unit
        if (tile == tiles - 1)
            for (int c = 32 * tiles; c < p.ip; c += 32) {
#pragma unroll
                for (int i = 0; i < kAPieces; ++i)
                    *reinterpret_cast<uint2*>(p.aq + ((int64_t)pair * kAPieces + i) * p.ip + c + 8 * q) = uint2{0, 0};
                if (q == 0) os[c / 32] = 127;
            }
    }
}

// ------------------------------------------------------------------ down
// A workgroup takes 16 rows of y for every token.  Its waves share the reached
// experts (and their K where those are few) in a fixed order, each with sums
// of its own in LDS, which are added in wave order at the end.
__global__ void __launch_bounds__(kDownThreads) k_moe_down(MoeArgs p)
{
    constexpr int kWaves = kDownThreads / 64;
    extern __shared__ __attribute__((aligned(16))) float ysum[];     // [waves, tokens, 16]
    __shared__ unsigned long long s_mask[kMaxExperts];
    __shared__ int16_t s_expert[kMaxExperts];
    __shared__ int32_t s_ids[64 * 16];
    __shared__ int s_count[kMaxExperts / 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row0 = 16 * blockIdx.x;
    const int pairs = p.tokens * p.top_k;
    if ((int)threadIdx.x < p.experts) s_mask[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < kWaves * p.tokens * 16; i += kDownThreads) ysum[i] = 0.0f;
    __syncthreads();
    if ((int)threadIdx.x < pairs) {
        const int e = p.ids[threadIdx.x];
        s_ids[threadIdx.x] = e;
        if ((uint32_t)e < (uint32_t)p.experts) atomicOr(&s_mask[e], 1ull << (threadIdx.x / p.top_k));
    }
    __syncthreads();
    // the reached experts in order
    const bool reached = (int)threadIdx.x < p.experts && s_mask[threadIdx.x] != 0;
    const uint64_t here = __ballot(reached);
    if (wave < kMaxExperts / 64 && lane == 0) s_count[wave] = __builtin_popcountll(here);
    __syncthreads();
    int before = 0, active = 0;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 64; ++i) {
        before += i < wave ? s_count[i] : 0;
        active += s_count[i];
    }
    if (reached) s_expert[before + __builtin_popcountll(here & ((1ull << lane) - 1))] = (int16_t)threadIdx.x;
    __syncthreads();

    const int c16 = lane & 15, q = lane >> 4;
    const int row = min(row0 + c16, p.hidden - 1);
    const int units = p.ip / kUnit;
    const int per = active >= 2 * kWaves ? units : 1;      // units of an item
    const int chunks = (units + per - 1) / per;
    float* mine = ysum + wave * p.tokens * 16;
    for (int item = wave; item < active * chunks; item += kWaves) {
        const int at = item / chunks, u0 = (item - at * chunks) * per, u1 = min(units, u0 + per);
        const int e = s_expert[at];
        const uint64_t mask = s_mask[e];
        const int n = __builtin_popcountll(mask);
        RowPtr w;
        w.q = p.q2 + e * p.eq2 + row * p.ldq2 + 16 * q;
        w.s = p.s2 + e * p.es2 + row * 16;
        uint64_t left = mask;
        for (int c0 = 0; c0 < n; c0 += 16) {
            // column c: the c-th token of the mask that is left, or its last
            uint64_t m = left;
            const int skip = min(c16, n - c0 - 1);
            for (int j = 0; j < skip; ++j) m &= m - 1;
            const int t = __builtin_ctzll(m);
            int pair = 0;
            for (int j = 0; j < p.top_k; ++j)
                if (s_ids[t * p.top_k + j] == e) pair = t * p.top_k + j;
            for (int j = 0; j < 16; ++j) left &= left - 1;
            const uint8_t* aq = p.aq + (int64_t)pair * kAPieces * p.ip + 16 * q;
            const uint8_t* as = p.as + (int64_t)pair * (p.ip / 32);
            v4f acc = {0, 0, 0, 0};
            for (int u = u0; u < u1; ++u) {
                UnitW uw;
                UnitX<kAPieces> ux;
                load_w(uw, w, p.ps2, u);
                load_x(ux, aq, p.ip, as, u);
                unit_mma(acc, uw, ux);
            }
            if (c0 + c16 < n) {
                v4f* s = reinterpret_cast<v4f*>(mine + t * 16 + 4 * q);
                *s += acc;
            }
        }
    }
    __syncthreads();
    uint32_t nonfinite = 0;
    for (int i = threadIdx.x; i < p.tokens * 16; i += kDownThreads) {
        const int t = i >> 4, r = row0 + (i & 15);
        float s = ysum[i];
        for (int w = 1; w < kWaves; ++w) s += ysum[w * p.tokens * 16 + i];
        if (r < p.hidden) {
            const uint16_t h = gemm::to_bf16(s);
            nonfinite += (h & 0x7F80u) == 0x7F80u;
            p.y[t * p.ldy + r] = h;
        }
    }
    flush_counters(p.ctr, 0, 0, 0, nonfinite);
}

struct MoeLayout {
    size_t logits, xq, xs, aq, as, total;
};
MoeLayout moe_layout(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inner)
{
    const auto up = [](int64_t v, int64_t a) { return (v + a - 1) / a * a; };
    const int64_t hp = up(hidden, kUnit), ip = up(inner, kUnit);
    MoeLayout m;
    int64_t at = 256;                                       // arrival counts
    const auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at = up(at + bytes, 256);
        return (size_t)o;
    };
    m.logits = take(tokens * experts * 8);
    m.xq = take(tokens * kXPieces * hp);
    m.xs = take(tokens * (hp / 32));
    m.aq = take(tokens * top_k * kAPieces * ip);
    m.as = take(tokens * top_k * (ip / 32));
    m.total = (size_t)at;
    return m;
}

}  // namespace

size_t mx4_moe_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inner)
{
    return moe_layout(tokens, experts, top_k, hidden, inner).total;
}

hipError_t launch_mx4_moe(const Mx4MoeArgs& g, hipStream_t stream)
{
    if (g.tokens == 0) return hipSuccess;
    const MoeLayout m = moe_layout(g.tokens, g.experts, g.top_k, g.hidden, g.inner);
    uint8_t* ws = static_cast<uint8_t*>(g.ws);
    MoeArgs p;
    p.x = static_cast<const uint16_t*>(g.x);
    p.ldx = g.ldx;
    p.router = static_cast<const uint16_t*>(g.router);
    p.ldr = g.ldr;
    p.tokens = (int)g.tokens;
    p.experts = (int)g.experts;
    p.top_k = (int)g.top_k;
    p.hidden = (int)g.hidden;
    p.inner = (int)g.inner;
    p.renormalize = g.renormalize;
    p.hp = (int)((g.hidden + kUnit - 1) / kUnit * kUnit);
    p.ip = (int)((g.inner + kUnit - 1) / kUnit * kUnit);
    p.q1 = g.w1.q;
    p.s1 = g.w1.s;
    p.ldq1 = g.w1.ldq;
    p.eq1 = g.w1.eq;
    p.ps1 = g.w1.ps;
    p.es1 = g.w1.es;
    p.q2 = g.w2.q;
    p.s2 = g.w2.s;
    p.ldq2 = g.w2.ldq;
    p.eq2 = g.w2.eq;
    p.ps2 = g.w2.ps;
    p.es2 = g.w2.es;
    p.y = static_cast<uint16_t*>(g.y);
    p.ldy = g.ldy;
    p.ids = g.ids;
    p.weights = g.weights;
    p.arrived = reinterpret_cast<uint32_t*>(ws);
    p.logits = reinterpret_cast<double*>(ws + m.logits);
    p.xq = ws + m.xq;
    p.xs = ws + m.xs;
    p.aq = ws + m.aq;
    p.as = ws + m.as;
    p.ctr = g.ctr;
    p.tiles_e = (p.experts + 15) / 16;
    p.tiles_t = (p.tokens + 15) / 16;
    p.by_pair = p.tokens * p.top_k <= p.experts;

    const auto al16 = [](const void* v) { return (reinterpret_cast<uintptr_t>(v) & 15u) == 0; };
    const bool vec = p.hidden % 8 == 0 && p.ldx % 8 == 0 && p.ldr % 8 == 0 && al16(g.x) && al16(g.router);
    const int items = p.tokens * ((p.hp + mx4::kPanel - 1) / mx4::kPanel);
    const int route = p.tiles_e * p.tiles_t + (items + kRouteThreads / 64 - 1) / (kRouteThreads / 64);
    if (vec)
        hipLaunchKernelGGL((k_moe_route<true>), dim3(route), dim3(kRouteThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((k_moe_route<false>), dim3(route), dim3(kRouteThreads), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int slots = p.by_pair ? p.tokens * p.top_k : p.experts;
    hipLaunchKernelGGL(k_moe_up, dim3(slots * ((p.inner + 31) / 32)), dim3(kUpThreads), 0, stream, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int lds = kDownThreads / 64 * p.tokens * 64;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_moe_down), hipFuncAttributeMaxDynamicSharedMemorySize,
                            kDownThreads / 64 * 64 * 64);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_moe_down, dim3((p.hidden + 15) / 16), dim3(kDownThreads), lds, stream, p);
    return hipGetLastError();
}

}  // namespace fp8mi
