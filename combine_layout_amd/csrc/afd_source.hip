// afd_source.hip -- gfx950 kernels of the source's side of a round: the norm
// with the residual's addition, the router's choice, the balance loss, and
// their gradients; and the HIP executor behind their be_* hooks.
//
// Nothing here is a dense contraction: every kernel reads its rows once, keeps
// them in registers, and is bound by HBM where there are many rows and by one
// trip to memory and the launch where there are few.  Sums cross lanes, then
// wavefronts, in an order that the sizes alone fix, so that the same inputs
// give the same bits; the only atomics are counts of integers.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "afd_plan.h"

namespace afd {
namespace {

constexpr int kWave = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

int launched() { return hipGetLastError() == hipSuccess ? 0 : 1; }

// ------------------------------------------------------------ across lanes ----

struct Sum {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumInt {
    __device__ __forceinline__ int operator()(int a, int b) const { return a + b; }
};
struct MaxInt {
    __device__ __forceinline__ int operator()(int a, int b) const { return max(a, b); }
};
struct MinInt {
    __device__ __forceinline__ int operator()(int a, int b) const { return min(a, b); }
};

template <int CTRL, typename T>
__device__ __forceinline__ T dpp(T v)
{
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// The reduction of every aligned group of LANES lanes, in each of its lanes; every
// lane of the wavefront has to take part.  Inside a row of 16 lanes by DPP (pairs,
// quads, then mirrored halves), across rows by swapping them with a copy.
template <int LANES, typename T, typename Op>
__device__ __forceinline__ T across(T v, Op op)
{
    v = op(v, dpp<0xB1>(v));    // lanes 1 0 3 2 of each four
    v = op(v, dpp<0x4E>(v));    // 2 3 0 1
    v = op(v, dpp<0x141>(v));   // each eight mirrored
    v = op(v, dpp<0x140>(v));   // each sixteen mirrored
    if constexpr (LANES > 16) {
        const unsigned u = __builtin_bit_cast(unsigned, v);
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const unsigned lo = r[0], hi = r[1];   // a bit cast of a vector's element takes its first
        v = op(__builtin_bit_cast(T, lo), __builtin_bit_cast(T, hi));
    }
    if constexpr (LANES > 32) {
        const unsigned u = __builtin_bit_cast(unsigned, v);
        const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        const unsigned lo = r[0], hi = r[1];   // a bit cast of a vector's element takes its first
        v = op(__builtin_bit_cast(T, lo), __builtin_bit_cast(T, hi));
    }
    return v;
}

// ------------------------------------------------------------- conversions ----

__device__ __forceinline__ uint32_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) { return to_bf16(lo) | (to_bf16(hi) << 16); }
__device__ __forceinline__ float from_bf16(uint32_t u) { return __builtin_bit_cast(float, u << 16); }

// Eight consecutive elements as they lie in memory: 16 bytes of bf16, or 32 of float32.
template <bool F32>
struct Eight;
template <>
struct Eight<false> {
    u32x4 a;
    __device__ __forceinline__ void load(const void *p, int64_t at) { a = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + at); }
    __device__ __forceinline__ void zero() { a = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w = a[i / 2];
        return __builtin_bit_cast(float, i % 2 ? w & 0xFFFF0000u : w << 16);
    }
};
template <>
struct Eight<true> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t at)
    {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + at);
        a = q[0];
        b = q[1];
    }
    __device__ __forceinline__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};

__device__ __forceinline__ u32x4 eight_bf16(const float *v)
{
    return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

template <bool F32>
__device__ __forceinline__ void store_eight(void *p, int64_t at, const float *v)
{
    if constexpr (F32) {
        f32x4 *q = reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at);
        q[0] = f32x4{v[0], v[1], v[2], v[3]};
        q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + at) = eight_bf16(v);
    }
}

// Scale of a block of E4M3 codes with the largest value m, and the factor to the codes;
// a scale below float32's smallest normal number counts as zero.
__device__ __forceinline__ float scale_of(float m, float &inv)
{
    const float s = m / 448.0f;
    if (s < 0x1p-126f) {
        inv = 0.f;
        return 0.f;
    }
    inv = 1.0f / s;
    return s;
}

__device__ __forceinline__ uint32_t four_codes(const float *v, float inv)
{
    const int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, c, true));
}

// The norm's weights, of either type.
struct Weights {
    u32x4 a, b;
    __device__ __forceinline__ void load(const void *p, int at, bool w32)
    {
        if (w32) {
            const u32x4 *q = reinterpret_cast<const u32x4 *>(static_cast<const float *>(p) + at);
            a = q[0];
            b = q[1];
        } else {
            a = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + at);
        }
    }
    __device__ __forceinline__ void values(float *v, bool w32) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h = a[i / 2], f = i < 4 ? a[i & 3] : b[i & 3];
            v[i] = __builtin_bit_cast(float, w32 ? f : i % 2 ? h & 0xFFFF0000u : h << 16);
        }
    }
};

// -------------------------------------------------------------------- norm ----

struct NormArgs {
    const void *x, *r, *w;
    void *out, *h;
    float *outs, *rstd;
    int64_t xs, rs, hs;
    int first, rows, H;   // rows [first, rows) in this launch
    float eps;
    bool w32;
};

// h = x + residual, y = h * rstd * weight, rstd = 1 / sqrt(mean(h^2) + eps).  A row is held
// by WPR wavefronts, C runs of eight columns a lane, from its one load to its last store, so
// that the bytes are the floor's.  RES: 0 no residual, 1 bf16, 2 float32.  Bound by HBM: 59
// MB in 11.7 us (4096 rows of 2048, FP8), 805 MB in 146 (16381 of 4096, float32 stream), where
// a copy takes 11.4 and 155; one row 2.2 us, the launch and a trip to memory.
template <bool X32, int RES, bool OUT8, int WPR, int C>
__global__ __launch_bounds__(WPR > 4 ? WPR *kWave : 256) void k_norm(NormArgs a)
{
    constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = (wave % WPR) * kWave + lane, runs = a.H / 8;
    const int64_t row = a.first + int64_t(blockIdx.x) * kRows + wave / WPR;
    if (row >= a.rows) return;   // a whole workgroup, or a wavefront with a row of its own
    Eight<X32> x[C];
    Eight<RES == 2> r[RES ? C : 1];
    Weights w[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = i * WPR * kWave + t;
        x[i].zero();
        if (RES) r[i].zero();
        if (c < runs) {
            x[i].load(a.x, row * a.xs + c * 8);
            if (RES) r[i].load(a.r, row * a.rs + c * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = i * WPR * kWave + t;
        if (c < runs) w[i].load(a.w, c * 8, a.w32);
    }
    float v[C][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = i * WPR * kWave + t;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] = x[i].get(j);
            if (RES) v[i][j] += r[i].get(j);
            if (RES == 1) v[i][j] = from_bf16(to_bf16(v[i][j]));   // normalised as stored
            ss = fmaf(v[i][j], v[i][j], ss);
        }
        if (RES && c < runs) store_eight<RES == 2>(a.h, row * a.hs + c * 8, v[i]);
    }
    ss = across<kWave>(ss, Sum());
    if constexpr (WPR > 1) {
        __shared__ float part[WPR];
        if (lane == 0) part[wave] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) ss += part[i];
    }
    const float rstd = __builtin_amdgcn_rsqf(ss / float(a.H) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = i * WPR * kWave + t;
        float y[8];
        w[i].values(y, a.w32);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = v[i][j] * rstd * y[j];
        if constexpr (OUT8) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[j]));
            m = across<16>(m, Max());   // 16 lanes hold a block of 128 columns
            float inv;
            const float s = scale_of(m, inv);
            if (c < runs) {
                *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.out) + row * a.H + c * 8) =
                    u32x2{four_codes(y, inv), four_codes(y + 4, inv)};
                if (lane % 16 == 0) a.outs[row * (a.H / 128) + c / 16] = s;
            }
        } else if (c < runs) {
            store_eight<false>(a.out, row * a.H + c * 8, y);
        }
    }
}

struct NormGradArgs {
    const void *g, *gr, *h, *w;
    const float *rstd;
    void *dh;
    float *part, *dw;
    int64_t hs;
    int rows, H, groups;   // workgroups of rows; with dw, those behind them have 64 columns of it each
    bool w32;
};

// 64 columns of dweight over all rows, eight a thread: few rows are read again, from the
// caches, rather than joined by a second launch.
template <bool H32, int THREADS>
__device__ __forceinline__ void norm_grad_columns(const NormGradArgs &a, int block)
{
    constexpr int kSlices = THREADS / 8;
    __shared__ f32x4 join[kSlices][16];
    const int slice = threadIdx.x / 8, c = block * 64 + threadIdx.x % 8 * 8;
    float s[8] = {};
    if (c < a.H) {
#pragma unroll 4
        for (int64_t row = slice; row < a.rows; row += kSlices) {
            Eight<false> g;
            Eight<H32> h;
            g.load(a.g, row * a.H + c);
            h.load(a.h, row * a.hs + c);
            const float rstd = a.rstd[row];
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = fmaf(g.get(j), h.get(j) * rstd, s[j]);
        }
    }
    join[slice][threadIdx.x % 8 * 2] = f32x4{s[0], s[1], s[2], s[3]};
    join[slice][threadIdx.x % 8 * 2 + 1] = f32x4{s[4], s[5], s[6], s[7]};
    __syncthreads();
    const int one = block * 64 + threadIdx.x;
    if (threadIdx.x < 64 && one < a.H) {
        float t = 0.f;
#pragma unroll 8
        for (int i = 0; i < kSlices; ++i) t += reinterpret_cast<const float *>(join[i])[threadIdx.x];
        a.dw[one] = t;
    }
}

// dh = rstd * (a - u * mean(a * u)) + grad_residual of every row, a = grad * weight and u =
// h * rstd, and the workgroup's sum of grad * u over its rows, which stays in registers from
// the first row to the last: dweight costs no second reading of many rows.  101 MB in 19 us
// (6144 rows of 2048, BF16; a copy's 19.4) and 4.1 for the launch behind it.
template <bool H32, int WPR, int C>
__global__ __launch_bounds__(WPR > 4 ? WPR *kWave : 256) void k_norm_grad(NormGradArgs a)
{
    constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = (wave % WPR) * kWave + lane, runs = a.H / 8;
    if (a.dw && int(blockIdx.x) >= a.groups) {
        norm_grad_columns<H32, (WPR > 4 ? WPR * kWave : 256)>(a, int(blockIdx.x) - a.groups);
        return;
    }
    __shared__ float sum[2][WPR];
    float dw[C][8] = {};
    int turn = 0;
    for (int64_t row = int64_t(blockIdx.x) * kRows + wave / WPR; row < a.rows; row += int64_t(a.groups) * kRows) {
        Eight<false> g[C];
        Eight<H32> h[C], gr[C];
        Weights w[C];
        const float rstd = a.rstd[row];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = i * WPR * kWave + t;
            g[i].zero();
            h[i].zero();
            gr[i].zero();
            if (c < runs) {
                g[i].load(a.g, row * a.H + c * 8);
                h[i].load(a.h, row * a.hs + c * 8);
                if (a.gr) gr[i].load(a.gr, row * a.H + c * 8);
                w[i].load(a.w, c * 8, a.w32);
            }
        }
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            float x[8];
            w[i].values(x, a.w32);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = h[i].get(j) * rstd;
                // columns behind the last hold whatever w holds: grad is 0 there
                x[j] = i * WPR * kWave + t < runs ? g[i].get(j) * x[j] : 0.f;
                m = fmaf(x[j], u, m);
                dw[i][j] = fmaf(g[i].get(j), u, dw[i][j]);
            }
        }
        m = across<kWave>(m, Sum());
        if constexpr (WPR > 1) {
            if (lane == 0) sum[turn][wave] = m;
            __syncthreads();
            m = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) m += sum[turn][i];
            turn ^= 1;   // the next row's sums go to the other half: one barrier a row
        }
        m /= float(a.H);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = i * WPR * kWave + t;
            if (c >= runs) continue;
            float x[8];
            w[i].values(x, a.w32);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = fmaf(rstd, g[i].get(j) * x[j] - h[i].get(j) * rstd * m, gr[i].get(j));
            store_eight<H32>(a.dh, row * a.H + c * 8, x);
        }
    }
    if (!a.part) return;
    float *part = a.part + int64_t(blockIdx.x) * a.H;
    if constexpr (WPR == 1) {
        // the four wavefronts hold the same columns: added one after another in LDS
        __shared__ f32x4 join[2 * C * kWave];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (wave == k) {
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    f32x4 *p = join + 2 * (i * kWave + lane);
                    f32x4 lo = {dw[i][0], dw[i][1], dw[i][2], dw[i][3]}, hi = {dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
                    if (k > 0) {
                        lo += p[0];
                        hi += p[1];
                    }
                    p[0] = lo;
                    p[1] = hi;
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.H / 4; c += 256) reinterpret_cast<f32x4 *>(part)[c] = join[c];
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = i * WPR * kWave + t;
            if (c < runs) store_eight<true>(part, c * 8, dw[i]);
        }
    }
}

// dweight: 64 columns a workgroup, four a thread, the partial rows over 64 of its threads.
__global__ __launch_bounds__(1024) void k_norm_grad_join(const float *part, float *dw, int H, int groups)
{
    __shared__ f32x4 join[64][16];
    const int col = threadIdx.x % 16, slice = threadIdx.x / 16, c = blockIdx.x * 64 + col * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (c < H) {
#pragma unroll
        for (int i = 0; i < kNormGradGroups / 64; ++i)
            if (i * 64 + slice < groups) s += *reinterpret_cast<const f32x4 *>(part + int64_t(i * 64 + slice) * H + c);
    }
    join[slice][col] = s;
    __syncthreads();
    const int one = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && one < H) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) t += reinterpret_cast<const float *>(join[i])[threadIdx.x];
        dw[one] = t;
    }
}

// ------------------------------------------------------------------ routes ----

constexpr float kMinusInf = -__builtin_inff();

// exp(x) for x <= 0.  The argument's rounding costs 1.2 |x| roundings of the result, which
// summands that are small beside 1 can bear; a second part of the product with log2(e) would
// be five instructions more of every logit, where the arithmetic bounds (balance loss of 32768
// tokens and 512 experts 20.5 -> 21.9 us, with sigmoids 22.2 -> 24.7; of 256 tokens and 128
// experts 7.0 -> 7.8).
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// exp(a - b) for a <= b, to three half steps however far they lie apart: a weight is the term
// itself and no summand, and a token has K of them, one or two a lane (32768 tokens of 512
// experts, routes 21.9 -> 22.4 us with it, 256 of 128 3.47 -> 3.53).  What the difference and its
// product with log2(e) lose is kept and multiplied on.  Below -120 it is 0; where both are the
// same infinity it is no number.
__device__ __forceinline__ float exp_between(float a, float b)
{
    const float d = a - b, back = d - a;
    const float lost = (a - (d - back)) - (b + back);
    const float hi = d * 1.44269504f;
    const float lo = fmaf(lost, 1.44269504f, fmaf(d, 1.92596300e-8f, fmaf(d, 1.44269504f, -hi)));
    const float e = __builtin_amdgcn_exp2f(hi);
    return d < -120.f ? 0.f : fmaf(e, lo * 0.693147181f, e);
}

// 1 / d for d in [1, 2]: the hardware's reciprocal and one step of Newton's.
__device__ __forceinline__ float inverse(float d)
{
    const float r = __builtin_amdgcn_rcpf(d);
    return fmaf(fmaf(-d, r, 1.0f), r, r);
}

// Integers in the order of the floats they stand for (the two zeros are one).
constexpr int kNoKey = int(0x807FFFFF);   // minus infinity
__device__ __forceinline__ int key_of(float v)
{
    const int b = __builtin_bit_cast(int, v + 0.f);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float of_key(int k) { return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7FFFFFFF)); }

struct RouteArgs {
    const void *l;
    const float *bias;
    const uint8_t *live;
    int32_t *ids;
    float *w;
    const float *g, *slope;
    void *dl;
    int64_t ls;
    int rows, E, K;
    float scale;
    bool sigmoid, renorm;
};

// A token's logits over LANES lanes, V a lane in runs of four, so that the lanes of a load or
// store touch one run of memory (eight consecutive ones a lane: 47 us instead of 31 for the
// balance loss's gradient of 32768 tokens and 512 experts).  Experts behind the last, and
// NaNs, are minus infinity.
template <bool L32, int LANES, int V, bool VEC>
struct Row {
    static constexpr int kLanes = LANES, kV = V;
    static constexpr int kRows = 256 / LANES;   // tokens of a workgroup of 256
    static constexpr int kSlots = (kMaxTopk + LANES - 1) / LANES;

    __device__ static __forceinline__ int lane() { return threadIdx.x & (LANES - 1); }
    __device__ static __forceinline__ int expert(int i) { return (i & 4) * LANES + 4 * lane() + (i & 3); }

    __device__ static __forceinline__ float one(const RouteArgs &a, int64_t at)
    {
        if (L32) return static_cast<const float *>(a.l)[at];
        return from_bf16(static_cast<const uint16_t *>(a.l)[at]);
    }

    // Logits as they lie in memory, so that nothing waits for a load before it is needed.
    struct Raw {
        typename std::conditional<L32, f32x4, u32x2>::type q[V / 4];

        __device__ __forceinline__ void load(const RouteArgs &a, int64_t row)
        {
            const int64_t base = row * a.ls;
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const int e = expert(i * 4);
                q[i] = {};
                if constexpr (VEC) {
                    if (e < a.E) {
                        if constexpr (L32) q[i] = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.l) + base + e);
                        else q[i] = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(a.l) + base + e);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (e + j >= a.E) continue;
                        if constexpr (L32) q[i][j] = static_cast<const float *>(a.l)[base + e + j];
                        else q[i][j / 2] |= uint32_t(static_cast<const uint16_t *>(a.l)[base + e + j]) << (16 * (j & 1));
                    }
                }
            }
        }

        __device__ __forceinline__ void values(const RouteArgs &a, float *v) const
        {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float x;
                if constexpr (L32) x = q[i / 4][i & 3];
                else x = from_bf16(i & 1 ? q[i / 4][(i & 3) / 2] >> 16 : q[i / 4][(i & 3) / 2] & 0xFFFFu);
                // (whole runs of four are inside or behind where they are loaded whole)
                v[i] = expert(VEC ? i & ~3 : i) < a.E && x == x ? x : kMinusInf;
            }
        }
    };

    __device__ static __forceinline__ void load(const RouteArgs &a, int64_t row, float *v)
    {
        Raw r;
        r.load(a, row);
        r.values(a, v);
    }

    __device__ static __forceinline__ void store(const RouteArgs &a, int64_t row, const float *d)
    {
        const int64_t base = row * a.E;
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const int e = expert(q * 4);
            const float *x = d + q * 4;
            if constexpr (VEC) {
                if (e < a.E) {
                    if (L32) *reinterpret_cast<f32x4 *>(static_cast<float *>(a.dl) + base + e) = f32x4{x[0], x[1], x[2], x[3]};
                    else *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.dl) + base + e) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (e + j >= a.E) continue;
                    if (L32) static_cast<float *>(a.dl)[base + e + j] = x[j];
                    else static_cast<uint16_t *>(a.dl)[base + e + j] = uint16_t(to_bf16(x[j]));
                }
            }
        }
    }

    __device__ static __forceinline__ float largest(const float *v)
    {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
        return of_key(across<LANES>(key_of(m), MaxInt()));   // as integers: no step has to look for NaNs
    }

    __device__ static __forceinline__ float total(const float *v)
    {
        float s = v[0];
#pragma unroll
        for (int i = 1; i < V; ++i) s += v[i];
        return across<LANES>(s, Sum());
    }

    // exp(l - m) of every logit and their sum (0 without an expert).  Where the largest
    // is infinite its holders have the term 1: an infinity less itself is no number.
    __device__ static __forceinline__ float terms(const float *v, float m, float *t)
    {
        const float top = m == kMinusInf ? -kMinusInf : m;   // without an expert every term is 0
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float e = exp_neg(v[i] - top);
            t[i] = v[i] == -kMinusInf ? 1.f : e;
        }
        return total(t);
    }

    // Sigmoids in the same proportions but for a common factor, and their sum: where every
    // logit is far below zero the largest is lifted to about 1, so that none vanishes.
    // left: 1 - sigmoid.
    __device__ static __forceinline__ float sigmoids(const float *v, float m, float *t, float *left)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = exp_neg(-fabsf(v[i])), d = inverse(1.0f + z);
            t[i] = (v[i] >= 0.f ? 1.f : z) * d;   // of minus infinity 0
            left[i] = (v[i] >= 0.f ? z : 1.f) * d;
        }
        if (__any(m < -40.f)) {
            const float top = m == kMinusInf ? -kMinusInf : m;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float e = exp_neg(v[i] - top);   // 1 - sigmoid is 1 here
                t[i] = m < -40.f ? e : t[i];
            }
        }
        return total(t);
    }
};

// The weights, but for the scale, of a token's chosen logits, one a lane and slot; m and sum
// of the softmax's terms where it is over all experts.
template <int LANES, int SLOTS>
__device__ __forceinline__ void weights_of(const RouteArgs &a, const float *l, const bool *on, float m, float sum, float *w)
{
    if (!a.sigmoid && !a.renorm) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            w[s] = !on[s] || l[s] == kMinusInf ? 0.f : (l[s] == m ? 1.f : exp_between(l[s], m)) / sum;
        return;
    }
    float top = kMinusInf;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
        if (on[s]) top = fmaxf(top, l[s]);
    top = across<LANES>(top, Max());
    float t = 0.f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        if (!a.sigmoid) {
            w[s] = l[s] == top ? 1.f : exp_between(l[s], top);
        } else {
            const float term = exp_between(a.renorm ? l[s] : -fabsf(l[s]), a.renorm ? fminf(top, 0.f) : 0.f);
            w[s] = (l[s] >= 0.f ? 1.f : term) * inverse(1.0f + exp_neg(-fabsf(l[s])));
        }
        if (!on[s] || l[s] == kMinusInf) w[s] = 0.f;
        t += w[s];
    }
    if (!a.renorm) return;
    t = across<LANES>(t, Sum());
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) w[s] = t > 0.f ? w[s] / t : 0.f;
}

// A lane's keys in falling order, and the place that each came from, four bits each.  Only
// neighbours change places, and only where the second is larger: equal keys stay in order.
template <int V>
__device__ __forceinline__ uint32_t sort_keys(int *k)
{
    int at[V];
#pragma unroll
    for (int i = 0; i < V; ++i) at[i] = i;
#pragma unroll
    for (int r = 0; r < V; ++r) {
#pragma unroll
        for (int i = r & 1; i + 1 < V; i += 2) {
            const int a = k[i], b = k[i + 1];
            // by differences: a choice between two elements becomes an index that is not
            // known, and 1000 instructions for the eight
            const int d = b > a ? at[i] ^ at[i + 1] : 0;
            k[i] = max(a, b);
            k[i + 1] = min(a, b);
            at[i] ^= d;
            at[i + 1] ^= d;
        }
    }
    uint32_t order = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) order |= uint32_t(at[i]) << (4 * i);
    return order;
}

struct Pick {
    int id, key;
};

// Orders one wavefront's accesses to LDS: its own lanes read what others of them wrote.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// What a token's choice leaves: up to kMost keys in falling order.
template <int LANES>
constexpr int kMost = LANES == 16 ? 48 : 64;

// Whether two keys with biases may be out of order.  A sigmoid is off by less than 4
// roundings of 1 (the exponential's argument and result, the sum, the reciprocal and the
// product), a softmax by less than 25 (its sum's 14 more); the sum with the bias by one of its
// own size.  Two keys that are 16, or 64, of both apart are in order (2^-20 = 16 roundings).
__device__ __forceinline__ bool too_near(int larger, int smaller, bool sigmoid)
{
    const float lo = of_key(smaller);
    return smaller != kNoKey && !(of_key(larger) - lo > (sigmoid ? 0x1p-20f : 0x1p-18f) * (1.f + fabsf(lo)));
}

struct Taken {
    int count;    // keys taken, the same for every token of the wavefront
    bool close;   // two of this token's follow each other too nearly to be in order
    bool open;    // so do the last two
};

// The largest keys of a token, one after another: the lanes' first keys are compared, the
// lane that holds the largest writes it down and goes on to its next; of several, the one
// with the lowest expert.  `rounds` of them, with NEAR one more for the border behind the
// last place, and as many as are too near to it.
template <typename R, int LANES, int V, bool NEAR>
__device__ __forceinline__ Taken take(int *k, int rounds, bool sigmoid, Pick *picks)
{
    uint32_t order = sort_keys<V>(k);
    Taken t{0, false, false};
    int before = 0x7F800000;
    const int base = (threadIdx.x & 63) & ~(LANES - 1);
    for (int r = 0; r < rounds || (NEAR && r <= rounds) || (NEAR && r < kMost<LANES> && __any(t.open)); ++r) {
        const int m = across<LANES>(k[0], MaxInt()), e = R::expert(order & 7);
        bool mine = k[0] == m;
        uint64_t hit = __ballot(mine) >> base;
        if (LANES < 64) hit &= (uint64_t(1) << (LANES & 63)) - 1;
        if (__any((hit & (hit - 1)) != 0)) {
            const int low = across<LANES>(mine ? e : INT32_MAX, MinInt());   // by every lane of the wavefront
            mine = mine && low == e;
        }
        mine = mine && m != kNoKey;
        if (mine) picks[r] = Pick{e, m};
        // by a mask: a choice between two elements becomes an index that is not known, and the keys go to scratch memory
        const int pop = mine ? -1 : 0;
        order = mine ? order >> 4 : order;
#pragma unroll
        for (int i = 0; i < V; ++i) k[i] = (pop & (i + 1 < V ? k[i + 1] : kNoKey)) | (~pop & k[i]);
        if constexpr (NEAR) {
            t.open = r > 0 && too_near(before, m, sigmoid);
            t.close = t.close || t.open;
            before = m;
        }
        t.count = r + 1;
    }
    return t;
}

// The 64-bit score of a logit; `sum` of the softmax's terms.
__device__ __forceinline__ double score(const RouteArgs &a, float l, float m, double sum)
{
    if (a.sigmoid) return 1.0 / (1.0 + exp(-double(l)));
    return (l == kMinusInf ? 0.0 : l == m ? 1.0 : exp(double(l) - double(m))) / sum;
}

template <typename R>
__device__ __forceinline__ double score_sum(const RouteArgs &a, const float *v, float m)
{
    if (a.sigmoid) return 1.0;
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < R::kV; ++i) t += score(a, v[i], m, 1.0);
    for (int d = 1; d < R::kLanes; d *= 2) t += __shfl_xor(t, d);
    return t;
}

// The order of the picked experts by their 64-bit scores: each compares itself with all.
template <typename R>
__device__ __forceinline__ void order_exactly(const RouteArgs &a, int64_t row, int count, Pick *picks)
{
    constexpr int LANES = R::kLanes, kEach = kMost<LANES> / LANES;
    float m = 0.f;
    double sum = 1.0;
    if (!a.sigmoid) {
        float v[R::kV];
        R::load(a, row, v);   // again, rather than held by all who need none of this
        m = R::largest(v);
        sum = score_sum<R>(a, v, m);
    }
    double key[kEach];
    int id[kEach], rank[kEach];
#pragma unroll
    for (int s = 0; s < kEach; ++s) {
        id[s] = s * LANES + R::lane() < count ? picks[s * LANES + R::lane()].id : -1;
        rank[s] = 0;
        key[s] = -__builtin_inf();
        if (id[s] >= 0) key[s] = score(a, R::one(a, row * a.ls + id[s]), m, sum) + double(a.bias[id[s]]);
    }
    for (int j = 0; j < count; ++j) {
        double x = 0.0;
        int e = -1;
#pragma unroll
        for (int s = 0; s < kEach; ++s) {
            if (j / LANES != s) continue;
            x = __shfl(key[s], j % LANES, LANES);
            e = __shfl(id[s], j % LANES, LANES);
        }
#pragma unroll
        for (int s = 0; s < kEach; ++s) rank[s] += e >= 0 && (x > key[s] || (x == key[s] && e < id[s]));
    }
    wave_sync();
#pragma unroll
    for (int s = 0; s < kEach; ++s)
        if (id[s] >= 0) picks[rank[s]].id = id[s];
}

// The choice by 64-bit scores from the start, where more than kMost follow each other too
// nearly.
template <typename R>
__device__ __forceinline__ void take_exactly(const RouteArgs &a, int64_t row, Pick *picks)
{
    constexpr int V = R::kV, LANES = R::kLanes;
    float v[V];
    R::load(a, row, v);
    const float m = R::largest(v);
    const double sum = score_sum<R>(a, v, m);
    double key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = R::expert(i);
        const double x = score(a, v[i], m, sum) + (e < a.E ? double(a.bias[e]) : 0.0);
        key[i] = v[i] == kMinusInf || !(x == x) ? -__builtin_inf() : x;
    }
    for (int k = 0; k < a.K; ++k) {
        double top = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = key[i] > top ? key[i] : top;
        for (int d = 1; d < LANES; d *= 2) {
            const double o = __shfl_xor(top, d);
            top = o > top ? o : top;
        }
        int e = INT32_MAX;
#pragma unroll
        for (int i = V - 1; i >= 0; --i) e = key[i] == top ? R::expert(i) : e;
        e = across<LANES>(e, MinInt());
        if (R::lane() == 0) picks[k].id = top == -__builtin_inf() ? -1 : e;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = R::expert(i) == e ? -__builtin_inf() : key[i];
    }
}

// The choice of a wavefront with one token: a border that at least K of the lanes' largest
// keys reach is found by halving, the keys that reach it (about K and a few; with NEAR those
// too that are too near to it) are brought together, one a lane, and each counts the larger
// ones.  Returns the lane's key and its rank, or false where more than 64 reach the border
// (many equal keys), with `k` as it was.
template <typename R, int V, bool NEAR>
__device__ __forceinline__ bool take_above(const int *k, int K, Pick *picks, Pick &mine, int &rank, int &count)
{
    int head = k[0];
#pragma unroll
    for (int i = 1; i < V; ++i) head = max(head, k[i]);
    int lo = __builtin_amdgcn_readfirstlane(across<kWave>(head, MinInt()));
    int hi = __builtin_amdgcn_readfirstlane(across<kWave>(head, MaxInt()));
    for (int i = 0; i < 12 && lo < hi; ++i) {
        const int mid = lo + int(((uint32_t(hi) - uint32_t(lo)) >> 1) + ((uint32_t(hi) - uint32_t(lo)) & 1));
        const int reach = __popcll(__ballot(head >= mid));
        if (reach >= K) {
            lo = mid;
            if (reach <= K + 2) break;
        } else {
            hi = mid - 1;
        }
    }
    if constexpr (NEAR) {
        const float f = of_key(lo);
        if (f - f == 0.f) lo = key_of(f - 0x1p-17f * (1.f + fabsf(f)));   // (twice what too_near allows)
    }
    lo = max(lo, kNoKey + 1);
    count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) count += __popcll(__ballot(k[i] >= lo));
    if (count > kWave) return false;
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint64_t in = __ballot(k[i] >= lo);
        const int to = at + __builtin_amdgcn_mbcnt_hi(uint32_t(in >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(in), 0));
        if (k[i] >= lo) picks[to] = Pick{R::expert(i), k[i]};
        at += __popcll(in);
    }
    wave_sync();
    mine = R::lane() < count ? picks[R::lane()] : Pick{-1, kNoKey};
    rank = 0;
    // key, then the lower expert, as one number
    const uint64_t self = uint64_t(uint32_t(mine.key) ^ 0x80000000u) << 32 | uint32_t(~mine.id);
    for (int j = 0; j < count; ++j) {
        const uint64_t other = uint64_t(uint32_t(__builtin_amdgcn_readlane(int(self >> 32), j))) << 32 |
                               uint32_t(__builtin_amdgcn_readlane(int(self), j));
        rank += other > self;
    }
    return true;
}

// One token per LANES lanes, its logits in registers from the load on.  What bounds it is
// the choice, which is arithmetic and not memory: a round of `take` is one reduction over
// the lanes, so a lane's logits are sorted once and only the first of them takes part; with
// a wavefront for a token a border is cheaper (take_above: 38 -> 29 us).  32768 tokens of 512
// experts, 8 chosen: 24 us, of which the logits' 67 MB are 13 and the vector instructions 18;
// 65536 tokens of 128: 19, 7 and 16, of 256: 34, 14 and 33 (with a bias 29, 7 and 25; 50, 14 and
// 50); 6144 tokens of 96 with a bias 7.1; 256 of 128 4.0, the launch, a trip to memory and the
// chain of eight rounds.
template <bool L32, int LANES, int V, bool VEC, bool BIAS>
__global__ __launch_bounds__(256) void k_route(RouteArgs a)
{
    using R = Row<L32, LANES, V, VEC>;
    __shared__ Pick picked[R::kRows][kMost<LANES>];
    const int lane = R::lane();
    const int64_t row_ = int64_t(blockIdx.x) * R::kRows + threadIdx.x / LANES, row = min(row_, int64_t(a.rows - 1));
    Pick *picks = picked[threadIdx.x / LANES];
    float v[V];
    R::load(a, row, v);
    const bool live = !a.live || a.live[row] != 0;
    float m = 0.f, sum = 1.f;
    int key[V];
    if constexpr (BIAS) {
        float b[V], t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = R::expert(i) < a.E ? a.bias[R::expert(i)] : 0.f;
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float z = exp_neg(-fabsf(v[i]));
                t[i] = (v[i] >= 0.f ? 1.f : z) * inverse(1.0f + z);
            }
        } else {
            m = R::largest(v);
            sum = R::terms(v, m, t);
            const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] *= inv;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = t[i] + b[i];
            key[i] = v[i] == kMinusInf || !(x == x) ? kNoKey : key_of(x);
        }
    } else {
        if (!a.sigmoid && !a.renorm) {
            float t[V];
            m = R::largest(v);
            sum = R::terms(v, m, t);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key_of(v[i]);
    }
    bool done = false;
    if constexpr (BIAS && LANES == kWave) {
        Pick mine;
        int rank, count;
        done = take_above<R, V, true>(key, a.K, picks, mine, rank, count);
        if (done) {
            wave_sync();
            picks[lane < count ? rank : lane] = mine;   // in order by the 32-bit scores
            wave_sync();
            const int below = lane + 1 < kWave ? picks[lane + 1].key : kNoKey;
            if (__any(lane < a.K && too_near(picks[lane].key, below, a.sigmoid))) {
                wave_sync();
                order_exactly<R>(a, row, count, picks);
            }
        }
    }
    if constexpr (!BIAS && LANES == kWave) {
        Pick mine;
        int rank, count;
        if (take_above<R, V, false>(key, a.K, picks, mine, rank, count)) {
            const bool on = lane < count && rank < a.K;
            const float l = of_key(mine.key);
            float w;
            weights_of<LANES, 1>(a, &l, &on, m, sum, &w);
            if (row_ < a.rows) {
                if (on) {
                    a.ids[row * a.K + rank] = live ? mine.id : -1;
                    a.w[row * a.K + rank] = live ? a.scale * w : 0.f;
                }
                if (lane >= count && lane < a.K) {
                    a.ids[row * a.K + lane] = -1;
                    a.w[row * a.K + lane] = 0.f;
                }
            }
            return;
        }
    }
    if (!done) {
#pragma unroll
        for (int s = 0; s < kMost<LANES> / LANES; ++s) picks[s * LANES + lane] = Pick{-1, kNoKey};
        wave_sync();
        const Taken taken = take<R, LANES, V, BIAS>(key, a.K, a.sigmoid, picks);
        if constexpr (BIAS) {
            if (__any(taken.close)) {
                wave_sync();
                if (__any(taken.open)) take_exactly<R>(a, row, picks);
                else order_exactly<R>(a, row, taken.count, picks);
            }
        }
    }
    wave_sync();
    bool on[R::kSlots];
    float w[R::kSlots], l[R::kSlots];
    int id[R::kSlots];
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) {
        const int k = s * LANES + lane;
        const Pick p = k < a.K ? picks[k] : Pick{-1, kNoKey};
        id[s] = p.id;
        on[s] = p.id >= 0;
        if (BIAS) l[s] = on[s] ? R::one(a, row * a.ls + p.id) : kMinusInf;
        else l[s] = of_key(p.key);
    }
    weights_of<LANES, R::kSlots>(a, l, on, m, sum, w);
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) {
        const int k = s * LANES + lane;
        if (k < a.K && row_ < a.rows) {
            a.ids[row * a.K + k] = live ? id[s] : -1;
            a.w[row * a.K + k] = live && on[s] ? a.scale * w[s] : 0.f;
        }
    }
}

// Slot k's value in every lane of its token.
template <int LANES, typename T>
__device__ __forceinline__ T slot(T v, int k)
{
    if constexpr (LANES == 64) return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), k));
    return __shfl(v, k % LANES, LANES);
}

// The weights' gradient by the chosen logits, and with DENSE (a softmax over all experts) by
// every other one.  Persistent, with the next token's logits (dense), ids and gradients on their
// way: 26 -> 24 us for 32768 tokens of 512 experts (dense; 137 MB, a copy's 26).  The chosen
// logits alone are gathered behind their ids: 65536 tokens of 128 experts 10.8 us, of 512 38,
// where the bytes that are written take 7 and 26.
template <bool L32, int LANES, int V, bool VEC, bool DENSE>
__global__ __launch_bounds__(256) void k_route_grad(RouteArgs a)
{
    using R = Row<L32, LANES, V, VEC>;
    constexpr int S = R::kSlots;
    __shared__ float spread[R::kRows][LANES * V];
    const int lane = R::lane();
    float *to = spread[threadIdx.x / LANES];
    const int64_t last = a.rows - 1, step = int64_t(gridDim.x) * R::kRows;
    int64_t row_ = int64_t(blockIdx.x) * R::kRows + threadIdx.x / LANES;
    typename R::Raw raw, raw_;
    int id[S], id_[S];
    float g[S], g_[S];
    const auto load = [&](int64_t r) {
        if (DENSE) raw_.load(a, r);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int k = s * LANES + lane;
            id_[s] = k < a.K ? a.ids[r * a.K + k] : -1;
            g_[s] = k < a.K ? a.g[r * a.K + k] : 0.f;
        }
    };
    load(min(row_, last));
    for (int64_t at = int64_t(blockIdx.x) * R::kRows; at < a.rows; at += step, row_ += step) {
        const int64_t row = min(row_, last);
        raw = raw_;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            id[s] = id_[s];
            g[s] = g_[s];
        }
        if (at + step < a.rows) load(min(row_ + step, last));
        bool on[S];
        float w[S], left[S], p[V], sum = 1.f, dot = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            on[s] = id[s] >= 0 && id[s] < a.E;
            id[s] = on[s] ? id[s] : -1;
            g[s] = on[s] ? g[s] * a.scale : 0.f;
            left[s] = 1.f;
        }
        if constexpr (DENSE) {
            float v[V];
            raw.values(a, v);
            sum = R::terms(v, R::largest(v), p);
            const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) to[R::expert(i)] = p[i] *= inv;
            wave_sync();
#pragma unroll
            for (int s = 0; s < S; ++s) w[s] = on[s] ? to[id[s]] : 0.f;
            wave_sync();
        } else {
            float l[S];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const float x = on[s] ? R::one(a, row * a.ls + id[s]) : kMinusInf;
                l[s] = x == x ? x : kMinusInf;
                if (a.sigmoid) {
                    const float z = exp_between(-fabsf(l[s]), 0.f);
                    left[s] = (l[s] >= 0.f ? z : 1.f) * inverse(1.0f + z);
                }
            }
            weights_of<LANES, S>(a, l, on, 0.f, 1.f, w);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) dot += w[s] > 0.f ? g[s] * w[s] : 0.f;
        dot = across<LANES>(dot, Sum());
        float c[S], all[S];   // what a slot adds to its expert's gradient, and every slot of that expert
#pragma unroll
        for (int s = 0; s < S; ++s) {
            c[s] = w[s] > 0.f ? w[s] * (a.renorm ? g[s] - dot : g[s]) * left[s] : 0.f;
            all[s] = 0.f;
        }
        for (int k = 0; k < a.K; ++k) {
            int e = 0;
            float x = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (k / LANES != s) continue;
                e = slot<LANES>(id[s], k);
                x = slot<LANES>(c[s], k);
            }
#pragma unroll
            for (int s = 0; s < S; ++s) all[s] += id[s] == e ? x : 0.f;
        }
        // to the experts' lanes through LDS; slots of one expert write the same sum
#pragma unroll
        for (int i = 0; i < V; ++i) to[R::expert(i)] = 0.f;
        wave_sync();
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (on[s]) to[id[s]] = all[s];
        wave_sync();
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = DENSE ? fmaf(p[i], -dot, to[R::expert(i)]) : to[R::expert(i)];
        wave_sync();
        if (row_ < a.rows) R::store(a, row, d);
    }
}

// ------------------------------------------------------------ balance loss ----

// What a token's shares come from, on its way.
template <typename R>
struct Token {
    typename R::Raw l;
    int32_t id[R::kSlots];
    __device__ __forceinline__ void load(const RouteArgs &a, int64_t row)
    {
        l.load(a, row);
#pragma unroll
        for (int s = 0; s < R::kSlots; ++s) {
            const int k = s * R::kLanes + R::lane();
            id[s] = k < a.K ? a.ids[row * a.K + k] : -1;
        }
    }
};

// A token's shares (0 where it does not count), with sigmoids the factors 1 - sigmoid, and
// whether it counts.  chosen: the lane's choices.
template <typename R>
__device__ __forceinline__ bool shares(const RouteArgs &a, const Token<R> &t, bool in, float *p, float *left, int32_t *hist,
                                       int &chosen)
{
    bool any = false;
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) {
        if (in && t.id[s] >= 0 && t.id[s] < a.E) {
            any = true;
            ++chosen;
            if (hist) atomicAdd(hist + t.id[s], 1);
        }
    }
    const uint64_t who = __ballot(any) >> ((threadIdx.x & 63) & ~(R::kLanes - 1));
    const bool on = R::kLanes == 64 ? who != 0 : (who & ((uint64_t(1) << (R::kLanes & 63)) - 1)) != 0;
    float v[R::kV];
    t.l.values(a, v);
    const float m = R::largest(v), sum = a.sigmoid ? R::sigmoids(v, m, p, left) : R::terms(v, m, p);
    const float inv = on && sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < R::kV; ++i) p[i] *= inv;
    return on;
}

struct BalanceArgs {
    RouteArgs r;
    float *share;
    int32_t *count, *totals;
    uint32_t *done;
    float *loss, *slope;   // with one workgroup
    int32_t *counts;
    float coefficient;
};

// The loss and the slope from an expert's sums, by the first E threads of a workgroup.
__device__ __forceinline__ float slope_of(float coefficient, int E, int count, int tokens, int chosen)
{
    const double n = double(tokens) * double(chosen);
    return n > 0.0 ? float(double(coefficient) * double(E) * double(count) / n) : 0.f;
}

// Sums of the shares over tokens in registers, counts in LDS; a token's logits and ids are
// on their way while the one before is worked on.  SOLO: one workgroup has all tokens, and
// ends with the results.  67 MB of logits in 15 us (32768 tokens of 512 experts; a copy's 13),
// with 1024 threads; 7 more for the launch that joins 256 workgroups' sums.
template <bool L32, int LANES, int V, bool VEC, int THREADS, bool SOLO>
__global__ __launch_bounds__(THREADS) void k_balance(BalanceArgs b)
{
    using R = Row<L32, LANES, V, VEC>;
    constexpr int kRows = THREADS / LANES;
    const RouteArgs &a = b.r;
    __shared__ int32_t hist[LANES * V], total[2];
    __shared__ float join[kRows][LANES * V];
    for (int e = threadIdx.x; e < LANES * V; e += THREADS) hist[e] = 0;
    if (threadIdx.x < 2) total[threadIdx.x] = 0;
    if (!SOLO && blockIdx.x == 0 && threadIdx.x == 0) *b.done = 0;   // for the launch behind this one
    __syncthreads();
    float acc[V] = {};
    int tokens = 0, chosen = 0;
    const int64_t last = a.rows - 1, step = int64_t(gridDim.x) * kRows;
    int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / LANES;
    Token<R> next;
    next.load(a, min(row, last));
    for (int64_t at = int64_t(blockIdx.x) * kRows; at < a.rows; at += step, row += step) {
        const Token<R> t = next;
        if (at + step < a.rows) next.load(a, min(row + step, last));
        float p[V], left[V];
        tokens += shares<R>(a, t, row <= last, p, left, hist, chosen);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += p[i];
    }
    tokens = across<kWave>(R::lane() == 0 ? tokens : 0, SumInt());
    chosen = across<kWave>(chosen, SumInt());
    if (threadIdx.x % kWave == 0) {
        atomicAdd(&total[0], tokens);
        atomicAdd(&total[1], chosen);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) join[threadIdx.x / LANES][R::expert(i)] = acc[i];
    __syncthreads();
    if constexpr (SOLO) {
        static_assert(THREADS >= kMaxExperts, "a thread for every expert");
        __shared__ double part[THREADS / kWave];
        const int e = threadIdx.x;
        double loss = 0.0;
        if (e < a.E) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kRows; ++i) s += join[i][e];
            const float slope = slope_of(b.coefficient, a.E, hist[e], total[0], total[1]);
            b.counts[e] = hist[e];
            b.slope[e] = slope;
            loss = double(slope) * double(s);
        }
        for (int d = 1; d < kWave; d *= 2) loss += __shfl_xor(loss, d);
        if (e % kWave == 0) part[e / kWave] = loss;
        __syncthreads();
        if (e != 0) return;
        loss = 0.0;
#pragma unroll
        for (int i = 0; i < THREADS / kWave; ++i) loss += part[i];
        b.loss[0] = float(loss);
        return;
    }
    for (int e = threadIdx.x; e < a.E; e += THREADS) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) s += join[i][e];
        b.share[int64_t(blockIdx.x) * a.E + e] = s;
        b.count[int64_t(blockIdx.x) * a.E + e] = hist[e];
    }
    if (threadIdx.x < 2) b.totals[blockIdx.x * 2 + threadIdx.x] = total[threadIdx.x];
}

struct BalanceJoinArgs {
    const float *share;
    const int32_t *count, *totals;
    double *part;
    uint32_t *done;
    float *loss, *slope;
    int32_t *counts;
    int E, groups;
    float coefficient;
};

// Sixteen experts a workgroup, sixteen threads for each; the workgroup that is done last
// adds the parts of the loss, in their order.
__global__ __launch_bounds__(256) void k_balance_join(BalanceJoinArgs a)
{
    __shared__ double share[16][16];
    __shared__ int count[16][16];
    __shared__ int2 totals[4];
    const int col = threadIdx.x % 16, slice = threadIdx.x / 16, e = blockIdx.x * 16 + col;
    // every load on its way before the first is used
    constexpr int kTurns = kBalanceGroups / 16;
    float sv[kTurns];
    int cv[kTurns];
    const int in = min(e, a.E - 1);
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int g = min(i * 16 + slice, a.groups - 1);
        sv[i] = a.share[int64_t(g) * a.E + in];
        cv[i] = a.count[int64_t(g) * a.E + in];
    }
    static_assert(kBalanceGroups <= 256, "a thread for every group's totals");
    int2 mine = {0, 0};
    if (int(threadIdx.x) < a.groups) mine = reinterpret_cast<const int2 *>(a.totals)[threadIdx.x];
    mine.x = across<kWave>(mine.x, SumInt());
    mine.y = across<kWave>(mine.y, SumInt());
    if (threadIdx.x % kWave == 0) totals[threadIdx.x / kWave] = mine;
    double s = 0.0;
    int c = 0;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const bool there = i * 16 + slice < a.groups;
        s += there ? double(sv[i]) : 0.0;
        c += there ? cv[i] : 0;
    }
    share[slice][col] = s;
    count[slice][col] = c;
    __syncthreads();
    if (threadIdx.x >= 16) return;
    s = 0.0;
    c = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        s += share[i][col];
        c += count[i][col];
    }
    int2 all = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        all.x += totals[i].x;
        all.y += totals[i].y;
    }
    const float slope = slope_of(a.coefficient, a.E, c, all.x, all.y);
    if (e < a.E) {
        a.counts[e] = c;
        a.slope[e] = slope;
    }
    double loss = e < a.E ? double(slope) * s : 0.0;
    for (int d = 1; d < 16; d *= 2) loss += __shfl_xor(loss, d);
    if (threadIdx.x != 0) return;
    __hip_atomic_store(a.part + blockIdx.x, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(a.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != gridDim.x - 1) return;
    loss = 0.0;
    for (unsigned i = 0; i < gridDim.x; ++i) loss += __hip_atomic_load(a.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.loss[0] = float(loss);
}

// No tokens.
__global__ __launch_bounds__(kMaxExperts) void k_balance_none(float *loss, float *slope, int32_t *counts, int E)
{
    if (threadIdx.x == 0) loss[0] = 0.f;
    if (int(threadIdx.x) < E) {
        slope[threadIdx.x] = 0.f;
        counts[threadIdx.x] = 0;
    }
}

// dlogits = grad * share * (slope - sum of share * slope), times 1 - sigmoid with sigmoids.  As
// k_balance; the slopes stay in registers over a workgroup's tokens (30 -> 22 us for 32768
// tokens of 512 experts, 134 MB; a copy's 26).
template <bool L32, int LANES, int V, bool VEC>
__global__ __launch_bounds__(256) void k_balance_grad(RouteArgs a)
{
    using R = Row<L32, LANES, V, VEC>;
    const int64_t last = a.rows - 1, step = int64_t(gridDim.x) * R::kRows;
    int64_t row = int64_t(blockIdx.x) * R::kRows + threadIdx.x / LANES;
    Token<R> next;
    next.load(a, min(row, last));
    const float g = a.g[0];
    float slope[V];
#pragma unroll
    for (int i = 0; i < V; ++i) slope[i] = R::expert(i) < a.E ? a.slope[R::expert(i)] : 0.f;
    for (int64_t at = int64_t(blockIdx.x) * R::kRows; at < a.rows; at += step, row += step) {
        const Token<R> t = next;
        if (at + step < a.rows) next.load(a, min(row + step, last));
        float p[V], left[V], d[V], dot = 0.f;
        int chosen = 0;
        const bool on = shares<R>(a, t, true, p, left, nullptr, chosen);
#pragma unroll
        for (int i = 0; i < V; ++i) dot = fmaf(p[i], slope[i], dot);
        dot = across<LANES>(dot, Sum());
#pragma unroll
        for (int i = 0; i < V; ++i) {
            d[i] = p[i] * (slope[i] - dot);
            if (a.sigmoid) d[i] *= left[i];
            d[i] = on ? g * d[i] : 0.f;
        }
        if (row <= last) R::store(a, row, d);
    }
}

// ---------------------------------------------------------------- launches ----

// Rows of one launch: up to 1024 threads each, and a launch has fewer than 2^32.
constexpr int kLaunchRows = 1 << 20;

template <bool X32, int RES, bool OUT8, int WPR, int C>
int norm_as(NormArgs a, hipStream_t st)
{
    constexpr int each = WPR >= 4 ? 1 : 4 / WPR;
    const int rows = a.rows;
    for (; a.first < rows; a.first += kLaunchRows) {
        a.rows = std::min(rows, a.first + kLaunchRows);
        hipLaunchKernelGGL((k_norm<X32, RES, OUT8, WPR, C>), dim3(unsigned((a.rows - a.first + each - 1) / each)),
                           dim3(WPR > 4 ? WPR * kWave : 256), 0, st, a);
        if (launched() != 0) return 1;
    }
    return 0;
}

// One run of eight columns a lane as far as it goes, which has the most loads on the way for
// few rows and costs many none (2048 columns, bf16, one wavefront with four runs and four with
// one: 256 rows 3.5 and 2.8 us, 4096 9.8 and 9.7; 4096 columns, four with two and eight with
// one: 64 rows 2.9 and 2.7, 4096 16.4 and 16.9; 8192, 16 with one: 3.5 and 3.2, 30.9 and 31.3).
template <bool X32, int RES, bool OUT8>
int norm_of(const NormArgs &a, hipStream_t st)
{
    if (a.H <= 512) return norm_as<X32, RES, OUT8, 1, 1>(a, st);
    if (a.H <= 1024) return norm_as<X32, RES, OUT8, 1, 2>(a, st);
    if (a.H <= 2048) return norm_as<X32, RES, OUT8, 4, 1>(a, st);
    if (a.H <= 4096) return norm_as<X32, RES, OUT8, 8, 1>(a, st);
    if (a.H <= 8192) return norm_as<X32, RES, OUT8, 16, 1>(a, st);
    static_assert(AFD_MAX_NORM_HIDDEN == 16 * kWave * 2 * 8, "the widest row");
    return norm_as<X32, RES, OUT8, 16, 2>(a, st);
}

template <bool X32, int RES>
int norm_out(const NormArgs &a, bool out8, hipStream_t st)
{
    return out8 ? norm_of<X32, RES, true>(a, st) : norm_of<X32, RES, false>(a, st);
}

template <bool H32, int WPR, int C>
int norm_grad_as(NormGradArgs a, int groups, hipStream_t st)
{
    constexpr int each = WPR >= 4 ? 1 : 4 / WPR;
    a.groups = a.part ? groups : std::min((a.rows + each - 1) / each, kNormGradGroups * 4 / each);
    const int columns = a.dw ? (a.H + 63) / 64 : 0;
    const dim3 threads(WPR > 4 ? WPR * kWave : 256);
    if (columns > 0 && a.dh == a.g) {   // dh in grad's place: dweight first
        NormGradArgs c = a;
        c.groups = 0;
        hipLaunchKernelGGL((k_norm_grad<H32, WPR, C>), dim3(unsigned(columns)), threads, 0, st, c);
        a.dw = nullptr;
        if (launched() != 0) return 1;
    }
    hipLaunchKernelGGL((k_norm_grad<H32, WPR, C>), dim3(unsigned(a.groups + (a.dw ? columns : 0))), threads, 0, st, a);
    return launched();
}

template <bool H32>
int norm_grad_of(const NormGradArgs &a, int groups, hipStream_t st)
{
    if (a.H <= 512) return norm_grad_as<H32, 1, 1>(a, groups, st);
    if (a.H <= 1024) return norm_grad_as<H32, 1, 2>(a, groups, st);
    // a wavefront with four runs, or four with one: bf16 64 rows 3.3 and 2.6 us, 1024 6.2 and 6.7,
    // 16384 37.0 and 39.8; float32 3.5 and 2.6, 10.3 and 11.8, 93.9 and 86.2.  By the rows and the type
    // alone, as the two add a row's products in another order: dh has the same bits without dweight.
    if (a.H <= 2048)
        return a.rows <= 512 || (H32 && groups > 0) ? norm_grad_as<H32, 4, 1>(a, groups, st) : norm_grad_as<H32, 1, 4>(a, groups, st);
    if (a.H <= 4096) return norm_grad_as<H32, 4, 2>(a, groups, st);
    if (a.H <= 8192) return norm_grad_as<H32, 4, 4>(a, groups, st);
    return norm_grad_as<H32, 16, 2>(a, groups, st);
}

RouteArgs route_args(const RoutePlan &p)
{
    RouteArgs a{};
    a.l = p.l;
    a.bias = p.bias;
    a.live = p.live;
    a.ids = p.ids;
    a.w = p.w;
    a.g = p.g;
    a.slope = p.slope;
    a.dl = p.dl;
    a.ls = p.ls;
    a.rows = int(p.rows);
    a.E = p.E;
    a.K = p.K;
    a.scale = p.scale;
    a.sigmoid = p.sigmoid;
    a.renorm = p.renorm;
    return a;
}

// The lanes of a token: 16 with four or eight logits each, then 32 and 64 with eight.
template <template <bool, int, int, bool> class Launch, bool L32, bool VEC, typename... Args>
int by_experts(int E, Args... args)
{
    if (E <= 64) return Launch<L32, 16, 4, VEC>::run(args...);
    if (E <= 128) return Launch<L32, 16, 8, VEC>::run(args...);
    if (E <= 256) return Launch<L32, 32, 8, VEC>::run(args...);
    return Launch<L32, 64, 8, VEC>::run(args...);
}

template <template <bool, int, int, bool> class Launch, typename... Args>
int by_logits(const RoutePlan &p, Args... args)
{
    // four logits at a time, where they and their gradients lie for it
    const uintptr_t each = p.l32 ? 16 : 8;
    const bool vec = p.E % 4 == 0 && p.ls % 4 == 0 && reinterpret_cast<uintptr_t>(p.l) % each == 0 &&
                     reinterpret_cast<uintptr_t>(p.dl) % each == 0;
    if (p.l32) return vec ? by_experts<Launch, true, true>(p.E, args...) : by_experts<Launch, true, false>(p.E, args...);
    return vec ? by_experts<Launch, false, true>(p.E, args...) : by_experts<Launch, false, false>(p.E, args...);
}

template <bool L32, int LANES, int V, bool VEC>
struct RouteLaunch {
    static int run(const RouteArgs &a, hipStream_t st)
    {
        // Few tokens of 65 to 128 experts: a shorter chain in twice the lanes (16 with eight logits
        // and 32 with four: 256 tokens 4.3 and 3.9 us, 4096 4.6 and 4.1, 65536 18.4 and 20.9; with
        // a bias 5.4 and 4.6, 8.2 and 7.0, 29.4 and 32.7).
        if constexpr (LANES == 16 && V == 8) {
            if (a.rows <= 8192) return as<32, 4>(a, st);
        }
        return as<LANES, V>(a, st);
    }

    template <int N, int EACH>
    static int as(const RouteArgs &a, hipStream_t st)
    {
        constexpr int rows = Row<L32, N, EACH, VEC>::kRows;
        const dim3 grid(unsigned((a.rows + rows - 1) / rows));
        if (a.bias) hipLaunchKernelGGL((k_route<L32, N, EACH, VEC, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_route<L32, N, EACH, VEC, false>), grid, dim3(256), 0, st, a);
        return launched();
    }
};

// Workgroups of the gradients: as many as are resident at once.
constexpr int kGradGroups = 256 * 8;

template <bool L32, int LANES, int V, bool VEC>
struct RouteGradLaunch {
    static int run(const RouteArgs &a, hipStream_t st)
    {
        constexpr int rows = Row<L32, LANES, V, VEC>::kRows;
        const dim3 grid(unsigned(std::min((a.rows + rows - 1) / rows, kGradGroups)));
        if (!a.sigmoid && !a.renorm) hipLaunchKernelGGL((k_route_grad<L32, LANES, V, VEC, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_route_grad<L32, LANES, V, VEC, false>), grid, dim3(256), 0, st, a);
        return launched();
    }
};

template <bool L32, int LANES, int V, bool VEC>
struct BalanceLaunch {
    static int run(const BalanceArgs &a, int groups, bool wide, hipStream_t st)
    {
        if (groups == 1) hipLaunchKernelGGL((k_balance<L32, LANES, V, VEC, 1024, true>), dim3(1), dim3(1024), 0, st, a);
        else if (wide) hipLaunchKernelGGL((k_balance<L32, LANES, V, VEC, 1024, false>), dim3(unsigned(groups)), dim3(1024), 0, st, a);
        else hipLaunchKernelGGL((k_balance<L32, LANES, V, VEC, 256, false>), dim3(unsigned(groups)), dim3(256), 0, st, a);
        return launched();
    }
};

template <bool L32, int LANES, int V, bool VEC>
struct BalanceGradLaunch {
    static int run(const RouteArgs &a, hipStream_t st)
    {
        constexpr int rows = Row<L32, LANES, V, VEC>::kRows;
        const dim3 grid(unsigned(std::min((a.rows + rows - 1) / rows, kGradGroups)));
        hipLaunchKernelGGL((k_balance_grad<L32, LANES, V, VEC>), grid, dim3(256), 0, st, a);
        return launched();
    }
};

}  // namespace

int be_launch_norm(const NormPlan &p, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    NormArgs a{p.x, p.r, p.w, p.out, p.h, p.outs, p.rstd, p.xs, p.rs, p.hs, 0, int(p.rows), p.H, p.eps, p.w32};
    if (!p.res) return p.x32 ? norm_out<true, 0>(a, p.out8, st) : norm_out<false, 0>(a, p.out8, st);
    if (!p.r32) return p.x32 ? norm_out<true, 1>(a, p.out8, st) : norm_out<false, 1>(a, p.out8, st);
    return p.x32 ? norm_out<true, 2>(a, p.out8, st) : norm_out<false, 2>(a, p.out8, st);
}

int be_launch_norm_grad(const NormGradPlan &p, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool join = p.dw && p.groups > 0;   // else the workgroups of the first launch have dweight as well
    if (p.rows > 0) {
        NormGradArgs a{p.g, p.gr, p.h, p.w, p.rstd, p.dh, join ? p.part : nullptr, join ? nullptr : p.dw, p.hs, int(p.rows), p.H, 0, p.w32};
        const int rc = p.h32 ? norm_grad_of<true>(a, p.groups, st) : norm_grad_of<false>(a, p.groups, st);
        if (rc != 0 || !join) return rc;
    }
    hipLaunchKernelGGL(k_norm_grad_join, dim3(unsigned((p.H + 63) / 64)), dim3(1024), 0, st, p.part, p.dw, p.H, p.groups);
    return launched();
}

int be_launch_route(const RoutePlan &p, void *stream)
{
    return by_logits<RouteLaunch>(p, route_args(p), static_cast<hipStream_t>(stream));
}

int be_launch_route_grad(const RoutePlan &p, void *stream)
{
    return by_logits<RouteGradLaunch>(p, route_args(p), static_cast<hipStream_t>(stream));
}

int be_launch_balance(const BalancePlan &p, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (p.groups == 0) {
        hipLaunchKernelGGL(k_balance_none, dim3(1), dim3(kMaxExperts), 0, st, p.loss, p.slope, p.counts, p.r.E);
        return launched();
    }
    BalanceArgs a{route_args(p.r), p.share, p.count, p.totals, p.done, p.loss, p.slope, p.counts, p.coefficient};
    const int rc = by_logits<BalanceLaunch>(p.r, a, p.groups, p.wide, st);
    if (rc != 0 || p.groups == 1) return rc;
    BalanceJoinArgs j{p.share, p.count, p.totals, p.part, p.done, p.loss, p.slope, p.counts, p.r.E, p.groups, p.coefficient};
    hipLaunchKernelGGL(k_balance_join, dim3(unsigned((p.r.E + 15) / 16)), dim3(256), 0, st, j);
    return launched();
}

int be_launch_balance_grad(const RoutePlan &p, void *stream)
{
    return by_logits<BalanceGradLaunch>(p, route_args(p), static_cast<hipStream_t>(stream));
}

}  // namespace afd
