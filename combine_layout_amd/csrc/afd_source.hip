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
struct Min {
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
    int rows, H;
    float eps;
    bool w32;
};

// A row is held by WPR wavefronts, C runs of eight columns a lane, from its load to its
// last store.  RES: 0 no residual, 1 bf16, 2 float32.
template <bool X32, int RES, bool OUT8, int WPR, int C>
__global__ __launch_bounds__(WPR > 4 ? WPR *kWave : 256) void k_norm(NormArgs a)
{
    constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = (wave % WPR) * kWave + lane, runs = a.H / 8;
    const int64_t row = int64_t(blockIdx.x) * kRows + wave / WPR;
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
    float *part;
    int64_t hs;
    int rows, H;
    bool w32;
};

// dh of every row, and the workgroup's sum of grad * u over its rows, which stays in
// registers from the first row to the last.
template <bool H32, int WPR, int C>
__global__ __launch_bounds__(WPR > 4 ? WPR *kWave : 256) void k_norm_grad(NormGradArgs a)
{
    constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = (wave % WPR) * kWave + lane, runs = a.H / 8;
    __shared__ float sum[2][WPR];
    float dw[C][8] = {};
    int turn = 0;
    for (int64_t row = int64_t(blockIdx.x) * kRows + wave / WPR; row < a.rows; row += int64_t(gridDim.x) * kRows) {
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
        float d[C][8], m = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            w[i].values(d[i], a.w32);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = h[i].get(j) * rstd;
                // columns behind the last hold whatever w holds: grad is 0 there
                d[i][j] = i * WPR * kWave + t < runs ? g[i].get(j) * d[i][j] : 0.f;
                m = fmaf(d[i][j], u, m);
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
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i][j] = fmaf(rstd, d[i][j] - h[i].get(j) * rstd * m, gr[i].get(j));
            if (c < runs) store_eight<H32>(a.dh, row * a.H + c * 8, d[i]);
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

// dweight: 64 columns a workgroup, 16 wavefronts that share the partial rows.
__global__ __launch_bounds__(1024) void k_norm_grad_join(const float *part, float *dw, int H, int groups)
{
    __shared__ float join[16][kWave];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * kWave + lane;
    float s = 0.f;
    if (c < H)
        for (int g = wave; g < groups; g += 16) s += part[int64_t(g) * H + c];
    join[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < H) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += join[i][lane];
        dw[c] = s;
    }
}

// ------------------------------------------------------------------ routes ----

constexpr float kMinusInf = -__builtin_inff();

// exp(x) for x <= 0, to about one float32 step; the argument's product with log2(e) is
// kept in two parts, since its rounding alone would cost |x| steps.  Below -120, and for
// a NaN, it is 0.
__device__ __forceinline__ float exp_neg(float x)
{
    x = fmaxf(x, -120.f);
    const float hi = x * 1.44269504f, lo = fmaf(x, 1.44269504f, -hi) + x * 1.92596300e-8f;
    return __builtin_amdgcn_exp2f(hi) * fmaf(lo, 0.693147181f, 1.0f);
}

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
    bool sigmoid, renorm, vec;
};

// A token's logits over LANES lanes, V a lane in runs of four: value i of a lane is of
// expert (i / 4) * 4 * LANES + 4 * lane + i % 4.  Experts behind the last, and NaNs, are
// minus infinity.
template <bool L32, int LANES, int V>
struct Row {
    static constexpr int kRows = 256 / LANES;   // tokens of a workgroup
    static constexpr int kSlots = (kMaxTopk + LANES - 1) / LANES;

    __device__ static __forceinline__ int lane() { return threadIdx.x & (LANES - 1); }
    __device__ static __forceinline__ int expert(int i) { return (i / 4) * 4 * LANES + 4 * lane() + i % 4; }

    __device__ static __forceinline__ float one(const RouteArgs &a, int64_t at)
    {
        if (L32) return static_cast<const float *>(a.l)[at];
        return from_bf16(static_cast<const uint16_t *>(a.l)[at]);
    }

    __device__ static __forceinline__ void load(const RouteArgs &a, int64_t row, float *v)
    {
        const int64_t base = row * a.ls;
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const int e = expert(q * 4);
            f32x4 x = {kMinusInf, kMinusInf, kMinusInf, kMinusInf};
            if (a.vec) {
                if (e < a.E) {
                    if (L32) {
                        x = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.l) + base + e);
                    } else {
                        const u32x2 u = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(a.l) + base + e);
                        x = f32x4{from_bf16(u[0] & 0xFFFFu), from_bf16(u[0] >> 16), from_bf16(u[1] & 0xFFFFu), from_bf16(u[1] >> 16)};
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j < a.E) x[j] = one(a, base + e + j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) v[q * 4 + j] = x[j] == x[j] ? x[j] : kMinusInf;
        }
    }

    __device__ static __forceinline__ void store(const RouteArgs &a, int64_t row, const float *d)
    {
        const int64_t base = row * a.E;
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const int e = expert(q * 4);
            const float *x = d + q * 4;
            if (a.vec) {
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
        return across<LANES>(m, Max());
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
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = v[i] == kMinusInf ? 0.f : v[i] == m ? 1.f : exp_neg(v[i] - m);
        return total(t);
    }

    // Sigmoids in the same proportions but for a common factor, and their sum: where every
    // logit is far below zero the largest is lifted to about 1, so that none vanishes.
    // left: 1 - sigmoid.
    __device__ static __forceinline__ float sigmoids(const float *v, float m, float *t, float *left)
    {
        const float lift = fminf(m, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = exp_neg(-fabsf(v[i])), d = 1.0f / (1.0f + z);
            t[i] = v[i] == kMinusInf ? 0.f : (v[i] >= 0.f ? 1.f : lift < -40.f ? exp_neg(v[i] - lift) : z) * d;
            left[i] = (v[i] >= 0.f ? z : 1.f) * d;
        }
        return total(t);
    }
};

__device__ __forceinline__ double across_max(double v, int lanes)
{
    for (int d = 1; d < lanes; d *= 2) v = fmax(v, __shfl_xor(v, d));
    return v;
}

// The weights of a token's chosen logits, one a lane and slot (NaN: none), and their
// relation to the scores: w = scale * weight.
template <int LANES, int SLOTS>
__device__ __forceinline__ void weights_of(const RouteArgs &a, const float *l, const bool *on, float m, float sum, float *w)
{
    if (!a.sigmoid && !a.renorm) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            w[s] = !on[s] || l[s] == kMinusInf ? 0.f : (l[s] == m ? 1.f : exp_neg(l[s] - m)) / sum;
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
            w[s] = l[s] == top ? 1.f : exp_neg(l[s] - top);
        } else {
            const float z = exp_neg(-fabsf(l[s])), lift = fminf(top, 0.f);
            w[s] = (l[s] >= 0.f ? 1.f : a.renorm ? exp_neg(l[s] - lift) : z) / (1.0f + z);
        }
        if (!on[s] || l[s] == kMinusInf) w[s] = 0.f;
        t += w[s];
    }
    if (!a.renorm) return;
    t = across<LANES>(t, Sum());
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) w[s] = t > 0.f ? w[s] / t : 0.f;
}

// One token per LANES lanes: its logits in registers, the largest key taken K times.
template <bool L32, int LANES, int V>
__global__ __launch_bounds__(256) void k_route(RouteArgs a)
{
    using R = Row<L32, LANES, V>;
    const int lane = R::lane();
    const int64_t row_ = int64_t(blockIdx.x) * R::kRows + threadIdx.x / LANES, row = min(row_, int64_t(a.rows - 1));
    float v[V];
    R::load(a, row, v);
    const bool live = !a.live || a.live[row] != 0;
    const float m = R::largest(v);
    float sum = 1.f, l[R::kSlots];
    int id[R::kSlots];
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) {
        id[s] = -1;
        l[s] = kMinusInf;
    }
    if (!a.bias) {
        if (!a.sigmoid && !a.renorm) {
            float t[V];
            sum = R::terms(v, m, t);
        }
        for (int k = 0; k < a.K; ++k) {
            const float top = R::largest(v);
            int e = INT32_MAX;
#pragma unroll
            for (int i = V - 1; i >= 0; --i) e = v[i] == top ? R::expert(i) : e;
            e = across<LANES>(e, Min());
#pragma unroll
            for (int s = 0; s < R::kSlots; ++s) {
                if (k == s * LANES + lane && top != kMinusInf) {
                    id[s] = e;
                    l[s] = top;
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = R::expert(i) == e ? kMinusInf : v[i];
        }
    } else {
        double key[V], t = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const double x = double(v[i]);
            if (a.sigmoid) key[i] = 1.0 / (1.0 + exp(-x));
            else key[i] = v[i] == kMinusInf ? 0.0 : v[i] == m ? 1.0 : exp(x - double(m));
            t += key[i];
        }
        for (int d = 1; d < LANES; d *= 2) t += __shfl_xor(t, d);
        sum = float(t);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = R::expert(i);
            const double b = e < a.E ? double(a.bias[e]) : 0.0, s = a.sigmoid ? key[i] : key[i] / t;
            const double x = s + b;
            key[i] = v[i] == kMinusInf || !(x == x) ? -__builtin_inf() : x;
        }
        for (int k = 0; k < a.K; ++k) {
            double top = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) top = fmax(top, key[i]);
            top = across_max(top, LANES);
            int e = INT32_MAX;
#pragma unroll
            for (int i = V - 1; i >= 0; --i) e = key[i] == top ? R::expert(i) : e;
            e = across<LANES>(e, Min());
#pragma unroll
            for (int s = 0; s < R::kSlots; ++s)
                if (k == s * LANES + lane && top != -__builtin_inf()) id[s] = e;
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = R::expert(i) == e ? -__builtin_inf() : key[i];
        }
#pragma unroll
        for (int s = 0; s < R::kSlots; ++s)
            if (id[s] >= 0) l[s] = R::one(a, row * a.ls + id[s]);
    }
    bool on[R::kSlots];
    float w[R::kSlots];
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) on[s] = id[s] >= 0;
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

template <bool L32, int LANES, int V>
__global__ __launch_bounds__(256) void k_route_grad(RouteArgs a)
{
    using R = Row<L32, LANES, V>;
    const int lane = R::lane();
    const int64_t row_ = int64_t(blockIdx.x) * R::kRows + threadIdx.x / LANES, row = min(row_, int64_t(a.rows - 1));
    const bool dense = !a.sigmoid && !a.renorm;   // every logit of the softmax's sum has a gradient
    float m = 0.f, sum = 1.f, p[V];
    if (dense) {
        float v[V];
        R::load(a, row, v);
        m = R::largest(v);
        sum = R::terms(v, m, p);
    }
    float l[R::kSlots], g[R::kSlots], w[R::kSlots], dot = 0.f;
    int id[R::kSlots];
    bool on[R::kSlots];
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) {
        const int k = s * LANES + lane;
        id[s] = k < a.K ? a.ids[row * a.K + k] : -1;
        on[s] = id[s] >= 0 && id[s] < a.E;
        g[s] = on[s] ? a.g[row * a.K + k] * a.scale : 0.f;
        const float x = on[s] ? R::one(a, row * a.ls + id[s]) : kMinusInf;
        l[s] = x == x ? x : kMinusInf;
    }
    weights_of<LANES, R::kSlots>(a, l, on, m, sum, w);
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) dot += w[s] > 0.f ? g[s] * w[s] : 0.f;
    dot = across<LANES>(dot, Sum());
    float c[R::kSlots];   // what a slot adds to its expert's gradient
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) {
        const float z = exp_neg(-fabsf(l[s])), left = (l[s] >= 0.f ? z : 1.f) / (1.0f + z);
        c[s] = w[s] * (a.renorm ? g[s] - dot : g[s]) * (a.sigmoid ? left : 1.f);
        if (!(w[s] > 0.f)) c[s] = 0.f;
    }
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = dense ? -(p[i] / sum) * dot : 0.f;
    if (dense && !(sum > 0.f)) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = 0.f;
    }
    for (int k = 0; k < a.K; ++k) {
        int e = -1;
        float x = 0.f;
#pragma unroll
        for (int s = 0; s < R::kSlots; ++s) {
            if (k / LANES != s) continue;
            e = __shfl(on[s] ? id[s] : -1, k % LANES, LANES);
            x = __shfl(c[s], k % LANES, LANES);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] += R::expert(i) == e ? x : 0.f;
    }
    if (row_ < a.rows) R::store(a, row, d);
}

// ------------------------------------------------------------ balance loss ----

// A token's shares, whether it counts, and with LEFT the factor 1 - sigmoid.
template <typename R, int LANES, int V>
__device__ __forceinline__ bool shares(const RouteArgs &a, int64_t row, bool in, float *p, float *left, int32_t *hist)
{
    float v[V];
    R::load(a, row, v);
    int none = 1;
#pragma unroll
    for (int s = 0; s < R::kSlots; ++s) {
        const int k = s * LANES + R::lane();
        const int id = k < a.K ? a.ids[row * a.K + k] : -1;
        if (in && id >= 0 && id < a.E) {
            none = 0;
            if (hist) atomicAdd(hist + id, 1);
        }
    }
    const bool on = across<LANES>(none, Min()) == 0;
    const float m = R::largest(v), sum = a.sigmoid ? R::sigmoids(v, m, p, left) : R::terms(v, m, p);
    const float inv = on && sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= inv;
    return on;
}

struct BalanceArgs {
    RouteArgs r;
    float *share;
    int32_t *count, *tokens;
};

template <bool L32, int LANES, int V>
__global__ __launch_bounds__(256) void k_balance(BalanceArgs b)
{
    using R = Row<L32, LANES, V>;
    const RouteArgs &a = b.r;
    __shared__ int32_t hist[LANES * V], live;
    __shared__ float join[R::kRows][LANES * V];
    for (int e = threadIdx.x; e < LANES * V; e += 256) hist[e] = 0;
    if (threadIdx.x == 0) live = 0;
    __syncthreads();
    float acc[V] = {};
    int mine = 0;
    for (int64_t at = int64_t(blockIdx.x) * R::kRows; at < a.rows; at += int64_t(gridDim.x) * R::kRows) {
        const int64_t row = at + threadIdx.x / LANES;
        float p[V], left[V];
        mine += shares<R, LANES, V>(a, min(row, int64_t(a.rows - 1)), row < a.rows, p, left, hist);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += p[i];
    }
    if (R::lane() == 0) atomicAdd(&live, mine);
#pragma unroll
    for (int i = 0; i < V; ++i) join[threadIdx.x / LANES][R::expert(i)] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < R::kRows; ++i) s += join[i][e];
        b.share[int64_t(blockIdx.x) * a.E + e] = s;
        b.count[int64_t(blockIdx.x) * a.E + e] = hist[e];
    }
    if (threadIdx.x == 0) b.tokens[blockIdx.x] = live;
}

struct BalanceJoinArgs {
    const float *share;
    const int32_t *count, *tokens;
    float *loss, *slope;
    int32_t *counts;
    int E, groups;
    float coefficient;
};

// One workgroup: every expert's sums, then the loss.
__global__ __launch_bounds__(1024) void k_balance_join(BalanceJoinArgs a)
{
    __shared__ double part[16];
    __shared__ int all[2];
    if (threadIdx.x < 2) all[threadIdx.x] = 0;
    __syncthreads();
    double share = 0.0;
    int count = 0, tokens = 0;
    const int e = threadIdx.x;
    if (e < a.E) {
        for (int g = 0; g < a.groups; ++g) {
            share += double(a.share[int64_t(g) * a.E + e]);
            count += a.count[int64_t(g) * a.E + e];
        }
        a.counts[e] = count;
        atomicAdd(&all[0], count);
    }
    for (int g = threadIdx.x; g < a.groups; g += 1024) tokens += a.tokens[g];
    atomicAdd(&all[1], tokens);
    __syncthreads();
    const double n = double(all[0]) * double(all[1]);
    float slope = 0.f;
    if (e < a.E) {
        slope = n > 0.0 ? float(double(a.coefficient) * double(a.E) * double(count) / n) : 0.f;
        a.slope[e] = slope;
    }
    double loss = double(slope) * share;
    for (int d = 1; d < kWave; d *= 2) loss += __shfl_xor(loss, d);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        loss = 0.0;
        for (int i = 0; i < 16; ++i) loss += part[i];
        a.loss[0] = float(loss);
    }
}

template <bool L32, int LANES, int V>
__global__ __launch_bounds__(256) void k_balance_grad(RouteArgs a)
{
    using R = Row<L32, LANES, V>;
    const int64_t row_ = int64_t(blockIdx.x) * R::kRows + threadIdx.x / LANES, row = min(row_, int64_t(a.rows - 1));
    float p[V], left[V], d[V], dot = 0.f;
    const float g = a.g[0];
    const bool on = shares<R, LANES, V>(a, row, true, p, left, nullptr);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = R::expert(i);
        d[i] = e < a.E ? a.slope[e] : 0.f;
        dot = fmaf(p[i], d[i], dot);
    }
    dot = across<LANES>(dot, Sum());
#pragma unroll
    for (int i = 0; i < V; ++i) {
        d[i] = p[i] * (d[i] - dot);
        if (a.sigmoid) d[i] *= left[i];
        d[i] = on ? g * d[i] : 0.f;
    }
    if (row_ < a.rows) R::store(a, row, d);
}

// ---------------------------------------------------------------- launches ----

template <bool X32, int RES, bool OUT8, int WPR, int C>
int norm_as(const NormArgs &a, hipStream_t st)
{
    constexpr int rows = WPR >= 4 ? 1 : 4 / WPR;
    hipLaunchKernelGGL((k_norm<X32, RES, OUT8, WPR, C>), dim3(unsigned((a.rows + rows - 1) / rows)), dim3(WPR > 4 ? WPR * kWave : 256),
                       0, st, a);
    return launched();
}

template <bool X32, int RES, bool OUT8>
int norm_of(const NormArgs &a, hipStream_t st)
{
    if (a.H <= 512) return norm_as<X32, RES, OUT8, 1, 1>(a, st);
    if (a.H <= 1024) return norm_as<X32, RES, OUT8, 1, 2>(a, st);
    if (a.H <= 2048) return norm_as<X32, RES, OUT8, 1, 4>(a, st);
    if (a.H <= 4096) return norm_as<X32, RES, OUT8, 4, 2>(a, st);
    if (a.H <= 8192) return norm_as<X32, RES, OUT8, 4, 4>(a, st);
    if (a.H <= 16384) return norm_as<X32, RES, OUT8, 16, 2>(a, st);
    if (a.H <= 32768) return norm_as<X32, RES, OUT8, 16, 4>(a, st);
    return norm_as<X32, RES, OUT8, 16, 8>(a, st);
}

template <bool X32, int RES>
int norm_out(const NormArgs &a, bool out8, hipStream_t st)
{
    return out8 ? norm_of<X32, RES, true>(a, st) : norm_of<X32, RES, false>(a, st);
}

template <bool H32, int WPR, int C>
int norm_grad_as(const NormGradArgs &a, int groups, hipStream_t st)
{
    hipLaunchKernelGGL((k_norm_grad<H32, WPR, C>), dim3(unsigned(groups)), dim3(WPR > 4 ? WPR * kWave : 256), 0, st, a);
    return launched();
}

template <bool H32>
int norm_grad_of(const NormGradArgs &a, int groups, hipStream_t st)
{
    if (a.H <= 512) return norm_grad_as<H32, 1, 1>(a, groups, st);
    if (a.H <= 1024) return norm_grad_as<H32, 1, 2>(a, groups, st);
    if (a.H <= 2048) return norm_grad_as<H32, 1, 4>(a, groups, st);
    if (a.H <= 4096) return norm_grad_as<H32, 4, 2>(a, groups, st);
    if (a.H <= 8192) return norm_grad_as<H32, 4, 4>(a, groups, st);
    if (a.H <= 16384) return norm_grad_as<H32, 16, 2>(a, groups, st);
    if (a.H <= 32768) return norm_grad_as<H32, 16, 4>(a, groups, st);
    return norm_grad_as<H32, 16, 8>(a, groups, st);
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
    const uintptr_t each = p.l32 ? 16 : 8;   // four logits at a time
    a.vec = p.E % 4 == 0 && p.ls % 4 == 0 && reinterpret_cast<uintptr_t>(p.l) % each == 0 &&
            reinterpret_cast<uintptr_t>(p.dl) % each == 0;
    return a;
}

// The lanes of a token: 16 with four or eight logits each, then 32 and 64 with eight.
template <template <bool, int, int> class Launch, typename... Args>
int by_experts(int E, bool l32, Args... args)
{
    if (E <= 64) return l32 ? Launch<true, 16, 4>::run(args...) : Launch<false, 16, 4>::run(args...);
    if (E <= 128) return l32 ? Launch<true, 16, 8>::run(args...) : Launch<false, 16, 8>::run(args...);
    if (E <= 256) return l32 ? Launch<true, 32, 8>::run(args...) : Launch<false, 32, 8>::run(args...);
    return l32 ? Launch<true, 64, 8>::run(args...) : Launch<false, 64, 8>::run(args...);
}

template <bool L32, int LANES, int V>
struct RouteLaunch {
    static int run(const RouteArgs &a, hipStream_t st)
    {
        constexpr int rows = Row<L32, LANES, V>::kRows;
        hipLaunchKernelGGL((k_route<L32, LANES, V>), dim3(unsigned((a.rows + rows - 1) / rows)), dim3(256), 0, st, a);
        return launched();
    }
};

template <bool L32, int LANES, int V>
struct RouteGradLaunch {
    static int run(const RouteArgs &a, hipStream_t st)
    {
        constexpr int rows = Row<L32, LANES, V>::kRows;
        hipLaunchKernelGGL((k_route_grad<L32, LANES, V>), dim3(unsigned((a.rows + rows - 1) / rows)), dim3(256), 0, st, a);
        return launched();
    }
};

template <bool L32, int LANES, int V>
struct BalanceLaunch {
    static int run(const BalanceArgs &a, int groups, hipStream_t st)
    {
        hipLaunchKernelGGL((k_balance<L32, LANES, V>), dim3(unsigned(groups)), dim3(256), 0, st, a);
        return launched();
    }
};

template <bool L32, int LANES, int V>
struct BalanceGradLaunch {
    static int run(const RouteArgs &a, hipStream_t st)
    {
        constexpr int rows = Row<L32, LANES, V>::kRows;
        hipLaunchKernelGGL((k_balance_grad<L32, LANES, V>), dim3(unsigned((a.rows + rows - 1) / rows)), dim3(256), 0, st, a);
        return launched();
    }
};

}  // namespace

int be_launch_norm(const NormPlan &p, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    NormArgs a{p.x, p.r, p.w, p.out, p.h, p.outs, p.rstd, p.xs, p.rs, p.hs, int(p.rows), p.H, p.eps, p.w32};
    if (!p.res) return p.x32 ? norm_out<true, 0>(a, p.out8, st) : norm_out<false, 0>(a, p.out8, st);
    if (!p.r32) return p.x32 ? norm_out<true, 1>(a, p.out8, st) : norm_out<false, 1>(a, p.out8, st);
    return p.x32 ? norm_out<true, 2>(a, p.out8, st) : norm_out<false, 2>(a, p.out8, st);
}

int be_launch_norm_grad(const NormGradPlan &p, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (p.groups > 0) {
        NormGradArgs a{p.g, p.gr, p.h, p.w, p.rstd, p.dh, p.dw ? p.part : nullptr, p.hs, int(p.rows), p.H, p.w32};
        const int rc = p.h32 ? norm_grad_of<true>(a, p.groups, st) : norm_grad_of<false>(a, p.groups, st);
        if (rc != 0) return rc;
    }
    if (!p.dw) return 0;
    hipLaunchKernelGGL(k_norm_grad_join, dim3(unsigned((p.H + kWave - 1) / kWave)), dim3(1024), 0, st, p.part, p.dw, p.H, p.groups);
    return launched();
}

int be_launch_route(const RoutePlan &p, void *stream)
{
    return by_experts<RouteLaunch>(p.E, p.l32, route_args(p), static_cast<hipStream_t>(stream));
}

int be_launch_route_grad(const RoutePlan &p, void *stream)
{
    return by_experts<RouteGradLaunch>(p.E, p.l32, route_args(p), static_cast<hipStream_t>(stream));
}

int be_launch_balance(const BalancePlan &p, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (p.groups > 0) {
        BalanceArgs a{route_args(p.r), p.share, p.count, p.tokens};
        const int rc = by_experts<BalanceLaunch>(p.r.E, p.r.l32, a, p.groups, st);
        if (rc != 0) return rc;
    }
    BalanceJoinArgs j{p.share, p.count, p.tokens, p.loss, p.slope, p.counts, p.r.E, p.groups, p.coefficient};
    hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(1024), 0, st, j);
    return launched();
}

int be_launch_balance_grad(const RoutePlan &p, void *stream)
{
    return by_experts<BalanceGradLaunch>(p.E, p.l32, route_args(p), static_cast<hipStream_t>(stream));
}

}  // namespace afd
