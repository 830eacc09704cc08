// afd_experts.hip -- gfx950 kernels of the experts' side of a round: products
// grouped by expert, their low-rank adapters, and the row tags; and the HIP
// executor behind their be_* hooks.
//
// Mathematics.  Expert j owns rows [align_up(ends[j-1], alpha), ends[j]).
//   product   out[r, n] = act( sum_k x[r, k] W[j, n, k] )
//   FP8       x = q * xs[r, k/128] and W = p * ws[j, n/128, k/128]: the codes of
//             one 128-column block are multiplied and summed by the matrix unit,
//             and each block's sum enters the float32 sum times xs * ws
//   adapters  t[r, :] = scaling[a] * A[a, j] x[r] (k_shrink, summed in float32), then
//             B[a, j] t[r] is added to row r's sums before the activation
//
// Orientation.  The matrix unit's A operand holds weight rows and its B operand
// rows of x, so that D's column, and with it everything a lane holds of a
// result, belongs to ONE row of x: a lane needs one row scale, one adapter and
// one bounds check, and rows cannot reach each other's results, whatever their
// values.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "afd_plan.h"

namespace afd {
namespace {

constexpr int kWave = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <typename T>
using gptr = __attribute__((address_space(1))) T *;
template <typename T>
using lptr = __attribute__((address_space(3))) T *;

// One lane's operand of a 128-byte step of k: two 16-byte pieces (two bf16
// products of 32 columns, or one E4M3 product of 128).  Both operands hold the
// same columns in the same places, so the order of the columns inside a step
// is free; lane group g (16 lanes) takes pieces g and 4 + g of the step's eight.
struct Frag {
    u32x4 p[2];
};

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// E4M3 x E4M3 over 128 columns; the block exponents are 127 (times one).  The unit sums
// eight consecutive columns on one grid, 13 bits below their largest exponent, and the
// eights in float32 (found with products that cancel but for one; 16x16x32 does the
// same): 1.5e-5 of the sums' size for normally distributed values, where float32 has
// 6e-8.  It is the unit's own and the price of its rate: BF16 products of the converted
// codes, whose sums are float32, run at half of it and convert every code first.
__device__ __forceinline__ f32x4 mfma_fp8(const Frag &a, const Frag &b, f32x4 c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, a), __builtin_bit_cast(i32x8, b), c,
                                                            0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
}

// float32 to bf16, nearest even, in the low half (NaN stays NaN).
__device__ __forceinline__ uint32_t to_bf16(float v)
{
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) { return to_bf16(lo) | (to_bf16(hi) << 16); }

// g / (1 + exp(-g)); the reciprocal is the hardware's, off by one float32 step.
__device__ __forceinline__ float silu(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// Scale of a block of E4M3 codes with the largest value m, and the factor to the
// codes.  A scale below float32's smallest normal number counts as zero: its
// reciprocal would be infinite.
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

// Four values times inv as E4M3 codes, nearest even.
__device__ __forceinline__ uint32_t codes_of(const f32x4 &v, float inv)
{
    const int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, c, true));
}

// ------------------------------------------------------------- row tiles ----

// The experts' rows as tiles, built by every workgroup in LDS from ends[]
// (512 experts at most: a few hundred bytes read, one wavefront's prefix sum).
// An expert's rows are split into as few tiles of at most MAX rows as hold
// them, of even heights in steps of STEP: 260 rows are two tiles of 160 and
// 100 rows, not of 256 and 4.
struct Tiles {
    int first[kMaxExperts + 1];   // tiles before expert e
    int start[kMaxExperts];       // first row
    int count[kMaxExperts];       // rows
};

struct Tile {
    int e, row0, nrows;
};

template <int MAX, int STEP>
__device__ __forceinline__ int tile_height(int count)
{
    const int n = (count + MAX - 1) / MAX;
    return n <= 1 ? MAX : ((count + n - 1) / n + STEP - 1) / STEP * STEP;
}

// The experts' rows, by wavefront 0; returns the rows and the experts that have
// any, in every lane.
__device__ int2 read_spans(Tiles &s, const int32_t *ends, int E, int alpha, int rows)
{
    const int lane = threadIdx.x, per = (E + kWave - 1) / kWave, lo = lane * per;
    int2 n = {0, 0};
    for (int i = 0; i < per; ++i) {
        const int e = lo + i;
        if (e >= E) break;
        const uint32_t prev = e == 0 ? 0u : uint32_t(min(max(ends[e - 1], 0), rows));
        const uint32_t st = (prev + uint32_t(alpha) - 1u) / uint32_t(alpha) * uint32_t(alpha);
        const int end = min(ends[e], rows);
        const int start = int(min(st, uint32_t(rows)));
        const int count = max(end - start, 0);
        s.start[e] = start;
        s.count[e] = count;
        n.x += count;
        n.y += count > 0;
    }
    for (int d = 1; d < kWave; d *= 2) {
        n.x += __shfl_xor(n.x, d);
        n.y += __shfl_xor(n.y, d);
    }
    return n;
}

// The tiles of the spans, by wavefront 0; the caller places a barrier behind it.
template <int MAX>
__device__ void build_tiles(Tiles &s, int E)
{
    const int lane = threadIdx.x, per = (E + kWave - 1) / kWave, lo = lane * per;
    int mine = 0;
    for (int i = 0; i < per && lo + i < E; ++i) mine += (s.count[lo + i] + MAX - 1) / MAX;
    int sum = mine;
    for (int d = 1; d < kWave; d *= 2) {
        const int o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
    }
    int run = sum - mine;
    for (int i = 0; i < per && lo + i < E; ++i) {
        s.first[lo + i] = run;
        run += (s.count[lo + i] + MAX - 1) / MAX;
    }
    if (lane == kWave - 1) s.first[E] = sum;
}

// Item `at` of the tiles times `nt` column tiles: an expert's items are together,
// and of these the row tiles of one column tile, so that the workgroups that read
// the same weights run at the same time.  The expert is the last one whose first
// item is at or before `at`, found by counting over the lanes of a wavefront.
template <int MAX, int STEP>
__device__ __forceinline__ Tile find_tile(const Tiles &s, int E, int nt, int at, int &column)
{
    const int lane = threadIdx.x & 63, t = at / nt;
    int e = -1;
    for (int i = 0; i < E; i += kWave) e += __popcll(__ballot(i + lane < E && s.first[min(i + lane, E)] <= t));
    const int first = s.first[e], row_tiles = s.first[e + 1] - first, in = at - first * nt, col = in / row_tiles;
    const int count = s.count[e], h = tile_height<MAX, STEP>(count), done = (in - col * row_tiles) * h;
    Tile r;
    r.e = __builtin_amdgcn_readfirstlane(e);
    r.row0 = __builtin_amdgcn_readfirstlane(s.start[e] + done);
    r.nrows = __builtin_amdgcn_readfirstlane(min(h, count - done));
    column = __builtin_amdgcn_readfirstlane(col);
    return r;
}

// Persistent workgroups: workgroup b runs on XCD b % 8, and each XCD takes a
// contiguous eighth of the items, so that the column tiles of one row tile
// find its rows (and the row tiles of one expert its weights) in one L2.
struct Items {
    int at, end, step;
};
__device__ __forceinline__ Items my_items(int total_)
{
    const int total = __builtin_amdgcn_readfirstlane(total_);   // read from LDS: the same in every lane
    const int nb = gridDim.x, b = blockIdx.x;   // nb is a multiple of 8
    const int per = (total + 7) / 8, x = b & 7;
    Items it;
    it.at = x * per + (b >> 3);
    it.end = min((x + 1) * per, total);
    it.step = nb >> 3;
    return it;
}

// --------------------------------------------------------------- product ----

struct ProductArgs {
    const uint8_t *x;
    const uint8_t *w;
    const float *xs, *ws;
    const int32_t *ends, *tags;
    const uint16_t *t;   // [rows][2][c * rank]: the two bf16 parts of every row's t
    const uint8_t *b;
    void *out;
    float *outs;
    int rows, E, alpha;
    int n;         // columns of out
    int m;         // weight rows of an expert: n, or 2n gated
    int kb;        // bytes of a row of x and of W
    int packed;    // W's layout
    int wstep;     // bytes from a step of 128 bytes of a weight row to the next: 128, or 2048 packed
    int nad, rank;
    int ntiles;    // column tiles
};

// t enters the matrix unit as two bf16 parts, t - hi - lo below 2^-16 of t: hi in the
// low half, lo in the high half.
__device__ __forceinline__ uint32_t split_t(float t)
{
    const uint32_t hi = to_bf16(t);
    const float rest = t - __uint_as_float(hi << 16);
    return hi | (fabsf(rest) < INFINITY ? to_bf16(rest) << 16 : 0u);   // an infinite t has no rest
}

// Adds B t of the adapters of MB row blocks to v (33 and 29 us on top of the 102 and
// 64 us FP8 products of 256 rows per expert with about five adapters of rank 32 in
// 64 rows: a chain of one load of t and one of B per adapter): per block, NQ column
// blocks per kind of 4 consecutive columns of one row per lane.  wrow[] are the weight
// rows of this lane's A-operand rows.  Per 32 ranks, every row's t is loaded once
// (each row has one adapter), in its two bf16 parts (split_t); the distinct adapters
// number sub, sub + nsub, .. are taken one after the other, the next one's B on its
// way meanwhile, and each lane adds only its own row's, by selection, so an adapter's
// infinities reach no other request.
template <int KINDS, int NQ, int MB>
__device__ __forceinline__ void add_adapters(const ProductArgs &a, int e, const int (&row)[MB], const int (&tag)[MB],
                                             const int (&wrow)[KINDS * NQ], f32x4 (&v)[MB][KINDS * NQ], int sub, int nsub)
{
    const int lane = threadIdx.x & 63, g = lane >> 4;
    for (int j0 = 0; j0 < a.rank; j0 += 32) {
        const int j = j0 + g * 8;
        u32x4 hi[MB][KINDS], lo[MB][KINDS];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int c = 0; c < KINDS; ++c) {
                const bool have = tag[i] >= 0 && j < a.rank;
                const gptr<const uint16_t> t = (gptr<const uint16_t>)a.t + int64_t(row[i]) * (2 * KINDS * a.rank) + c * a.rank + j;
                hi[i][c] = have ? *(gptr<const u32x4>)t : u32x4{0u, 0u, 0u, 0u};
                lo[i][c] = have ? *(gptr<const u32x4>)(t + KINDS * a.rank) : u32x4{0u, 0u, 0u, 0u};
            }
        uint32_t left[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) left[i] = uint32_t(__ballot(tag[i] >= 0)) & 0xFFFFu;
        struct Pick {
            int ad;              // -1: none
            uint32_t hit[MB];    // its rows
        };
        int skip = sub;
        auto pick = [&]() {
            Pick p;
            for (;;) {
                p.ad = -1;
#pragma unroll
                for (int i = MB - 1; i >= 0; --i)
                    if (left[i]) p.ad = __builtin_amdgcn_readlane(tag[i], __builtin_ctz(left[i]));
                if (p.ad < 0) break;
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    p.hit[i] = uint32_t(__ballot(tag[i] == p.ad)) & 0xFFFFu;
                    left[i] &= ~p.hit[i];
                }
                if (skip == 0) {
                    skip = nsub - 1;
                    break;
                }
                --skip;
            }
            return p;
        };
        auto load_b = [&](u32x4 (&bf)[KINDS * NQ], int ad) {
            const gptr<const uint8_t> base = (gptr<const uint8_t>)a.b + (int64_t(ad) * a.E + e) * (int64_t(a.m) * a.rank * 2);
#pragma unroll
            for (int q = 0; q < KINDS * NQ; ++q)
                bf[q] = j < a.rank ? *(gptr<const u32x4>)(base + (int64_t(wrow[q]) * a.rank + j) * 2) : u32x4{0u, 0u, 0u, 0u};
        };
        Pick p = pick();
        u32x4 bf[KINDS * NQ];
        if (p.ad >= 0) load_b(bf, p.ad);
        while (p.ad >= 0) {
            const Pick next = pick();
            u32x4 bn[KINDS * NQ];
            if (next.ad >= 0) load_b(bn, next.ad);
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                if (!p.hit[i]) continue;
                const bool mine = tag[i] == p.ad;
#pragma unroll
                for (int q = 0; q < KINDS * NQ; ++q) {
                    const f32x4 d = mfma_bf16(bf[q], hi[i][q / NQ], mfma_bf16(bf[q], lo[i][q / NQ], f32x4{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i][q][k] = mine ? v[i][q][k] + d[k] : v[i][q][k];
                }
            }
            p = next;
#pragma unroll
            for (int q = 0; q < KINDS * NQ; ++q) bf[q] = bn[q];
        }
    }
}

// Products of few rows per expert: bound by reading every expert's weights
// once.  A workgroup computes up to 32 rows by 16 CS NB weight rows; its KS x CS
// wavefronts split k (step u of 128 bytes goes to wavefront u % KS) and the
// weight rows, so every byte of W is loaded straight into the registers of the
// one wavefront that uses it, with no staging and no barrier until the sums are
// joined in LDS.  A step is loaded while the one before is multiplied.  Measured:
// one row for each of 96 experts (H 2048, inner 768, BF16) 154 us for the network's
// 906 MB, 5.9 TB/s; 8 rows on 8 experts (25 MB) 8 us, of which 3 are the launch and
// finding the tile.
template <bool FP8, bool GATED, bool OUT8, bool LOW, int NB, int KS, int CS>
struct Few {
    static constexpr int G = GATED ? NB / 2 : NB;   // blocks of one kind of a wavefront
    static constexpr int BN = CS * G * 16;          // columns of out per tile
    static constexpr int waves = KS * CS, threads = waves * kWave;
    static constexpr int rows = 32;

    struct Shared {
        Tiles tiles;
        f32x4 red[KS][CS * NB][kWave];
        float amax[OUT8 ? waves : 1][16];
    };
    template <int MB>
    struct Step {
        Frag w[NB], x[MB];
        float sx[MB], s0, s1;
    };

    const ProductArgs &a;
    Shared &sh;
    int lane, g, r16, wave, kw, cw, nu;

    __device__ __forceinline__ Few(const ProductArgs &a_, Shared &s_) : a(a_), sh(s_)
    {
        lane = threadIdx.x & 63;
        g = lane >> 4;
        r16 = lane & 15;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        kw = wave % KS;
        cw = wave / KS;
        nu = a.kb / 128;   // steps of k (FP8: scale blocks)
    }

    template <int MB>
    __device__ __forceinline__ void run(const Tile &t, int c0)
    {
        const gptr<const uint8_t> wb = (gptr<const uint8_t>)a.w + int64_t(t.e) * a.m * a.kb;
        const gptr<const uint8_t> xb = (gptr<const uint8_t>)a.x + int64_t(t.row0) * a.kb;
        uint32_t wo[NB], xo[MB];
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int c = min(c0 + cw * (16 * G) + q % G * 16, a.n - 16) + (q < G ? 0 : a.n);   // the block's first row
            wo[q] = uint32_t(c) * uint32_t(a.kb) + (a.packed ? lane * 16 : uint32_t(r16) * uint32_t(a.kb) + g * 16);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) xo[i] = uint32_t(min(i * 16 + r16, t.nrows - 1)) * uint32_t(a.kb) + g * 16;
        const uint32_t piece = a.packed ? 1024 : 64;   // from a lane's first piece of a step to its second
        f32x4 acc[MB][NB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int q = 0; q < NB; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        const gptr<const float> wsp =
            FP8 ? (gptr<const float>)a.ws + (int64_t(t.e) * ((a.m + 127) / 128) + c0 / 128) * nu : nullptr;
        auto load = [&](Step<MB> &st, int u) {
#pragma unroll
            for (int q = 0; q < NB; ++q)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    st.w[q].p[p] = *(gptr<const u32x4>)(wb + (wo[q] + uint32_t(u) * uint32_t(a.wstep) + p * piece));
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int p = 0; p < 2; ++p) st.x[i].p[p] = *(gptr<const u32x4>)(xb + xo[i] + u * 128 + p * 64);
            if constexpr (FP8) {
                st.s0 = wsp[u];
                st.s1 = GATED ? wsp[(a.n / 128) * nu + u] : 0.f;
#pragma unroll
                for (int i = 0; i < MB; ++i)
                    st.sx[i] = ((gptr<const float>)a.xs)[int64_t(t.row0 + min(i * 16 + r16, t.nrows - 1)) * nu + u];
            }
        };
        auto multiply = [&](const Step<MB> &st) {
#pragma unroll
            for (int q = 0; q < NB; ++q)
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    if constexpr (FP8) {
                        const f32x4 d = mfma_fp8(st.w[q], st.x[i], f32x4{0.f, 0.f, 0.f, 0.f});
                        const float f = st.sx[i] * (q < G ? st.s0 : st.s1);
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][q][j] = fmaf(d[j], f, acc[i][q][j]);
                    } else {
#pragma unroll
                        for (int p = 0; p < 2; ++p) acc[i][q] = mfma_bf16(st.w[q].p[p], st.x[i].p[p], acc[i][q]);
                    }
                }
        };
        if (kw < nu) {
            // the steps two at a time, so that each has registers of its own
            Step<MB> s0, s1;
            int u = kw;
            load(s0, u);
            for (; u + 2 * KS < nu; u += 2 * KS) {
                load(s1, u + KS);
                __builtin_amdgcn_sched_barrier(0);
                multiply(s0);
                load(s0, u + 2 * KS);
                __builtin_amdgcn_sched_barrier(0);
                multiply(s1);
            }
            if (u + KS < nu) {
                load(s1, u + KS);
                __builtin_amdgcn_sched_barrier(0);
                multiply(s0);
                multiply(s1);
            } else {
                multiply(s0);
            }
        }
        if constexpr (LOW) {
            // each of the KS wavefronts along k adds its share of the adapters
            int row[MB], tag[MB], wrow[NB];
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                row[i] = t.row0 + min(i * 16 + r16, t.nrows - 1);
                tag[i] = i * 16 + r16 < t.nrows ? ((gptr<const int32_t>)a.tags)[row[i]] : -1;
                if (tag[i] >= a.nad) tag[i] = -1;
            }
#pragma unroll
            for (int q = 0; q < NB; ++q) {
                const int c = min(c0 + cw * (16 * G) + q % G * 16 + r16, a.n - 1);
                wrow[q] = q < G ? c : a.n + c;
            }
            add_adapters<GATED ? 2 : 1, G, MB>(a, t.e, row, tag, wrow, acc, kw, KS);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) join(t, c0, i, acc[i]);
    }

    // Row block i: the wavefronts' sums joined, and on to out.
    __device__ __forceinline__ void join(const Tile &t, int c0, int i, const f32x4 (&acc)[NB])
    {
#pragma unroll
        for (int q = 0; q < NB; ++q) sh.red[kw][cw * NB + q][lane] = acc[q];
        __syncthreads();
        constexpr int own = (CS * G + waves - 1) / waves;   // column blocks per wavefront
        f32x4 res[own];
        const int r = i * 16 + r16;
        const bool in = r < t.nrows;
        const int row = t.row0 + min(r, t.nrows - 1);
        float big = 0.f;
#pragma unroll
        for (int o = 0; o < own; ++o) {
            const int idx = o * waves + wave, s = idx / G, q = idx - s * G;
            if (idx < CS * G) {
                f32x4 v[GATED ? 2 : 1];
#pragma unroll
                for (auto &z : v) z = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const f32x4 p = sh.red[k][s * NB + q][lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[0][j] += p[j];
                    if constexpr (GATED) {
                        const f32x4 p1 = sh.red[k][s * NB + G + q][lane];
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[1][j] += p1[j];
                    }
                }
                if constexpr (GATED)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[0][j] = silu(v[0][j]) * v[1][j];
                const int c = c0 + s * (16 * G) + q * 16 + g * 4;
                if constexpr (!OUT8) {
                    if (in && c < a.n)
                        *(gptr<u32x2>)((gptr<uint16_t>)a.out + int64_t(row) * a.n + c) =
                            u32x2{pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3])};
                } else {
                    res[o] = v[0];
#pragma unroll
                    for (int j = 0; j < 4; ++j) big = fmaxf(big, fabsf(v[0][j]));
                }
            }
        }
        if constexpr (OUT8) {
            // one scale per row and tile (a tile is one 128-column block)
            static_assert(BN == 128 && CS * G % waves == 0, "a tile is one scale block");
            big = fmaxf(big, __shfl_xor(big, 16));
            big = fmaxf(big, __shfl_xor(big, 32));
            if (g == 0) sh.amax[wave][r16] = big;
            __syncthreads();
            float m = 0.f;
#pragma unroll
            for (int w = 0; w < waves; ++w) m = fmaxf(m, sh.amax[w][r16]);
            float inv;
            const float sc = scale_of(m, inv);
            if (in && wave == 0 && g == 0) ((gptr<float>)a.outs)[int64_t(row) * (a.n / 128) + c0 / 128] = sc;
#pragma unroll
            for (int o = 0; o < own; ++o) {
                const int idx = o * waves + wave, s = idx / G, q = idx - s * G;
                const uint32_t code = codes_of(res[o], inv);
                if (in) *(gptr<uint32_t>)((gptr<uint8_t>)a.out + int64_t(row) * a.n + c0 + s * (16 * G) + q * 16 + g * 4) = code;
            }
        }
        __syncthreads();   // red and amax are written again
    }
};

template <bool FP8, bool GATED, bool OUT8, bool LOW, int NB, int KS, int CS>
__global__ __launch_bounds__(KS * CS * kWave) void k_product_few(ProductArgs a)
{
    typedef Few<FP8, GATED, OUT8, LOW, NB, KS, CS> F;
    __shared__ typename F::Shared sh;
    if (threadIdx.x < kWave) {
        read_spans(sh.tiles, a.ends, a.E, a.alpha, a.rows);
        build_tiles<F::rows>(sh.tiles, a.E);
    }
    __syncthreads();
    F f(a, sh);
    for (Items it = my_items(sh.tiles.first[a.E] * a.ntiles); it.at < it.end; it.at += it.step) {
        int c0;
        const Tile t = find_tile<F::rows, 16>(sh.tiles, a.E, a.ntiles, it.at, c0);
        c0 *= F::BN;
        if (t.nrows <= 16) f.template run<1>(t, c0);
        else f.template run<2>(t, c0);
    }
}

// Products of many rows per expert: WM x WN wavefronts compute a tile of up to
// 32 MX rows by 64 WN weight rows, each MB (at most MX) by 4 blocks of 16 x 16.
// Steps of 128 bytes of k of both operands go from global memory straight into a
// ring of ST stages in LDS (no registers, no address arithmetic: per-lane offsets
// are fixed, each item is a few buffer descriptors, and rows behind the tile read
// as zero by the descriptor's bound).  ST - 1 steps are on their way while one is
// computed, across the borders of items.
//
// In LDS a row's step is eight pieces of 16 bytes, piece p of row r at p ^ (r % 8):
// the rows that one cycle of a 16-byte read touches then lie in different banks,
// while the writes, whose order the hardware fixes, stay whole rows.  Packed
// weights lie as they come, sixteen rows in the order in which the lanes read them.
//
// Measured (64 experts, H 2048, inner 768, first and second product of the network):
// BF16 16 rows each 72 and 38 us (5.6 and 5.2 TB/s of weights), 256 rows 138 and
// 90 us (0.74 and 0.58 PFLOP/s), 485 rows of 96 experts 339 and 214 us (0.86 and
// 0.69); FP8 16 rows 43 and 25 us, 256 rows 103 and 65 us.  Few rows are bound by
// HBM.  Many are bound by the loads' latency times the distinct bytes on their way,
// which LDS limits, and by the activation and stores at a tile's end, under which
// only the next item's loads run.
struct ManyItem {
    Tile t;
    int c0;
    u32x4 xr, wr, sr;   // buffer descriptors of the tile's rows, weight rows and (by wavefront) scales
};

// The same in every lane, told to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return uint32_t(__builtin_amdgcn_readfirstlane(int(v))); }
__device__ __forceinline__ u32x4 uniform(u32x4 v) { return u32x4{uniform(v[0]), uniform(v[1]), uniform(v[2]), uniform(v[3])}; }

// The descriptor of `bytes` bytes from p on; reads behind them give zero.
__device__ __forceinline__ u32x4 buffer_of(const void *p, uint32_t bytes)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    return uniform(u32x4{uint32_t(v), uint32_t(v >> 32) & 0xFFFFu, bytes, 0x00020000u});
}

// A lane's four columns of blocks q and q + 1 (columns 4g .. of each) to eight of one
// block: odd lane groups take theirs of block q + 1, even ones of block q, from each
// other, so that a row's stores are whole 64-byte pieces.  Afterwards a holds the
// first four columns and b the last; returns the first one, from block q's first on.
__device__ __forceinline__ int pair_up(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
    const int g = (threadIdx.x & 63) >> 4;
    return (g & 1) * 16 + (g >> 1) * 8;
}

// N loads of 64 lanes x 16 bytes (or one of 64 x 4) of buffer `r`, lane by lane at
// voff[i] + soff, to LDS from `lds` + i STEP on.  In assembly, because the compiler
// waits for every such load it knows of before any LDS read that it cannot tell apart,
// which would end the overlap of one step's arithmetic with the next one's loads; the
// waits are written out where a stage is first read.
//
// The compiler places no wait states inside assembly, nor does the hardware: a vector
// memory instruction may read a scalar register five wait states after a vector
// instruction (the v_readfirstlane of uniform(), a register spilled to lanes) wrote it,
// and use M0 one after.  All of a block's registers are written before it, so the wait
// stands once per block, ahead of its first load: s_mov and s_nop 3.  (All of a step's
// loads in one block: no difference.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // that M0, which the compiler sets where it needs it, is named as written
__device__ __forceinline__ void to_lds4(u32x4 r, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(uniform(lds)), "v"(voff),
                 "s"(uniform(r)), "s"(uniform(soff))
                 : "m0");
}
template <uint32_t STEP>
__device__ __forceinline__ void to_lds16(u32x4 r, const uint32_t (&voff)[2], uint32_t soff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %3, %4 offen lds\n\t"
                 "s_add_u32 m0, m0, %5\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds" ::"s"(uniform(lds)),
                 "v"(voff[0]), "v"(voff[1]), "s"(uniform(r)), "s"(uniform(soff)), "n"(STEP)
                 : "m0", "scc");
}
template <uint32_t STEP>
__device__ __forceinline__ void to_lds16(u32x4 r, const uint32_t (&voff)[4], uint32_t soff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %5, %6 offen lds\n\t"
                 "s_add_u32 m0, m0, %7\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %5, %6 offen lds\n\t"
                 "s_add_u32 m0, m0, %7\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %5, %6 offen lds\n\t"
                 "s_add_u32 m0, m0, %7\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %5, %6 offen lds" ::"s"(uniform(lds)),
                 "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3]), "s"(uniform(r)), "s"(uniform(soff)), "n"(STEP)
                 : "m0", "scc");
}
#pragma clang diagnostic pop

template <int WM_, int WN_, int MX_, int ST_>
struct Shape {
    static constexpr int WM = WM_, WN = WN_, MX = MX_, ST = ST_;
    static constexpr int waves = WM * WN, threads = waves * kWave;
    static constexpr int rows = WM * MX * 16, wrows = WN * 64;
    static constexpr int nx = rows / 8 / waves, nw = wrows / 8 / waves;   // loads (1 KiB) of a wavefront and step
    static constexpr uint32_t xbytes = rows * 128, scales = (rows + wrows) * 128;
    static_assert(nx * waves * 8 == rows && nw * waves * 8 == wrows, "whole loads");
};

template <class S, bool FP8, bool GATED, bool OUT8, bool LOW>
struct Many {
    static constexpr int G = GATED ? 2 : 4;               // blocks of one kind per wavefront
    static constexpr int BN = S::wrows / (GATED ? 2 : 1); // columns of out per tile
    static constexpr uint32_t stage_bytes = S::scales + (FP8 ? S::waves * 256 : 0);
    static constexpr int loads = S::nx + S::nw + (FP8 ? 1 : 0);
    static_assert(!FP8 || S::rows <= 64 * S::waves / 2, "half the wavefronts bring the rows' scales");

    const ProductArgs &a;
    Tiles &tiles;
    float *amax;                   // LDS [WN][rows]
    lptr<unsigned char> stages;
    uint32_t lds;                  // LDS address of the first stage
    int lane, g, r16, wave, wm, wn;
    uint32_t xo[S::nx], wo[S::nw], so;     // this lane's offsets of a step's pieces in memory
    int xp[2], wp[2];                      // and of its own two of a block in LDS
    int nu;

    // the next load: its place among the items, its item and stage
    LoadCursor next;
    ManyItem ahead;
    int ahead_stage;

    static __device__ __forceinline__ int key(int row) { return row & 7; }

    __device__ __forceinline__ Many(const ProductArgs &a_, Tiles &t_, float *amax_, lptr<unsigned char> stages_)
        : a(a_), tiles(t_), amax(amax_), stages(stages_)
    {
        lds = uint32_t(reinterpret_cast<uintptr_t>(stages));
        lane = threadIdx.x & 63;
        g = lane >> 4;
        r16 = lane & 15;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wm = wave / S::WN;
        wn = wave % S::WN;
        nu = a.kb / 128;
#pragma unroll
        for (int i = 0; i < S::nx; ++i) {
            const int row = ((i * S::waves + wave) * 64 + lane) / 8;
            xo[i] = uint32_t(row) * uint32_t(a.kb) + uint32_t(((lane & 7) ^ key(row)) * 16);
        }
#pragma unroll
        for (int i = 0; i < S::nw; ++i) {
            const int at = ((i * S::waves + wave) * 64 + lane) * 16, row = at / 128;   // in the stage's weights
            // wavefront wn's rows of the stage are its four blocks in order
            const int q = row >> 4 & 3, c = (row >> 6) * (16 * G) + q % G * 16 + (q < G ? 0 : a.n);
            wo[i] = uint32_t(c) * uint32_t(a.kb) +
                    (a.packed ? uint32_t(at % 2048)
                              : uint32_t(row & 15) * uint32_t(a.kb) + uint32_t(((lane & 7) ^ key(row)) * 16));
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            xp[p] = r16 * 128 + ((4 * p + g) ^ key(r16)) * 16;
            wp[p] = a.packed ? p * 1024 + lane * 16 : xp[p];
        }
        // the first half of the wavefronts bring 64 row scales each, the others the weights' two
        if (FP8) so = wave < S::waves / 2 ? uint32_t(wave * 64 + lane) * uint32_t(nu) * 4u
                                          : uint32_t(GATED ? (lane & 1) * (a.n / 128) : (lane & 1)) * uint32_t(nu) * 4u;
    }

    __device__ __forceinline__ Tile tile_of(int at, int &c0) const
    {
        const Tile t = find_tile<S::rows, 16 * S::WM>(tiles, a.E, a.ntiles, at, c0);
        c0 *= BN;
        return t;
    }

    __device__ __forceinline__ void load_item()
    {
        const bool live = next.live;
        ahead.t = tile_of(next.at, ahead.c0);
        const Tile &t = ahead.t;
        const int c0 = ahead.c0;
        // behind the last item the loads go on without a byte, so that their number stays the same
        ahead.xr = buffer_of(a.x + int64_t(t.row0) * a.kb, live ? uint32_t(t.nrows) * uint32_t(a.kb) : 0u);
        ahead.wr = buffer_of(a.w + (int64_t(t.e) * a.m + c0) * a.kb, live ? uint32_t(a.m - c0) * uint32_t(a.kb) : 0u);
        if (FP8) {
            const int mb = (a.m + 127) / 128;   // scale rows of an expert
            if (wave < S::waves / 2)
                ahead.sr = buffer_of(a.xs + int64_t(t.row0) * nu, live ? uint32_t(t.nrows) * uint32_t(nu) * 4u : 0u);
            else
                ahead.sr = buffer_of(a.ws + (int64_t(t.e) * mb + c0 / 128) * nu,
                                     live ? uint32_t(mb - c0 / 128) * uint32_t(nu) * 4u : 0u);
        }
    }

    // The next step's loads on their way.
    __device__ __forceinline__ void issue(const Items &it)
    {
        const uint32_t at = lds + uint32_t(ahead_stage) * stage_bytes, xu = uint32_t(next.u) * 128u, wu = uint32_t(next.u) * uint32_t(a.wstep);
        to_lds16<S::waves * 1024>(ahead.wr, wo, wu, at + S::xbytes + uint32_t(wave) * 1024u);
        to_lds16<S::waves * 1024>(ahead.xr, xo, xu, at + uint32_t(wave) * 1024u);
        if (FP8) to_lds4(ahead.sr, so, uint32_t(next.u) * 4u, at + S::scales + uint32_t(wave) * 256u);
        ahead_stage = ahead_stage + 1 == S::ST ? 0 : ahead_stage + 1;
        if (next.advance(nu, it.end, it.step)) load_item();
    }

    __device__ __forceinline__ void begin(const Items &it)
    {
        next = LoadCursor{it.at, 0, true};
        ahead_stage = 0;
        load_item();
#pragma unroll
        for (int i = 0; i < S::ST - 1; ++i) issue(it);
    }

    // A block of sixteen rows, this lane's pieces of it at `at`.
    __device__ __forceinline__ Frag read(lptr<const unsigned char> block, const int (&at)[2]) const
    {
        Frag o;
#pragma unroll
        for (int p = 0; p < 2; ++p) o.p[p] = *(lptr<const u32x4>)(block + at[p]);
        return o;
    }

    template <int MB>
    __device__ __forceinline__ void tile(const Tile &t, int c0, const Items &it, int &stage)
    {
        f32x4 acc[MB][4];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int row = wm * MB * 16 + r16;
        for (int u = 0; u < nu; ++u) {
            // this wavefront's part of the step has come; behind the barrier all of
            // it has, and every read of the stage that is loaded next is over
            asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S::ST - 2) * loads) : "memory");
            issue(it);
            const lptr<const unsigned char> st = stages + stage * stage_bytes, xb = st + wm * MB * 2048,
                                            wb = st + S::xbytes + wn * 4 * 2048;
            Frag wf[4], xf[MB];
            f32x4 d[2][4];   // FP8: a row block's sums are scaled under the next one's products
#pragma unroll
            for (int q = 0; q < 4; ++q) wf[q] = read(wb + q * 2048, wp);
            float s0 = 0.f, s1 = 0.f, sx[MB];
            const lptr<const float> sc = (lptr<const float>)(st + S::scales);
            if (FP8) {
                s0 = sc[S::waves * 32 + (GATED ? 0 : wn >> 1)];
                s1 = sc[S::waves * 32 + 1];
#pragma unroll
                for (int i = 0; i < MB; ++i) sx[i] = sc[row + i * 16];
            }
            xf[0] = read(xb, xp);
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                if (i + 1 < MB) xf[i + 1] = read(xb + (i + 1) * 2048, xp);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (FP8) {
                        d[i & 1][q] = mfma_fp8(wf[q], xf[i], f32x4{0.f, 0.f, 0.f, 0.f});
                        if (i > 0) {
                            const float s = sx[i - 1] * (q < G ? s0 : s1);
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[i - 1][q][j] = fmaf(d[(i - 1) & 1][q][j], s, acc[i - 1][q][j]);
                        }
                    } else {
#pragma unroll
                        for (int p = 0; p < 2; ++p) acc[i][q] = mfma_bf16(wf[q].p[p], xf[i].p[p], acc[i][q]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (FP8)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float s = sx[MB - 1] * (q < G ? s0 : s1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[MB - 1][q][j] = fmaf(d[(MB - 1) & 1][q][j], s, acc[MB - 1][q][j]);
                }
            stage = stage + 1 == S::ST ? 0 : stage + 1;
        }
        finish<MB>(t, c0, acc);
    }

    template <int MB>
    __device__ __forceinline__ void finish(const Tile &t, int c0, f32x4 (&acc)[MB][4]) const
    {
        if constexpr (LOW) {
            int row[MB], tag[MB], wrow[4];
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                const int r = (wm * MB + i) * 16 + r16;
                row[i] = t.row0 + min(r, t.nrows - 1);
                tag[i] = r < t.nrows ? ((gptr<const int32_t>)a.tags)[row[i]] : -1;
                if (tag[i] >= a.nad) tag[i] = -1;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = min(c0 + wn * (16 * G) + q % G * 16 + r16, a.n - 1);
                wrow[q] = q < G ? c : a.n + c;
            }
            add_adapters<GATED ? 2 : 1, G, MB>(a, t.e, row, tag, wrow, acc, 0, 1);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int r = (wm * MB + i) * 16 + r16;
            const bool in = r < t.nrows;
            const int row = t.row0 + min(r, t.nrows - 1);
            if constexpr (GATED)
#pragma unroll
                for (int q = 0; q < G; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][q][j] = silu(acc[i][q][j]) * acc[i][q + G][j];
            if constexpr (!OUT8) {
#pragma unroll
                for (int h = 0; h < G / 2; ++h) {
                    uint32_t v[2][2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        v[q][0] = pack_bf16(acc[i][2 * h + q][0], acc[i][2 * h + q][1]);
                        v[q][1] = pack_bf16(acc[i][2 * h + q][2], acc[i][2 * h + q][3]);
                    }
                    const int c = c0 + wn * (16 * G) + h * 32 + pair_up(v[0][0], v[1][0]);
                    pair_up(v[0][1], v[1][1]);
                    if (in && c < a.n)
                        *(gptr<u32x4>)((gptr<uint16_t>)a.out + int64_t(row) * a.n + c) = u32x4{v[0][0], v[0][1], v[1][0], v[1][1]};
                }
            } else {
                float v = 0.f;
#pragma unroll
                for (int q = 0; q < G; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v = fmaxf(v, fabsf(acc[i][q][j]));
                v = fmaxf(v, __shfl_xor(v, 16));
                v = fmaxf(v, __shfl_xor(v, 32));
                if (g == 0) amax[wn * S::rows + r] = v;
            }
        }
        if constexpr (OUT8) {
            static_assert(BN == 128, "a tile is one scale block");
            // the tile's 128 columns are one scale block, spread over the four
            // wavefronts along the weights
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                const int r = (wm * MB + i) * 16 + r16;
                float v = amax[r];
#pragma unroll
                for (int w = 1; w < S::WN; ++w) v = fmaxf(v, amax[w * S::rows + r]);
                float inv;
                const float sc = scale_of(v, inv);
                const int64_t row = t.row0 + r;
                if (r < t.nrows && wn == 0 && g == 0) ((gptr<float>)a.outs)[row * (a.n / 128) + c0 / 128] = sc;
                uint32_t code[2] = {codes_of(acc[i][0], inv), codes_of(acc[i][1], inv)};
                const int c = c0 + wn * 32 + pair_up(code[0], code[1]);
                if (r < t.nrows) *(gptr<u32x2>)((gptr<uint8_t>)a.out + row * a.n + c) = u32x2{code[0], code[1]};
            }
            // (amax is written again behind the next item's step barriers)
        }
    }
};

// All items of a workgroup, in tiles of shape S.
template <class S, bool FP8, bool GATED, bool OUT8, bool LOW>
__device__ __forceinline__ void run_many(const ProductArgs &a, Tiles &tiles, float *amax, lptr<unsigned char> stages)
{
    Many<S, FP8, GATED, OUT8, LOW> k(a, tiles, amax, stages);
    Items it = my_items(tiles.first[a.E] * a.ntiles);
    if (it.at >= it.end) return;
    const Items all = it;
    k.begin(all);
    int stage = 0;
    for (; it.at < it.end; it.at += it.step) {
        int c0;
        const Tile t = k.tile_of(it.at, c0);
        const int mb = (t.nrows + 16 * S::WM - 1) / (16 * S::WM);
        if constexpr (S::MX == 4) {
            switch (mb) {
            case 1: k.template tile<1>(t, c0, all, stage); break;
            case 2: k.template tile<2>(t, c0, all, stage); break;
            case 3: k.template tile<3>(t, c0, all, stage); break;
            default: k.template tile<4>(t, c0, all, stage); break;
            }
        } else {
            switch (mb) {
            case 1: k.template tile<1>(t, c0, all, stage); break;
            case 2: k.template tile<2>(t, c0, all, stage); break;
            case 3: k.template tile<3>(t, c0, all, stage); break;
            case 4: k.template tile<4>(t, c0, all, stage); break;
            case 5: k.template tile<5>(t, c0, all, stage); break;
            case 6: k.template tile<6>(t, c0, all, stage); break;
            case 7: k.template tile<7>(t, c0, all, stage); break;
            default: k.template tile<8>(t, c0, all, stage); break;
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load may come after the LDS is another workgroup's
}

// One workgroup per CU: 128 x 256 tiles with three stages, or 256 x 256 with two.
// The taller ones read and move less per product, the others wait less for the
// weights and leave fewer CUs idle at the end; FP8 (which holds the sums of one scale
// block beside the scaled ones) and the adapters have no registers for 256 rows.
typedef Shape<2, 4, 4, 3> Low;
typedef Shape<2, 4, 8, 2> Tall;

// Rows per expert (of those that have any) from which BF16 products take the tall tiles.
// (64 experts, H 2048, inner 768: at 256 rows 259 us instead of 228, at 320 258 and
// 262, at 384 275 and 326, at 512 378 and 406.  Measured at this width and number of
// experts only; at 256 rows the 384 tall items are 1.5 rounds of the CUs, the 768 low ones
// three.)
constexpr int kTallFrom = 320;

template <bool FP8, bool GATED, bool OUT8, bool LOW>
__global__ __launch_bounds__(Low::threads, 2) void k_product_many(ProductArgs a)
{
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ Tiles tiles;
    __shared__ float amax[OUT8 ? Low::WN * Low::rows : 1];
    __shared__ int tall;
    constexpr bool both = !FP8 && !LOW;
    if (threadIdx.x < kWave) {
        const int2 n = read_spans(tiles, a.ends, a.E, a.alpha, a.rows);
        const bool t = both && int64_t(n.x) >= int64_t(kTallFrom) * n.y;
        if (t) build_tiles<Tall::rows>(tiles, a.E);
        else build_tiles<Low::rows>(tiles, a.E);
        if (threadIdx.x == 0) tall = t;
    }
    __syncthreads();
    if constexpr (both) {
        if (__builtin_amdgcn_readfirstlane(tall)) {
            run_many<Tall, FP8, GATED, OUT8, LOW>(a, tiles, amax, (lptr<unsigned char>)stages);
            return;
        }
    }
    run_many<Low, FP8, GATED, OUT8, LOW>(a, tiles, amax, (lptr<unsigned char>)stages);
}

// -------------------------------------------------------------- adapters ----

struct ShrinkArgs {
    const uint8_t *x;
    const float *xs;
    const int32_t *ends, *tags;
    const uint8_t *a;
    const float *scaling;
    uint16_t *t;   // [rows][2][c]
    int rows, E, alpha;
    int k;
    int c;       // rows of one adapter's A: rank, or 2 rank gated
    int nad;
    int share;   // workgroups per expert
    int spread;  // experts side by side: 8, or all of fewer
};

// Eight E4M3 codes to bf16 (exact: four significant bits).
__device__ __forceinline__ u32x4 fp8_to_bf16(uint32_t q0, uint32_t q1)
{
    u32x4 r;
    const uint32_t q[2] = {q0, q1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[i]), false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[i]), true);
        r[2 * i] = (__float_as_uint(lo[0]) >> 16) | (__float_as_uint(lo[1]) & 0xFFFF0000u);
        r[2 * i + 1] = (__float_as_uint(hi[0]) >> 16) | (__float_as_uint(hi[1]) & 0xFFFF0000u);
    }
    return r;
}

// t[r, :] = scaling[i] A[i, j] x[r] for every row r of expert j with an adapter i.
// Meant to be bound by reading the A of every (adapter, expert) pair once.  An
// expert's workgroups find its distinct adapters from a bit map of the rows' tags;
// the pairs of an adapter and 32 rows of its A go round them.  For each, the expert's
// tags are read again (rows times distinct adapters in all) and the
// adapter's rows are gathered, 32 (FP8 64) at a time, and multiplied as in
// k_product_few: the A operand holds rows of A, the wavefronts split k.
// Measured: 32 adapters of rank 16, 1024 rows over 64 experts (813 pairs, 106 MB of
// A) 41 us for the first product; FP8, 8 of rank 32, 16384 rows (134 MB) 56 us
// (68 with x read 8 bytes at a time).
template <bool FP8>
struct Shrink {
    static constexpr int KS = 4, threads = KS * kWave, NB = 2, CH = 16 * NB;
    static constexpr int step = FP8 ? 128 : 64;         // columns of k
    static constexpr int NP = FP8 ? 4 : 2;              // products of 32 columns per step
    static constexpr int MAXB = FP8 ? 4 : 2, GROUP = 16 * MAXB;   // row blocks and rows at a time
    static constexpr int words = AFD_MAX_ADAPTERS / 32;

    struct Shared {
        uint32_t bits[words];
        int sums[threads];
        int list[threads + GROUP];   // gathered rows
        int waves[KS], found;
        f32x4 red[KS][MAXB * NB][kWave];
    };
    template <int MB>
    struct Step {
        u32x4 a[NB][NP];
        u32x4 x[MB][2];   // FP8: 16 codes, of two products
        float s[MB];
    };

    const ShrinkArgs &a;
    Shared &sh;
    int lane, g, r16, wave, nu;

    __device__ __forceinline__ Shrink(const ShrinkArgs &a_, Shared &s_) : a(a_), sh(s_)
    {
        lane = threadIdx.x & 63;
        g = lane >> 4;
        r16 = lane & 15;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        nu = a.k / step;
    }

    // n rows from list[first], columns c0 .. of the adapter.
    template <int MB>
    __device__ __forceinline__ void multiply(int e, int ad, int c0, int first, int n)
    {
        int row[MB];
        gptr<const uint8_t> xp[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            row[i] = sh.list[first + min(i * 16 + r16, n - 1)];
            xp[i] = (gptr<const uint8_t>)a.x + int64_t(row[i]) * a.k * (FP8 ? 1 : 2) + g * 16;
        }
        gptr<const uint8_t> ap[NB];
#pragma unroll
        for (int q = 0; q < NB; ++q)
            ap[q] = (gptr<const uint8_t>)a.a +
                    ((int64_t(ad) * a.E + e) * a.c + min(c0 + q * 16 + r16, a.c - 1)) * int64_t(a.k) * 2 + g * (FP8 ? 32 : 16);
        f32x4 acc[MB][NB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int q = 0; q < NB; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto load = [&](Step<MB> &st, int u) {
#pragma unroll
            for (int q = 0; q < NB; ++q)
#pragma unroll
                for (int p = 0; p < NP; ++p) st.a[q][p] = *(gptr<const u32x4>)(ap[q] + u * (step * 2) + (FP8 ? p / 2 * 128 + p % 2 * 16 : p * 64));
#pragma unroll
            for (int i = 0; i < MB; ++i) {
#pragma unroll
                for (int p = 0; p < 2; ++p) st.x[i][p] = *(gptr<const u32x4>)(xp[i] + u * 128 + p * 64);
                if (FP8) st.s[i] = ((gptr<const float>)a.xs)[int64_t(row[i]) * nu + u];
            }
        };
        auto use = [&](const Step<MB> &st) {
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                if constexpr (FP8) {
                    f32x4 d[NB];
#pragma unroll
                    for (int q = 0; q < NB; ++q) d[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const u32x4 xv = fp8_to_bf16(st.x[i][p / 2][p % 2 * 2], st.x[i][p / 2][p % 2 * 2 + 1]);
#pragma unroll
                        for (int q = 0; q < NB; ++q) d[q] = mfma_bf16(st.a[q][p], xv, d[q]);
                    }
#pragma unroll
                    for (int q = 0; q < NB; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][q][j] = fmaf(d[q][j], st.s[i], acc[i][q][j]);
                } else {
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int q = 0; q < NB; ++q) acc[i][q] = mfma_bf16(st.a[q][p], st.x[i][p], acc[i][q]);
                }
            }
        };
        if constexpr (FP8) {   // 64 rows' steps leave no registers for two
            for (int u = wave; u < nu; u += KS) {
                Step<MB> s0;
                load(s0, u);
                __builtin_amdgcn_sched_barrier(0);
                use(s0);
            }
        } else if (wave < nu) {
            Step<MB> s0, s1;
            int u = wave;
            load(s0, u);
            for (; u + 2 * KS < nu; u += 2 * KS) {
                load(s1, u + KS);
                __builtin_amdgcn_sched_barrier(0);
                use(s0);
                load(s0, u + 2 * KS);
                __builtin_amdgcn_sched_barrier(0);
                use(s1);
            }
            if (u + KS < nu) {
                load(s1, u + KS);
                __builtin_amdgcn_sched_barrier(0);
                use(s0);
                use(s1);
            } else {
                use(s0);
            }
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int q = 0; q < NB; ++q) sh.red[wave][i * NB + q][lane] = acc[i][q];
        __syncthreads();
        for (int b = wave; b < MB * NB; b += KS) {
            const int i = b / NB, q = b % NB, c = c0 + q * 16 + g * 4;
            f32x4 v = sh.red[0][b][lane];
#pragma unroll
            for (int w = 1; w < KS; ++w)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += sh.red[w][b][lane][j];
            const float f = ((gptr<const float>)a.scaling)[ad];
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = split_t(v[j] * f);
            if (i * 16 + r16 < n && c < a.c) {
                const gptr<uint16_t> t = (gptr<uint16_t>)a.t + int64_t(sh.list[first + i * 16 + r16]) * (2 * a.c) + c;
                *(gptr<u32x2>)t = u32x2{(h[0] & 0xFFFFu) | h[1] << 16, (h[2] & 0xFFFFu) | h[3] << 16};
                *(gptr<u32x2>)(t + a.c) = u32x2{h[0] >> 16 | (h[1] & 0xFFFF0000u), h[2] >> 16 | (h[3] & 0xFFFF0000u)};
            }
        }
        __syncthreads();   // red is written again, and the list may be
    }

    // The number (from 0) `want` of the set bits of the map.
    __device__ __forceinline__ int nth_adapter(int want)
    {
        const int tid = threadIdx.x, per = words / threads;
        const int before = tid ? sh.sums[tid - 1] : 0;
        if (want >= before && want < sh.sums[tid]) {
            int k = want - before;
            for (int i = 0; i < per; ++i) {
                uint32_t w = sh.bits[tid * per + i];
                const int n = __popc(w);
                if (k >= n) {
                    k -= n;
                    continue;
                }
                while (k--) w &= w - 1;
                sh.found = (tid * per + i) * 32 + __builtin_ctz(w);
                break;
            }
        }
        __syncthreads();
        const int r = __builtin_amdgcn_readfirstlane(sh.found);
        __syncthreads();
        return r;
    }

    __device__ __forceinline__ void run(int e, int y, int start, int count)
    {
        const int tid = threadIdx.x, per = words / threads;
        const gptr<const int32_t> tags = (gptr<const int32_t>)a.tags + start;
        for (int i = tid; i < words; i += threads) sh.bits[i] = 0;
        __syncthreads();
        for (int i = tid; i < count; i += threads) {
            const int tag = tags[i];
            if (tag >= 0 && tag < a.nad) atomicOr(&sh.bits[tag >> 5], 1u << (tag & 31));
        }
        __syncthreads();
        int n = 0;
        for (int i = 0; i < per; ++i) n += __popc(sh.bits[tid * per + i]);
        for (int d = 1; d < kWave; d *= 2) {
            const int o = __shfl_up(n, d);
            if (lane >= d) n += o;
        }
        if (lane == kWave - 1) sh.waves[wave] = n;
        __syncthreads();
        for (int w = 0; w < wave; ++w) n += sh.waves[w];
        sh.sums[tid] = n;
        __syncthreads();
        const int chunks = (a.c + CH - 1) / CH, total = __builtin_amdgcn_readfirstlane(sh.sums[threads - 1]) * chunks;
        for (int z = y; z < total; z += a.share) {
            const int ad = nth_adapter(z / chunks), c0 = (z % chunks) * CH;
            int have = 0;
            for (int base = 0; base < count; base += threads) {
                const bool mine = base + tid < count && tags[base + tid] == ad;
                const uint64_t m = __ballot(mine);
                if (lane == 0) sh.waves[wave] = __popcll(m);
                __syncthreads();
                int at = have + __popcll(m & ((uint64_t(1) << lane) - 1)), all = have;
                for (int w = 0; w < KS; ++w) {
                    if (w < wave) at += sh.waves[w];
                    all += sh.waves[w];
                }
                if (mine) sh.list[at] = start + base + tid;
                have = __builtin_amdgcn_readfirstlane(all);
                __syncthreads();
                const bool last = base + threads >= count;
                int first = 0;
                while (have - first >= GROUP || (last && have > first)) {
                    const int n = min(have - first, GROUP);
                    if (n <= 16) multiply<1>(e, ad, c0, first, n);
                    else if (n <= 32 || MAXB == 2) multiply<2>(e, ad, c0, first, n);
                    else multiply<MAXB>(e, ad, c0, first, n);
                    first += n;
                }
                // fewer rows left than a group: to the front, for the next tags
                const int rest = have - first;
                int keep = 0;
                if (tid < rest) keep = sh.list[first + tid];
                __syncthreads();
                if (tid < rest) sh.list[tid] = keep;
                have = rest;
                __syncthreads();
            }
        }
    }
};

// Workgroup b runs on XCD b % 8: from eight experts on, an expert's share one L2 for
// its rows; of fewer, each has workgroups on every XCD (the network of 60 rows, one
// expert, 64 adapters of rank 64: 60 us instead of 91).
template <bool FP8>
__global__ __launch_bounds__(Shrink<FP8>::threads, FP8 ? 3 : 4) void k_shrink(ShrinkArgs a)
{
    __shared__ typename Shrink<FP8>::Shared sh;
    const int i = blockIdx.x / a.spread, e = i / a.share * a.spread + blockIdx.x % a.spread, y = i % a.share;
    if (e >= a.E) return;
    const int prev = e == 0 ? 0 : min(max(a.ends[e - 1], 0), a.rows);
    const uint32_t st = (uint32_t(prev) + uint32_t(a.alpha) - 1u) / uint32_t(a.alpha) * uint32_t(a.alpha);
    const int start = int(min(st, uint32_t(a.rows))), count = min(a.ends[e], a.rows) - start;
    if (count <= 0) return;
    Shrink<FP8> k(a, sh);
    k.run(e, y, start, count);
}

// --------------------------------------------------------------- packing ----

struct PackArgs {
    const u32x4 *w;
    u32x4 *out;
    int64_t n;       // 16-byte pieces of all experts
    int pieces;      // of a row
};

// One 16-byte piece per thread and turn, in the order of the packed weights
// (m is a multiple of 16, so groups of sixteen rows do not cross experts).
__global__ __launch_bounds__(256) void k_pack(PackArgs a)
{
    const int64_t group = int64_t(a.pieces) * 16;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < a.n; i += int64_t(gridDim.x) * 256) {
        const int64_t gr = i / group;
        const int in = int(i - gr * group), step = in >> 7, piece = in >> 4 & 7, row = in & 15;
        a.out[i] = a.w[gr * group + int64_t(row) * a.pieces + step * 8 + piece];
    }
}

// ------------------------------------------------------------------ tags ----

struct TagArgs {
    const int32_t *slot;   // [ntok][K] {part << 24 | row, weight bits}, -1 skipped
    int32_t *out;
    const int32_t *tags[kMaxSources];
    int off[kMaxSources + 1];
    int n;                 // ntok * K
    int K, N, f;
};

// One thread per choice: bound by one dependent pair of loads (3 us, mostly launch).
__global__ __launch_bounds__(256) void k_tags(TagArgs a)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.n) return;
    const int sl = a.slot[2 * int64_t(i)];
    if (sl < 0 || (sl >> 24) != a.f) return;
    const int g = i / a.K;
    const int32_t *p = a.tags[0] + g;
    for (int s = 1; s < a.N; ++s)
        if (g >= a.off[s]) p = a.tags[s] + (g - a.off[s]);
    a.out[sl & 0xFFFFFF] = *p;
}

int launched() { return hipGetLastError() == hipSuccess ? 0 : 1; }

// Workgroups of a persistent launch: one per item, at most `most`, a multiple
// of 8 (my_items).  The host knows only the bound of the items: every expert can
// end inside a tile.
unsigned persistent_grid(int64_t tiles, int64_t per_tile, int most)
{
    const int64_t items = (tiles * per_tile + 7) / 8 * 8;
    return unsigned(items < most ? items : most);
}
int64_t tile_bound(int E, int64_t rows, int height) { return std::min(E + rows / height, rows); }

constexpr int kComputeUnits = 256;

template <bool FP8, bool GATED, bool OUT8, bool LOW, int NB, int KS, int CS>
int launch_few(const ProductPlan &p, ProductArgs a, hipStream_t st)
{
    typedef Few<FP8, GATED, OUT8, LOW, NB, KS, CS> F;
    a.ntiles = (p.n + F::BN - 1) / F::BN;
    const unsigned grid = persistent_grid(tile_bound(p.E, p.rows, F::rows), a.ntiles, kComputeUnits * 8);
    hipLaunchKernelGGL((k_product_few<FP8, GATED, OUT8, LOW, NB, KS, CS>), dim3(grid), dim3(F::threads), 0, st, a);
    return launched();
}

// A launch whose dynamic LDS exceeds 64 KiB; the kernel is told once per device.
template <bool FP8, bool GATED, bool OUT8, bool LOW>
int launch_many(const ProductPlan &p, ProductArgs a, hipStream_t st)
{
    typedef Many<Low, FP8, GATED, OUT8, LOW> M;
    constexpr int lds = std::max(Low::ST * M::stage_bytes, Tall::ST * Tall::scales);
    static_assert(Low::threads == Tall::threads, "one launch");
    a.ntiles = (p.n + M::BN - 1) / M::BN;
    static std::atomic<uint64_t> told{0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 1;
    if (!(told.load() >> dev & 1)) {
        if (hipFuncSetAttribute(reinterpret_cast<const void *>(&k_product_many<FP8, GATED, OUT8, LOW>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
            return 1;
        told.fetch_or(uint64_t(1) << dev);
    }
    const unsigned grid = persistent_grid(tile_bound(p.E, p.rows, Low::rows), a.ntiles, kComputeUnits);
    hipLaunchKernelGGL((k_product_many<FP8, GATED, OUT8, LOW>), dim3(grid), dim3(Low::threads), lds, st, a);
    return launched();
}

// The tiled product runs from this many expected rows per expert on (rows_of_expert),
// unless the few-row kernel's items fit side by side.
// 64 experts, H 2048, inner 768, network, us few and tiled: BF16 with 1 row each 79 and
// 97, 2 96 and 102, 4 108 and 108, 8 113 and 109, 32 162 and 115, 64 221 and 124; FP8 59
// and 61, 66 and 63, 69 and 66, 71 and 67, 100 and 74, 131 and 80.  With adapters (32 of
// rank 16) the few-row kernel's wavefronts share a tile's adapters: BF16 with 16 rows 188
// and 199, 24 235 and 228, 32 304 and 252, 64 413 and 296; FP8 161 and 166, 191 and 193,
// 239 and 213, 323 and 264.
constexpr int kManyFrom = 4, kManyFromLow = 24;

// Items of the few-row kernel, per CU, that run side by side.  Up to there the tiled
// product, whose larger tiles occupy few CUs, waits longer for each tile's chain of
// steps than the few-row kernel for reading rows and weights again.
// K 2048, N 768 gated, BF16 (items: few, tiled, us): 432: 13.2, 30.0; 1584: 32.3,
// 46.8; 2304: 31.2, 23.9.  K 768, N 2048: 1280: 11.4, 16.0; 2304: 19.8, 16.6; FP8 640:
// 7.9, 12.8; 1152: 13.0, 13.3; 1536: 13.2, 10.7; FP8 output (eight wavefronts for 256
// weight rows) 240: 35.3, 41.7; 408: 38.0, 24.9.
template <bool FP8, bool OUT8>
constexpr int kSideBySide = OUT8 ? 1 : FP8 ? 4 : 8;

template <bool FP8, bool GATED, bool OUT8, bool LOW, int NB, int KS, int CS>
int launch_either(const ProductPlan &p, const ProductArgs &a, hipStream_t st)
{
    typedef Few<FP8, GATED, OUT8, LOW, NB, KS, CS> F;
    const int64_t items = tile_bound(p.E, p.live, F::rows) * ((p.n + F::BN - 1) / F::BN);
    if (p.each >= (LOW ? kManyFromLow : kManyFrom) && items > kComputeUnits * kSideBySide<FP8, OUT8>)
        return launch_many<FP8, GATED, OUT8, LOW>(p, a, st);
    return launch_few<FP8, GATED, OUT8, LOW, NB, KS, CS>(p, a, st);
}

template <bool LOW>
int launch_product(const ProductPlan &p, const ProductArgs &a, hipStream_t st)
{
    // Few rows: workgroups of four wavefronts leave the most loads in flight per CU: 32
    // weight rows (BF16; 64 take 133 us instead of 129 for 1024 rows over 64
    // experts, H 2048, inner 768) or 64 (FP8: 32 take 35 us instead of 32 for the
    // second product).  An FP8 output needs 256 weight rows, one scale block.
    if (!p.fp8)
        return p.gated ? launch_either<false, true, false, LOW, 2, 4, 1>(p, a, st)
                       : launch_either<false, false, false, LOW, 2, 4, 1>(p, a, st);
    if (p.out8) return launch_either<true, true, true, LOW, 4, 2, 4>(p, a, st);
    return p.gated ? launch_either<true, true, false, LOW, 4, 4, 1>(p, a, st)
                   : launch_either<true, false, false, LOW, 4, 4, 1>(p, a, st);
}

}  // namespace

int be_launch_product(const ProductPlan &p, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (p.nad > 0) {
        ShrinkArgs s{};
        s.x = static_cast<const uint8_t *>(p.x);
        s.xs = p.xs;
        s.ends = p.ends;
        s.tags = p.tags;
        s.a = static_cast<const uint8_t *>(p.w.a);
        s.scaling = p.w.scaling;
        s.t = p.t;
        s.rows = int(p.rows);
        s.E = p.E;
        s.alpha = p.alpha;
        s.k = p.k;
        s.c = p.rank * (p.gated ? 2 : 1);
        s.nad = p.nad;
        // about eight workgroups per CU, all resident at once; no more per expert
        // than it can have pairs of an adapter and 32 rows of A
        const int pairs = std::min(p.nad, int(std::min<int64_t>(p.rows, AFD_MAX_ADAPTERS))) * ((s.c + 31) / 32);
        s.share = std::max(1, std::min(kComputeUnits * 8 / p.E, pairs));
        s.spread = std::min(p.E, 8);
        const unsigned grid = unsigned((p.E + s.spread - 1) / s.spread * s.spread * s.share);
        if (p.fp8) hipLaunchKernelGGL(k_shrink<true>, dim3(grid), dim3(Shrink<true>::threads), 0, st, s);
        else hipLaunchKernelGGL(k_shrink<false>, dim3(grid), dim3(Shrink<false>::threads), 0, st, s);
        if (launched() != 0) return 1;
    }
    ProductArgs a{};
    a.x = static_cast<const uint8_t *>(p.x);
    a.w = static_cast<const uint8_t *>(p.w.w);
    a.xs = p.xs;
    a.ws = p.w.w_scales;
    a.ends = p.ends;
    a.tags = p.tags;
    a.t = p.t;
    a.b = static_cast<const uint8_t *>(p.w.b);
    a.out = p.out;
    a.outs = p.outs;
    a.rows = int(p.rows);
    a.E = p.E;
    a.alpha = p.alpha;
    a.n = p.n;
    a.m = p.n * (p.gated ? 2 : 1);
    a.kb = p.k * (p.fp8 ? 1 : 2);
    a.packed = p.packed;
    a.wstep = p.packed ? 2048 : 128;
    a.nad = p.nad;
    a.rank = p.rank;
    return p.nad > 0 ? launch_product<true>(p, a, st) : launch_product<false>(p, a, st);
}

int be_launch_pack(const void *w, void *out, int64_t rows, int64_t row_bytes, void *stream)
{
    PackArgs a{static_cast<const u32x4 *>(w), static_cast<u32x4 *>(out), rows * row_bytes / 16, int(row_bytes / 16)};
    const int64_t blocks = std::min<int64_t>((a.n + 255) / 256, kComputeUnits * 32);
    hipLaunchKernelGGL(k_pack, dim3(unsigned(blocks)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return launched();
}

int be_launch_tags(const RoundPlan &p, int f, const int32_t *const *tags, int32_t *out, void *stream)
{
    TagArgs a{};
    a.slot = p.slot;
    a.out = out;
    for (int s = 0; s < p.N; ++s) {
        a.tags[s] = tags[s];
        a.off[s] = p.tok_off[s];
    }
    a.n = p.ntok * p.K;
    a.K = p.K;
    a.N = p.N;
    a.f = f;
    hipLaunchKernelGGL(k_tags, dim3(unsigned((a.n + 255) / 256)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return launched();
}

}  // namespace afd
