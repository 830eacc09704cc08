// afd_plan.h -- host-side plan of one round, shared by the host core and the
// backends (the HIP executor, or the recording backend used by CPU tests).
// Plain C++17; no HIP types.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "../../include/afd.h"

namespace afd {

constexpr int kMaxSources = AFD_MAX_SOURCES;
constexpr int kMaxParts = AFD_MAX_PARTITIONS;
constexpr int kMaxExperts = AFD_MAX_EXPERTS;
constexpr int kMaxTopk = AFD_MAX_TOPK;

// Tokens handled by one workgroup of the layout kernel: 1, 2 or 4
// wavefronts of 64 lanes, one token per lane (a wavefront's 64 tokens form
// one chunk).
constexpr int kLayoutTileMin = 64;
constexpr int kLayoutTile = 256;
// Tile counts of an expert the scatter requests at entry (beyond this many
// tiles it sums them in a loop), and the number of tile records the layout
// kernel's arguments carry (rounds with more tiles find each tile's source
// from the source offsets instead).
constexpr int kLayoutMaxTiles = 32;
// Small rounds rebuild the layout inside every scatter workgroup (one kernel
// for the whole dispatch): at most this many tokens, ids (staged in LDS) and
// experts, and rows of at most this many 16-byte columns.
constexpr int kFusedMaxTokens = 512;
constexpr int kFusedMaxIds = 4096;
constexpr int kFusedMaxExperts = 256;
constexpr int kFusedMaxCols = 2048;

// Sticky route-error word: (s << 56) | (t << 24) | (k << 16) | code, so the
// numeric minimum is the first offender in (source, token, k) order.
constexpr uint64_t kNoError = ~0ull;

// The workspace's first 256 bytes: the route-error word at 0, and the
// one-launch dispatch's words (uint32) at byte 64: launch counter at index
// 0, finished workgroup groups at 16, the sticky gave-up flag at 32.
constexpr size_t kSyncOffset = 64;
constexpr int kSyncDone = 16;
constexpr int kSyncStall = 32;
constexpr int kDefaultWaitPolls = 1000000;
// The one-launch dispatch's ready flag, in this many copies one 128-byte
// line apart, so that the scatter workgroups' polls spread over many lines
// instead of all reading one word.
constexpr int kReadyCopies = 64;
constexpr int kReadyStride = 32;   // uint32 words between copies (and between group counters)
// Finished workgroups of a one-launch dispatch are counted in this many
// group counters (workgroup b in group b % kDoneGroups), each on a line of
// its own after the flag copies; the last of a group counts the group in
// the workspace's finished-group word.
constexpr int kDoneGroups = 16;
// Experts of a round the one-launch dispatch takes (its hand-off reads four
// experts' words per lane of one wavefront).
constexpr int kMaxExpertsOneLaunch = 256;

// Largest combine output (bytes) written with streaming stores.
constexpr int64_t kCombineStreamOutBytes = int64_t(4) << 20;

// Words between consecutive tiles' runs of the one-launch dispatch's tile
// counts (tile-major, each run on whole 128-byte lines).
#ifdef __HIPCC__
__host__ __device__
#endif
inline int tcount_pitch(int E) { return (E + 31) / 32 * 32; }

inline int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// Larger rounds place every source on a tile boundary of a "tiled" token
// space: source s occupies slots [voff[s], voff[s] + T[s]), and the slots up
// to the next boundary are empty.  Every layout tile, and every scatter
// workgroup inside it, then holds the tokens of a single source, whose
// record a kernel reads once.  The tile is the smallest of 64, 128 and 256
// tokens that keeps the round within kLayoutMaxTiles tiles, so mid-size
// rounds spread their layout over more workgroups.  Returns the tile.
inline int place_sources(const int *T, int N, int *voff)
{
    for (int tile = kLayoutTileMin;; tile *= 2) {
        voff[0] = 0;
        for (int s = 0; s < N; ++s) voff[s + 1] = voff[s] + int(align_up(T[s], tile));
        if (tile == kLayoutTile || voff[N] / tile <= kLayoutMaxTiles) return tile;
    }
}

// Bytes of one stage-one row of the per-stage combine: BF16 [H], or H E4M3
// codes followed by H/128 scale bytes, padded to a multiple of 32.
inline int64_t partial_row_bytes(int combine, int H)
{
    return combine == AFD_COMBINE_PER_STAGE_FP8 ? H + align_up(H / 128, 32) : int64_t(H) * 2;
}

// Byte offsets of the workspace regions (each 256-byte aligned).
struct WorkspacePlan {
    size_t err = 0;        // uint64 sticky route-error word
    size_t ends = 0;       // int32 [E]
    size_t blkcnt = 0;     // int32 [E][pitch] live choices per layout tile (expert-major;
                           // pitch = tiles rounded up to 4)
    size_t packed = 0;     // int32 [N*capacity*K] (expert << 16 | rank in tile), -1 skipped
    size_t slot = 0;       // int32x2 [N*capacity*K] {part << 24 | row, weight bits}, then 64
                           // bytes of slack (the combine reads slots 64 bytes at a time)
    size_t inbox = 0;      // BF16 [N][capacity][H] (one partition only)
    size_t partials = 0;   // per-stage combine: [F][N][capacity] rows of partial_row_bytes
    size_t tcount = 0;     // one-launch dispatch: uint32 [kLayoutMaxTiles][tcount_pitch(E)] tagged tile counts,
                           // then uint64 [kLayoutMaxTiles + 1][tcount_pitch(E)] tagged first rows per tile and
                           // expert, and the ends
    size_t ready = 0;      // one-launch dispatch: uint32 ready flag, kReadyCopies copies kReadyStride apart,
                           // then kDoneGroups finished-workgroup counters at the same stride
    size_t total = 0;
    int nblk_max = 0;
};

// Everything a backend needs to run one round; pointers are device
// addresses recorded from the caller.
struct RoundPlan {
    // configuration
    int N = 0, F = 0, E = 0, E_loc = 0, K = 0, H = 0, alpha = 1, fp8 = 0, capacity = 0;
    int combine = AFD_COMBINE_ONCE;
    int64_t prow = 0;        // per-stage combine: bytes of one partial row
    int64_t row_bytes = 0;   // H * bytes per activation
    int G = 0;               // H / 128 scale blocks per row
    // tokens, concatenated over sources in order
    int ntok = 0;
    int tok_off[kMaxSources + 1] = {};
    bool fused = false;      // one-kernel dispatch
    bool empty = false;      // no tokens: the dispatch only clears ends[]
    bool onepass = false;    // one-launch dispatch (counting and scatter in one kernel)
    bool cached = false;     // scatter from the slot map of the last layout
    int nblk = 0;            // layout tiles (split path)
    int tile = 0;            // tokens per layout tile
    int voff[kMaxSources + 1] = {};   // first tiled slot of each source (voff[N]: slots)
    // per source
    const void *x[kMaxSources] = {};
    const int32_t *ids[kMaxSources] = {};
    const float *w[kMaxSources] = {};
    const float *scale[kMaxSources] = {};
    int64_t sst[kMaxSources] = {}, ssg[kMaxSources] = {};
    void *out[kMaxSources] = {};       // combine destination (out_bf16 or inbox)
    // per partition
    void *rows[kMaxParts] = {};
    float *scales[kMaxParts] = {};
    float *roww[kMaxParts] = {};
    const void *reply[kMaxParts] = {};
    // workspace
    uint64_t *err = nullptr;
    int32_t *ends = nullptr;
    int32_t *blkcnt = nullptr;
    int32_t *packed = nullptr;
    int32_t *slot = nullptr;
    // per-stage combine: row (f, s, t) at partials + ((f * N + s) * capacity + t) * prow
    uint8_t *partials = nullptr;
    // one-launch dispatch
    uint32_t *tcount = nullptr;   // [kLayoutMaxTiles][tcount_pitch(E)]
    uint32_t *ready = nullptr;    // [(kReadyCopies + kDoneGroups) * kReadyStride]
    uint32_t *sync = nullptr;     // launch counter, finished workgroups, gave-up flag
    int wait_polls = kDefaultWaitPolls;
};

// Layout tile records of a round of at most kLayoutMaxTiles tiles: tile b
// holds tokens t0 .. t0 + n - 1 of source src, the first of them token g0 of
// the round.  The layout kernel reads its tile's record instead of finding
// its source.  Returns the number of records; 0 when no layout kernel runs
// (one-kernel or cached dispatch) or the round has more tiles.
struct TileRec {
    int src, t0, n, g0;
};

inline int layout_tiles(const RoundPlan &p, TileRec *out)
{
    if (p.fused || p.cached || p.empty || p.nblk > kLayoutMaxTiles) return 0;
    for (int b = 0; b < p.nblk; ++b) {
        int s = 0;   // the last source whose span starts at or before the tile (empty spans are skipped)
        while (s + 1 < p.N && b * p.tile >= p.voff[s + 1]) ++s;
        const int t0 = b * p.tile - p.voff[s];
        const int T = p.tok_off[s + 1] - p.tok_off[s];
        out[b] = TileRec{s, t0, T - t0 < p.tile ? T - t0 : p.tile, p.tok_off[s] + t0};
    }
    return p.nblk;
}

// Rows that an expert is expected to have, which the kernel is chosen by: what the caller
// says, no more than rows has room for; or else half of the rows' bound without what
// alignment alone can add (the bound counts every choice for this partition).
inline int rows_of_expert(const afd_product_config &c, int64_t rows)
{
    const int64_t E = c.num_experts;
    if (c.rows_per_expert > 0) return int(std::min<int64_t>(c.rows_per_expert, (rows + E - 1) / E));
    return int(std::max<int64_t>((rows - E * (c.alignment - 1)) / E / 2, 0));
}

// One grouped product (and its adapters' first halves); pointers are device
// addresses recorded from the caller.
struct ProductPlan {
    int E = 0, alpha = 1, k = 0, n = 0;
    bool fp8 = false, out8 = false, gated = false, packed = false;
    int nad = 0, rank = 0;           // adapters (0: none) and their rank
    int64_t rows = 0;
    int each = 0;                    // rows that an expert is expected to have (rows_of_expert)
    int64_t live = 0;                // and all experts together; rows where nobody says
    const void *x = nullptr;
    const float *xs = nullptr;
    const int32_t *ends = nullptr;
    const int32_t *tags = nullptr;   // [rows] adapter of every row
    afd_product_weights w{};
    void *out = nullptr;
    float *outs = nullptr;
    uint16_t *t = nullptr;           // [rows][2][(gated ? 2 : 1) * rank] two bf16 parts of every row's scaling * A x
};

// Where the tiled product's next load stands: step u of its item `at` (the workgroup's
// are at, at + step, .. below end), of nu steps each.  Loads run ahead of the arithmetic,
// and their number is the same for every step; behind the last item they go on without
// a byte (an empty buffer) and at step 0: a step's scalar offset may be no larger than its
// buffer, because the hardware's range check is given as offset >= size - scalar offset.
struct LoadCursor {
    int at, u;
    bool live;   // false: behind the last item
    // To the next step; true if another item begins, or the last one has ended.
    constexpr bool advance(int nu, int end, int step)
    {
        if (!live || ++u < nu) return false;
        u = 0;
        live = at + step < end;
        if (live) at += step;
        return true;
    }
};

// ---- the source's side: norms, routes, the balance loss ----

struct NormPlan {
    int H = 0;
    bool x32 = false, r32 = false, res = false, w32 = false, out8 = false;
    float eps = 0.f;
    int64_t rows = 0;
    const void *x = nullptr, *r = nullptr, *w = nullptr;
    int64_t xs = 0, rs = 0, hs = 0;   // row strides (elements) of x, the residual and h
    void *out = nullptr, *h = nullptr;
    float *outs = nullptr, *rstd = nullptr;
};

// Workgroups of the norm's gradient: each sums dweight over its rows in registers and
// leaves one partial row of float32, and a second launch adds these up.  Few rows (0 here)
// take one launch, in which other workgroups read them again for dweight (us, one and two
// launches, BF16: 2048 columns, 512 rows 4.0 and 7.3, 1024 6.4 and 9.0, 2048 14.8 and 12.2;
// 8192, 1024 rows 15.9 and 18.8, 1500 24.8 and 21.1; 16384, 512 rows 18.3 and 18.4, 700 22.9
// and 21.1).
constexpr int kNormGradGroups = 512;
inline int norm_grad_groups(int64_t rows, int H)
{
    return rows <= (H <= 8192 ? 1024 : 512) ? 0 : int(std::min<int64_t>((rows + 3) / 4, kNormGradGroups));
}

struct NormGradPlan {
    int H = 0;
    bool h32 = false, w32 = false;
    int64_t rows = 0, hs = 0;
    const void *g = nullptr, *gr = nullptr, *h = nullptr, *w = nullptr;
    const float *rstd = nullptr;
    void *dh = nullptr;
    float *dw = nullptr, *part = nullptr;   // part: [groups][H]
    int groups = 0;
};

struct RoutePlan {
    int E = 0, K = 0;
    bool l32 = false, sigmoid = false, renorm = false;
    float scale = 1.f;
    int64_t rows = 0, ls = 0;
    const void *l = nullptr;
    const float *bias = nullptr;
    const uint8_t *live = nullptr;
    int32_t *ids = nullptr;
    float *w = nullptr;
    const float *g = nullptr;      // the gradient calls': of the weights, or of the loss
    const float *slope = nullptr;  // (balance)
    void *dl = nullptr;
};

// Lanes that hold a token's logits.
inline int lanes_of(int E) { return E <= 128 ? 16 : E <= 256 ? 32 : 64; }

// Workgroups of the balance loss's first launch: each leaves its sums of the shares, its
// counts, and its numbers of counting tokens and of choices.  Few tokens are one
// workgroup's of 1024 threads, which has the results without a second launch, up to six
// turns of it (384 tokens of 128 experts).  The eager call, which the host bounds, takes 10 us
// instead of 14 by it.  A captured one, in us: one turn to six 3.9, 4.9, 6.0, 7.0, 8.1 and 9.2
// with up to 128 experts, where two launches take 7.1 to 7.6 (512 experts: four turns 7.3, two
// launches 10.3): turns five and six cost it 1 to 2, less than they save the eager one.
constexpr int kBalanceGroups = 256;
constexpr int kBalanceSolo = 6;
inline int balance_groups(int64_t rows, int E)
{
    const int64_t each = 256 / lanes_of(E);
    if (rows > 0 && rows <= kBalanceSolo * 4 * each) return 1;
    return int(std::min<int64_t>((rows + each - 1) / each, kBalanceGroups));
}
// Workgroups of 1024 threads instead of 256 where those would take more than two turns (us, 256
// and 1024 threads: 128 experts, 8192 tokens 9.1 and 9.1, 16384 10.4 and 9.2; 512 experts,
// 2048 tokens 11.9 and 12.1, 4096 13.2 and 12.5, 32768 30.5 and 21.6).
inline bool balance_wide(int64_t rows, int E) { return rows > int64_t(2) * kBalanceGroups * (256 / lanes_of(E)); }

struct BalancePlan {
    RoutePlan r;
    float coefficient = 1.f;
    float *loss = nullptr;
    int32_t *counts = nullptr;
    float *slope = nullptr;
    int groups = 0;
    bool wide = false;
    float *share = nullptr;       // [groups][E]
    int32_t *count = nullptr;     // [groups][E]
    int32_t *totals = nullptr;    // [groups][2] counting tokens, choices
    double *part = nullptr;       // [(E + 15) / 16] of the loss
    uint32_t *done = nullptr;     // workgroups of the second launch that have left theirs
};

// Contexts made by afd_create_static use a static scratch array of this many
// bytes per GPU as their workspace (one such context per device at a time).
constexpr size_t kStaticScratchBytes = size_t(AFD_STATIC_SCRATCH_BYTES);
constexpr int kMaxDevices = 64;

// ---- backend: implemented by the HIP executor or the recording fake ----
// Each returns 0 on success, nonzero on a runtime failure.
int be_init_workspace(void *workspace, const WorkspacePlan &wp);
int be_is_capturing(void *stream, int *capturing);
int be_launch_dispatch(const RoundPlan &p, void *stream);
int be_read_ends(const RoundPlan &p, void *stream, int32_t *host_ends, uint64_t *err_word);
int be_launch_combine(const RoundPlan &p, void *stream);
int be_launch_partial(const RoundPlan &p, int f, void *stream);   // per-stage combine, stage one
int be_launch_last(const RoundPlan &p, int f, void *stream);      // per-stage: the last reply's stage one + stage two
int be_launch_copy(const void *src, void *dst, int64_t bytes, void *stream);
int be_read_error(uint64_t *dev_err, void *stream, int clear, uint64_t *word);
// The one-launch dispatch's gave-up flag (and clears it when asked).
int be_read_stall(uint32_t *dev_sync, void *stream, int clear, int *stalled);
// A grouped product: with adapters a launch for A x, then the product.
int be_launch_product(const ProductPlan &p, void *stream);
// Row-major weight rows (of all experts) into the packed order.
int be_launch_pack(const void *w, void *out, int64_t rows, int64_t row_bytes, void *stream);
// tags[s][t] to the receive rows of partition f, from the round's slot map.
int be_launch_tags(const RoundPlan &p, int f, const int32_t *const *tags, int32_t *out, void *stream);
// The source's side.
int be_launch_norm(const NormPlan &p, void *stream);
int be_launch_norm_grad(const NormGradPlan &p, void *stream);
int be_launch_route(const RoutePlan &p, void *stream);
int be_launch_route_grad(const RoutePlan &p, void *stream);
int be_launch_balance(const BalancePlan &p, void *stream);
int be_launch_balance_grad(const RoutePlan &p, void *stream);
int be_device_sync();
// The current device and the address of its static scratch array (found
// once per device); no allocation.
int be_static_scratch(int *device, void **ptr);
// Initialise a static scratch workspace (the error word) with a kernel on
// the null stream and wait for it; no allocation, no host-to-device copy.
int be_init_static(void *workspace, const WorkspacePlan &wp);

}  // namespace afd
