// How the scaled and gated products and the gradients are cut into units of work: tile widths, parts of
// the reductions, which kernel takes a call, and which unit a CTA pair or a cluster does when. Plain
// arithmetic on sizes, the same on host and device; it includes nothing of CUDA, so that the CPU
// tests compile it and walk through every unit.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstddef>

#ifdef __CUDACC__
#define QG_PLAN_FN __host__ __device__ __forceinline__
#else
#define QG_PLAN_FN inline
#endif

namespace qg {

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tile width and parts of the reductions of a launch of gradient tiles; us: estimate for a B200
struct GradTiles {
    int bn, parts_x, parts_w;
    double us;
};
// How the gradients are computed: by the sizes alone, not by what is asked for, so that dX or the
// weights' gradients by themselves are those of the whole call, bit for bit.
struct GradPlan {
    bool few;               // dX by the few-token kernel, only the weights' gradients by tiles
    bool together;          // tiles of dX and of the weights' gradients in one launch
    GradTiles x, w;
};

// ------------------------------------------------------------------------------------------
// Large tiles (ffn_tile.cu)
// ------------------------------------------------------------------------------------------
namespace tile {

enum Form { kScaled, kGated, kDx, kDw, kBoth };

constexpr int kTileM = 256;                    // rows of the result of a CTA pair
constexpr int kMaxBn = 256;
constexpr int kRasterM = 8;                    // row tiles per raster group (4, 16: no faster)

// One product of a launch (gradients: dX, and the two weights' gradients together)
struct Work {
    int M, tiles_m;         // the result's rows, and tiles of them
    int slabs;              // slabs of the reduction
    int parts, part_slabs;  // parts of the reduction and slabs of each (the last may have fewer)
    int units;              // results x tiles x parts; 0: not computed
};

struct Shape {
    int N, tiles_n;         // the result's columns (of H for kGated)
    int bn;                 // the MMA's N: columns of a tile (kGated: of gate and up together)
    int seg_slabs;          // slabs of one of dX's two products
    int act;
    Work x, w;              // the product, or dX; the weights' gradients
    int full, rem;          // units of x: `full` a pair, one more for the first `rem` pairs
    int extra;              // tiles of w that pairs with one tile of x less take for it, first of all
};

struct Unit {
    int which, m0, n0, part, s0, ns;    // result, origin of the tile, part, first slab, slabs
};

// Tiles in groups of kRasterM row tiles, rows fastest: the pairs at work at one time share a block
// of about kRasterM x 9 tiles whose operands stay in L2.
QG_PLAN_FN Unit unit_of(int u, const Work &k, int tiles_n, int ncol)
{
    Unit w;
    w.part = u % k.parts;
    int t = u / k.parts;
    const int per = k.tiles_m * tiles_n;
    w.which = t / per;
    t -= w.which * per;
    const int group = t / (kRasterM * tiles_n);
    const int first = group * kRasterM;
    const int gm = k.tiles_m - first < kRasterM ? k.tiles_m - first : kRasterM;
    t -= group * kRasterM * tiles_n;
    w.m0 = (first + t % gm) * kTileM;
    w.n0 = (t / gm) * ncol;
    w.s0 = w.part * k.part_slabs;
    w.ns = k.slabs - w.s0 < k.part_slabs ? k.slabs - w.s0 : k.part_slabs;
    return w;
}

// The j-th unit of a pair out of `pairs`, in *w; false behind its last one.
template <int FORM>
QG_PLAN_FN bool unit_at(int j, int pairs, int pair, const Shape &s, int ncol, Unit *w)
{
    const int u = j * pairs + pair;
    if (FORM != kDw && u < s.x.units) {
        *w = unit_of(u, s.x, s.tiles_n, ncol);
        return true;
    }
    if constexpr (FORM != kDw && FORM != kBoth) return false;
    // The weights' units go on where x's end, at the pairs that have one of x less; or `extra` rounds
    // over those pairs alone, then rounds over all.
    int v = u - s.x.units;
    if (s.extra > 0) {
        const int i = j - s.full - (pair < s.rem ? 1 : 0), lacking = pairs - s.rem;
        if (pair < s.rem) v = i * pairs + pair + s.extra * lacking;
        else if (i < s.extra) v = i * lacking + pair - s.rem;
        else v = (i - s.extra) * pairs + pair + s.extra * lacking;
    }
    if (v >= s.w.units) return false;
    *w = unit_of(v, s.w, s.tiles_n, ncol);
    w->which += 1;
    return true;
}

// Tiles of w that a pair takes in place of its missing last tile of x
inline int extra_tiles(const Work &x, const Work &w, int pairs)
{
    const int rem = x.units % pairs;
    if (rem == 0 || w.units == 0) return 0;
    const int fit = (x.part_slabs + w.part_slabs / 2) / w.part_slabs;
    return std::min(fit, w.units / (pairs - rem));
}

// How the units of x and w are shared out over the pairs
inline void share_units(Shape *s, int pairs)
{
    s->full = s->x.units / pairs;
    s->rem = s->x.units % pairs;
    s->extra = extra_tiles(s->x, s->w, pairs);
}

// Widths that the MMA of a pair takes: multiples of 32 for int8 and of 16 for 16-bit types. The
// gradients' MN-major operands come in whole chunks of 64 values a CTA: 128 or 256 columns.
constexpr int kStepI8 = 32, kStep16 = 16;
constexpr int kPairs = 74;             // of a B200
constexpr int kMaxParts = 16;

inline Work work_of(int M, int N, int ncol, int results, int slabs, int parts)
{
    Work k = {};
    k.M = M;
    k.tiles_m = ceil_div(M, kTileM);
    k.slabs = slabs;
    k.part_slabs = ceil_div(slabs, parts);
    k.parts = ceil_div(slabs, k.part_slabs);        // no empty part
    const long long units = (long long)results * k.tiles_m * ceil_div(N, ncol) * k.parts;
    k.units = units > 0x7fffffffLL ? -1 : (int)units;
    return k;
}

// Estimate of a slab in a wave that fills the device, nearly whatever the width (the 256-row operand
// passes through the MMA either way, and L2 delivers little more than 90 GB/s to an SM): 0.34 us at
// 256 columns, 0.32 at 128. Measured between reductions of 4096 and 8192 int8 values: 0.33 us at 256
// columns (72 tiles), 0.29 at 128 (64 tiles); between 8192 and 16384, with the clock lower: 0.35 and
// 0.33.
inline double slab_us(int bn) { return 0.34 * (0.88 + 0.12 * bn / kMaxBn); }

struct Plan {
    int bn;
    double us;                         // estimate for a B200
};

// Tile width of the scaled and gated products: whole waves of tiles over the CTA pairs. Fewest
// waves win, and among them the narrower tile, whose epilogue is shorter: 2 x 43 tiles of 256
// columns on 74 pairs, say, leave most of a second wave idle; 2 x 69 tiles of 160 take the same two
// waves 15 % faster (509 x 11007 x 4080: 38.3 -> 32.4 us). The estimate is for comparisons: it leaves
// out rows that are not 16-byte aligned and 3 us of the first loads and the last epilogue (24 us for
// that call, 16.7 measured for 14.4 estimated at 2048 x 2304 x 4096).
inline Plan plan_tiles(int M, int N, bool gated, int step, int slabs)
{
    const long long tm = ceil_div(M, kTileM);
    Plan best{kMaxBn, 1e30};
    for (int bn = kMaxBn; bn >= 64; bn -= step) {
        const long long units = tm * ceil_div(N, gated ? bn / 2 : bn);
        const double us = 3.5 + (double)((units + kPairs - 1) / kPairs) * slabs * slab_us(bn);
        if (us < best.us - 1e-9) best = Plan{bn, us};
    }
    return best;
}

inline Shape shape_of(int M, int N, int bn, int ncol, int slabs, int act)
{
    Shape s = {};
    s.N = N;
    s.tiles_n = ceil_div(N, ncol);
    s.bn = bn;
    s.act = act;
    s.x = work_of(M, N, ncol, 1, slabs, 1);
    return s;
}

// Tile width and parts of the gradients of one launch. Parts cost their fp32 sums' way to memory and
// back and a second kernel; they are tried while the pairs have at most two tiles each. Both products
// in one launch count a tenth more a slab: 3 to 8 % that theirs take longer, and a margin. Joined
// against two launches, us, where the estimates choose two: 2843 x 1357 x 3888 134 against 128,
// 2048 x 11008 x 4096 611 against 597, 2048 x 2048 x 2048 59.5 against 60.2, 512 x 11008 x 512 49
// against 52; where they choose one: 3000 x 1500 x 696 33.1 against 48.8, 1024 x 4096 x 2048 63
// against 68, 300 x 4096 x 512 26.7 against 28.3.
inline GradTiles grad_tiles(int M, int F, int K, bool dx, bool dw)
{
    const int slabs_x = 2 * ceil_div(F, 64), slabs_w = ceil_div(M, 64);
    const int most = dx && dw ? 2 * kPairs : kPairs * 3 / 2;     // units: 256 KB of sums each
    GradTiles best{kMaxBn, 1, 1, 1e30};
    for (int bn = kMaxBn; bn >= kMaxBn / 2; bn /= 2) {
        const Work x1 = work_of(M, K, bn, 1, slabs_x, 1), w1 = work_of(F, K, bn, 2, slabs_w, 1);
        if (x1.units < 0 || w1.units < 0) continue;
        auto consider = [&](int px, int pw) {
            // parts keep eight slabs
            if ((px > 1 && slabs_x < 8 * px) || (pw > 1 && slabs_w < 8 * pw)) return;
            const long long units =
                (dx ? (long long)x1.units * px : 0) + (dw ? (long long)w1.units * pw : 0);
            if ((px > 1 || pw > 1) && units > most) return;
            const Work x = dx ? (px > 1 ? work_of(M, K, bn, 1, slabs_x, px) : x1) : Work{};
            const Work w = dw ? (pw > 1 ? work_of(F, K, bn, 2, slabs_w, pw) : w1) : Work{};
            const int pairs = (int)std::min<long long>((long long)x.units + w.units, kPairs);
            const int full = x.units / pairs, rem = x.units % pairs;
            const int extra = extra_tiles(x, w, pairs);
            long long slabs = (long long)full * x.part_slabs;
            if (rem > 0) slabs += std::max(x.part_slabs, extra * w.part_slabs);
            const int left = w.units - (rem > 0 ? extra * (pairs - rem) : 0);
            slabs += (long long)ceil_div(left, pairs) * w.part_slabs;
            double us = 3.5 + slabs * slab_us(bn) * (dx && dw ? 1.10 : 1.0);
            if (x.parts > 1) us += 2.5 + (double)M * K * 8 * x.parts / 5e6;
            if (w.parts > 1) us += 2.5 + (double)2 * F * K * 8 * w.parts / 5e6;
            if (us < best.us - 1e-9)
                best = GradTiles{bn, std::max(1, x.parts), std::max(1, w.parts), us};
        };
        consider(1, 1);
        const long long least =
            std::min(dx ? x1.units : 0x7fffffff, dw ? w1.units : 0x7fffffff);
        for (int parts = 2; parts <= kMaxParts && least * parts <= most; ++parts) {
            if (dx) consider(parts, 1);
            if (dw) consider(1, parts);
            if (dx && dw) consider(parts, parts);
        }
    }
    return best;
}

inline Shape grad_shape(const GradTiles &t, int M, int F, int K, bool of_x, bool of_w)
{
    Shape s = {};
    s.N = K;
    s.bn = t.bn;
    s.tiles_n = ceil_div(K, t.bn);
    s.seg_slabs = ceil_div(F, 64);
    if (of_x) s.x = work_of(M, K, t.bn, 1, 2 * s.seg_slabs, t.parts_x);
    if (of_w) s.w = work_of(F, K, t.bn, 2, ceil_div(M, 64), t.parts_w);
    return s;
}

} // namespace tile

// ------------------------------------------------------------------------------------------
// Few tokens (ffn_small.cu)
// ------------------------------------------------------------------------------------------
namespace few {

enum Form { kScaled, kGated, kDx };

constexpr int kTokens = 128, kSlab = 128, kMmaM = 128;
constexpr int kWeightMajor = 64;       // up to so many tokens the weights are the MMA's M side
constexpr int kRingBytes = 108 * 1024;
constexpr int kMaxStages = 16;

struct Shape {
    int M, N;               // tokens; columns of the result
    int cols;               // result columns of a tile, a multiple of 4
    int second;             // first row of up in a slab, a multiple of 8 (kGated)
    int used;               // weight rows in a slab that reach a result
    int slab_rows;          // weight rows in a slab, a multiple of 8
    int box_tokens;         // token rows in a slab, a multiple of 8
    int stages;
    int pitch;              // words a token of a partial tile: 4 x odd, no bank conflicts
    int seg_slabs, slabs;   // slabs of the reduction: of one product, of all
    int act;
};

inline int round_up(int a, int b) { return ceil_div(a, b) * b; }

// Stages of the ring: its bytes, and the whole blocks of 128 rows that the MMA reads from the last
// slab of the M side.
inline int stages_of(int used, int box, int M)
{
    const int w = round_up(used, 8) * kSlab, x = box * kSlab;
    int st = std::min(kMaxStages, kRingBytes / (w + x));
    const bool wm = M <= kWeightMajor;
    const int first = wm ? w : x, read = wm ? round_up(used, kMmaM) * kSlab : kMmaM * kSlab;
    while (st > 2 && (st - 1) * first + read > kRingBytes) --st;
    return st;
}

struct Plan {
    int cols, parts;
    double us;                // estimate for a B200
};

// Clusters of 1, 2, 4 and 8 CTAs that run at once on a B200 with one CTA an SM (larger clusters
// leave SMs of a partly filled processing cluster idle) and with two.
constexpr int kClusters[2][4] = {{148, 74, 33, 15}, {296, 148, 71, 33}};

// Columns of a tile and parts of the reduction: for every cluster size and one or two CTAs an SM,
// the columns that divide the weights evenly over the clusters that run at once (more waves of them
// if a tile's columns would not fit), by the estimated time of
//   - a slab: its MMAs with their waits (0.29 us of one CTA on an SM, 0.40 us of two CTAs together;
//     more with a second block or a wide N side), what L2 delivers to an SM (115 GB/s), or the
//     memory's 2 us over the slabs in flight;
//   - the stream: the slabs of a CTA against HBM, the two slowing each other near balance;
//   - joining: a barrier, and partial tiles through shared memory at 35 GB/s (60 GB/s unsplit).
// Times in us of columns x parts, measured over a sweep: one token, 11008 gate and up columns, 4096
// deep, 76x2: 17.1, 76x1: 17.8, 40x1: 17.8, 64x1: 19.1, 128x1: 19.4; 16 tokens in 16 bits, 76x2:
// 30.6, 40x1: 32.7, 64x1: 33.4, 76x1: 34.7; 128 tokens, 4096 columns, 128x4: 9.0, 128x8: 11.5,
// 64x2: 10.6.
inline Plan plan_small(int form, int M, int N, int slabs)
{
    const int tiles_t = ceil_div(M, kTokens), box = round_up(std::min(M, kTokens), 8);
    const int halves = form == kGated ? 2 : 1;
    const int grain = form == kDx ? 64 : 4;
    // the MMA's 256 rows; and the partial tile fits in the ring
    int most = 256 / halves / 8 * 8;
    while (most > grain && (most * halves + 8) * std::min(M, kTokens) * 4 > kRingBytes) most -= 8;
    most = std::max(grain, most / grain * grain);
    Plan best{grain, 1, 1e30};
    for (int per_sm = 1; per_sm <= 2; ++per_sm)
        for (int i = 0; i < 4; ++i) {
            const int parts = 1 << i, slots = kClusters[per_sm - 1][i];
            if (parts > 1 && slabs < 4 * parts) break;
            // even columns over the fewest whole waves
            const long long least = (long long)ceil_div(N, most) * tiles_t;
            const long long waves = (least + slots - 1) / slots;
            const long long tiles = std::max(1LL, slots * waves / tiles_t);
            const int cols = round_up((int)((N + tiles - 1) / tiles), grain);
            const long long ctas = (long long)ceil_div(N, cols) * tiles_t * parts;
            const double on_sm = std::max(1.0, std::min(2.0, std::ceil(ctas / 148.0)));
            const double rounds = std::max(1.0, ctas / ((double)kClusters[1][i] * parts));
            const int used = form == kGated ? round_up(cols, 8) + cols : cols;
            const int tokens = std::min(M, kTokens);
            const int blocks = M <= kWeightMajor ? ceil_div(used, kMmaM) : 1;
            const double mma = on_sm < 2 ? (blocks > 1 ? 0.40 : (used > 128 ? 0.35 : 0.29))
                                         : (blocks > 1 ? 0.50 : 0.40 * std::max(1.0, used / 170.0));
            const double slab = std::max({mma, on_sm * (used + box) * kSlab / 115e3,
                                          2.0 / stages_of(used, box, M)});
            const double sm = ceil_div(slabs, parts) * slab * rounds;
            const double hbm = (double)slabs * kSlab * ((double)N * halves + M) / 6.4e6;
            const double stream = std::sqrt(std::sqrt(sm * sm * sm * sm + hbm * hbm * hbm * hbm));
            const double tile = on_sm * tokens * used * 4.0;
            const double join = parts > 1 ? 0.5 + 0.15 * parts + tile / 35e3 : tile / 60e3;
            const double us = 2.5 + stream + join * rounds;
            if (us < best.us) best = Plan{cols, parts, us};
        }
    return best;
}

// The slab and the partial tile of a call with `cols` columns a tile; false: they do not fit
inline bool lay_out(Shape *s, int cols, int form)
{
    s->cols = cols;
    s->second = form == kGated ? round_up(cols, 8) : 0;
    const int used = s->used = s->second + cols;
    s->box_tokens = round_up(std::min(s->M, kTokens), 8);
    s->pitch = used / 4 % 2 ? used : used + 4;
    s->slab_rows = round_up(used, 8);
    s->stages = stages_of(used, s->box_tokens, s->M);
    return std::min(s->M, kTokens) * s->pitch * 4 <= kRingBytes && used <= 256 && s->stages >= 2;
}

inline Shape shape_of(int M, int N, int seg_slabs, int segs, int act)
{
    Shape s = {};
    s.M = M;
    s.N = N;
    s.seg_slabs = seg_slabs;
    s.slabs = segs * seg_slabs;
    s.act = act;
    return s;
}

} // namespace few

// ------------------------------------------------------------------------------------------
// Which kernel: estimates in microseconds; slabs: 128-byte steps of the reduction
// ------------------------------------------------------------------------------------------
inline double tile_us(int M, int N, bool gated, bool i8, int slabs)
{
    return tile::plan_tiles(M, N, gated, i8 ? tile::kStepI8 : tile::kStep16, slabs).us;
}

inline double small_us(int M, int N, bool gated, int slabs)
{
    return few::plan_small(gated ? few::kGated : few::kScaled, M, N, slabs).us;
}

inline double small_dx_us(int M, int F, int K)
{
    return few::plan_small(few::kDx, M, K, 2 * ceil_div(F, 64)).us;
}

// Up to here the few-token kernel without asking the estimates: the weights' stream is the bound (at
// 100 tokens, 512 to 11008 columns by 2048 to 11008: 6 to 36 us against 9 to 48 us of the tiles).
constexpr int kFewTokens = 64;

inline bool few_tokens(int M, int N, bool gated, bool i8, int slabs)
{
    return M <= kFewTokens || small_us(M, N, gated, slabs) < tile_us(M, N, gated, i8, slabs);
}

inline GradPlan plan_gated_backward(int M, int F, int K)
{
    GradPlan p = {};
    p.w = tile::grad_tiles(M, F, K, false, true);
    p.few = M <= kFewTokens;
    if (p.few) return p;
    p.x = tile::grad_tiles(M, F, K, true, false);
    const GradTiles both = tile::grad_tiles(M, F, K, true, true);
    p.together = both.us < p.x.us + p.w.us;
    p.few = small_dx_us(M, F, K) + p.w.us < (p.together ? both.us : p.x.us + p.w.us);
    if (p.few) p.together = false;
    else if (p.together) p.x = p.w = both;
    return p;
}

inline size_t grad_part_bytes(const GradPlan &p, int M, int F, int K)
{
    size_t n = p.w.parts_w > 1 ? (size_t)p.w.parts_w * 2 * F * K : 0;
    if (!p.few && p.x.parts_x > 1) n += (size_t)p.x.parts_x * M * K;
    return n * 4;
}

} // namespace qg
