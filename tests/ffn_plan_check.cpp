// Walks through the units of the scaled and gated products and of the gradients, as ffn_plan.cuh
// cuts them, on the CPU. One case a line of standard input:
//   grad M F K               plan of the gradients; every unit of the whole call, of dX alone and of
//                            the weights' gradients alone
//   prod M N slabs gated i8  tiles of a forward product, by either kernel
//   sweep N SEED             N random sizes of both kinds, checked and not printed
// A line of numbers for each grad and prod; "bad ..." and status 1 for what does not add up.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <tuple>

#include "ffn_plan.cuh"

using namespace qg;

static int bad = 0;
#define CHECK(x, ...)                                                                              \
    do {                                                                                           \
        if (!(x)) {                                                                                \
            std::printf("bad %s: ", #x);                                                           \
            std::printf(__VA_ARGS__);                                                              \
            std::printf("\n");                                                                     \
            bad = 1;                                                                               \
        }                                                                                          \
    } while (0)

constexpr long long kWalk = 300000;        // units that are walked through one by one

// Every unit of one launch exactly once, inside the result and the reduction; returns the most units
// of a pair.
template <int FORM> static int walk(tile::Shape s, int ncol)
{
    const long long units = (long long)s.x.units + s.w.units;
    CHECK(s.x.units >= 0 && s.w.units >= 0 && units > 0, "units %d %d", s.x.units, s.w.units);
    if (units > kWalk) return 0;
    const int pairs = (int)std::min<long long>(units, tile::kPairs);
    tile::share_units(&s, pairs);
    std::set<std::tuple<int, int, int, int>> seen;
    int most = 0, least = 1 << 30;
    for (int pair = 0; pair < pairs; ++pair) {
        tile::Unit w;
        int j = 0;
        for (; tile::unit_at<FORM>(j, pairs, pair, s, ncol, &w); ++j) {
            const bool weights = FORM == tile::kDw || (FORM == tile::kBoth && w.which > 0);
            const tile::Work &k = weights ? s.w : s.x;
            // the kernel tells the kinds of unit apart by their place alone
            if (FORM == tile::kBoth) CHECK(weights == (j * pairs + pair >= s.x.units), "unit %d of pair %d", j, pair);
            CHECK(weights ? w.which == 1 || w.which == 2 : w.which == 0, "which %d", w.which);
            CHECK(seen.insert({w.which, w.part, w.m0, w.n0}).second, "twice: %d %d %d %d", w.which, w.part, w.m0, w.n0);
            CHECK(w.m0 >= 0 && w.m0 < k.M && w.n0 >= 0 && w.n0 < s.N, "origin %d %d", w.m0, w.n0);
            CHECK(w.part < k.parts && w.ns >= 1 && w.s0 >= 0 && w.s0 + w.ns <= k.slabs, "slabs %d + %d", w.s0, w.ns);
        }
        most = std::max(most, j);
        least = std::min(least, j);
    }
    CHECK(least > 0, "a pair without a unit");
    // no rounds of their own for the pairs that have a tile of dX less: units are dealt out evenly
    if (s.extra == 0) CHECK(most - least <= 1, "%d units for a pair, %d for another", most, least);
    CHECK((long long)seen.size() == units, "%lld units, %zu done", units, seen.size());
    return most;
}

static void few_case(int form, int M, int N, int slabs)
{
    const few::Plan plan = few::plan_small(form, M, N, slabs);
    few::Shape s = few::shape_of(M, N, form == few::kDx ? slabs / 2 : slabs, form == few::kDx ? 2 : 1, 0);
    CHECK(few::lay_out(&s, plan.cols, form), "M %d N %d slabs %d cols %d", M, N, slabs, plan.cols);
    const bool wm = M <= few::kWeightMajor;
    const int w = s.slab_rows * few::kSlab, x = s.box_tokens * few::kSlab;
    const int first = wm ? w : x, read = wm ? ceil_div(s.used, few::kMmaM) * few::kMmaM * few::kSlab : few::kMmaM * few::kSlab;
    CHECK(s.stages * (w + x) <= few::kRingBytes, "ring: %d stages of %d", s.stages, w + x);
    CHECK((s.stages - 1) * first + read <= few::kRingBytes, "M side past the ring");
    CHECK(s.cols % (form == few::kDx ? 64 : 4) == 0 && s.second % 8 == 0, "cols %d", s.cols);
    CHECK(form == few::kGated ? s.second >= s.cols : s.second == 0, "second %d", s.second);
    const int mma_n = ((wm ? s.box_tokens : s.used) + 15) / 16 * 16;
    CHECK(mma_n <= 256 && mma_n * (wm ? ceil_div(s.used, few::kMmaM) : 1) <= 256, "accumulator columns");
    // every part has a slab, and every column and token a tile
    for (int r = 0; r < plan.parts; ++r)
        CHECK((long long)s.slabs * (r + 1) / plan.parts > (long long)s.slabs * r / plan.parts, "empty part");
    CHECK((long long)ceil_div(N, s.cols) * s.cols >= N, "columns");
}

static tile::Shape forward(int M, int N, int slabs, bool gated, bool i8, int *ncol)
{
    const int bn = tile::plan_tiles(M, N, gated, i8 ? tile::kStepI8 : tile::kStep16, slabs).bn;
    CHECK(bn >= 64 && bn <= tile::kMaxBn && bn % (i8 ? 32 : 16) == 0, "width %d", bn);
    *ncol = gated ? bn / 2 : bn;
    return tile::shape_of(M, N, bn, *ncol, slabs, 0);
}

static void prod(int M, int N, int slabs, bool gated, bool i8, bool print)
{
    int ncol = 0;
    const tile::Shape s = forward(M, N, slabs, gated, i8, &ncol);
    const int most = gated ? walk<tile::kGated>(s, ncol) : walk<tile::kScaled>(s, ncol);
    few_case(gated ? few::kGated : few::kScaled, M, N, slabs);
    if (print) std::printf("%d %d %d %d\n", (int)few_tokens(M, N, gated, i8, slabs), s.bn, s.x.units, most);
}

static void grad(int M, int F, int K, bool print)
{
    const GradPlan p = plan_gated_backward(M, F, K);
    few_case(few::kDx, M, K, 2 * ceil_div(F, 64));
    tile::Shape both = {};
    int most = 0, most_x = 0, extra = -1;
    for (const GradTiles *t : {&p.x, &p.w})
        CHECK((p.few && t == &p.x) || (t->bn == 128 || t->bn == 256), "width %d", t->bn);
    if (p.together) {
        both = tile::grad_shape(p.x, M, F, K, true, true);
        most = walk<tile::kBoth>(both, p.x.bn);
        const int pairs = (int)std::min<long long>((long long)both.x.units + both.w.units, tile::kPairs);
        extra = tile::extra_tiles(both.x, both.w, pairs);
    }
    const tile::Shape w = tile::grad_shape(p.w, M, F, K, false, true);
    const int most_w = walk<tile::kDw>(w, p.w.bn);
    CHECK(w.w.parts == p.w.parts_w, "parts of w");
    tile::Shape x = {};
    if (!p.few) {
        x = tile::grad_shape(p.x, M, F, K, true, false);
        most_x = walk<tile::kDx>(x, p.x.bn);
        CHECK(x.x.parts == p.x.parts_x, "parts of x");
    }
    // partial sums of the workspace
    const size_t need = (p.w.parts_w > 1 ? (size_t)w.w.parts * 2 * F * K * 4 : 0) +
                        (!p.few && p.x.parts_x > 1 ? (size_t)x.x.parts * M * K * 4 : 0);
    CHECK(need == grad_part_bytes(p, M, F, K), "partial sums");
    if (print)
        std::printf("%d %d %d %d %d %d %d %d %d %d\n", (int)p.few, (int)p.together, p.few ? 0 : p.x.bn,
                    p.few ? 0 : p.x.parts_x, p.w.bn, p.w.parts_w, extra, most, most_x, most_w);
}

int main()
{
    char kind[16];
    while (std::scanf("%15s", kind) == 1) {
        int a = 0, b = 0, c = 0, d = 0, e = 0;
        if (!std::strcmp(kind, "grad") && std::scanf("%d %d %d", &a, &b, &c) == 3) {
            grad(a, b, c, true);
        } else if (!std::strcmp(kind, "prod") && std::scanf("%d %d %d %d %d", &a, &b, &c, &d, &e) == 5) {
            prod(a, b, c, d, e, true);
        } else if (!std::strcmp(kind, "sweep") && std::scanf("%d %d", &a, &b) == 2) {
            std::srand((unsigned)b);
            auto size = [](double hi) { return (int)std::exp(std::log(hi) * (std::rand() / (double)RAND_MAX)); };
            for (int i = 0; i < a; ++i) {
                grad(size(20000), size(20000), (size(12000) + 7) / 8 * 8, false);
                prod(size(20000), size(100000), size(1500), std::rand() & 1, std::rand() & 1, false);
            }
        } else {
            return 2;
        }
    }
    return bad;
}
