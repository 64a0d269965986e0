// w8a8_plan.h -- how a launch of the 8-bit products is laid out: the forms of
// the kernel, which of them a problem takes and how its tiles are cut.  Host
// code without HIP, so that tests can compile it alone.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace vq {

constexpr int KC = 128;  // k of a group's chunk: a 128-byte line of a row (half lines, 64 k, doubled the L2 requests)
constexpr int kMaxGroups = 512;          // persistent workgroups of a launch
// A tile cut between workgroups has one arrival counter per wave, at zero
// between calls; the pieces begin where the verify GEMMs' do, so that a
// workspace shared with them keeps their counters too.
constexpr size_t kCounterBytes = 64 * 1024;
static_assert(kMaxGroups * 8 * 4 <= kCounterBytes, "counters");

// The forms of the kernel (template arguments and workgroups per CU) and what
// each costs, in us: `begin` per launch, `tile` per tile of a workgroup (its
// outputs), `join` + `piece` per piece where tiles are cut, and each round of
// workgroups the longest of three: `chunk` per chunk, the bytes into LDS at
// `l2` TB/s, its share of the weights at `hbm` TB/s, `again` of them for each
// further row of tiles.  Fitted to 11,000 launches of 870 problems, before the
// loads were spread between the matrix instructions and the weights' cache policy
// was what it is.  The form with the least sum is launched.  On the kernel as it
// is, over 928 problems (1 to 4,093 rows, 128 to 17,408 features, k 256 to 17,408,
// plain and gated; 17,600 launches of every form and cut), that took 1.7% more than
// the best one in the mean and 1.34 times at worst (24 rows 17408 to 5120, 30.8 us
// for 23.0); one form for each row count had taken up to twice the best.
struct Form {
    int rt, ft, wr, wf, wk, stages, per_cu;
    float begin, chunk, tile, join, piece, hbm, again, l2;
    constexpr int rows() const { return 16 * rt * wr; }
    constexpr int feats() const { return 16 * ft * wf; }
};
constexpr Form kForms[] = {
    {1, 2, 1, 1, 4, 3, 2, 5.0f, 0.25f, 1.0f, 1.0f, 0.16f, 6.3f, 0.34f, 18.6f},  // 16 x 32
    {1, 2, 1, 4, 1, 6, 1, 5.2f, 0.26f, 1.0f, 1.3f, 0.21f, 6.2f, 0.24f, 14.6f},  // 16 x 128
    {2, 2, 1, 1, 4, 2, 2, 5.2f, 0.34f, 1.0f, 1.0f, 0.28f, 4.3f, 0.07f, 19.3f},  // 32 x 32
    {4, 2, 1, 2, 2, 3, 1, 5.0f, 0.41f, 2.0f, 1.1f, 0.48f, 5.9f, 0.43f, 18.7f},  // 64 x 64
    {4, 2, 1, 4, 1, 4, 1, 4.9f, 0.36f, 1.9f, 1.6f, 0.51f, 6.0f, 0.34f, 16.3f},  // 64 x 128
    {4, 2, 2, 2, 1, 4, 1, 5.0f, 0.34f, 1.9f, 1.4f, 0.62f, 4.7f, 0.64f, 17.7f},  // 128 x 64
    {4, 2, 2, 4, 1, 4, 1, 5.2f, 0.46f, 2.4f, 2.8f, 0.68f, 5.0f, 0.39f, 15.7f},  // 128 x 128
    {8, 2, 2, 4, 1, 3, 1, 6.0f, 0.74f, 3.3f, 3.3f, 1.19f, 5.0f, 0.50f, 13.5f},  // 256 x 128
    {8, 4, 2, 4, 1, 2, 1, 6.8f, 1.28f, 5.1f, 6.7f, 2.35f, 4.0f, 0.10f, 10.6f},  // 256 x 256
};
constexpr int kFormCount = sizeof(kForms) / sizeof(kForms[0]);

// Forms whose tiles are at most half padding.
inline bool fits_rows(const Form &f, int N) { return f.rows() == 16 || f.rows() < 2 * N; }

inline int groups_of(const Form &f, int cus) { return std::min(cus * f.per_cu, kMaxGroups); }
inline size_t pieces_bytes(const Form &f, int cus) {
    return kCounterBytes + (size_t)groups_of(f, cus) * f.rows() * f.feats() * 4;
}

// Whether a launch loads its weights past the caches.  Only where the 256 MB
// behind them could not keep them for the next call beside the rest of a layer
// (42 MB, one row, three matrices in turn: 11.1 us past them, 10.3 with), and
// where no workgroup reads what another has read before:
//  - One row of tiles reads each weight once: gated 17408 x 5120 (178 MB) of 16
//    rows 39.9 us past the caches and 43.4 with, of 61 rows 38.8 and 43.0, of 256
//    in 256 x 128 tiles 73.7 and 76.8.
//  - More rows of tiles find them in L2 only while they keep together, and a last
//    row of few rows, with less to load, runs ahead: 17 rows 17408 to 8192 in 16 x
//    32 tiles 44.2 us past and 33.9 with, gated 65 rows in 64 x 128 tiles 63.1 and
//    50.9, 129 rows in 128 x 64 tiles 107 and 74.
//  - Two rows of 16 x 128 tiles do keep together, nine tenths of their loads being
//    weights: gated 17 rows 41.6 and 45.7, 32 rows 42.6 and 47.6; three do not (48
//    rows 70.5 and 67.1).
inline bool past_caches(const Form &f, int N, int M, int K, bool gated) {
    const int rows = (N + f.rows() - 1) / f.rows();
    return (int64_t)M * K * (gated ? 2 : 1) >= (int64_t)128 << 20 &&
           (rows == 1 || (rows == 2 && f.rows() == 16 && f.feats() == 128));
}

// How a launch cuts its tiles: `whole` of them by single workgroups, each of
// the rest in `cuts` pieces.  Without room for the pieces every tile is whole.
struct Plan {
    int form, groups, whole, cuts;
};

// `room`: bytes of the workspace, 0 without one.
inline Plan plan_of(int N, int M, int K, bool gated, int cus, size_t room) {
    Plan best{};
    float least = 0.f;
    for (int i = 0; i < kFormCount; ++i) {
        const Form &f = kForms[i];
        if (!fits_rows(f, N))
            continue;
        const int G = groups_of(f, cus), feats = gated ? f.feats() / 2 : f.feats();
        const int64_t rows = (N + f.rows() - 1) / f.rows(), cols = (M + feats - 1) / feats, tiles = rows * cols;
        const int nch = (K + f.wk * KC - 1) / (f.wk * KC), rest = (int)(tiles % G);
        const bool fits = room >= pieces_bytes(f, cus);
        const float weights = (float)M * (float)K * (gated ? 2.f : 1.f) * (1.f + f.again * (float)(rows - 1)) /
                              (f.hbm * 1e6f * (float)tiles);  // us for a tile's share of them
        const float chunk = (float)((f.rows() + f.feats()) * f.wk * KC) / (f.l2 * 1e6f);  // us for a chunk into LDS
        const auto round = [&](int chunks, int groups, float tiles_in) {
            return std::max({f.chunk * (float)chunks, chunk * (float)chunks * (float)groups, weights * tiles_in});
        };
        const float fixed = f.begin + f.tile * (float)((tiles + G - 1) / G) + (float)(tiles / G) * round(nch, G, (float)G);
        const int most = rest && fits ? std::min({G / rest, nch, 12}) : 1;
        for (int cuts = 1; cuts <= most; ++cuts) {
            const float us = fixed + (rest ? round((nch + cuts - 1) / cuts, rest * cuts, (float)rest) : 0.f) +
                             (cuts == 1 ? 0.f : f.join + f.piece * (float)cuts);
            if (best.groups == 0 || us < least) {
                least = us;
                best = cuts == 1 ? Plan{i, (int)std::min<int64_t>(tiles, G), (int)tiles, 0}
                                 : Plan{i, tiles > G ? G : rest * cuts, (int)(tiles - rest), cuts};
            }
        }
    }
    return best;
}

// Rows per launch: the tile numbers of a launch stay in 32 bits.
inline int rows_at_once(int N, int M) {
    const int64_t cols = (M + 15) / 16;
    return (int)std::min<int64_t>(N, std::max<int64_t>(256, ((int64_t)1 << 30) / cols / 16 * 256));
}

// Bytes that a launch writes of a workspace with room for every form.
inline size_t plan_bytes(const Plan &p, int N, int M, bool gated) {
    if (p.cuts == 0)
        return 0;
    const Form &f = kForms[p.form];
    const int feats = gated ? f.feats() / 2 : f.feats();
    const int64_t tiles = (int64_t)((N + f.rows() - 1) / f.rows()) * ((M + feats - 1) / feats);
    return kCounterBytes + (size_t)(tiles - p.whole) * p.cuts * f.rows() * f.feats() * 4;
}

}  // namespace vq
