// Host enumeration of the work decomposition of swa_prefill_weights_kernel: in
// each pass every (query, key) pair of every window is computed exactly once,
// by a unit whose tiles lie inside the tensors, and no other pair counts; a tile
// that is not masked needs no mask.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../sliding_window_gqa_prefill_b200/csrc/weights_plan.cuh"

using namespace swa;

static int fails = 0;
static long long cleared = 0;
#define EXPECT(c, ...)                      \
    do {                                    \
        if (!(c) && ++fails < 20) {         \
            std::printf("FAIL: " __VA_ARGS__); \
            std::printf("\n");              \
        }                                   \
    } while (0)

template <int MODE>
void check(WeightsParams p, int splits, const std::vector<int> &lens) {
    constexpr bool row_is_query = MODE == kWeightsLse, q_stays = MODE != kWeightsByKey;
    p.splits = splits;
    const int pairs = weights_pairs<MODE>(p.nqt, p.nkt);
    p.num_units = p.B * p.Hkv * splits * pairs;
    std::vector<std::vector<unsigned char>> seen((size_t)p.B * p.Hkv,
                                                 std::vector<unsigned char>((size_t)p.T * p.G * p.N, 0));
    std::vector<int> taken((size_t)p.num_units, 0), pair_taken((size_t)p.num_units, 0);
    const int blocks = 1 + std::rand() % 20;
    for (int c = 0; c < blocks; ++c) {
        long long u;
        for (int k = 0; (u = weights_unit_of(k, c, blocks)) < p.num_units; ++k) taken[u]++;
    }
    for (int u = 0; u < p.num_units; ++u) {
        EXPECT(taken[u] == 1, "unit %d taken %d times by %d blocks", u, taken[u], blocks);
        const int b = u / p.Hkv % p.B;
        const int len = weights_len(lens[b], p.N);
        const WeightsUnit U = weights_unit<MODE>(p, u, len);
        EXPECT(U.b == b, "unit %d: sequence %d, warps use %d", u, U.b, b);
        const int na = q_stays ? p.nqt : p.nkt, ns = q_stays ? p.nkt : p.nqt;
        EXPECT(U.a >= 0 && U.a + U.act1 < na && U.g >= 0 && U.g < p.Hkv && U.split >= 0 && U.split < splits, "unit %d", u);
        EXPECT(U.act1 == (U.a + 1 < na), "unit %d: second tile", u);
        pair_taken[(((size_t)U.b * p.Hkv + U.g) * splits + U.split) * pairs + U.a / 2]++;
        if (MODE == kWeightsByQuery && U.n) {
            int lo, hi;                                  // what the joining kernel takes as written
            weights_key_tiles(p, U.base, 0, p.nqt - 1, lo, hi);
            EXPECT(U.first >= lo && U.first + U.n - 1 <= hi, "unit %d: tiles outside the queries' range", u);
        }
        for (int j = 0; j < U.n; ++j)
            for (int i = 0; i <= (int)U.act1; ++i) {
                const int tile = U.first + j;
                EXPECT(tile >= 0 && tile < ns, "unit %d: tile %d of %d", u, tile, ns);
                const int qt = q_stays ? U.a + i : tile, kt = q_stays ? tile : U.a + i;
                const WeightsClear C = weights_clear<q_stays>(p, U, i);
                const bool clear = tile >= C.lo && tile <= C.hi;
                cleared += clear;
                for (int row = 0; row < 128; ++row) {
                    const WeightsMask M = weights_mask<row_is_query>(p, U, qt, kt, row, row / p.G);
                    for (int c = 0; c < 128; ++c) {
                        const int qr = row_is_query ? row : c, key = kt * 128 + (row_is_query ? c : row);
                        const int tt = qr / p.G, t = qt * p.TQ + tt, at = len - p.T + t;
                        const bool query = tt < p.TQ && t < p.T && at >= 0;   // else its lse removes it
                        const bool visible = clear || (c >= M.lo && c < M.hi);
                        const bool want = key <= at && key > at - p.W;
                        if (!query) continue;
                        EXPECT(visible == want, "mode %d unit %d row %d column %d: visible %d, want %d", MODE, u, row, c,
                               visible, want);
                        if (visible && key < p.N)
                            seen[(size_t)U.b * p.Hkv + U.g][((size_t)t * p.G + qr % p.G) * p.N + key]++;
                    }
                }
            }
    }
    for (size_t i = 0; i < pair_taken.size(); ++i)
        EXPECT(pair_taken[i] == 1, "stationary pair %zu taken %d times", i, pair_taken[i]);
    for (int b = 0; b < p.B; ++b)
        for (int g = 0; g < p.Hkv; ++g)
            for (int t = 0; t < p.T; ++t)
                for (int h = 0; h < p.G; ++h)
                    for (int k = 0; k < p.N; ++k) {
                        const int len = weights_len(lens[b], p.N), at = len - p.T + t;
                        const int want = at >= 0 && k <= at && k > at - p.W;
                        const int got = seen[(size_t)b * p.Hkv + g][((size_t)t * p.G + h) * p.N + k];
                        EXPECT(got == want, "mode %d: query %d head %d key %d counted %d times, want %d", MODE, t, h, k,
                               got, want);
                    }
}

int main() {
    std::srand(7);
    auto rnd = [](int lo, int hi) { return lo + std::rand() % (hi - lo + 1); };
    int by_query = 0;
    const int groups[] = {1, 2, 3, 4, 5, 7, 8, 12, 40, 128};
    for (int n = 0; n < 120; ++n) {
        WeightsParams p{};
        p.G = groups[rnd(0, 9)];
        p.Hkv = rnd(1, 2);
        p.B = rnd(1, 3);
        p.N = rnd(1, n % 3 ? 300 : 900);
        p.T = n % 4 == 0 ? p.N : n % 4 == 1 ? 1 : rnd(1, p.N);
        if ((long long)p.T * p.N * p.G > 600000) p.T = 1 + 600000 / (p.N * p.G) % p.N;
        p.W = n % 5 ? rnd(1, p.N) : p.N;
        p.TQ = 128 / p.G;
        p.nqt = (p.T + p.TQ - 1) / p.TQ;
        p.nkt = (p.N + 127) / 128;
        std::vector<int> lens;
        for (int b = 0; b < p.B; ++b) lens.push_back(b == 0 ? p.N : rnd(-1, p.N + 1));
        check<kWeightsLse>(p, rnd(1, 5), lens);
        check<kWeightsByKey>(p, rnd(1, 5), lens);
        if (p.nqt <= 2) check<kWeightsByQuery>(p, rnd(1, 5), lens), ++by_query;
    }
    EXPECT(cleared > 100, "%lld tiles without a mask", cleared);
    EXPECT(by_query > 20, "%d cases with resident queries", by_query);
    std::printf(fails ? "%d failures\n" : "ok\n", fails);
    return fails != 0;
}
