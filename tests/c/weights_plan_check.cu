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
#define EXPECT(c, ...)                      \
    do {                                    \
        if (!(c) && ++fails < 20) {         \
            std::printf("FAIL: " __VA_ARGS__); \
            std::printf("\n");              \
        }                                   \
    } while (0)

template <int PASS>
void check(WeightsParams p, int splits, const std::vector<int> &lens) {
    p.splits = splits;
    p.num_units = p.B * p.Hkv * splits * (PASS == 1 ? p.nqt : p.nkt);
    // pairs of one (sequence, KV head): query row (t, h) x key
    std::vector<std::vector<unsigned char>> seen((size_t)p.B * p.Hkv,
                                                 std::vector<unsigned char>((size_t)p.T * p.G * p.N, 0));
    std::vector<int> stationary((size_t)p.B * p.Hkv * splits * (PASS == 1 ? p.nqt : p.nkt), 0);
    for (int u = 0; u < p.num_units; ++u) {
        const int b = u / p.Hkv % p.B;
        const int len = weights_len(lens[b], p.N);
        const WeightsUnit U = weights_unit<PASS>(p, u, len);
        EXPECT(U.b == b, "unit %d: sequence %d, warps use %d", u, U.b, b);
        const int na = PASS == 1 ? p.nqt : p.nkt, ns = PASS == 1 ? p.nkt : p.nqt;
        EXPECT(U.a >= 0 && U.a < na && U.g >= 0 && U.g < p.Hkv && U.split >= 0 && U.split < splits, "unit %d", u);
        stationary[(((size_t)U.b * p.Hkv + U.g) * splits + U.split) * na + U.a]++;
        for (int j = 0; j < U.n; ++j) {
            const int tile = U.first + j;
            EXPECT(tile >= 0 && tile < ns, "unit %d: tile %d of %d", u, tile, ns);
            for (int row = 0; row < 128; ++row) {
                const WeightsMask M = weights_mask<PASS>(p, U, tile, row);
                for (int c = 0; c < 128; ++c) {
                    const int qr = PASS == 1 ? row : c, kr = PASS == 1 ? c : row;
                    const int qt = PASS == 1 ? U.a : tile, key = (PASS == 1 ? tile : U.a) * 128 + kr;
                    const int tt = qr / p.G, t = qt * p.TQ + tt;
                    const int at = len - p.T + t;
                    const bool query = tt < p.TQ && t < p.T && at >= 0;   // else its lse removes it
                    const bool visible = !M.masked || (c >= M.lo && c < M.hi);
                    const bool want = key <= at && key > at - p.W;
                    if (!query) continue;
                    EXPECT(visible == want, "pass %d unit %d row %d column %d: visible %d, want %d", PASS, u, row, c,
                           visible, want);
                    if (visible && key < p.N) seen[(size_t)U.b * p.Hkv + U.g][((size_t)t * p.G + qr % p.G) * p.N + key]++;
                }
            }
        }
    }
    for (size_t i = 0; i < stationary.size(); ++i)
        EXPECT(stationary[i] == 1, "stationary tile %zu taken %d times", i, stationary[i]);
    for (int b = 0; b < p.B; ++b)
        for (int g = 0; g < p.Hkv; ++g)
            for (int t = 0; t < p.T; ++t)
                for (int h = 0; h < p.G; ++h)
                    for (int k = 0; k < p.N; ++k) {
                        const int len = weights_len(lens[b], p.N), at = len - p.T + t;
                        const int want = at >= 0 && k <= at && k > at - p.W;
                        const int got = seen[(size_t)b * p.Hkv + g][((size_t)t * p.G + h) * p.N + k];
                        EXPECT(got == want, "pass %d: query %d head %d key %d counted %d times, want %d", PASS, t, h, k,
                               got, want);
                    }
}

int main() {
    std::srand(7);
    auto rnd = [](int lo, int hi) { return lo + std::rand() % (hi - lo + 1); };
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
        check<1>(p, rnd(1, 5), lens);
        check<2>(p, rnd(1, 5), lens);
    }
    std::printf(fails ? "%d failures\n" : "ok\n", fails);
    return fails != 0;
}
