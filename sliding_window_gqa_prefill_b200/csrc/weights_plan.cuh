// weights_plan.cuh -- work decomposition of the passes of
// swa_prefill_weights_kernel: units, streamed tiles and masks, callable on the
// host as well as on the device.
#pragma once

#include "device_common.cuh"

namespace swa {

// What a launch of the kernel computes, and which operand stays in shared
// memory while the other is streamed.
constexpr int kWeightsLse = 1;       // lse of each query; query tiles stay, key tiles are streamed
constexpr int kWeightsByKey = 2;     // weights; key tiles stay, query tiles are streamed
constexpr int kWeightsByQuery = 3;   // weights; all query tiles (at most two) stay, key tiles are streamed

struct WeightsParams {
    int B, N, T, Hkv, G, TQ;     // TQ positions (times G heads) per query tile
    int W;                       // window, at most N
    int nqt, nkt;                // query tiles, key tiles
    int splits;                  // of the streamed tiles of a unit
    int num_units;
    float scale_log2;
    const int32_t *lens;
    float2 *ml;                  // lse pass: [B, Hkv, nqt, 128][2 splits] {max, sum}
    const float *lse;            // weights passes: [B, Hkv, nqt, 128]
    float *part;                 // weights passes: planes of [B, Hkv, N]
};

// One unit: up to two stationary tiles a, a+1 and the run of streamed tiles of
// one split.
struct WeightsUnit {
    int b, g, a, split;
    bool act1;                   // tile a+1 exists
    int first, n;                // streamed tiles first .. first+n-1
    int base;                    // position of query t is base + t
};

// Key tiles lo .. hi that the queries of tiles a0 .. a1 see (hi < lo: none).
__host__ __device__ inline void weights_key_tiles(const WeightsParams &p, int base, int a0, int a1, int &lo, int &hi) {
    const long long t1 = (long long)(a1 + 1) * p.TQ < p.T ? (long long)(a1 + 1) * p.TQ : p.T;
    const int pmin = base + a0 * p.TQ > 0 ? base + a0 * p.TQ : 0, pmax = base + (int)t1 - 1;
    lo = (pmin - p.W + 1 > 0 ? pmin - p.W + 1 : 0) / 128;
    hi = pmax >= 0 ? pmax / 128 : -1;
}

// Stationary pairs of a (sequence, KV head).
template <int MODE>
__host__ __device__ inline int weights_pairs(int nqt, int nkt) {
    return MODE == kWeightsLse ? (nqt + 1) / 2 : MODE == kWeightsByKey ? (nkt + 1) / 2 : 1;
}

template <int MODE>
__host__ __device__ inline WeightsUnit weights_unit(const WeightsParams &p, int u, int len) {
    WeightsUnit U;
    // stationary pair slowest, those with the most work first: late queries see
    // the most keys, early keys are seen by the most queries
    const int pairs = weights_pairs<MODE>(p.nqt, p.nkt);
    U.g = u % p.Hkv;
    int r = u / p.Hkv;
    U.b = r % p.B;
    r /= p.B;
    U.split = r % p.splits;
    const int pair = MODE == kWeightsLse ? pairs - 1 - r / p.splits : r / p.splits;
    U.a = 2 * pair;
    U.act1 = U.a + 1 < (MODE == kWeightsByKey ? p.nkt : p.nqt);
    U.base = len - p.T;
    long long lo, hi;            // streamed tiles lo .. hi
    if (MODE != kWeightsByKey) {
        int l, h;
        weights_key_tiles(p, U.base, U.a, U.a + U.act1, l, h);
        lo = l;
        hi = h;
    } else {
        const long long k0 = (long long)U.a * 128, k1 = k0 + (U.act1 ? 255 : 127);
        long long t_lo = k0 - U.base, t_hi = k1 + p.W - 1 - U.base;
        if (t_lo < -U.base) t_lo = -(long long)U.base;
        if (t_lo < 0) t_lo = 0;
        if (t_hi > p.T - 1) t_hi = p.T - 1;
        if (k0 >= len) t_hi = t_lo - 1;
        lo = t_lo / p.TQ;
        hi = t_hi >= t_lo ? t_hi / p.TQ : lo - 1;
    }
    const long long count = hi >= lo ? hi - lo + 1 : 0;
    const long long per = (count + p.splits - 1) / p.splits;
    const long long f = lo + U.split * per, l = f + per - 1 < hi ? f + per - 1 : hi;
    U.first = (int)f;
    U.n = l >= f ? (int)(l - f + 1) : 0;
    return U;
}

// Streamed tiles lo .. hi whose product with stationary tile a + i needs no mask:
// every query of it sees every key of it.
struct WeightsClear {
    int lo, hi;
};

__host__ __device__ inline int weights_floordiv(long long x, int by) {
    return (int)(x >= 0 ? x / by : -((-x + by - 1) / by));
}

template <bool Q_STAYS>
__host__ __device__ inline WeightsClear weights_clear(const WeightsParams &p, const WeightsUnit &U, int i) {
    WeightsClear C;
    if (Q_STAYS) {               // keys k0 .. k0+127 with k0 + 127 <= first query, k0 > last query - W
        const int qt = U.a + i;
        const int p0 = U.base + qt * p.TQ;
        const int last = (qt + 1) * p.TQ < p.T ? (qt + 1) * p.TQ : p.T;
        C.lo = weights_floordiv((long long)U.base + last - 1 - p.W, 128) + 1;
        C.hi = weights_floordiv((long long)p0 - 127, 128);
    } else {                     // the same of the query tiles
        const long long k0 = (long long)(U.a + i) * 128;
        C.lo = weights_floordiv(k0 + 127 - U.base + p.TQ - 1, p.TQ);
        C.hi = (long long)U.base + p.T - 1 < k0 + p.W ? p.nqt - 1 : weights_floordiv(k0 + p.W - U.base, p.TQ) - 1;
    }
    return C;
}

// Which columns of a product of query tile qt and key tile kt a row sees: lo <=
// c < hi.  row_pos: row / G.
struct WeightsMask {
    int lo, hi;
};

template <bool ROW_IS_QUERY>
__host__ __device__ inline WeightsMask weights_mask(const WeightsParams &p, const WeightsUnit &U, int qt, int kt,
                                                    int row, int row_pos) {
    const int k0 = kt * 128, p0 = U.base + qt * p.TQ;
    WeightsMask M;
    if (ROW_IS_QUERY) {          // keys (at - W, at]
        const int at = p0 + row_pos;
        M.lo = at - p.W + 1 - k0;
        M.hi = at + 1 - k0;
    } else {                     // queries [key, key + W), column c at position p0 + c / G
        const int key = k0 + row;
        const int from = key - p0 < -1 ? -1 : key - p0 > 128 ? 128 : key - p0;
        const long long to = (long long)key - p0 + p.W;
        M.lo = from * p.G;
        M.hi = (int)(to < 0 ? 0 : to > 128 ? 128 : to) * p.G;
    }
    return M;
}

// A sequence's length as the kernels use it: outside [0, N] it counts as 0.
__host__ __device__ inline int weights_len(int len, int N) { return len < 0 || len > N ? 0 : len; }

// The unit of a persistent block's round k: forward in even rounds, backward in
// odd ones, so that blocks with heavier units in one round get lighter ones in
// the next.
__host__ __device__ inline long long weights_unit_of(int k, int c, int blocks) {
    return (long long)k * blocks + ((k & 1) ? blocks - 1 - c : c);
}

}  // namespace swa
