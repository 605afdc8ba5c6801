// weights_plan.cuh -- work decomposition of the two passes of
// swa_prefill_weights_kernel: units, streamed tiles and masks, callable on the
// host as well as on the device.
#pragma once

#include "device_common.cuh"

namespace swa {

struct WeightsParams {
    int B, N, T, Hkv, G, TQ;     // TQ positions (times G heads) per query tile
    int W;                       // window, at most N
    int nqt, nkt;                // query tiles, key tiles
    int splits;                  // of the streamed tiles of a unit
    int num_units;
    float scale_log2;
    const int32_t *lens;
    float2 *ml;                  // pass 1: [B, Hkv, nqt, 128][2 splits] {max, sum}
    const float *lse;            // pass 2: [B, Hkv, nqt, 128]
    float *part;                 // pass 2: [2 splits][B, Hkv, N]
};

// One unit: the stationary tile and the run of streamed tiles of one split.
struct WeightsUnit {
    int b, g, a, split;          // a: stationary tile (query tile / key tile)
    int first, n;                // streamed tiles first .. first+n-1
    int base;                    // position of query t is base + t
};

template <int PASS>
__host__ __device__ inline WeightsUnit weights_unit(const WeightsParams &p, int u, int len) {
    WeightsUnit U;
    // stationary tile slowest, those with the most work first: late queries see
    // the most keys, early keys are seen by the most queries
    const int na = PASS == 1 ? p.nqt : p.nkt;
    U.g = u % p.Hkv;
    int r = u / p.Hkv;
    U.b = r % p.B;
    r /= p.B;
    U.split = r % p.splits;
    U.a = r / p.splits;
    if (PASS == 1) U.a = na - 1 - U.a;
    U.base = len - p.T;
    long long lo, hi;            // streamed tiles lo .. hi
    if (PASS == 1) {
        const int t1 = (U.a + 1) * p.TQ < p.T ? (U.a + 1) * p.TQ : p.T;
        const int pmin = U.base + U.a * p.TQ > 0 ? U.base + U.a * p.TQ : 0, pmax = U.base + t1 - 1;
        const int k_lo = pmin - p.W + 1 > 0 ? pmin - p.W + 1 : 0;
        lo = k_lo / 128;
        hi = pmax >= 0 ? pmax / 128 : -1;
    } else {
        const long long k0 = (long long)U.a * 128;
        long long t_lo = k0 - U.base, t_hi = k0 + 127 + p.W - 1 - U.base;
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

// Which columns of a streamed tile a row of the stationary tile sees: lo <= c
// < hi, or all if not `masked` (the same for the whole tile).
struct WeightsMask {
    bool masked;
    int lo, hi;
};

template <int PASS>
__host__ __device__ inline WeightsMask weights_mask(const WeightsParams &p, const WeightsUnit &U, int tile, int row) {
    // positions of the tile of queries, and first key of the tile of keys
    const int qt = PASS == 1 ? U.a : tile, k0 = (PASS == 1 ? tile : U.a) * 128;
    const int p0 = U.base + qt * p.TQ;
    const int last = (qt + 1) * p.TQ < p.T ? (qt + 1) * p.TQ : p.T;
    const int pmax = U.base + last - 1;
    WeightsMask M;
    M.masked = !(k0 + 127 <= p0 && k0 > pmax - p.W);
    if (PASS == 1) {             // a query: keys (at - W, at]
        const int at = p0 + row / p.G;
        M.lo = at - p.W + 1 - k0;
        M.hi = at + 1 - k0;
    } else {                     // a key: queries [key, key + W), column c at position p0 + c / G
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

}  // namespace swa
