// weights_kernel.cuh -- the softmax weight each key of a prompt receives from
// the prompt's last T queries:
//     weights[j] = sum over the group's heads h and the queries i of
//                  2^(x_hij - lse_hi),   x = scale log2(e) q_hi . k_j,
//     lse_hi = log2 sum_j 2^(x_hij)   over the window i-W < j <= i.
//
// The sum over queries needs lse, which needs every key of the window first, so
// there are two passes over Q K^T, each a persistent tcgen05 kernel of one
// shape: up to two 128-row tiles stay in shared memory, tiles of the other
// operand are streamed past them through a ring by TMA, the products go to
// tensor memory, and one thread per row of a product reduces along its row, so
// that no reduction crosses threads and no score is ever written:
//  * lse: rows are queries; a row keeps a running maximum and sum;
//  * weights: rows are keys; a row adds 2^(x - lse), lse coming along with the
//    queries.  Each key is owned by one thread: no atomics, and the order of
//    the sum is fixed.  Either two key tiles stay and the queries are streamed,
//    or, when all queries fit in two tiles, they stay and the keys are streamed.
// A tile of queries holds TQ = floor(128 / G) positions times the G heads of
// the group (position-major), one TMA box.
//
// Warps: 0 TMA, 1 MMA (one thread each), 2 tensor-memory allocation, 4-19 the
// four reducing warpgroups.  Warpgroup w reduces columns 64 (w >> 1) .. + 63 of
// the products of stationary tile w & 1.  Tensor memory holds two 128 x 128 fp32
// products of each stationary tile; a warpgroup reads its 64 columns in two
// loads and gives the product back halfway through, so the tensor core is up to
// a step and a half ahead.  (One product per warpgroup, given back at three
// quarters, is as fast; the stationary tiles as the products' operand in tensor
// memory, three products beside them, slower: 738 against 683 us at the time.)
//
// What bounds it: one exponential per score and pass, 16 per clock and SM on the
// special-function unit: 1024 clocks for a 128 x 128 product whose MMA takes 512.
// kWeightsPoly of 16 pairs therefore go to a polynomial on the FMA pipe (none
// 726, 4 of 16 698, 5 720, 8 798 us).  T = N = 8192, 32 / 8 heads, D=128, both
// passes: 694 us (687 to 702), 0.40 PFLOP/s of one pass's products.  At 1.55 GHz a product
// takes 1200 clocks, in which the schedulers issue 62% of the time and no pipe is
// above 62% busy: 6.9 instructions per score against the 4.4 of its arithmetic,
// the rest barriers, masks and loads per 64 columns; without the exponentials it
// still takes 880.  T = 64 of N = 16384, two sequences: 59 us.
#pragma once

#include "weights_plan.cuh"

namespace swa {

template <int D, int MODE>
struct WeightsCfg {
    static constexpr int NREG = D / 64;
    static constexpr int REGION_BYTES = 128 * 128;
    static constexpr int TILE_BYTES = NREG * REGION_BYTES;
    static constexpr int STAGES = 4;
    static constexpr int OFF_A = 0;                                      // two stationary tiles
    static constexpr int OFF_B = 2 * TILE_BYTES;
    static constexpr int OFF_LSE = OFF_B + STAGES * TILE_BYTES;          // 128 floats per stage / stationary tile
    static constexpr int OFF_BAR = OFF_LSE + STAGES * 512;
    // a_full, a_empty, b_full[STAGES], b_empty[STAGES], s_full[4], s_empty[4], drain
    static constexpr int NBAR = 2 + 2 * STAGES + 8 + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM_ALLOC = OFF_MISC + 16 + 1024;              // slack for 1024-byte alignment
    static constexpr int THREADS = 640;
    static constexpr uint32_t IDESC = make_idesc_bf16(128, 128, 0);
    static_assert(D == 64 || D == 128, "head_dim 64 or 128");
    static_assert(SMEM_ALLOC <= 232448, "dynamic shared memory of one block (227 KB)");
};

// 1-D bulk copy global -> shared, completion on an mbarrier; addresses and size
// multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// The largest of three; a NaN among them stays one.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float4 lds_f32x4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ float2 lds_f32x2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}

// 2^x for two values on the FMA pipe, as exp2_poly2 but to about the accuracy of
// the special-function unit: degree 5, fitted in the same way (relative error
// 1.6e-7, with fp32 steps 2.2e-7, both at the ends of a binade).  x is clamped at
// -126; a NaN becomes 2^-126.
__device__ __forceinline__ float2 exp2_poly2_fine(float2 x) {
    constexpr float kShift = 12582912.0f;                       // 1.5 * 2^23
    constexpr float c1 = 0.69314694f, c2 = 0.24022120f, c3 = 0.055507131f, c4 = 0.0096755410f, c5 = 0.0013276471f;
    x.x = fmaxf(x.x, -126.0f);
    x.y = fmaxf(x.y, -126.0f);
    const float2 t = fadd2(x, make_float2(kShift, kShift));
    const float2 n = fadd2(t, make_float2(-kShift, -kShift));    // round(x), exact
    const float2 f = ffma2(n, make_float2(-1.0f, -1.0f), x);     // x - n, exact
    float2 p = ffma2(f, make_float2(c5, c5), make_float2(c4, c4));
    p = ffma2(p, f, make_float2(c3, c3));
    p = ffma2(p, f, make_float2(c2, c2));
    p = ffma2(p, f, make_float2(c1, c1));
    p = ffma2(p, f, make_float2(1.0f, 1.0f));
    return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                       __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

// which of the 16 column pairs of 32 columns take the polynomial
constexpr uint32_t kWeightsPoly = 0x1111u;

template <int D, int MODE>
__global__ void __launch_bounds__(640, 1)
swa_prefill_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const WeightsParams p) {
    using Cfg = WeightsCfg<D, MODE>;
    constexpr int NREG = Cfg::NREG, RB = Cfg::REGION_BYTES, TB = Cfg::TILE_BYTES, ST = Cfg::STAGES;
    constexpr bool Q_STAYS = MODE != kWeightsByKey, ROW_IS_QUERY = MODE == kWeightsLse;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t sA = sbase + Cfg::OFF_A, sB = sbase + Cfg::OFF_B;
    const uint32_t bar_a_full = sbase + Cfg::OFF_BAR, bar_a_empty = bar_a_full + 8;
    const uint32_t bar_b_full = bar_a_empty + 8, bar_b_empty = bar_b_full + 8 * ST;
    const uint32_t bar_s_full = bar_b_empty + 8 * ST, bar_s_empty = bar_s_full + 32;
    const uint32_t bar_drain = bar_s_empty + 32;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = g_wait_limit_ns;
    const int qrows = p.TQ * p.G;                    // rows of a query tile
    const uint32_t q_bytes = (uint32_t)NREG * qrows * 128;

    if (threadIdx.x == 0) {
        mbar_init(bar_a_full, 1);
        // the tensor core, and where lse comes with the stationary queries the
        // 16 reducing warps, which read it
        mbar_init(bar_a_empty, MODE == kWeightsByQuery ? 17 : 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(bar_b_full + 8 * s, 1);
            // where lse comes with the streamed queries, the 16 warps that reduce
            // the stage's two products (8, arriving for 16, if there is one)
            mbar_init(bar_b_empty + 8 * s, MODE == kWeightsByKey ? 17 : 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar_s_full + 8 * s, 1);
            mbar_init(bar_s_empty + 8 * s, 8);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        mbar_init_fence();
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
    }
    // rows of a query tile past TQ * G are never written by TMA: zeros
    for (int t = Q_STAYS ? 0 : 2; t < (Q_STAYS ? 2 : 2 + ST); ++t)
        for (int r = 0; r < NREG; ++r)
            for (int i = qrows * 8 + threadIdx.x; i < 1024; i += Cfg::THREADS)
                reinterpret_cast<uint4 *>(smem + t * TB + r * RB)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 2) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto unit = [&](long long u) {
        return weights_unit<MODE>(p, (int)u, weights_len(__ldg(p.lens + (int)(u / p.Hkv % p.B)), p.N));
    };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t bc = 0, uc = 0, b_cnt[ST] = {};
            bool ok = true;
            auto load_k = [&](uint32_t dst, uint32_t bar, const WeightsUnit &U, int tile) {
                for (int r = 0; r < NREG; ++r)
                    tma_load_4d(dst + r * RB, &tm_k, bar, r * 64, checked_coord(U.g, p.Hkv),
                                checked_coord(tile * 128, p.N), checked_coord(U.b, p.B));
            };
            auto load_q = [&](uint32_t dst, uint32_t bar, const WeightsUnit &U, int tile) {
                for (int r = 0; r < NREG; ++r)
                    tma_load_4d(dst + r * RB, &tm_q, bar, r * 64, checked_coord(U.g * p.G, p.Hkv * p.G),
                                checked_coord(tile * p.TQ, p.T), checked_coord(U.b, p.B));
            };
            auto load_lse = [&](int slot, uint32_t bar, const WeightsUnit &U, int tile) {
                bulk_load(sbase + Cfg::OFF_LSE + slot * 512,
                          p.lse + (((size_t)U.b * p.Hkv + U.g) * p.nqt + checked_coord(tile, p.nqt)) * 128, 512, bar);
            };
            long long u;
            for (int k = 0; (u = weights_unit_of(k, blockIdx.x, gridDim.x)) < p.num_units && ok; ++k) {
                const WeightsUnit U = unit(u);
                if (U.n == 0) continue;
                if (!mbar_wait_bounded(bar_a_empty, (uc & 1) ^ 1, abort_flag, limit)) { ok = false; break; }
                ++uc;
                const uint32_t lse_bytes = MODE == kWeightsByQuery ? 512u : 0u;
                mbar_arrive_expect_tx(bar_a_full, (1 + U.act1) * ((Q_STAYS ? q_bytes : (uint32_t)TB) + lse_bytes));
                for (int i = 0; i <= (int)U.act1; ++i) {
                    if (Q_STAYS) load_q(sA + i * TB, bar_a_full, U, U.a + i);
                    else load_k(sA + i * TB, bar_a_full, U, U.a + i);
                    if (MODE == kWeightsByQuery) load_lse(i, bar_a_full, U, U.a + i);
                }
                for (int j = 0; j < U.n; ++j, ++bc) {
                    const uint32_t s = bc % ST, bar = bar_b_full + 8 * s;
                    if (!mbar_wait_bounded(bar_b_empty + 8 * s, ((bc / ST) & 1) ^ 1, abort_flag, limit)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(bar, Q_STAYS ? (uint32_t)TB : q_bytes + 512u);
                    if (Q_STAYS) {
                        load_k(sB + s * TB, bar, U, U.first + j);
                    } else {
                        load_q(sB + s * TB, bar, U, U.first + j);
                        load_lse(s, bar, U, U.first + j);
                    }
                    ++b_cnt[s];
                }
            }
            if (!ok) {          // let every copy this thread started land before the block exits
                if (uc) mbar_drain_bounded(bar_a_full, (uc - 1) & 1, kDrainLimitNs);
                for (int s = 0; s < ST; ++s)
                    if (b_cnt[s]) mbar_drain_bounded(bar_b_full + 8 * s, (b_cnt[s] - 1) & 1, kDrainLimitNs);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t kDescHi = smem_desc_hi(1024);
            const uint32_t adesc = smem_desc_lo(sA, 16), bdesc = smem_desc_lo(sB, 16);
            uint32_t bc = 0, uc = 0, cnt[2] = {0, 0};
            bool ok = true;
            long long u;
            for (int k = 0; (u = weights_unit_of(k, blockIdx.x, gridDim.x)) < p.num_units && ok; ++k) {
                const WeightsUnit U = unit(u);
                if (U.n == 0) continue;
                if (!mbar_wait_bounded(bar_a_full, uc & 1, abort_flag, limit)) { ok = false; break; }
                ++uc;
                for (int j = 0; j < U.n && ok; ++j, ++bc) {
                    const uint32_t s = bc % ST;
                    if (!mbar_wait_bounded(bar_b_full + 8 * s, (bc / ST) & 1, abort_flag, limit)) { ok = false; break; }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i == 1 && !U.act1) break;
                        const uint32_t d = i + 2 * (cnt[i] & 1);
                        if (!mbar_wait_bounded(bar_s_empty + 8 * d, ((cnt[i] >> 1) & 1) ^ 1, abort_flag, limit)) {
                            ok = false;
                            break;
                        }
                        ++cnt[i];
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * RB + (kk & 3) * 32) >> 4;
                            const uint64_t st = smem_desc64(adesc + i * (TB >> 4) + off, kDescHi);
                            const uint64_t fl = smem_desc64(bdesc + s * (TB >> 4) + off, kDescHi);
                            // rows: the stationary tile, or the streamed keys
                            if (MODE == kWeightsByQuery) mma_ss(tmem + d * 128, fl, st, Cfg::IDESC, kk > 0);
                            else mma_ss(tmem + d * 128, st, fl, Cfg::IDESC, kk > 0);
                        }
                        mma_commit(bar_s_full + 8 * d);
                    }
                    if (!ok) break;
                    mma_commit(bar_b_empty + 8 * s);
                    if (j == U.n - 1) mma_commit(bar_a_empty);
                }
            }
            if (!ok) {
                mma_commit(bar_drain);
                mbar_drain_bounded(bar_drain, 0, kDrainLimitNs);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ reducing warpgroups
        const int wg = (warp - 4) >> 2;
        const int i = wg & 1, half = wg >> 1;                // stationary tile; columns of its products
        const int row = (warp & 3) * 32 + lane;              // row of the product
        const int row_pos = row / p.G;
        const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + i * 128 + half * 64;
        const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
        uint32_t cnt = 0, bc0 = 0, uc = 0;
        bool ok = true;
        long long u;
        for (int k = 0; (u = weights_unit_of(k, blockIdx.x, gridDim.x)) < p.num_units && ok; ++k) {
            const WeightsUnit U = unit(u);
            const bool active = i == 0 || U.act1;
            const size_t bg = (size_t)U.b * p.Hkv + U.g;
            const WeightsClear clear = weights_clear<Q_STAYS>(p, U, i);
            float m = -INFINITY, l = 0.f;                    // weights: l alone
            if (MODE == kWeightsByQuery && U.n > 0) {        // lse came with the stationary queries
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_a_full, uc & 1, abort_flag, limit))) {
                    ok = false;
                    break;
                }
                ++uc;
            }
            for (int j = 0; active && j < U.n; ++j) {
                const uint32_t s = (bc0 + j) % ST, d = i + 2 * ((cnt + j) & 1);
                bool got = mbar_wait_bounded(bar_s_full + 8 * d, ((cnt + j) >> 1) & 1, abort_flag, limit);
                // lse came with the stage's queries
                if (MODE == kWeightsByKey && got)
                    got = mbar_wait_bounded(bar_b_full + 8 * s, ((bc0 + j) / ST) & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int tile = U.first + j;
                const uint32_t lse_s = sbase + Cfg::OFF_LSE + (MODE == kWeightsByKey ? s : (uint32_t)i) * 512 + half * 256;
                // a product with a query that is not finite (-lse: +infinity) keeps
                // off the polynomial too: a score that is NaN, or -infinity, makes
                // the exponent NaN, which the polynomial's clamp would hide
                bool masked = tile < clear.lo || tile > clear.hi;
                if (!ROW_IS_QUERY) {
                    const float2 v = lds_f32x2(lse_s + lane * 8);
                    masked |= __any_sync(0xffffffffu, fmaxf(v.x, v.y) == INFINITY);
                }
                const uint32_t tD = tS + 256 * ((cnt + j) & 1);
                uint32_t r[2][32];
                tmem_ld32(tD, r[0]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t(&x)[32] = r[c & 1];
                    tmem_wait_ld();
                    reg_fence32(x);
                    if (c == 0) {
                        tmem_ld32(tD + 32, r[1]);
                    } else {                                 // the product is in registers: give it back
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_s_empty + 8 * d);
                    }
                    int lo = 0, hi = 32;                     // columns of these 32 that the row sees
                    if (masked) {
                        const WeightsMask M = weights_mask<ROW_IS_QUERY>(p, U, Q_STAYS ? U.a + i : tile,
                                                                         Q_STAYS ? tile : U.a + i, row, row_pos);
                        lo = M.lo - half * 64 - c * 32;
                        hi = M.hi - half * 64 - c * 32;
                        if (ROW_IS_QUERY) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (e < lo || e >= hi) x[e] = 0xFF800000u;                        // -inf
                        }
                    }
                    float2 off = make_float2(0.f, 0.f);
                    if (ROW_IS_QUERY) {
                        float mx[2] = {__uint_as_float(x[0]), __uint_as_float(x[1])};
#pragma unroll
                        for (int e = 2; e < 30; e += 4) {
                            mx[0] = fmax3_nan(mx[0], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                            mx[1] = fmax3_nan(mx[1], __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                        }
                        mx[0] = fmax3_nan(mx[0], __uint_as_float(x[30]), __uint_as_float(x[31]));
                        const float mt = fmax3_nan(mx[0], mx[1], mx[1]) * sl2.x;
                        // the offset is raised when a score exceeds it by more than
                        // 2^8: the sum keeps its 24 bits either way.  A NaN (which the
                        // polynomial would not show) makes offset and sum NaN for good.
                        if (!(mt <= m + 8.0f)) {
                            l *= ex2_approx(m - mt);
                            m = mt;
                        }
                        off.x = off.y = m == -INFINITY ? 0.f : -m;
                    }
                    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    // 2^-inf of a masked score is to be 0 exactly: not the polynomial;
                    // where the rows are keys the exponent is masked, as the -lse of a
                    // query that is not finite is +infinity
                    auto add = [&](uint32_t poly, bool mask) {
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (!ROW_IS_QUERY && e % 2 == 0) v = lds_f32x4(lse_s + c * 128 + e * 8);     // -lse
                            const float2 o = ROW_IS_QUERY ? off : e % 2 ? make_float2(v.z, v.w) : make_float2(v.x, v.y);
                            float2 y = ffma2(
                                make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sl2, o);
                            if (!ROW_IS_QUERY && mask) {
                                if (2 * e < lo || 2 * e >= hi) y.x = -INFINITY;
                                if (2 * e + 1 < lo || 2 * e + 1 >= hi) y.y = -INFINITY;
                            }
                            acc[e & 1] = fadd2(acc[e & 1], ((poly >> e) & 1u)
                                                               ? exp2_poly2_fine(y)
                                                               : make_float2(ex2_approx(y.x), ex2_approx(y.y)));
                        }
                    };
                    if (masked) add(0u, true);
                    else add(kWeightsPoly, false);
                    const float2 sum = fadd2(acc[0], acc[1]);
                    l += sum.x + sum.y;
                }
                if (MODE == kWeightsByKey) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive_n(bar_b_empty + 8 * s, U.act1 ? 1u : 2u);
                }
                if (MODE == kWeightsByQuery) {
                    // a key behind the prompt may hold anything, and meets the tiles'
                    // zero rows: its sum counts for nothing
                    const int key = tile * 128 + row;
                    if (key < p.N)
                        p.part[(size_t)(2 * i + half) * p.B * p.Hkv * p.N + bg * p.N + key] =
                            key < U.base + p.T ? l : 0.f;
                    l = 0.f;
                }
            }
            if (!ok) break;
            bc0 += U.n;
            if (active) cnt += U.n;
            if (MODE == kWeightsByQuery && U.n > 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_a_empty);
            }
            if (MODE == kWeightsLse && active)
                p.ml[((bg * p.nqt + U.a + i) * 128 + row) * (2 * p.splits) + 2 * U.split + half] = make_float2(m, l);
            if (MODE == kWeightsByKey && active) {
                const int key = (U.a + i) * 128 + row;
                if (key < p.N)
                    p.part[(size_t)(2 * U.split + half) * p.B * p.Hkv * p.N + bg * p.N + key] =
                        key < U.base + p.T ? l : 0.f;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the lse pass's partial {max, sum} of each row: -lse, or -infinity for a
// row that is no query (so that it gives 2^-inf = 0, or the polynomial's least,
// 2^-126).  A query whose scores are not finite gets +infinity, with which every
// weight it gives is not finite either: the weights pass takes no polynomial
// beside it.
__global__ void __launch_bounds__(128)
swa_weights_lse_kernel(const float2 *__restrict__ ml, float *__restrict__ lse, const int32_t *__restrict__ lens, int N,
                       int T, int Hkv, int G, int TQ, int nqt, int parts) {
    const int qt = blockIdx.x % nqt;
    const long long bg = blockIdx.x / nqt;
    const int b = (int)(bg / Hkv), r = threadIdx.x;
    const int raw = __ldg(lens + b);
    if (raw < 0 || raw > N) {
        if (r == 0) record_status(kStatusInvalid);
    }
    const int len = weights_len(raw, N);
    const int tt = r / G, t = qt * TQ + tt;
    const size_t row = (size_t)blockIdx.x * 128 + r;
    float out = -INFINITY;
    if (tt < TQ && t < T && len - T + t >= 0) {
        const float2 *src = ml + row * parts;
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < parts; ++i) m = fmaxf(m, src[i].x);
        for (int i = 0; i < parts; ++i) l += src[i].x == -INFINITY ? src[i].y : src[i].y * ex2_approx(src[i].x - m);
        out = -(m + __log2f(l));
        // (a query sees its own key at least: no maximum means that all scores are -infinity)
        if (!(fabsf(out) < INFINITY)) out = INFINITY;
    }
    lse[row] = out;
}

// weights[i] = the sum of the partial planes, in order.  by_query: the planes
// hold only the key tiles that the queries see.
__global__ void swa_weights_sum_kernel(const WeightsParams p, float *__restrict__ weights, int planes, int by_query) {
    const long long n = (long long)p.B * p.Hkv * p.N;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        float w = 0.f;
        bool there = true;
        if (by_query) {
            const int key = (int)(i % p.N), b = (int)(i / p.N / p.Hkv);
            int lo, hi;
            weights_key_tiles(p, weights_len(__ldg(p.lens + b), p.N) - p.T, 0, p.nqt - 1, lo, hi);
            there = key / 128 >= lo && key / 128 <= hi;
        }
        if (there)
            for (int s = 0; s < planes; ++s) w += __ldg(p.part + s * n + i);
        weights[i] = w;
    }
}

}  // namespace swa
