// weights_kernel.cuh -- the softmax weight each key of a prompt receives from
// the prompt's last T queries:
//     weights[j] = sum over the group's heads h and the queries i of
//                  2^(x_hij - lse_hi),   x = scale log2(e) q_hi . k_j,
//     lse_hi = log2 sum_j 2^(x_hij)   over the window i-W < j <= i.
//
// The sum over queries needs lse, which needs every key of the window first, so
// there are two passes over Q K^T, each a persistent tcgen05 kernel of one
// shape: a stationary 128-row tile A in shared memory, tiles B streamed through
// a ring by TMA, D = A B^T in tensor memory, and one thread per row of A that
// reduces along its row, so that no reduction crosses threads:
//  * pass 1 (lse): A = 128 (query, head) rows of one KV head's group, B = key
//    tiles; a row keeps a running maximum and sum;
//  * pass 2 (weights): A = 128 keys, B = tiles of (query, head) rows; a row (a
//    key) adds 2^(x - lse), lse coming along with the tile.  Each key is owned
//    by one thread: no atomics, and the order of the sum is fixed.
// A tile of queries holds TQ = floor(128 / G) positions times the G heads of
// the group (position-major), one TMA box.  Neither pass writes the scores.
//
// Warps: 0 TMA, 1 MMA (one thread each), 2 tensor-memory allocation, 4-7 and
// 8-11 the two reducing warpgroups, which take the tiles of a unit in turn.
// Tensor memory holds four 128 x 128 fp32 results, so the tensor core runs up
// to four tiles ahead of the reduction.  Each warpgroup leaves its own partial
// result; small kernels join them.
#pragma once

#include "weights_plan.cuh"

namespace swa {

template <int D, int PASS>
struct WeightsCfg {
    static constexpr int NREG = D / 64;
    static constexpr int REGION_BYTES = 128 * 128;
    static constexpr int TILE_BYTES = NREG * REGION_BYTES;
    static constexpr int STAGES = 4;
    static constexpr int BUFS = 4;                       // results in tensor memory
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = TILE_BYTES;
    static constexpr int OFF_LSE = OFF_B + STAGES * TILE_BYTES;          // [STAGES][128] floats
    static constexpr int OFF_BAR = OFF_LSE + STAGES * 512;
    // a_full, a_empty, b_full[STAGES], b_empty[STAGES], s_full[BUFS], s_empty[BUFS], drain
    static constexpr int NBAR = 2 + 2 * STAGES + 2 * BUFS + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM_ALLOC = OFF_MISC + 16 + 1024;              // slack for 1024-byte alignment
    static constexpr int THREADS = 384;
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

template <int D, int PASS>
__global__ void __launch_bounds__(384, 1)
swa_prefill_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const WeightsParams p) {
    using Cfg = WeightsCfg<D, PASS>;
    constexpr int NREG = Cfg::NREG, RB = Cfg::REGION_BYTES, TB = Cfg::TILE_BYTES, ST = Cfg::STAGES, NB = Cfg::BUFS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t sA = sbase + Cfg::OFF_A, sB = sbase + Cfg::OFF_B;
    const uint32_t bar_a_full = sbase + Cfg::OFF_BAR, bar_a_empty = bar_a_full + 8;
    const uint32_t bar_b_full = bar_a_empty + 8, bar_b_empty = bar_b_full + 8 * ST;
    const uint32_t bar_s_full = bar_b_empty + 8 * ST, bar_s_empty = bar_s_full + 8 * NB;
    const uint32_t bar_drain = bar_s_empty + 8 * NB;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = g_wait_limit_ns;
    const int qrows = p.TQ * p.G;                    // rows of a query tile
    const uint32_t q_bytes = (uint32_t)NREG * qrows * 128;

    if (threadIdx.x == 0) {
        mbar_init(bar_a_full, 1);
        mbar_init(bar_a_empty, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(bar_b_full + 8 * s, 1);
            // pass 2: the reducing warps read the stage's lse as well
            mbar_init(bar_b_empty + 8 * s, PASS == 2 ? 5 : 1);
        }
        for (int s = 0; s < NB; ++s) {
            mbar_init(bar_s_full + 8 * s, 1);
            mbar_init(bar_s_empty + 8 * s, 4);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        mbar_init_fence();
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
    }
    // rows of a query tile past TQ * G are never written by TMA: zeros
    for (int t = PASS == 1 ? 0 : 1; t < (PASS == 1 ? 1 : 1 + ST); ++t)
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

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t bc = 0, uc = 0, b_cnt[ST] = {};
            bool ok = true;
            // rows of a tile of keys, or of a tile of queries
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
            for (int u = blockIdx.x; u < p.num_units && ok; u += gridDim.x) {
                const int b = u / p.Hkv % p.B;
                const WeightsUnit U = weights_unit<PASS>(p, u, weights_len(__ldg(p.lens + b), p.N));
                if (U.n == 0) continue;
                if (!mbar_wait_bounded(bar_a_empty, (uc & 1) ^ 1, abort_flag, limit)) { ok = false; break; }
                ++uc;
                mbar_arrive_expect_tx(bar_a_full, PASS == 1 ? q_bytes : (uint32_t)TB);
                if (PASS == 1) load_q(sA, bar_a_full, U, U.a);
                else load_k(sA, bar_a_full, U, U.a);
                for (int j = 0; j < U.n; ++j, ++bc) {
                    const uint32_t s = bc % ST;
                    if (!mbar_wait_bounded(bar_b_empty + 8 * s, ((bc / ST) & 1) ^ 1, abort_flag, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = bar_b_full + 8 * s;
                    mbar_arrive_expect_tx(bar, PASS == 1 ? (uint32_t)TB : q_bytes + 512u);
                    if (PASS == 1) {
                        load_k(sB + s * TB, bar, U, U.first + j);
                    } else {
                        load_q(sB + s * TB, bar, U, U.first + j);
                        const int qt = checked_coord(U.first + j, p.nqt);
                        bulk_load(sbase + Cfg::OFF_LSE + s * 512,
                                  p.lse + ((((size_t)U.b * p.Hkv + U.g) * p.nqt) + qt) * 128, 512, bar);
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
            uint32_t bc = 0, uc = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < p.num_units && ok; u += gridDim.x) {
                const int b = u / p.Hkv % p.B;
                const WeightsUnit U = weights_unit<PASS>(p, u, weights_len(__ldg(p.lens + b), p.N));
                if (U.n == 0) continue;
                if (!mbar_wait_bounded(bar_a_full, uc & 1, abort_flag, limit)) { ok = false; break; }
                ++uc;
                for (int j = 0; j < U.n; ++j, ++bc) {
                    const uint32_t s = bc % ST, d = bc % NB;
                    if (!mbar_wait_bounded(bar_b_full + 8 * s, (bc / ST) & 1, abort_flag, limit) ||
                        !mbar_wait_bounded(bar_s_empty + 8 * d, ((bc / NB) & 1) ^ 1, abort_flag, limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * RB + (kk & 3) * 32) >> 4;
                        mma_ss(tmem + d * 128, smem_desc64(adesc + off, kDescHi),
                               smem_desc64(bdesc + s * (TB >> 4) + off, kDescHi), Cfg::IDESC, kk > 0);
                    }
                    mma_commit(bar_s_full + 8 * d);
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
        const int row = (warp & 3) * 32 + lane;              // row of the stationary tile
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const float sl2 = p.scale_log2;
        uint32_t bc0 = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < p.num_units && ok; u += gridDim.x) {
            const int b = u / p.Hkv % p.B;
            const WeightsUnit U = weights_unit<PASS>(p, u, weights_len(__ldg(p.lens + b), p.N));
            float m = -INFINITY, l = 0.f;                    // pass 2: l alone
            for (int j = wg; j < U.n; j += 2) {
                const uint32_t bc = bc0 + j, d = bc % NB, s = bc % ST;
                bool got = mbar_wait_bounded(bar_s_full + 8 * d, (bc / NB) & 1, abort_flag, limit);
                // the tile's lse came by the same barrier as its rows
                if (PASS == 2 && got) got = mbar_wait_bounded(bar_b_full + 8 * s, (bc / ST) & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tmem + lane_off + d * 128 + c * 32, r[c]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) reg_fence32(r[c]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_s_empty + 8 * d);

                const WeightsMask M = weights_mask<PASS>(p, U, U.first + j, row);
                if (M.masked) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c < M.lo || c >= M.hi) r[c >> 5][c & 31] = 0xFF800000u;      // -inf
                }
                if (PASS == 1) {
                    float mx[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e] = __uint_as_float(r[0][e]);
#pragma unroll
                    for (int c = 8; c < 128; ++c) mx[c & 7] = fmaxf(mx[c & 7], __uint_as_float(r[c >> 5][c & 31]));
                    float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                     fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sl2;
                    // the offset is raised when the tile exceeds it by more than
                    // 2^8: the sum keeps its 24 bits either way
                    if (mt > m + 8.0f) {
                        l *= ex2_approx(m - mt);
                        m = mt;
                    }
                }
                const float off = PASS == 1 ? (m == -INFINITY ? 0.f : m) : 0.f;
                const float2 sl2x2 = make_float2(sl2, sl2), noff = make_float2(-off, -off);
                const uint32_t lse_s = sbase + Cfg::OFF_LSE + s * 512;
                float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                 make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 128; c += 4) {
                    float2 n0 = noff, n1 = noff;
                    if (PASS == 2) {                         // lse is kept negated
                        float4 v;
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                                     : "r"(lse_s + c * 4)
                                     : "memory");
                        n0 = make_float2(v.x, v.y);
                        n1 = make_float2(v.z, v.w);
                    }
                    const uint32_t *x = &r[c >> 5][c & 31];
                    const float2 a = ffma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), sl2x2, n0);
                    const float2 e = ffma2(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), sl2x2, n1);
                    acc[(c >> 2) & 1] = fadd2(acc[(c >> 2) & 1], make_float2(ex2_approx(a.x), ex2_approx(a.y)));
                    acc[2 + ((c >> 2) & 1)] = fadd2(acc[2 + ((c >> 2) & 1)], make_float2(ex2_approx(e.x), ex2_approx(e.y)));
                }
                const float2 sum = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
                l += sum.x + sum.y;
                if (PASS == 2) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_b_empty + 8 * s);
                }
            }
            if (!ok) break;
            bc0 += U.n;
            if (PASS == 1) {
                const size_t rows = ((((size_t)U.b * p.Hkv + U.g) * p.nqt) + U.a) * 128 + row;
                p.ml[rows * (2 * p.splits) + 2 * U.split + wg] = make_float2(m, l);
            } else if (U.a * 128 + row < p.N) {
                // a key behind the prompt may hold anything, and meets the tiles' zero
                // rows: its sum counts for nothing
                const int at = U.a * 128 + row;
                if (at >= U.base + p.T) l = 0.f;
                const size_t plane = (size_t)p.B * p.Hkv * p.N;
                p.part[(2 * U.split + wg) * plane + ((size_t)U.b * p.Hkv + U.g) * p.N + at] = l;
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

// Joins pass 1's partial {max, sum} of each row: -lse, or -infinity for a row
// that is no query (so that its weights are 2^-inf = 0).
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
        out = -((m == -INFINITY ? 0.f : m) + __log2f(l));
    }
    lse[row] = out;
}

// weights[i] = the sum of the partial results, in order.
__global__ void swa_weights_sum_kernel(const float *__restrict__ part, float *__restrict__ weights, long long n,
                                       int parts) {
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        float w = 0.f;
        for (int s = 0; s < parts; ++s) w += __ldg(part + s * n + i);
        weights[i] = w;
    }
}

}  // namespace swa
