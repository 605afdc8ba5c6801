// evict_kernel.cuh -- the fixed-size KV cache: each KV head of a sequence has M
// slots of its own, and what leaves is chosen by accumulated attention weight.
//
// State per (sequence, KV head): slot_pos[M], the position each slot holds (-1:
// free), and weights[M], the softmax weight the slot has received so far,
// summed over the query heads of the group and over the queries.
#pragma once

#include "decode_kernel.cuh"

namespace swa {

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// ---------------------------------------------------------------------------
// Decode that keeps the scores.  As swa_decode_kernel over the slots
// 0 .. min(pos+1, M)-1 that hold a position up to pos (a sequence that was taken
// back leaves later ones; here they are as free slots), and each block also keeps
// its scores (base 2, scaled; -inf for a free slot), from which the weights follow
// once the softmax sums are known.  What free slots hold never meets the
// products: their scores are replaced, and in a 16-key block that has one (a
// branch the whole warp takes) their values are cleared.  slot_pos comes through
// the rings, 4 bytes per key beside the 4 D of K and V.
//  * CLUSTER: the slots are cut over the 4 blocks of a cluster, the scores stay
//    in shared memory, the sums are exchanged through distributed shared memory,
//    and every block adds its own slots' weights: one launch, no workspace.
//    The host takes it where all blocks run at once and the group is not cut:
//    past that, the time a block spends on its weights is time its share of the
//    memory system is idle (B=18, M=1000: 27.0 against 20.1 us; B=9: 16.0 both;
//    3 sequences of 701 slots: 5.9 against 11.3).
//  * else the scores (4 bytes written and read per slot and query head, against
//    4 D bytes of K and V per KV head) and partial results go to the workspace
//    and swa_weights_finish_kernel does the rest.
template <int D, int G>
struct DecodeScoresCfg {
    using Base = DecodeCfg<D, G>;
    static constexpr int ROW = D + 3;                            // {o[D], m, l, l of the rounded weights}
    static constexpr int STAGE_BYTES = Base::STAGE_BYTES + kDecodeBlk * 4;      // K, V, slot_pos
    static constexpr int WARP_RING = kDecodeStages * STAGE_BYTES;
    static constexpr int OFF_HEAD = kDecodeWarps * WARP_RING;    // per head {m, 1 / l, 1 / l rounded}
    static constexpr int OFF_SCORES = OFF_HEAD + 8 * 16;         // CLUSTER: [G][keys of the block]
    static constexpr int SMEM_BYTES = OFF_SCORES;
    static constexpr int MAX_SMEM = OFF_SCORES + kDecodeSplit * G * 4;
    static_assert((kDecodeWarps + 1) * G * ROW * 4 <= OFF_HEAD, "the merge reuses the rings");
};

// weights_in, weights_out, out: CLUSTER only.  score_stride: slots per row of
// scores (CLUSTER: per block, in shared memory).
template <int D, int G, bool CLUSTER>
__global__ void __launch_bounds__(kDecodeWarps * 32, 2)
swa_decode_scores_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ kc,
                         const __nv_bfloat16 *__restrict__ vc, const int32_t *__restrict__ slot_pos,
                         const int32_t *__restrict__ pos, float4 *__restrict__ ws_ml, float *__restrict__ ws_o,
                         float *__restrict__ scores, int score_stride, int Hkv, int M, int nsplit_max,
                         float scale_log2, int split_len, int kv_rep, const float *weights_in, float *weights_out,
                         __nv_bfloat16 *__restrict__ out) {
    using Cfg = DecodeCfg<D, G>;
    using SCfg = DecodeScoresCfg<D, G>;
    constexpr int CH = Cfg::CH, RB = Cfg::ROW_BYTES;
    extern __shared__ __align__(128) uint8_t smem[];

    const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int Hq = Hkv * G;
    const int p = __ldg(pos + b);
    if (p < 0) {                                    // invalid position: record, write nothing
        if (threadIdx.x == 0 && split == 0 && g == 0) record_status(kStatusInvalid);
        return;
    }
    const int L = (p >= M - 1) ? M : p + 1;
    constexpr int kClusterKeys = kDecodeClusterSplits * kDecodeBlk;
    const int split_keys = CLUSTER ? (L + kClusterKeys - 1) / kClusterKeys * kDecodeBlk : split_len;
    // a cluster block past the last slot still takes part in the merge
    if (!CLUSTER && (long long)split * split_keys >= L) return;
    const int begin = (int)min((long long)split * split_keys, (long long)L);
    const int end = min(L, begin + split_keys);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hr = lane >> 2, t4 = lane & 3;
    const bool head_ok = hr < G;
    const uint32_t ring = smem_addr(smem) + warp * SCfg::WARP_RING;
    const int Hkv_mem = Hkv / kv_rep, gk = g / kv_rep;
    const int32_t *sp = slot_pos + ((size_t)b * Hkv_mem + gk) * M;

    uint32_t qa[Cfg::KSTEPS][2];
    {
        const __nv_bfloat16 *qp = q + ((size_t)b * Hq + g * G + (head_ok ? hr : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < Cfg::KSTEPS; ++kk)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                qa[kk][hf] =
                    head_ok ? __ldg(reinterpret_cast<const uint32_t *>(qp + kk * 16 + hf * 8 + 2 * t4)) : 0u;
    }
    const size_t row_stride = (size_t)Hkv_mem * D;
    const __nv_bfloat16 *kbase = kc + ((size_t)b * M * Hkv_mem + gk) * D;
    const __nv_bfloat16 *vbase = vc + ((size_t)b * M * Hkv_mem + gk) * D;
    // this head's row of scores: in the workspace from slot 0, in shared memory
    // from the block's first slot
    float *srow = CLUSTER ? reinterpret_cast<float *>(smem + SCfg::OFF_SCORES) + hr * score_stride
                          : scores + ((size_t)b * Hq + g * G + hr) * score_stride + begin;

    const int nblk = (end - begin + kDecodeBlk - 1) / kDecodeBlk;
    const int my_blocks = (nblk > warp) ? (nblk - warp + kDecodeWarps - 1) / kDecodeWarps : 0;

    auto issue = [&](int i_local, int stage) {
        const int key0 = begin + (warp + i_local * kDecodeWarps) * kDecodeBlk;
        const uint32_t st = ring + stage * SCfg::STAGE_BYTES;
#pragma unroll
        for (int c = 0; c < Cfg::CPL; ++c) {
            const int id = c * 32 + lane;
            const int r = id / CH, ch = id % CH;
            const int key = min(key0 + r, end - 1);            // clamp: always in bounds
            if (!in_bounds(key, M)) continue;
            const uint32_t off = swz_off(r, ch, RB);
            const size_t rowi = (size_t)key * row_stride + ch * 8;
            cp_async16(st + off, kbase + rowi);
            cp_async16(st + Cfg::BLK_BYTES + off, vbase + rowi);
        }
        if (lane < kDecodeBlk) {
            const int key = min(key0 + lane, end - 1);
            if (in_bounds(key, M)) cp_async4(st + Cfg::STAGE_BYTES + 4 * lane, sp + key);
        }
    };

    float m_run = -INFINITY, l_run = 0.f;
    float2 lr2 = make_float2(0.f, 0.f);
    float o[Cfg::NB][2];
#pragma unroll
    for (int nb = 0; nb < Cfg::NB; ++nb) o[nb][0] = o[nb][1] = 0.f;
#pragma unroll
    for (int s = 0; s < kDecodeStages - 1; ++s) {
        if (s < my_blocks) issue(s, s);
        cp_async_commit();
    }

    for (int i = 0; i < my_blocks; ++i) {
        const int stage = i % kDecodeStages;
        cp_async_wait<kDecodeStages - 2>();
        __syncwarp();
        {
            const int nxt = i + kDecodeStages - 1;
            if (nxt < my_blocks) issue(nxt, nxt % kDecodeStages);
            cp_async_commit();
        }
        const uint32_t sk = ring + stage * SCfg::STAGE_BYTES, sv = sk + Cfg::BLK_BYTES;
        const int rel = (warp + i * kDecodeWarps) * kDecodeBlk;
        // which of the block's 16 slots hold a token up to p; >> 2 t4: bit 0, 1, 8, 9 are
        // this lane's keys
        uint32_t held;
        {
            int32_t at = -1;
            if (lane < kDecodeBlk && begin + rel + lane < end)
                asm volatile("ld.shared.s32 %0, [%1];" : "=r"(at) : "r"(sk + Cfg::STAGE_BYTES + 4 * lane) : "memory");
            held = __ballot_sync(0xffffffffu, (uint32_t)at <= (uint32_t)p);      // p >= 0; -1: free
        }
        const uint32_t bits = held >> (2 * t4);

        float s[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int c4 = 0; c4 < CH / 4; ++c4) {
                const int r = nb * 8 + (lane & 7), ch = c4 * 4 + (lane >> 3);
                uint32_t kb[4];
                ldsm_x4(sk + swz_off(r, ch, RB), kb);
                mma_rows8(s[nb][0], s[nb][1], qa[2 * c4][0], qa[2 * c4][1], kb[0], kb[1]);
                mma_rows8(s[nb][0], s[nb][1], qa[2 * c4 + 1][0], qa[2 * c4 + 1][1], kb[2], kb[3]);
            }
        float sc[4] = {s[0][0], s[0][1], s[1][0], s[1][1]};
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sc[e] = ((bits >> ((e & 1) + (e >> 1) * 8)) & 1u) ? sc[e] * scale_log2 : -INFINITY;
            mx = fmaxf(mx, sc[e]);
        }
        if (head_ok && in_bounds((CLUSTER ? 0 : begin) + rel + 15, score_stride)) {
            float2 *dst = reinterpret_cast<float2 *>(srow + rel + 2 * t4);
            dst[0] = make_float2(sc[0], sc[1]);
            dst[4] = make_float2(sc[2], sc[3]);
        }
        if (__any_sync(0xffffffffu, head_ok && mx > m_run + 8.0f)) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (mx > m_run) {                    // uniform across the quad
                const float alpha = ex2_approx(m_run - mx);
                l_run *= alpha;
                lr2.x *= alpha;
                lr2.y *= alpha;
#pragma unroll
                for (int nb = 0; nb < Cfg::NB; ++nb) {
                    o[nb][0] *= alpha;
                    o[nb][1] *= alpha;
                }
                m_run = mx;
            }
        }
        // no slot held so far: weights of 2^(-inf - 0) = 0
        const float off = (m_run == -INFINITY) ? 0.f : m_run;
        float pw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pw[e] = head_ok ? ex2_approx(sc[e] - off) : 0.f;
        // two sums: of the weights as they are, by which the accumulated
        // weights are normalised, and of the weights as rounded to bf16 for the
        // product with V, by which the output is (see swa_decode_kernel)
        const uint32_t pa0 = pack_bf16x2(pw[0], pw[1]), pa2 = pack_bf16x2(pw[2], pw[3]);
        l_run += (pw[0] + pw[1]) + (pw[2] + pw[3]);
        lr2 = add_bf16x2(add_bf16x2(lr2, pa0), pa2);
        auto add_pv = [&](auto masked) {
            const uint32_t keep0 = ((bits & 1u) ? 0xFFFFu : 0u) | ((bits & 2u) ? 0xFFFF0000u : 0u);
            const uint32_t keep1 = ((bits & 256u) ? 0xFFFFu : 0u) | ((bits & 512u) ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int c2 = 0; c2 < CH / 2; ++c2) {
                const int mi = lane >> 3;
                const int r = (mi & 1) * 8 + (lane & 7), ch = c2 * 2 + (mi >> 1);
                uint32_t vb[4];
                ldsm_x4_trans(sv + swz_off(r, ch, RB), vb);
                if constexpr (decltype(masked)::value) {
                    vb[0] &= keep0, vb[2] &= keep0;
                    vb[1] &= keep1, vb[3] &= keep1;
                }
                mma_rows8(o[2 * c2][0], o[2 * c2][1], pa0, pa2, vb[0], vb[1]);
                mma_rows8(o[2 * c2 + 1][0], o[2 * c2 + 1][1], pa0, pa2, vb[2], vb[3]);
            }
        };
        if (held == 0xFFFFu) add_pv(Flag<false>{});
        else add_pv(Flag<true>{});
        __syncwarp();
    }
    cp_async_wait<0>();
    float lr_run = lr2.x + lr2.y;
#pragma unroll
    for (int x = 1; x <= 2; x *= 2) {
        l_run += __shfl_xor_sync(0xffffffffu, l_run, x);
        lr_run += __shfl_xor_sync(0xffffffffu, lr_run, x);
    }

    // merge the warps in shared memory (over the rings) into the block's
    // {o[D], m, l, l of the rounded weights} per head
    constexpr int ROW = SCfg::ROW;
    __syncthreads();
    float *mg = reinterpret_cast<float *>(smem);
    float *part = mg + kDecodeWarps * G * ROW;      // [G][ROW], read by the cluster
    if (head_ok) {
        float *dst = mg + (warp * G + hr) * ROW;
#pragma unroll
        for (int nb = 0; nb < Cfg::NB; ++nb) {
            dst[nb * 8 + 2 * t4] = o[nb][0];
            dst[nb * 8 + 2 * t4 + 1] = o[nb][1];
        }
        if (t4 == 0) {
            dst[D] = m_run;
            dst[D + 1] = l_run;
            dst[D + 2] = lr_run;
        }
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < G * D; idx += blockDim.x) {
        const int h = idx / D, d = idx % D;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w) m = fmaxf(m, mg[(w * G + h) * ROW + D]);
        float l = 0.f, lr = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w) {
            const float *src = mg + (w * G + h) * ROW;
            const float sc = (src[D] == -INFINITY) ? 0.f : ex2_approx(src[D] - m);
            l += src[D + 1] * sc;
            lr += src[D + 2] * sc;
            acc += src[d] * sc;
        }
        if (CLUSTER) {
            part[h * ROW + d] = acc;
            if (d == 0) {
                part[h * ROW + D] = m;
                part[h * ROW + D + 1] = l;
                part[h * ROW + D + 2] = lr;
            }
        } else if (in_bounds(split, nsplit_max)) {
            const size_t slot = (((size_t)b * Hkv + g) * nsplit_max + split) * G + h;
            ws_o[slot * D + d] = acc;
            if (d == 0) ws_ml[slot] = make_float4(m, l, lr, 0.f);
        }
    }
    if constexpr (CLUSTER) {
        // every block of the cluster reaches both barriers: the only return above
        // depends on b alone, which the cluster shares
        cluster_sync_all();
        float4 *head = reinterpret_cast<float4 *>(smem + SCfg::OFF_HEAD);
        if (threadIdx.x < G) {
            const uint32_t row = smem_addr(part + threadIdx.x * ROW + D);
            float mr[kDecodeClusterSplits], m = -INFINITY, l = 0.f, lr = 0.f;
#pragma unroll
            for (int r = 0; r < kDecodeClusterSplits; ++r) {
                mr[r] = ld_peer_f32(row, r);
                m = fmaxf(m, mr[r]);
            }
            if (m == -INFINITY) m = 0.f;            // nothing held: every 2^(-inf - 0) is 0
#pragma unroll
            for (int r = 0; r < kDecodeClusterSplits; ++r) {
                const float sc = ex2_approx(mr[r] - m);
                l += ld_peer_f32(row + 4, r) * sc;
                lr += ld_peer_f32(row + 8, r) * sc;
            }
            // a KV head without a token gives an output of 0
            head[threadIdx.x] = make_float4(m, l == 0.f ? 0.f : 1.f / l, lr == 0.f ? 0.f : 1.f / lr, 0.f);
        }
        __syncthreads();
        static_assert((G * D) % kDecodeClusterSplits == 0, "outputs per block");
        constexpr int kPer = G * D / kDecodeClusterSplits;
        const int i0 = (int)cluster_rank() * kPer;
        for (int idx = i0 + threadIdx.x; idx < i0 + kPer; idx += blockDim.x) {
            const int h = idx / D, d = idx % D;
            const uint32_t row = smem_addr(part + h * ROW);
            float acc = 0.f;
#pragma unroll
            for (int r = 0; r < kDecodeClusterSplits; ++r)
                acc += ld_peer_f32(row + d * 4, r) * ex2_approx(ld_peer_f32(row + D * 4, r) - head[h].x);
            const size_t oi = ((size_t)b * Hq + g * G + h) * D + d;
            if (in_bounds((long long)oi, (long long)gridDim.z * Hq * D)) out[oi] = __float2bfloat16_rn(acc * head[h].z);
        }
        // the weights of this block's slots, and a share of the slots behind the
        // last, which keep theirs
        const size_t wrow = ((size_t)b * Hkv + g) * M;
        const float *sc = reinterpret_cast<const float *>(smem + SCfg::OFF_SCORES);
        for (int s = begin + threadIdx.x; s < end; s += blockDim.x) {
            float w = weights_in ? weights_in[wrow + s] : 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h) w += ex2_approx(sc[h * score_stride + s - begin] - head[h].x) * head[h].y;
            weights_out[wrow + s] = w;
        }
        for (int s = L + split * blockDim.x + threadIdx.x; s < M; s += kDecodeClusterSplits * blockDim.x)
            weights_out[wrow + s] = weights_in ? weights_in[wrow + s] : 0.f;
        cluster_sync_all();                          // peers' shared memory stays until read
    }
}

// Joins the splits of swa_decode_scores_kernel: the output rows, and
// weights_out[s] = weights_in[s] + sum over the group's heads of
// 2^(score - m) / l.  Each block takes kFinishSlots slots of one (sequence,
// KV head) and every gridDim.x-th head's output row; heads are added in
// order, so the sums do not depend on the schedule.  G heads in the group,
// held as rep groups of G / rep in the partial results.
constexpr int kFinishSlots = 1024, kFinishThreads = 256;

__global__ void __launch_bounds__(kFinishThreads)
swa_weights_finish_kernel(const int32_t *__restrict__ pos, const float4 *__restrict__ ws_ml,
                          const float *__restrict__ ws_o, const float *__restrict__ scores, int score_stride,
                          const float *weights_in, float *weights_out, __nv_bfloat16 *__restrict__ out, int Hkv,
                          int G, int rep, int D, int M, int nsplit_max, int split_len) {
    extern __shared__ float4 head[];                // {m, 1 / l, 1 / l rounded} per head of the group
    const int g = blockIdx.y, b = blockIdx.z;
    const int p = __ldg(pos + b);
    if (p < 0) return;
    const int L = (p >= M - 1) ? M : p + 1;
    const int nsplit = (L + split_len - 1) / split_len;
    if (!in_bounds(nsplit - 1, nsplit_max)) return;
    const int gt = G / rep;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this thread's four slots: their weights, and the scores of the first heads,
    // on their way while the sums are joined (the rows of scores are padded to
    // whole fours)
    static_assert(kFinishSlots == 4 * kFinishThreads, "four slots per thread");
    const size_t row = ((size_t)b * Hkv + g) * M;
    const float *srow = scores + ((size_t)b * Hkv + g) * G * score_stride;
    const long long s0 = (long long)blockIdx.x * kFinishSlots + 4 * threadIdx.x;
    constexpr int kFirst = 4;
    float w[4];
    float4 first[kFirst];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = weights_in && s0 + i < M ? weights_in[row + s0 + i] : 0.f;
#pragma unroll
    for (int h = 0; h < kFirst; ++h)
        first[h] = s0 < L && h < G ? __ldg(reinterpret_cast<const float4 *>(srow + (size_t)h * score_stride + s0))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
    // partial results of head h: slot(h) + s * gt
    auto slot = [&](int h) -> size_t {
        return (((size_t)b * Hkv + g) * rep + h / gt) * nsplit_max * gt + h % gt;
    };
    for (int h = warp; h < G; h += kFinishThreads / 32) {
        const float4 *src = ws_ml + slot(h);
        float m = -INFINITY;
        for (int s = lane; s < nsplit; s += 32) m = fmaxf(m, src[(size_t)s * gt].x);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (m == -INFINITY) m = 0.f;                // nothing held: every 2^(-inf - 0) is 0
        float l = 0.f, lr = 0.f;
        for (int s = lane; s < nsplit; s += 32) {
            const float4 v = src[(size_t)s * gt];
            const float sc = ex2_approx(v.x - m);
            l += v.y * sc;
            lr += v.z * sc;
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) {
            l += __shfl_xor_sync(0xffffffffu, l, x);
            lr += __shfl_xor_sync(0xffffffffu, lr, x);
        }
        // a KV head without a token gives an output of 0
        if (lane == 0) head[h] = make_float4(m, l == 0.f ? 0.f : 1.f / l, lr == 0.f ? 0.f : 1.f / lr, 0.f);
    }
    __syncthreads();
    const int mine = (G - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    for (int idx = threadIdx.x; idx < mine * D; idx += kFinishThreads) {
        const int h = (int)blockIdx.x + idx / D * (int)gridDim.x, d = idx % D;
        const size_t s0 = slot(h);
        float acc = 0.f;
        for (int s = 0; s < nsplit; ++s)
            acc += ws_o[(s0 + (size_t)s * gt) * D + d] * ex2_approx(ws_ml[s0 + (size_t)s * gt].x - head[h].x);
        out[((size_t)b * Hkv * G + g * G + h) * D + d] = __float2bfloat16_rn(acc * head[h].z);
    }
    auto add = [&](const float4 &x, int h) {
        const float m = head[h].x, inv = head[h].y;
        w[0] += ex2_approx(x.x - m) * inv;
        if (s0 + 1 < L) w[1] += ex2_approx(x.y - m) * inv;
        if (s0 + 2 < L) w[2] += ex2_approx(x.z - m) * inv;
        if (s0 + 3 < L) w[3] += ex2_approx(x.w - m) * inv;
    };
    if (s0 < L) {
#pragma unroll
        for (int h = 0; h < kFirst; ++h)
            if (h < G) add(first[h], h);
#pragma unroll 4
        for (int h = kFirst; h < G; ++h)
            add(__ldg(reinterpret_cast<const float4 *>(srow + (size_t)h * score_stride + s0)), h);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (s0 + i < M && in_bounds(s0 + i, M)) weights_out[row + s0 + i] = w[i];
}

// ---------------------------------------------------------------------------
// Eviction.  A weight's place in the order, as an unsigned number: larger
// weights give larger numbers, -0 and 0 the same one, NaN that of infinity.
__device__ __forceinline__ uint32_t weight_order(float w) {
    if (w != w) w = INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One new token per sequence at position p = pos[b]; in each KV head it takes
// the slot that already holds p, else the first that is free or holds a position
// behind p (of a sequence that was taken back; the decode does not see it), else
// the slot of least weight among those whose position q is neither a sink nor
// recent (S <= q <= p - R; ties: the lowest slot).  The slots before the first of
// the second kind hold different positions below p, so its index is at most p and
// the decode, which looks at slots 0 .. p, finds it.  One block per (sequence, KV
// head): the choice is the minimum over the slots of one 64-bit number, {kind,
// order of the weight, slot}, so it does not depend on the schedule.  8 bytes
// are read per slot; the kernel is bound by that and, for small batches, by
// the latency of one pass.
constexpr int kEvictThreads = 256;
constexpr int kEvictBatch = 16;                     // slots loaded side by side per thread
constexpr int kEvictMaxSlots = 1 << 30;             // the slot's 30 bits

// VEC: M is a multiple of 4 and both arrays are 16-byte aligned, so four slots
// come in one load (B=64, M=4096: 6.6 us; one slot at a time, four in flight, 10.0).
template <bool VEC>
__global__ void __launch_bounds__(kEvictThreads)
swa_evict_append_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, uint4 *__restrict__ k_cache,
                        uint4 *__restrict__ v_cache, int32_t *__restrict__ slot_pos, float *__restrict__ weights,
                        const int32_t *__restrict__ pos, int32_t *__restrict__ slots, int Hkv, int M, int head_vec,
                        int S, int R) {
    __shared__ unsigned long long best_of[kEvictThreads / 32];
    const int g = blockIdx.x, b = blockIdx.y;
    const size_t bg = (size_t)b * Hkv + g;
    const int32_t *sp = slot_pos + bg * M;
    const float *wt = weights + bg * M;
    constexpr int V = VEC ? 4 : 1, LOADS = kEvictBatch / V;
    const int p = __ldg(pos + b);
    const int last = max(p, 0) - R;                 // the newest position that may go (R >= 1)
    unsigned long long best = ~0ull;
    for (int s0 = 0; s0 < M; s0 += kEvictThreads * kEvictBatch) {
        int32_t at[kEvictBatch];
        float w[kEvictBatch];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {           // every load before the first use
            const int s = s0 + (i * kEvictThreads + threadIdx.x) * V;
            if constexpr (VEC) {
                int4 a = make_int4(0, 0, 0, 0);
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s < M) {
                    a = *reinterpret_cast<const int4 *>(sp + s);
                    x = *reinterpret_cast<const float4 *>(wt + s);
                }
                at[4 * i] = a.x, at[4 * i + 1] = a.y, at[4 * i + 2] = a.z, at[4 * i + 3] = a.w;
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            } else {
                at[i] = s < M ? sp[s] : 0;
                w[i] = s < M ? wt[s] : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kEvictBatch; ++i) {
            const int s = s0 + (i / V * kEvictThreads + threadIdx.x) * V + i % V;
            unsigned long long key = ~0ull;
            if (at[i] >= S && at[i] <= last)
                key = (2ull << 62) | ((unsigned long long)weight_order(w[i]) << 30) | (unsigned)s;
            if ((unsigned)at[i] > (unsigned)p) key = (1ull << 62) | (unsigned)s;      // free, or behind p
            if (at[i] == p) key = (unsigned)s;
            if (s < M) best = key < best ? key : best;
        }
    }
    if (p < 0) {                                    // invalid position: record, write nothing
        if (threadIdx.x == 0) {
            record_status(kStatusInvalid);
            if (slots) slots[bg] = -1;
        }
        return;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, x);
        best = o < best ? o : best;
    }
    if ((threadIdx.x & 31) == 0) best_of[threadIdx.x >> 5] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kEvictThreads / 32; ++w) best = best_of[w] < best ? best_of[w] : best;
    const int slot = (int)(best & (unsigned long long)(kEvictMaxSlots - 1));
    if (best == ~0ull || !in_bounds(slot, M)) {     // every slot is protected: record, write nothing
        if (threadIdx.x == 0) {
            record_status(kStatusInvalid);
            if (slots) slots[bg] = -1;
        }
        return;
    }
    if (threadIdx.x == 0) {
        slot_pos[bg * M + slot] = p;
        weights[bg * M + slot] = 0.f;
        if (slots) slots[bg] = slot;
    }
    for (int i = threadIdx.x; i < 2 * head_vec; i += kEvictThreads) {
        const int c = i % head_vec;
        const size_t dst = (((size_t)b * M + slot) * Hkv + g) * head_vec + c;
        if (i < head_vec) k_cache[dst] = __ldg(k_new + bg * head_vec + c);
        else v_cache[dst] = __ldg(v_new + bg * head_vec + c);
    }
}

// The slots a prompt of n = lens[b] positions keeps in each KV head: all if
// n <= M; else the first S, the last R and, between, the M - S - R of largest
// weight (ties: the lowest position), in the order of their positions.  One
// block per (sequence, KV head).  The smallest weight kept is found by three
// passes over the middle positions, each fixing 11 (the last 10) bits of its
// order number by a histogram; then every warp counts, and after one exchange of
// the counts writes, the positions it keeps in its own contiguous part of the
// prompt.  Digits of 11 bits, because weights lie in a few binades: with 8 bits
// (sign and most of the exponent) the first pass put a warp's 32 counts on a
// handful of addresses.  The order numbers stay in shared memory between the
// passes where they fit.  N=16384, M=2048, 32 blocks: 8 bits and every pass from
// L2 26.6 us, from shared memory 20.9, this 18.4 (and 11.8 for the copy of the rows).
constexpr int kKeepThreads = 1024, kKeepWarps = kKeepThreads / 32;
constexpr int kKeepBins = 2048;
constexpr int kKeepHists = 4;                       // each counted into by 8 warps
constexpr int kKeepCached = 40 * 1024;
inline int keep_smem(int N) { return (kKeepHists * kKeepBins + (N <= kKeepCached ? N : 0)) * 4; }
constexpr int kKeepMaxSmem = (kKeepHists * kKeepBins + kKeepCached) * 4;

__global__ void __launch_bounds__(kKeepThreads)
swa_keep_select_kernel(const float *__restrict__ weights, const int32_t *__restrict__ lens,
                       int32_t *__restrict__ slot_pos, float *__restrict__ weights_out, int N, int Hkv, int M, int S,
                       int R) {
    extern __shared__ uint32_t hist[];              // [kKeepHists][kKeepBins], then the order numbers
    __shared__ uint32_t warp_sum[kKeepWarps];
    __shared__ uint32_t pick_digit, pick_left;
    __shared__ int2 part[kKeepWarps];               // per warp: {kept for sure, at the smallest weight}
    const int g = blockIdx.x, b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int n = __ldg(lens + b);
    if (n < 0 || n > N) {                           // invalid length: record, keep nothing
        if (threadIdx.x == 0) record_status(kStatusInvalid);
        n = 0;
    }
    const size_t bg = (size_t)b * Hkv + g;
    const float *w = weights + bg * N;
    int32_t *sp = slot_pos + bg * M;
    float *wo = weights_out + bg * M;
    if (n <= M) {
        for (int s = threadIdx.x; s < M; s += kKeepThreads) {
            sp[s] = s < n ? s : -1;
            wo[s] = s < n ? w[s] : 0.f;
        }
        return;
    }
    const int lo = S, hi = n - R;                   // the middle: n > M >= S + R, so it has more than M - S - R
    uint32_t left = (uint32_t)(M - S - R);          // still to choose among those that match `prefix`
    uint32_t prefix = 0, mask = 0;
    uint32_t *cached = hist + kKeepHists * kKeepBins;
    const bool cache = N <= kKeepCached;
    if (cache) {
#pragma unroll 8
        for (int j = threadIdx.x; j < n; j += kKeepThreads) cached[j] = weight_order(__ldg(w + j));
    }
    auto order = [&](int j) -> uint32_t { return cache ? cached[j] : weight_order(__ldg(w + j)); };
    if (left > 0) {
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            for (int i = threadIdx.x; i < kKeepHists * kKeepBins / 4; i += kKeepThreads)
                reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            uint32_t *mine = hist + (warp % kKeepHists) * kKeepBins;
#pragma unroll 4
            for (int j = lo + threadIdx.x; j < hi; j += kKeepThreads) {
                const uint32_t u = order(j);
                if ((u & mask) == prefix) atomicAdd(&mine[(u >> shift) & digits], 1u);
            }
            __syncthreads();
            // thread t holds bins 2047 - 2t and 2046 - 2t, largest first
            const int bin = kKeepBins - 2 - 2 * (int)threadIdx.x;
            uint2 c = make_uint2(0, 0);              // .y the larger bin
#pragma unroll
            for (int i = 0; i < kKeepHists; ++i) {
                const uint2 x = *reinterpret_cast<const uint2 *>(hist + i * kKeepBins + bin);
                c.x += x.x;
                c.y += x.y;
            }
            uint32_t before = c.x + c.y;             // inclusive sum over the threads so far
#pragma unroll
            for (int x = 1; x < 32; x *= 2) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, before, x);
                if (lane >= x) before += o;
            }
            if (lane == 31) warp_sum[warp] = before;
            before -= c.x + c.y;
            __syncthreads();
            before += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
            if (before < left && before + c.x + c.y >= left) {       // one thread: the counts reach `left` here
                const bool upper = before + c.y >= left;
                pick_digit = upper ? bin + 1 : bin;
                pick_left = left - before - (upper ? 0 : c.y);
            }
            __syncthreads();
            prefix |= pick_digit << shift;
            mask |= digits << shift;
            left = pick_left;
        }
    }
    __syncthreads();
    // `prefix` is the smallest order number kept, `left` of its holders are
    // (lowest positions first); with nothing to choose, none
    const bool none = M - S - R == 0;
    const int per = (n + kKeepThreads - 1) / kKeepThreads * 32;       // positions per warp
    const int w0 = min(n, warp * per), w1 = min(n, w0 + per);
    auto kind = [&](int j) -> int {                 // 2: kept, 1: at the smallest weight kept, 0: not
        if (j < lo || j >= hi) return 2;
        if (none) return 0;
        const uint32_t u = order(j);
        return u > prefix ? 2 : u == prefix ? 1 : 0;
    };
    int sure = 0, tie = 0;
#pragma unroll 4
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int k = j0 + lane < w1 ? kind(j0 + lane) : 0;
        sure += __popc(__ballot_sync(0xffffffffu, k == 2));
        tie += __popc(__ballot_sync(0xffffffffu, k == 1));
    }
    if (lane == 0) part[warp] = make_int2(sure, tie);
    __syncthreads();
    const int2 ahead = lane < warp ? part[lane] : make_int2(0, 0);
    int ties = __reduce_add_sync(0xffffffffu, ahead.y);
    int at = __reduce_add_sync(0xffffffffu, ahead.x) + min(ties, (int)left);
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 4
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        int k = j < w1 ? kind(j) : 0;
        const float value = j < w1 ? __ldg(w + j) : 0.f;       // on its way before it is known to be kept
        const uint32_t tb = __ballot_sync(0xffffffffu, k == 1);
        if (k == 1 && ties + __popc(tb & below) >= (int)left) k = 0;
        const uint32_t kb = __ballot_sync(0xffffffffu, k != 0);
        if (k != 0) {
            const int s = at + __popc(kb & below);
            if (in_bounds(s, M)) {
                sp[s] = j;
                wo[s] = value;
            }
        }
        at += __popc(kb);
        ties += __popc(tb);
    }
}

// Copies the kept rows: slot s of KV head g from row slot_pos[b, g, s] of the
// prompt; free slots stay as they are.  16 bytes of K and of V per thread and
// step; grid y the sequence, x strides over its vectors, slot and vector of the
// row carried along.
__global__ void __launch_bounds__(256)
swa_keep_copy_kernel(const uint4 *__restrict__ k, const uint4 *__restrict__ v, const int32_t *__restrict__ slot_pos,
                     uint4 *__restrict__ k_cache, uint4 *__restrict__ v_cache, int N, int Hkv, int M, int head_vec) {
    const int row_vec = Hkv * head_vec;
    const int b = blockIdx.y;
    const size_t to = (size_t)b * M * row_vec, from = (size_t)b * N * row_vec;
    const int32_t *at = slot_pos + (size_t)b * Hkv * M;
    const long long first = blockIdx.x * (long long)blockDim.x + threadIdx.x, step = (long long)gridDim.x * blockDim.x;
    int c = (int)(first % row_vec);
    long long s = first / row_vec;
    const int step_c = (int)(step % row_vec);
    const long long step_s = step / row_vec;
    for (; s < M; s += step_s, c += step_c) {
        if (c >= row_vec) {
            c -= row_vec;
            if (++s >= M) break;
        }
        const int j = __ldg(at + (size_t)(c / head_vec) * M + s);
        if (j < 0 || !in_bounds(j, N)) continue;
        const size_t src = from + (size_t)j * row_vec + c, dst = to + (size_t)s * row_vec + c;
        k_cache[dst] = __ldg(k + src);
        v_cache[dst] = __ldg(v + src);
    }
}

}  // namespace swa
