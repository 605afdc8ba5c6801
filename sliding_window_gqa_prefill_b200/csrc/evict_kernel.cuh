// evict_kernel.cuh -- the fixed-size KV cache: each KV head of a sequence has M
// slots of its own, and what leaves is chosen by accumulated attention weight.
//
// State per (sequence, KV head): slot_pos[M], the position each slot holds (-1:
// free), and weights[M], the softmax weight the slot has received so far,
// summed over the query heads of the group and over the queries.
#pragma once

#include "decode_kernel.cuh"

namespace swa {

// 16-byte copy, or 16 zero bytes where `there` is false (src is not read).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// ---------------------------------------------------------------------------
// Decode that keeps the scores.  As swa_decode_kernel over the slots
// 0 .. min(pos+1, M)-1 that hold a position, and each block also writes its
// scores (base 2, scaled; -inf for a free slot) to the workspace, from which
// swa_weights_finish_kernel takes the weights once the softmax sums are known.
// A score costs 4 bytes written and read per query head against the 4 D bytes
// of K and V per KV head; at B=64, M=4096 they stay in L2.  Free slots
// are copied as zeros, so what they hold never meets the products.
template <int D, int G>
struct DecodeScoresCfg {
    using Base = DecodeCfg<D, G>;
    static constexpr int OFF_MASK = Base::SMEM_BYTES;            // one bit per key of the split
    static constexpr int SMEM_BYTES = OFF_MASK + kDecodeSplit / 8;
};

template <int D, int G>
__global__ void __launch_bounds__(kDecodeWarps * 32, 2)
swa_decode_scores_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ kc,
                         const __nv_bfloat16 *__restrict__ vc, const int32_t *__restrict__ slot_pos,
                         const int32_t *__restrict__ pos, float4 *__restrict__ ws_ml, float *__restrict__ ws_o,
                         float *__restrict__ scores, int score_stride, int Hkv, int M, int nsplit_max,
                         float scale_log2, int split_len, int kv_rep) {
    using Cfg = DecodeCfg<D, G>;
    constexpr int CH = Cfg::CH, RB = Cfg::ROW_BYTES;
    extern __shared__ __align__(128) uint8_t smem[];
    uint32_t *mask = reinterpret_cast<uint32_t *>(smem + DecodeScoresCfg<D, G>::OFF_MASK);

    const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int Hq = Hkv * G;
    const int p = __ldg(pos + b);
    if (p < 0) {                                    // invalid position: record, write nothing
        if (threadIdx.x == 0 && split == 0 && g == 0) record_status(kStatusInvalid);
        return;
    }
    const int L = (p >= M - 1) ? M : p + 1;
    if ((long long)split * split_len >= L) return;
    const int begin = split * split_len;
    const int end = min(L, begin + split_len);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hr = lane >> 2, t4 = lane & 3;
    const bool head_ok = hr < G;
    const uint32_t ring = smem_addr(smem) + warp * Cfg::WARP_RING;
    const int Hkv_mem = Hkv / kv_rep, gk = g / kv_rep;

    // which slots of the split hold a token: bit i of word w is slot begin + 32 w + i
    const int32_t *sp = slot_pos + ((size_t)b * Hkv_mem + gk) * M;
    for (int w = warp; w < (end - begin + 31) / 32; w += kDecodeWarps) {
        const int key = begin + w * 32 + lane;
        const uint32_t bits = __ballot_sync(0xffffffffu, key < end && in_bounds(key, M) && __ldg(sp + key) >= 0);
        if (lane == 0) mask[w] = bits;
    }

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
    float *srow = scores + ((size_t)b * Hq + g * G + hr) * score_stride;
    __syncthreads();

    const int nblk = (end - begin + kDecodeBlk - 1) / kDecodeBlk;
    const int my_blocks = (nblk > warp) ? (nblk - warp + kDecodeWarps - 1) / kDecodeWarps : 0;
    auto held = [&](int rel) -> uint32_t { return mask[rel >> 5] >> (rel & 31); };   // rel: a multiple of 16

    auto issue = [&](int i_local, int stage) {
        const int rel = (warp + i_local * kDecodeWarps) * kDecodeBlk;
        const uint32_t bits = held(rel);
        const uint32_t st = ring + stage * Cfg::STAGE_BYTES;
#pragma unroll
        for (int c = 0; c < Cfg::CPL; ++c) {
            const int id = c * 32 + lane;
            const int r = id / CH, ch = id % CH;
            const int key = min(begin + rel + r, end - 1);     // clamp: always in bounds
            if (!in_bounds(key, M)) continue;
            const bool there = (bits >> r) & 1u;
            const uint32_t off = swz_off(r, ch, RB);
            const size_t rowi = (size_t)key * row_stride + ch * 8;
            cp_async16_zfill(st + off, kbase + rowi, there);
            cp_async16_zfill(st + Cfg::BLK_BYTES + off, vbase + rowi, there);
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
        const uint32_t sk = ring + stage * Cfg::STAGE_BYTES, sv = sk + Cfg::BLK_BYTES;
        const int rel = (warp + i * kDecodeWarps) * kDecodeBlk;
        const uint32_t bits = held(rel) >> (2 * t4);       // bit 0, 1, 8, 9: this lane's keys

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
        if (head_ok && in_bounds(begin + rel + 15, score_stride)) {
            float2 *dst = reinterpret_cast<float2 *>(srow + begin + rel + 2 * t4);
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
#pragma unroll
        for (int c2 = 0; c2 < CH / 2; ++c2) {
            const int mi = lane >> 3;
            const int r = (mi & 1) * 8 + (lane & 7), ch = c2 * 2 + (mi >> 1);
            uint32_t vb[4];
            ldsm_x4_trans(sv + swz_off(r, ch, RB), vb);
            mma_rows8(o[2 * c2][0], o[2 * c2][1], pa0, pa2, vb[0], vb[1]);
            mma_rows8(o[2 * c2 + 1][0], o[2 * c2 + 1][1], pa0, pa2, vb[2], vb[3]);
        }
        __syncwarp();
    }
    cp_async_wait<0>();
    float lr_run = lr2.x + lr2.y;
#pragma unroll
    for (int x = 1; x <= 2; x *= 2) {
        l_run += __shfl_xor_sync(0xffffffffu, l_run, x);
        lr_run += __shfl_xor_sync(0xffffffffu, lr_run, x);
    }

    // merge the warps in shared memory (over the rings) into the split's
    // partial result {m, l, l of the rounded weights}, o[D] per head
    constexpr int ROW = D + 3;
    __syncthreads();
    float *mg = reinterpret_cast<float *>(smem);
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
    if (!in_bounds(split, nsplit_max)) return;
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
        const size_t slot = (((size_t)b * Hkv + g) * nsplit_max + split) * G + h;
        ws_o[slot * D + d] = acc;
        if (d == 0) ws_ml[slot] = make_float4(m, l, lr, 0.f);
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
    const size_t row = ((size_t)b * Hkv + g) * M;
    const float *srow = scores + ((size_t)b * Hkv + g) * G * score_stride;
#pragma unroll
    for (int i = 0; i < kFinishSlots / kFinishThreads; ++i) {
        const long long s = (long long)blockIdx.x * kFinishSlots + i * kFinishThreads + threadIdx.x;
        if (s >= M || !in_bounds(s, M)) break;
        float w = weights_in ? weights_in[row + s] : 0.f;
        if (s < L)
            for (int h = 0; h < G; ++h)
                w += ex2_approx(__ldg(srow + (size_t)h * score_stride + s) - head[h].x) * head[h].y;
        weights_out[row + s] = w;
    }
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
// the slot that already holds p, else the first free slot, else the slot of
// least weight among those whose position q is neither a sink nor recent
// (S <= q <= p - R; ties: the lowest slot).  One block per (sequence, KV
// head): the choice is the minimum over the slots of one 64-bit number, {kind,
// order of the weight, slot}, so it does not depend on the schedule.  8 bytes
// are read per slot; the kernel is bound by that and, for small batches, by
// the latency of one pass.
constexpr int kEvictThreads = 256;
constexpr int kEvictMaxSlots = 1 << 30;             // the slot's 30 bits

__global__ void __launch_bounds__(kEvictThreads)
swa_evict_append_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, uint4 *__restrict__ k_cache,
                        uint4 *__restrict__ v_cache, int32_t *__restrict__ slot_pos, float *__restrict__ weights,
                        const int32_t *__restrict__ pos, int32_t *__restrict__ slots, int Hkv, int M, int head_vec,
                        int S, int R) {
    __shared__ unsigned long long best_of[kEvictThreads / 32];
    const int g = blockIdx.x, b = blockIdx.y;
    const int p = __ldg(pos + b);
    const size_t bg = (size_t)b * Hkv + g;
    if (p < 0) {                                    // invalid position: record, write nothing
        if (threadIdx.x == 0) {
            record_status(kStatusInvalid);
            if (slots) slots[bg] = -1;
        }
        return;
    }
    const int32_t *sp = slot_pos + bg * M;
    const float *wt = weights + bg * M;
    unsigned long long best = ~0ull;
#pragma unroll 4
    for (int s = threadIdx.x; s < M; s += kEvictThreads) {
        const int at = sp[s];
        const uint32_t w = weight_order(wt[s]);
        unsigned long long key;
        if (at == p) key = 0;
        else if (at < 0) key = 1ull << 62;
        else if (at >= S && (long long)at <= (long long)p - R) key = (2ull << 62) | ((unsigned long long)w << 30);
        else continue;
        key |= (unsigned long long)s;
        best = key < best ? key : best;
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
// block per (sequence, KV head).  The smallest weight kept is found by four
// passes over the middle positions, each fixing 8 bits of its order number by
// a histogram (private to each warp, so the counts meet little contention);
// then every warp counts, and after one exchange of the counts writes, the
// positions it keeps in its own contiguous part of the prompt.
constexpr int kKeepThreads = 1024, kKeepWarps = kKeepThreads / 32;
constexpr int kKeepSmem = (kKeepWarps * 256 + 256) * 4;

__global__ void __launch_bounds__(kKeepThreads)
swa_keep_select_kernel(const float *__restrict__ weights, const int32_t *__restrict__ lens,
                       int32_t *__restrict__ slot_pos, float *__restrict__ weights_out, int N, int Hkv, int M, int S,
                       int R) {
    extern __shared__ uint32_t hist[];              // [warp][256], then the block's 256 sums
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
    uint32_t *sums = hist + kKeepWarps * 256;
    if (left > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = threadIdx.x; i < kKeepWarps * 256; i += kKeepThreads) hist[i] = 0;
            __syncthreads();
            for (int j = lo + threadIdx.x; j < hi; j += kKeepThreads) {
                const uint32_t u = weight_order(__ldg(w + j));
                if ((u & mask) == prefix) atomicAdd(&hist[warp * 256 + ((u >> shift) & 255)], 1u);
            }
            __syncthreads();
            if (threadIdx.x < 256) {
                uint32_t c = 0;
                for (int i = 0; i < kKeepWarps; ++i) c += hist[i * 256 + threadIdx.x];
                sums[threadIdx.x] = c;
            }
            __syncthreads();
            if (warp == 0) {
                // lane l holds digits 255 - 8l .. 248 - 8l, largest first
                uint32_t c[8], mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] = sums[255 - 8 * lane - i];
                    mine += c[i];
                }
                uint32_t before = mine;
#pragma unroll
                for (int x = 1; x < 32; x *= 2) {
                    const uint32_t o = __shfl_up_sync(0xffffffffu, before, x);
                    if (lane >= x) before += o;
                }
                before -= mine;                     // how many have a larger digit than this lane's
                if (before < left && before + mine >= left) {
                    int i = 0;
                    while (before + c[i] < left) before += c[i++];
                    pick_digit = 255 - 8 * lane - i;
                    pick_left = left - before;
                }
            }
            __syncthreads();
            prefix |= pick_digit << shift;
            mask |= 255u << shift;
            left = pick_left;
        }
    }
    // `prefix` is the smallest order number kept, `left` of its holders are
    // (lowest positions first); with nothing to choose, none
    const bool none = M - S - R == 0;
    const int per = (n + kKeepThreads - 1) / kKeepThreads * 32;       // positions per warp
    const int w0 = min(n, warp * per), w1 = min(n, w0 + per);
    auto kind = [&](int j) -> int {                 // 2: kept, 1: at the smallest weight kept, 0: not
        if (j < lo || j >= hi) return 2;
        if (none) return 0;
        const uint32_t u = weight_order(__ldg(w + j));
        return u > prefix ? 2 : u == prefix ? 1 : 0;
    };
    int sure = 0, tie = 0;
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int k = j0 + lane < w1 ? kind(j0 + lane) : 0;
        sure += __popc(__ballot_sync(0xffffffffu, k == 2));
        tie += __popc(__ballot_sync(0xffffffffu, k == 1));
    }
    if (lane == 0) part[warp] = make_int2(sure, tie);
    __syncthreads();
    int at = 0, ties = 0;
    for (int i = 0; i < warp; ++i) {
        at += part[i].x;
        ties += part[i].y;
    }
    at += min(ties, (int)left);
    const uint32_t below = (1u << lane) - 1;
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        int k = j < w1 ? kind(j) : 0;
        const uint32_t tb = __ballot_sync(0xffffffffu, k == 1);
        if (k == 1 && ties + __popc(tb & below) >= (int)left) k = 0;
        const uint32_t kb = __ballot_sync(0xffffffffu, k != 0);
        if (k != 0) {
            const int s = at + __popc(kb & below);
            if (in_bounds(s, M)) {
                sp[s] = j;
                wo[s] = __ldg(w + j);
            }
        }
        at += __popc(kb);
        ties += __popc(tb);
    }
}

// Copies the kept rows: slot s of KV head g from row slot_pos[b, g, s] of the
// prompt; free slots stay as they are.  16 bytes of K and of V per thread.
__global__ void swa_keep_copy_kernel(const uint4 *__restrict__ k, const uint4 *__restrict__ v,
                                     const int32_t *__restrict__ slot_pos, uint4 *__restrict__ k_cache,
                                     uint4 *__restrict__ v_cache, int B, int N, int Hkv, int M, int head_vec) {
    const long long total = (long long)B * M * Hkv * head_vec;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const int c = (int)(i % head_vec);
        const long long bsg = i / head_vec;
        const int g = (int)(bsg % Hkv);
        const long long bs = bsg / Hkv;
        const int s = (int)(bs % M), b = (int)(bs / M);
        const int j = __ldg(slot_pos + ((size_t)b * Hkv + g) * M + s);
        if (j < 0 || !in_bounds(j, N)) continue;
        const size_t src = (((size_t)b * N + j) * Hkv + g) * head_vec + c;
        k_cache[i] = __ldg(k + src);
        v_cache[i] = __ldg(v + src);
    }
}

}  // namespace swa
