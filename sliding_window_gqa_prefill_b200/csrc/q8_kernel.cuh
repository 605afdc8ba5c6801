// q8_kernel.cuh -- the rolling-buffer KV cache held in 8 bits: append,
// single-token decode, and the widening that feeds the chunk pre-fill.
//
// Format.  The code c of an element is an e4m3 value (4 exponent bits, 3
// mantissa bits, largest 448, no infinity); the elements of one block of
// `block` consecutive slots of one KV head share one scale s, K and V apart.
// The element is c * s.  s is a power of two (or 0 for a block of zeros):
//  * e4m3 is a floating-point format, so a scale that is not a power of two
//    would not make any code more precise; the up to one binade of headroom a
//    power of two leaves costs only the smallest values, 2^-9 s apart;
//  * c * s is exact in bf16 and fp32, so the widened cache is exactly what
//    the codes stand for;
//  * changing a block's scale moves the exponents of the codes it holds and
//    rounds only those that become subnormal, so tokens that stay in a block
//    while others join it are not degraded by repeated rounding.
// s = 2^e with the smallest e such that max |x| <= 448 * 2^e over the block's
// finite elements, e held to [-117, 119] (the widened values stay normal and
// finite).  A NaN or an infinity is stored as NaN.
#pragma once

#include "decode_kernel.cuh"

namespace swa {

// Two e4m3 codes (low byte first) widened to two f16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

// Two values rounded to e4m3 (nearest, ties to even; above 448: 448).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
    float2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The scale of a block whose largest finite magnitude is `top` (0 for 0), and
// its inverse: 448 = 1.75 * 2^8, so top = m * 2^x needs e = x - 8 where
// m <= 1.75 and x - 7 above.
__device__ __forceinline__ float q8_scale(float top, float &inv) {
    if (!(top > 0.f)) {
        inv = 0.f;
        return 0.f;
    }
    const uint32_t u = __float_as_uint(top);
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = max(-117, min(119, e));
    inv = __uint_as_float((uint32_t)(127 - e) << 23);
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

// A bf16 value times the inverse scale, ready for the conversion to e4m3:
// infinities become NaN (e4m3 has none, and 448 would hide them).
__device__ __forceinline__ float q8_scaled(float x, float inv) {
    return (fabsf(x) < INFINITY) ? x * inv : __uint_as_float(0x7FC00000u);
}

// Blocks of a cache of W slots that T consecutive positions can touch: the
// first may be entered at its last slot, and so may the short last block.
__host__ __device__ inline int q8_blocks_touched(int T, int block, int nblk) {
    if (T == 1) return 1;
    const long long n = ((long long)T - 2 + block - 1) / block + 2;
    return n < nblk ? (int)n : nblk;
}

// Append.  One thread block owns one (cache block, KV head, K or V) of one
// sequence, so nothing is shared and no atomic is needed: it reads the new
// tokens of its slots and the codes that stay, takes the largest magnitude of
// both, and writes the new codes -- and the others too, if the scale moved.
// Slots that no token has reached yet (a sequence shorter than the buffer)
// count for nothing and stay as they are.  Each thread holds 4 pieces of 8
// elements (16 bytes of bf16, 8 of codes), so the block is read once and
// stays in registers between the maximum and the rounding.
template <int BLOCK, int D>
__global__ void __launch_bounds__(BLOCK * D / 32)
swa_append_q8_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                     uint2 *__restrict__ k_cache, uint2 *__restrict__ v_cache, float *__restrict__ k_scale,
                     float *__restrict__ v_scale, const int32_t *__restrict__ pos, int T, int W, int Hkv,
                     int nblk, int ntouch) {
    constexpr int PIECES = D / 8;             // 8-element pieces per row
    constexpr int ROWS = BLOCK / 4;           // rows per pass, 4 passes
    constexpr int WARPS = BLOCK * D / 1024;
    __shared__ uint32_t red[2][WARPS > 0 ? WARPS : 1];
    const int b = blockIdx.y;
    // heads and K / V vary fastest: the rows of one slot are read together
    const int hv = blockIdx.x % (2 * Hkv), i_blk = blockIdx.x / (2 * Hkv);
    const int h = hv >> 1;
    const bool is_v = hv & 1;
    const int p0 = __ldg(pos + b);
    if (p0 < 0) {                             // invalid position: record, skip
        if (threadIdx.x == 0 && blockIdx.x == 0) record_status(kStatusInvalid);
        return;
    }
    const int first = p0 % W;
    int blk = first / BLOCK + i_blk;
    if (blk >= nblk) blk -= nblk;
    if (!in_bounds(blk, nblk) || i_blk >= ntouch) return;

    const uint4 *src = is_v ? v_new : k_new;
    uint2 *cache = is_v ? v_cache : k_cache;
    float *sc = (is_v ? v_scale : k_scale) + ((size_t)b * nblk + blk) * Hkv + h;
    const float old_scale = *sc;

    const int piece = threadIdx.x % PIECES, r0 = threadIdx.x / PIECES;
    uint4 fresh[4];
    uint2 held[4];
    int state[4];                             // 0: leave alone, 1: holds a token, 2: new token
    uint32_t top_new = 0, top_old = 0;        // magnitudes: bf16 bits, e4m3 bits
    int any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int slot = blk * BLOCK + i * ROWS + r0;
        state[i] = 0;
        if (slot >= W) continue;
        int t = slot - first;
        if (t < 0) t += W;
        if (t < T) {
            state[i] = 2;
            any = 1;
            fresh[i] = __ldg(src + (((size_t)b * T + t) * Hkv + h) * PIECES + piece);
        } else if (slot < p0) {
            state[i] = 1;
            held[i] = cache[(((size_t)b * W + slot) * Hkv + h) * PIECES + piece];
        }
    }
    if (!__syncthreads_or(any)) return;       // the last of `ntouch` blocks may be untouched
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (state[i] == 2) {
            const uint32_t w[4] = {fresh[i].x, fresh[i].y, fresh[i].z, fresh[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
                top_new = max(top_new, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
            }
        } else if (state[i] == 1) {
            const uint32_t w[2] = {held[i].x & 0x7F7F7F7Fu, held[i].y & 0x7F7F7F7Fu};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t c = (w[e >> 2] >> (8 * (e & 3))) & 0x7Fu;
                top_old = max(top_old, c != 0x7Fu ? c : 0u);
            }
        }
    }
    top_new = __reduce_max_sync(0xffffffffu, top_new);
    top_old = __reduce_max_sync(0xffffffffu, top_old);
    if (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) {
            red[0][threadIdx.x >> 5] = top_new;
            red[1][threadIdx.x >> 5] = top_old;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            top_new = max(top_new, red[0][w]);
            top_old = max(top_old, red[1][w]);
        }
    }
    // the scale of a block that holds nothing yet may be anything: used only
    // where a held code is not zero
    float top = __uint_as_float(top_new << 16);
    if (top_old) top = fmaxf(top, f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)top_old)).x * old_scale);
    float inv;
    const float scale = q8_scale(top, inv);
    const bool moved = scale != old_scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (state[i] == 0 || (state[i] == 1 && !moved)) continue;
        const int slot = blk * BLOCK + i * ROWS + r0;
        if (!in_bounds(slot, W)) continue;
        uint32_t c[4];
        if (state[i] == 2) {
            const uint32_t w[4] = {fresh[i].x, fresh[i].y, fresh[i].z, fresh[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c[e] = f32x2_to_e4m3x2(q8_scaled(__uint_as_float(w[e] << 16), inv),
                                       q8_scaled(__uint_as_float(w[e] & 0xFFFF0000u), inv));
        } else {
            const uint32_t w[2] = {held[i].x, held[i].y};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[e >> 1] >> (16 * (e & 1)))));
                // two products, not one by old_scale * inv: that may overflow
                c[e] = f32x2_to_e4m3x2(x.x * old_scale * inv, x.y * old_scale * inv);
            }
        }
        cache[(((size_t)b * W + slot) * Hkv + h) * PIECES + piece] =
            make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    if (threadIdx.x == 0 && moved) *sc = scale;
}

// The cached window widened to bf16 (exact) for the chunk pre-fill: kd, vd
// [B, W, Hkv, D].  Slots no token has reached become zeros, so that the
// attention's masked products there stay 0.  16 codes per thread and step.
__global__ void swa_widen_q8_kernel(const uint4 *__restrict__ k_cache, const uint4 *__restrict__ v_cache,
                                    const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                                    const int32_t *__restrict__ pos, uint4 *__restrict__ kd,
                                    uint4 *__restrict__ vd, int B, int W, int Hkv, int head_vec, int block,
                                    int nblk) {
    const int row_vec = Hkv * head_vec;                  // 16-code vectors per slot
    const long long total = (long long)B * W * row_vec;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const int c = (int)(i % row_vec);
        const long long bs = i / row_vec;
        const int slot = (int)(bs % W), b = (int)(bs / W);
        const bool there = slot < __ldg(pos + b);
        const size_t si = ((size_t)b * nblk + slot / block) * Hkv + c / head_vec;
        if (!in_bounds(b, B) || !in_bounds(slot / block, nblk)) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (there) {
                const uint4 w4 = __ldg((kv ? v_cache : k_cache) + i);
                const float s = __ldg((kv ? v_scale : k_scale) + si);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 x = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[e >> 1] >> (16 * (e & 1)))));
                    o[e] = pack_bf16x2(x.x * s, x.y * s);
                }
            }
            uint4 *dst = (kv ? vd : kd) + 2 * i;
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

// ---------------------------------------------------------------------------
// Decode over the 8-bit buffer: out = sum_j softmax_j(scale q.k_j) v_j over
// the slots 0 .. min(pos+1, W)-1, as swa_decode_kernel, at half its bytes.
//
// Arithmetic.  Codes widen exactly to f16, so both products run as f16
// tensor-core tiles (mma.sync m16n8k16) on unrounded codes, with the block
// scales applied in fp32 afterwards:
//  * S = (q 2^-x) . c_k, times scale 2^x s_k.  x brings each head's largest
//    |q| to [2^14, 2^15): q rounds in f16 only below 2^-28 of that;
//  * O += s_v (P . c_v): the product of one 16-key block starts from zero and
//    joins O by one fp32 FMA with the block's scale;
//  * P is rounded to f16 (2^-11 relative; bf16's 2^-8 in the 16-bit cache's
//    kernel) and l sums it as rounded.  P is 2^7 larger than 2^(s - offset),
//    at most 2^15, so weights down to 2^-21 of the largest keep all their bits
//    and those down to 2^-31 some: a long tail of small weights is not lost.
// The order of d inside a product is free as long as q and k agree, and the
// order of the output columns is free until they are written; both are chosen
// so that a lane's fragment is 16 consecutive codes of one row: K is read by
// one 16-byte shared load per row and half, V by one per key, and the bytes
// of two keys are interleaved with byte permutes.
template <int D, int G>
struct DecodeQ8Cfg {
    static constexpr int CH = D / 16;                          // 16-byte chunks per key row
    static constexpr int BLK_BYTES = kDecodeBlk * D;           // K (or V) codes of one 16-key block
    static constexpr int STAGE_BYTES = 2 * BLK_BYTES;
    static constexpr int STAGES = 6;                           // 16-key blocks in flight per warp
    static constexpr int WARP_RING = STAGES * STAGE_BYTES;
    static constexpr int RING_BYTES = kDecodeWarps * WARP_RING;
    static constexpr int CPL = kDecodeBlk * CH / 32;           // 16-byte copies per lane, K or V
    static constexpr int KSTEPS = D / 16;
    static constexpr int NB = D / 8;
    static constexpr int MERGE_BYTES = (kDecodeWarps + 1) * G * (D + 2) * 4;
    static constexpr int SMEM_BYTES = RING_BYTES > MERGE_BYTES ? RING_BYTES : MERGE_BYTES;
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(G >= 1 && G <= 8, "group size 1 to 8 (the rows 0..7 of the MMA tile)");
    static_assert(CPL * 32 == kDecodeBlk * CH, "copies per lane");
};

// Shared-memory offset of 16-byte chunk `ch` of code row `r`.  A line of 128
// bytes (one row of D = 128, two of D = 64) has its 8 chunks permuted by XOR
// so that the eight lanes of a phase hit eight different 16-byte bank groups
// both when they read 2 rows x 4 chunks (K) and 4 rows, two apart, x 2 chunks
// (V).
template <int D>
__device__ __forceinline__ uint32_t q8_off(int r, int ch) {
    if (D == 128) return (uint32_t)(r * 128 + ((ch ^ (((r >> 1) & 3) << 1) ^ ((r & 1) << 2)) << 4));
    return (uint32_t)((r >> 1) * 128 + (((((r & 1) << 2) | ch) ^ (((r >> 1) & 3) << 1)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// As mma_rows8, f16 operands: rows 0..7 of the tile only.
__device__ __forceinline__ void mma_rows8_f16(float &d0, float &d1, uint32_t a0, uint32_t a2, uint32_t b0,
                                              uint32_t b1) {
    [[maybe_unused]] float u2, u3;
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d0), "=f"(d1), "=f"(u2), "=f"(u3)
        : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1), "f"(d0), "f"(d1), "f"(0.f), "f"(0.f));
}

// MODE kDecodeWindow (splits merged by swa_decode_combine_kernel) or
// kDecodeWindowCluster (the splits of a window are the blocks of a cluster).
template <int D, int G, int MODE>
__global__ void __launch_bounds__(kDecodeWarps * 32, 2)
swa_decode_q8_kernel(const __nv_bfloat16 *__restrict__ q, const uint8_t *__restrict__ kc,
                     const uint8_t *__restrict__ vc, const float *__restrict__ k_scale,
                     const float *__restrict__ v_scale, const int32_t *__restrict__ pos,
                     __nv_bfloat16 *__restrict__ out, float2 *__restrict__ ws_ml, float *__restrict__ ws_o, int Hkv,
                     int W, int nsplit_max, float scale_log2, int split_len, int kv_rep, int block_log2, int nblk) {
    constexpr bool CLUSTER = MODE == kDecodeWindowCluster;
    using Cfg = DecodeQ8Cfg<D, G>;
    constexpr int CH = Cfg::CH;
    extern __shared__ __align__(128) uint8_t smem[];

    const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int Hq = Hkv * G;
    const int p = __ldg(pos + b);
    if (p < 0) {                                    // invalid position: record, write nothing
        if (threadIdx.x == 0 && split == 0 && g == 0) record_status(kStatusInvalid);
        return;
    }
    const int L = (p >= W - 1) ? W : p + 1;
    constexpr int kClusterKeys = kDecodeClusterSplits * kDecodeBlk;
    const int split_keys = CLUSTER ? (L + kClusterKeys - 1) / kClusterKeys * kDecodeBlk : split_len;
    if (!CLUSTER && (long long)split * split_keys >= L) return;
    const int begin = (int)min((long long)split * split_keys, (long long)L);
    const int end = min(L, begin + split_keys);
    const int nsplit = (L + split_keys - 1) / split_keys;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hr = lane >> 2, t4 = lane & 3;
    const bool head_ok = hr < G;
    const uint32_t ring = smem_addr(smem) + warp * Cfg::WARP_RING;

    const int Hkv_mem = Hkv / kv_rep, gk = g / kv_rep;
    const size_t row_stride = (size_t)Hkv_mem * D;
    const uint8_t *kbase = kc + ((size_t)b * W * Hkv_mem + gk) * D;
    const uint8_t *vbase = vc + ((size_t)b * W * Hkv_mem + gk) * D;
    const float *ksb = k_scale + (size_t)b * nblk * Hkv_mem + gk;
    const float *vsb = v_scale + (size_t)b * nblk * Hkv_mem + gk;

    const int nblk16 = (end - begin + kDecodeBlk - 1) / kDecodeBlk;
    const int my_blocks = (nblk16 > warp) ? (nblk16 - warp + kDecodeWarps - 1) / kDecodeWarps : 0;

    auto issue = [&](int i_local, int stage) {
        const int blk = warp + i_local * kDecodeWarps;
        const uint32_t st = ring + stage * Cfg::STAGE_BYTES;
#pragma unroll
        for (int c = 0; c < Cfg::CPL; ++c) {
            const int id = c * 32 + lane;
            const int r = id / CH, ch = id % CH;
            const int key = min(begin + blk * kDecodeBlk + r, end - 1);     // clamp: always in bounds
            if (!in_bounds(key, W)) continue;
            const uint32_t off = q8_off<D>(r, ch);
            const size_t rowi = (size_t)key * row_stride + ch * 16;
            cp_async16(st + off, kbase + rowi);
            cp_async16(st + Cfg::BLK_BYTES + off, vbase + rowi);
        }
    };
#pragma unroll
    for (int s = 0; s < Cfg::STAGES - 1; ++s) {
        if (s < my_blocks) issue(s, s);
        cp_async_commit();
    }

    // q of head hr scaled by 2^-x into f16; fragment j of the products takes
    // d = (4c + t4) * 16 + 4w + {0, 1 | 2, 3}, j = 4c + w
    uint32_t qa[Cfg::KSTEPS][2];
    float qfac;                                     // scale log2(e) 2^x
    {
        const __nv_bfloat16 *qp = q + ((size_t)b * Hq + g * G + (head_ok ? hr : 0)) * D;
        uint32_t raw[Cfg::KSTEPS][2];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < Cfg::KSTEPS; ++j)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int d = (4 * (j >> 2) + t4) * 16 + 4 * (j & 3) + 2 * hf;
                raw[j][hf] = head_ok ? __ldg(reinterpret_cast<const uint32_t *>(qp + d)) : 0u;
                const uint32_t lo = raw[j][hf] & 0x7FFFu, hi = (raw[j][hf] >> 16) & 0x7FFFu;
                top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
            }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent field of the largest |q| (at least 15: below that q is 0 to
        // any key that fits), brought to that of 2^14
        const int ef = max(15, (int)(top >> 7));
        const float down = __uint_as_float((uint32_t)(268 - ef) << 23);
        qfac = scale_log2 * __uint_as_float((uint32_t)(ef - 14) << 23);
#pragma unroll
        for (int j = 0; j < Cfg::KSTEPS; ++j)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                qa[j][hf] = pack_f16x2(__uint_as_float(raw[j][hf] << 16) * down,
                                       __uint_as_float(raw[j][hf] & 0xFFFF0000u) * down);
    }

    float m_run = -INFINITY, l_run = 0.f;
    float o[Cfg::NB][2];
#pragma unroll
    for (int nb = 0; nb < Cfg::NB; ++nb) o[nb][0] = o[nb][1] = 0.f;

    // scales of the current block, loaded one block ahead
    float ks_next = 0.f, vs_next = 0.f;
    auto load_scales = [&](int i_local) {
        const int key0 = begin + (warp + i_local * kDecodeWarps) * kDecodeBlk;
        const size_t si = (size_t)(key0 >> block_log2) * Hkv_mem;
        if (!in_bounds(key0 >> block_log2, nblk)) return;
        ks_next = __ldg(ksb + si);
        vs_next = __ldg(vsb + si);
    };
    if (my_blocks > 0) load_scales(0);

    for (int i = 0; i < my_blocks; ++i) {
        const int stage = i % Cfg::STAGES;
        cp_async_wait<Cfg::STAGES - 2>();
        __syncwarp();
        const float kf = ks_next * qfac, vs = vs_next;
        {
            const int nxt = i + Cfg::STAGES - 1;
            if (nxt < my_blocks) issue(nxt, nxt % Cfg::STAGES);
            cp_async_commit();
        }
        if (i + 1 < my_blocks) load_scales(i + 1);
        const uint32_t sk = ring + stage * Cfg::STAGE_BYTES, sv = sk + Cfg::BLK_BYTES;
        const int key0 = begin + (warp + i * kDecodeWarps) * kDecodeBlk;

        float s[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int c = 0; c < CH / 4; ++c) {
                const uint4 w4 = lds128(sk + q8_off<D>(nb * 8 + hr, c * 4 + t4));
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mma_rows8_f16(s[nb][0], s[nb][1], qa[4 * c + e][0], qa[4 * c + e][1],
                                  e4m3x2_to_f16x2((uint16_t)w[e]), e4m3x2_to_f16x2((uint16_t)(w[e] >> 16)));
            }
        float sc[4] = {s[0][0], s[0][1], s[1][0], s[1][1]};
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int key = key0 + 2 * t4 + (e & 1) + (e >> 1) * 8;
            sc[e] = (key < end) ? sc[e] * kf : -INFINITY;
            mx = fmaxf(mx, sc[e]);
        }
        if (__any_sync(0xffffffffu, head_ok && mx > m_run + 8.0f)) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (mx > m_run) {                    // uniform across the quad
                const float alpha = ex2_approx(m_run - mx);
                l_run *= alpha;
#pragma unroll
                for (int nb = 0; nb < Cfg::NB; ++nb) {
                    o[nb][0] *= alpha;
                    o[nb][1] *= alpha;
                }
                m_run = mx;
            }
        }
        float pw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pw[e] = head_ok ? ex2_approx(sc[e] - m_run + 7.0f) : 0.f;
        const uint32_t pa0 = pack_f16x2(pw[0], pw[1]), pa2 = pack_f16x2(pw[2], pw[3]);
        {
            const float2 l0 = f16x2_to_f32x2(pa0), l1 = f16x2_to_f32x2(pa2);
            l_run += (l0.x + l0.y) + (l1.x + l1.y);
        }
        // V: this lane's 4 keys (2 t4 + {0, 1, 8, 9}), codes hr * NB .. + NB-1
        uint32_t vw[4][Cfg::NB / 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 2 * t4 + (e & 1) + (e >> 1) * 8;
            if (D == 128) {
                const uint4 w4 = lds128(sv + q8_off<D>(r, hr));
                vw[e][0] = w4.x;
                vw[e][1] = w4.y;
                vw[e][Cfg::NB / 4 - 2] = w4.z;
                vw[e][Cfg::NB / 4 - 1] = w4.w;
            } else {
                const uint2 w2 = lds64(sv + q8_off<D>(r, hr >> 1) + (hr & 1) * 8);
                vw[e][0] = w2.x;
                vw[e][1] = w2.y;
            }
        }
#pragma unroll
        for (int w = 0; w < Cfg::NB / 4; ++w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {     // byte columns 4w + 2hf, + 1
                const uint32_t sel = hf ? 0x7362u : 0x5140u;
                const uint32_t x = __byte_perm(vw[0][w], vw[1][w], sel), y = __byte_perm(vw[2][w], vw[3][w], sel);
                const int nb = 4 * w + 2 * hf;
                float t0 = 0.f, t1 = 0.f, u0 = 0.f, u1 = 0.f;
                mma_rows8_f16(t0, t1, pa0, pa2, e4m3x2_to_f16x2((uint16_t)x), e4m3x2_to_f16x2((uint16_t)y));
                mma_rows8_f16(u0, u1, pa0, pa2, e4m3x2_to_f16x2((uint16_t)(x >> 16)),
                              e4m3x2_to_f16x2((uint16_t)(y >> 16)));
                o[nb][0] = fmaf(vs, t0, o[nb][0]);
                o[nb][1] = fmaf(vs, t1, o[nb][1]);
                o[nb + 1][0] = fmaf(vs, u0, o[nb + 1][0]);
                o[nb + 1][1] = fmaf(vs, u1, o[nb + 1][1]);
            }
        __syncwarp();
    }
    cp_async_wait<0>();
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);

    __syncthreads();
    float *mg = reinterpret_cast<float *>(smem);    // [warp][G][D+2]
    if (head_ok) {
        float *dst = mg + (warp * G + hr) * (D + 2);
#pragma unroll
        for (int nb = 0; nb < Cfg::NB; ++nb) {      // column n of byte nb is d = n * NB + nb
            dst[(2 * t4) * Cfg::NB + nb] = o[nb][0];
            dst[(2 * t4 + 1) * Cfg::NB + nb] = o[nb][1];
        }
        if (t4 == 0) {
            dst[D] = m_run;
            dst[D + 1] = l_run;
        }
    }
    decode_merge<D, G, CLUSTER>(mg, b, b, (long long)gridDim.z, g, Hkv, split, nsplit, nsplit_max, out, ws_ml, ws_o);
}

}  // namespace swa
