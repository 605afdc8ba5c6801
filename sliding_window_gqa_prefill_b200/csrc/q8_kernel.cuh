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

// Two bf16 magnitudes at once: the larger of each half; a NaN in either half of
// either operand stays one.
__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
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

// The larger of `top` and the magnitudes of 8 bf16 (two halves kept apart).
__device__ __forceinline__ uint32_t q8_top(uint32_t top, const uint4 &x) {
    top = bf16x2_max_nan(bf16x2_max_nan(top, x.x & 0x7FFF7FFFu), x.y & 0x7FFF7FFFu);
    return bf16x2_max_nan(bf16x2_max_nan(top, x.z & 0x7FFF7FFFu), x.w & 0x7FFF7FFFu);
}

// The largest finite magnitude of 8 bf16, element by element (rare: where
// q8_top met a NaN or an infinity).
__device__ __forceinline__ uint32_t q8_top_finite(uint32_t top, const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
        top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
    return top;
}

// 8 bf16 as codes.  finite: none of the thread's elements is a NaN or infinite.
__device__ __forceinline__ uint2 q8_codes(const uint4 &x, float inv, bool finite) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[4];
    if (finite) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c[e] = f32x2_to_e4m3x2(__uint_as_float(w[e] << 16) * inv, __uint_as_float(w[e] & 0xFFFF0000u) * inv);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c[e] = f32x2_to_e4m3x2(q8_scaled(__uint_as_float(w[e] << 16), inv),
                                   q8_scaled(__uint_as_float(w[e] & 0xFFFF0000u), inv));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The largest value of `v` over the thread block.
template <int WARPS>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        v = __reduce_max_sync(0xffffffffu, lane < WARPS ? red[lane] : 0u);
    }
    return v;
}

// Append.  One thread block owns one (cache block, KV head, K or V) of one
// sequence, so nothing is shared and no atomic is needed: it reads the new
// tokens of its slots and the codes that stay, takes the largest magnitude of
// both, and writes the new codes -- and the others too, if the scale moved.
// Slots that no token has reached yet (a sequence shorter than the buffer)
// count for nothing and stay as they are.  Each thread holds 4 pieces of 8
// elements (16 bytes of bf16, 8 of codes), so the block is read once and
// stays in registers between the maximum and the rounding.
//
// Bound by memory for long appends if the arithmetic per piece stays small: 4 x
// 4000 tokens, 8 heads, D=128 (99 MB): 31 us with one path for every block and
// scalar maxima (170 instructions a piece), 23.3 with packed maxima, 19.2 with
// whole blocks apart.  A step of one token for 64 sequences takes 7.5 us, mostly
// the latency of position -> block -> scale.
template <int BLOCK, int D>
__global__ void __launch_bounds__(BLOCK * D / 32)
swa_append_q8_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                     uint2 *__restrict__ k_cache, uint2 *__restrict__ v_cache, float *__restrict__ k_scale,
                     float *__restrict__ v_scale, const int32_t *__restrict__ pos, int T, int W, int Hkv,
                     int nblk, int ntouch) {
    constexpr int PIECES = D / 8;             // 8-element pieces per row
    constexpr int ROWS = BLOCK / 4;           // rows per pass, 4 passes
    constexpr int WARPS = BLOCK * D / 1024;
    static_assert(WARPS >= 1 && WARPS <= 32, "whole warps");
    __shared__ uint32_t red[2][WARPS];
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
    // the block's slots s0 .. s1-1, and the token t0 that would go to the first
    const int s0 = blk * BLOCK, s1 = min(W, s0 + BLOCK);
    int t0 = s0 - first;
    if (t0 < 0) t0 += W;
    if (t0 >= T && !(first >= s0 && first < s1)) return;          // no new token here

    const int piece = threadIdx.x % PIECES, r0 = threadIdx.x / PIECES;
    const size_t slot_pieces = (size_t)Hkv * PIECES;
    const uint4 *src = (is_v ? v_new : k_new) + ((size_t)b * T * Hkv + h) * PIECES + piece;
    uint2 *cache = (is_v ? v_cache : k_cache) + ((size_t)b * W * Hkv + h) * PIECES + piece;
    float *sc = (is_v ? v_scale : k_scale) + ((size_t)b * nblk + blk) * Hkv + h;
    uint4 x[4];                               // 8 bf16, or 8 codes in .x, .y
    uint32_t top_new = 0;                     // magnitude, as bf16 bits
    float inv;

    // a block that new tokens fill needs nothing of what it held: most blocks of
    // a long append, so it has code of its own
    if ((long long)t0 + BLOCK <= T && s0 + BLOCK <= W) {
        src += (size_t)(t0 + r0) * slot_pieces;
        cache += (size_t)(s0 + r0) * slot_pieces;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __ldg(src + (size_t)(i * ROWS) * slot_pieces);
#pragma unroll
        for (int i = 0; i < 4; ++i) top_new = q8_top(top_new, x[i]);
        top_new = max(top_new & 0xFFFFu, top_new >> 16);
        const bool finite = top_new < 0x7F80u;
        if (!finite) {
            top_new = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top_new = q8_top_finite(top_new, x[i]);
        }
        top_new = block_max<WARPS>(top_new, red[0]);
        const float scale = q8_scale(__uint_as_float(top_new << 16), inv);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (in_bounds(s0 + r0 + i * ROWS, W))
                cache[(size_t)(i * ROWS) * slot_pieces] = q8_codes(x[i], inv, finite);
        if (threadIdx.x == 0) *sc = scale;
        return;
    }

    const float old_scale = *sc;
    int state[4];                             // 0: leave alone, 1: holds a token, 2: new token
    uint32_t top_old = 0;                     // magnitude, as e4m3 bits
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int slot = s0 + i * ROWS + r0;
        state[i] = 0;
        if (slot >= W) continue;
        int t = slot - first;
        if (t < 0) t += W;
        if (t < T) {
            state[i] = 2;
            x[i] = __ldg(src + (size_t)t * slot_pieces);
        } else if (slot < p0) {
            state[i] = 1;
            const uint2 c = cache[(size_t)slot * slot_pieces];
            x[i].x = c.x;
            x[i].y = c.y;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (state[i] == 2) {
            top_new = q8_top(top_new, x[i]);
        } else if (state[i] == 1) {
            const uint32_t w[2] = {x[i].x & 0x7F7F7F7Fu, x[i].y & 0x7F7F7F7Fu};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t c = (w[e >> 2] >> (8 * (e & 3))) & 0x7Fu;
                top_old = max(top_old, c != 0x7Fu ? c : 0u);
            }
        }
    }
    top_new = max(top_new & 0xFFFFu, top_new >> 16);
    const bool finite = top_new < 0x7F80u;    // of this thread's new elements
    if (!finite) {
        top_new = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (state[i] == 2) top_new = q8_top_finite(top_new, x[i]);
    }
    top_new = block_max<WARPS>(top_new, red[0]);
    top_old = block_max<WARPS>(top_old, red[1]);
    // the scale of a block that holds nothing yet may be anything: used only
    // where a held code is not zero
    float top = __uint_as_float(top_new << 16);
    if (top_old) top = fmaxf(top, f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)top_old)).x * old_scale);
    const float scale = q8_scale(top, inv);
    const bool moved = scale != old_scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (state[i] == 0 || (state[i] == 1 && !moved)) continue;
        const int slot = s0 + i * ROWS + r0;
        if (!in_bounds(slot, W)) continue;
        uint2 codes;
        if (state[i] == 2) {
            codes = q8_codes(x[i], inv, finite);
        } else {
            const uint32_t w[2] = {x[i].x, x[i].y};
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[e >> 1] >> (16 * (e & 1)))));
                // two products, not one by old_scale * inv: that may overflow
                c[e] = f32x2_to_e4m3x2(v.x * old_scale * inv, v.y * old_scale * inv);
            }
            codes = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        }
        cache[(size_t)slot * slot_pieces] = codes;
    }
    if (threadIdx.x == 0 && moved) *sc = scale;
}

// The cached window widened to bf16 (exact) for the chunk pre-fill: kd, vd
// [B, W, Hkv, D].  Slots that no query of the chunk sees -- those no token has
// reached, and of a full buffer the one that holds position start - W -- become
// zeros, so that the attention's masked products there stay 0 whatever they
// hold.  16 codes of K and of V per thread and step; grid y the sequence, x
// strides over its vectors, slot and vector of the row carried along rather than
// divided out of an index each step (13.6 us at B=2, W=4096, 8 heads of 128; now
// 11.8); the scale's index still takes two divisions, by `block` and head_vec.
__global__ void __launch_bounds__(256)
swa_widen_q8_kernel(const uint4 *__restrict__ k_cache, const uint4 *__restrict__ v_cache,
                    const float *__restrict__ k_scale, const float *__restrict__ v_scale,
                    const int32_t *__restrict__ pos, uint4 *__restrict__ kd, uint4 *__restrict__ vd, int W, int Hkv,
                    int head_vec, int block, int nblk) {
    const int row_vec = Hkv * head_vec;                  // 16-code vectors per slot
    const int b = blockIdx.y;
    const int p = __ldg(pos + b);
    const int unseen = p < W ? -1 : p % W;
    const size_t base = (size_t)b * W * row_vec;
    const long long first = blockIdx.x * (long long)blockDim.x + threadIdx.x, step = (long long)gridDim.x * blockDim.x;
    int c = (int)(first % row_vec);
    long long slot = first / row_vec;
    const int step_c = (int)(step % row_vec);
    const long long step_slot = step / row_vec;
    for (; slot < W; slot += step_slot, c += step_c) {
        if (c >= row_vec) {
            c -= row_vec;
            if (++slot >= W) break;
        }
        const bool there = slot < p && slot != unseen;
        const size_t i = base + (size_t)slot * row_vec + c;
        const size_t si = ((size_t)b * nblk + slot / block) * Hkv + c / head_vec;
        if (!in_bounds(slot / block, nblk)) continue;
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
// Arithmetic, per 16 keys and warp (G query heads of the group, at most 8):
//  * S = Q K^T on the codes themselves (mma.sync m16n8k32, e4m3): q, brought by a
//    power of two to a largest magnitude in [2^7, 2^8), is the sum of two e4m3
//    numbers, hi + lo / 16, exactly but for what lies below 2^-21 of that
//    largest element (a bf16 has 8 significant bits, e4m3 two times 4).  hi are
//    rows 0..7 of the 16-row tile, lo rows 8..15, so the split costs nothing.
//    The K scale, the softmax scale and the power of two are one fp32 factor.
//  * P is rounded to f16 (2^-11 relative; bf16's 2^-8 in the 16-bit cache's
//    kernel) and l sums it as rounded.  P is 2^7 larger than 2^(s - offset), at
//    most 2^15, so weights down to 2^-21 of the largest keep all their bits and
//    those down to 2^-31 some: a long tail of small weights is not lost, as it
//    would be in 8 bits.
//  * O^T = V^T P^T (mma.sync m16n8k16, f16): V^T as the 16-row operand fills the
//    tile (16 columns of d by 16 keys), and the P of a lane is its fragment of
//    P^T as it stands.  Codes widen exactly to f16; the product of 16 keys starts
//    from zero and joins O by one fp32 FMA with the block's scale.
// The order of d inside a product is free as long as both operands agree, and
// the order of O's rows is free until they are written; both are chosen so that
// a lane's fragments are 16 consecutive codes of one row: K is read by one
// 16-byte shared load per row and half, V by one per key, and the bytes of two
// keys are paired by byte permutes.
//
// Measured at B=64, W=4096, 32 / 8 heads, D=128: 88 us, 6.1 TB/s (100 to 104 in
// loops of a tenth of a second and more, where the power cap lowers the clock:
// the ALU is half busy with the conversions).  With four
// splits to a window instead of one (3.46 rounds of blocks instead of less than
// one, and their merge) 99 to 101 us, and the following on top of that: with
// both products in f16 and the heads as rows of both it took 114 to 142 us (the
// 16-bit copies of K cost registers, and the O product half its rows); with K
// alone in f16 104 us.  Four blocks of four warps to an SM, 3 stages of 16 keys:
// two blocks with more stages 117 to 121 us, stages of 32 keys 100 us.
//
// The codes of kQ8Stage keys come into a warp's own ring as two TMA boxes (rows
// of one head, K and V) that one lane issues, so copying costs the warp a
// handful of instructions.
constexpr int kQ8Stage = 16;           // keys per TMA box
constexpr int kQ8Warps = 4;
// O sums up to 2^24 keys of P up to 2^15 times 448 V scales: below 2^108 for
// scales up to 2^60.  From the first larger one on a warp holds O 2^-60 times, so
// that scales up to 2^119 stay below 2^107; only beside such values do those
// below 2^-73 lose bits.
constexpr float kQ8LargeScale = 1152921504606846976.f, kQ8DownLog2 = 60.f, kQ8Down = 1.f / kQ8LargeScale;

template <int D, int G>
struct DecodeQ8Cfg {
    static constexpr int CH = D / 16;                          // 16-byte chunks per key row
    static constexpr int TILE_BYTES = kQ8Stage * D;            // K (or V) codes of one stage
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int STAGES = 3;
    static constexpr int WARP_RING = STAGES * STAGE_BYTES;
    static constexpr int RING_BYTES = kQ8Warps * WARP_RING;
    static constexpr int KSTEPS = D / 32;                      // MMA k-steps of S
    static constexpr int MT = D / 16;                          // 16-row tiles of O^T
    static constexpr int MERGE_BYTES = (kQ8Warps + 1) * G * (D + 2) * 4;
    static constexpr int OFF_BAR = RING_BYTES > MERGE_BYTES ? RING_BYTES : MERGE_BYTES;
    static constexpr int OFF_ABORT = OFF_BAR + kQ8Warps * STAGES * 8;
    static constexpr int SMEM_BYTES = OFF_ABORT + 8 + 1024;    // slack for 1024-byte alignment
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(G >= 1 && G <= 8, "group size 1 to 8 (the rows 0..7 of the MMA tile)");
    static_assert(OFF_BAR % 8 == 0, "barrier alignment");
};

// Shared-memory offset of 16-byte chunk `ch` of code row `r`, as TMA places it:
// 128-byte swizzle for D = 128 (chunk ^ row mod 8), 64-byte for D = 64 (chunk ^
// (row / 2) mod 4).  The V loads of a phase (4 rows, two apart, x 2 chunks) and
// the K loads (2 rows x 4 chunks) meet at most two to a bank.
template <int D>
__device__ __forceinline__ uint32_t q8_off(int r, int ch) {
    if (D == 128) return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4));
    return (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
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

// D(16x8, fp32) += A(16x32, e4m3) B(32x8, e4m3), warp-wide.
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A(16x16, f16) B(16x8, f16), warp-wide, fp32.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// MODE kDecodeWindow (splits merged by swa_decode_combine_kernel) or
// kDecodeWindowCluster (the splits of a window are the blocks of a cluster).
template <int D, int G, int MODE>
__global__ void __launch_bounds__(kQ8Warps * 32, 4)
swa_decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __nv_bfloat16 *__restrict__ q, const float *__restrict__ k_scale,
                     const float *__restrict__ v_scale, const int32_t *__restrict__ pos,
                     __nv_bfloat16 *__restrict__ out, float2 *__restrict__ ws_ml, float *__restrict__ ws_o, int Hkv,
                     int W, int nsplit_max, float scale_log2, int split_len, int kv_rep, int block_log2, int nblk) {
    constexpr bool CLUSTER = MODE == kDecodeWindowCluster;
    using Cfg = DecodeQ8Cfg<D, G>;
    constexpr int CH = Cfg::CH;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));

    const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int Hq = Hkv * G;
    const int p = __ldg(pos + b);
    if (p < 0) {                                    // invalid position: record, write nothing
        if (threadIdx.x == 0 && split == 0 && g == 0) record_status(kStatusInvalid);
        return;
    }
    const int L = (p >= W - 1) ? W : p + 1;
    constexpr int kClusterKeys = kDecodeClusterSplits * kQ8Stage;
    const int split_keys = CLUSTER ? (L + kClusterKeys - 1) / kClusterKeys * kQ8Stage : split_len;
    if (!CLUSTER && (long long)split * split_keys >= L) return;
    const int begin = (int)min((long long)split * split_keys, (long long)L);
    const int end = min(L, begin + split_keys);
    const int nsplit = (L + split_keys - 1) / split_keys;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hr = lane >> 2, t4 = lane & 3;
    const bool head_ok = hr < G;
    const uint32_t ring = smem_addr(smem) + warp * Cfg::WARP_RING;
    const uint32_t bars = smem_addr(smem) + Cfg::OFF_BAR + warp * Cfg::STAGES * 8;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Cfg::OFF_ABORT);
    const unsigned long long limit = g_wait_limit_ns;

    const int Hkv_mem = Hkv / kv_rep, gk = g / kv_rep;
    const float *ksb = k_scale + (size_t)b * nblk * Hkv_mem + gk;
    const float *vsb = v_scale + (size_t)b * nblk * Hkv_mem + gk;

    const int nst = (end - begin + kQ8Stage - 1) / kQ8Stage;      // stages of the split; this warp's:
    const int mine = (nst > warp) ? (nst - warp + kQ8Warps - 1) / kQ8Warps : 0;

    // lane 0: the next of this warp's stages into ring slot `slot`
    int issue_key = begin + warp * kQ8Stage;
    auto issue = [&](int slot) {
        const uint32_t st = ring + slot * Cfg::STAGE_BYTES, bar = bars + slot * 8;
        mbar_arrive_expect_tx(bar, Cfg::STAGE_BYTES);
        const int k0 = checked_coord(issue_key, W);               // rows past W arrive as zeros
        tma_load_4d(st, &tm_k, bar, 0, gk, k0, b);
        tma_load_4d(st + Cfg::TILE_BYTES, &tm_v, bar, 0, gk, k0, b);
        issue_key += kQ8Warps * kQ8Stage;
    };
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int s = 0; s < kQ8Warps * Cfg::STAGES; ++s) mbar_init(smem_addr(smem) + Cfg::OFF_BAR + 8 * s, 1);
        mbar_init_fence();
    }
    __syncthreads();
    if (lane == 0)
        for (int i = 0; i < Cfg::STAGES && i < mine; ++i) issue(i);
    __syncwarp();

    // q of head hr times 2^-x as hi + lo / 16: k-step j = 2c + n takes d = (4c +
    // t4) * 16 + 8n + {0..3 | 4..7}
    uint32_t qa[Cfg::KSTEPS][4];
    float qfac;                                     // scale log2(e) 2^x
    {
        const __nv_bfloat16 *qp = q + ((size_t)b * Hq + g * G + (head_ok ? hr : 0)) * D;
        uint32_t raw[Cfg::KSTEPS][4];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < Cfg::KSTEPS; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int d = (4 * (j >> 1) + t4) * 16 + 8 * (j & 1) + 2 * w;
                raw[j][w] = head_ok ? __ldg(reinterpret_cast<const uint32_t *>(qp + d)) : 0u;
                const uint32_t lo = raw[j][w] & 0x7FFFu, hi = (raw[j][w] >> 16) & 0x7FFFu;
                top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
            }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent field of the largest |q| (at least 8: below that q is 0 to any
        // key that fits), brought to that of 2^7
        const int ef = max(8, (int)(top >> 7));
        const float down = __uint_as_float((uint32_t)(261 - ef) << 23);
        qfac = scale_log2 * __uint_as_float((uint32_t)(ef - 7) << 23);
#pragma unroll
        for (int j = 0; j < Cfg::KSTEPS; ++j)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t hi = 0, lo = 0;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t x = raw[j][2 * hf + w];
                    // not finite: NaN, as neither part could say so otherwise
                    const float2 y = make_float2(q8_scaled(__uint_as_float(x << 16), down),
                                                 q8_scaled(__uint_as_float(x & 0xFFFF0000u), down));
                    const uint32_t c = f32x2_to_e4m3x2(y.x, y.y);
                    const float2 r = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)c));
                    hi |= c << (16 * w);
                    lo |= f32x2_to_e4m3x2((y.x - r.x) * 16.f, (y.y - r.y) * 16.f) << (16 * w);
                }
                qa[j][2 * hf] = hi;
                qa[j][2 * hf + 1] = lo;
            }
    }

    float m_run = -INFINITY, l_run = 0.f;           // of head hr, this lane's keys
    // O^T: rows d = hr * MT * 2 + 2 mt (o[mt][0], [1]) and + 1 ([2], [3]), heads 2 t4 + {0, 1}
    float2 o[Cfg::MT][2];
#pragma unroll
    for (int mt = 0; mt < Cfg::MT; ++mt) o[mt][0] = o[mt][1] = make_float2(0.f, 0.f);

    // byte offsets of this lane's fragments in a stage: K rows hr (+ 8), V rows
    // 2 t4 + {0, 1, 8, 9}; 16 rows further on the swizzle repeats
    uint32_t koff[2][CH / 4], voff[4];
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int c = 0; c < CH / 4; ++c) koff[nb][c] = ring + q8_off<D>(nb * 8 + hr, c * 4 + t4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int r = 2 * t4 + (e & 1) + (e >> 1) * 8;
        voff[e] = ring + Cfg::TILE_BYTES + (D == 128 ? q8_off<D>(r, hr) : q8_off<D>(r, hr >> 1) + (hr & 1) * 8);
    }
    float vfac = 1.f;                               // O is held vfac times
    constexpr int HALVES = kQ8Stage / 16;
    float ks[HALVES], vs[HALVES];
    // one scale per 16 keys, loaded a stage ahead of its use
    auto load_scales = [&](int stage0) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            const int blk = min(stage0 + 16 * h, end - 1) >> block_log2;
            if (!in_bounds(blk, nblk)) continue;
            // below 2^32: more scales would stand for over 4 TB of codes
            const uint32_t at = (uint32_t)blk * (uint32_t)Hkv_mem;
            ks[h] = __ldg(ksb + at);
            vs[h] = __ldg(vsb + at);
        }
    };
    int stage0 = begin + warp * kQ8Stage;
    if (mine > 0) load_scales(stage0);
    uint32_t slot = 0, phase = 0;
    for (int i = 0; i < mine; ++i) {
        const uint32_t st = slot * Cfg::STAGE_BYTES;
        float kf[HALVES];
        float2 vs2[HALVES];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            kf[h] = ks[h] * qfac;
            if (vs[h] * vfac > kQ8LargeScale) {      // uniform; at most once
                vfac = kQ8Down;
#pragma unroll
                for (int mt = 0; mt < Cfg::MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        o[mt][r].x *= kQ8Down;
                        o[mt][r].y *= kQ8Down;
                    }
            }
            vs2[h] = make_float2(vs[h] * vfac, vs[h] * vfac);
        }
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bars + slot * 8, phase, abort_flag, limit))) {
            // let what this warp started land before the block goes on
            if (lane == 0)
                for (int j = i; j < min(mine, i + Cfg::STAGES); ++j)
                    mbar_drain_bounded(bars + (j % Cfg::STAGES) * 8, (j / Cfg::STAGES) & 1, kDrainLimitNs);
            __syncwarp();
            break;
        }
        if (i + 1 < mine) load_scales(stage0 + kQ8Warps * kQ8Stage);
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            const int key0 = stage0 + 16 * h;
            if (key0 >= end) break;
            const uint32_t at = st + h * 16 * D;
            // rows 0..7: q hi, rows 8..15: q lo, of keys 8 nb + 2 t4 + {0, 1}
            float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int c = 0; c < CH / 4; ++c) {
                    const uint4 w = lds128(koff[nb][c] + at);
                    mma_e4m3(s[nb], qa[2 * c], w.x, w.y);
                    mma_e4m3(s[nb], qa[2 * c + 1], w.z, w.w);
                }
            const bool tail = key0 + 16 > end;       // uniform; a branch, not predication, keeps it off the others
            float sc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[e] = fmaf(s[e >> 1][2 + (e & 1)], 0.0625f, s[e >> 1][e & 1]) * kf[h];
            if (tail) {
                asm volatile("" ::: "memory");
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key0 + 2 * t4 + (e & 1) + (e >> 1) * 8 >= end) sc[e] = -INFINITY;
            }
            float mx = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
            if (__any_sync(0xffffffffu, mx > m_run + 8.0f)) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                float alpha = 1.f;
                if (mx > m_run) {                    // uniform across the quad
                    alpha = ex2_approx(m_run - mx);
                    l_run *= alpha;
                    m_run = mx;
                }
                // O^T has the heads across the lanes of a quad
                const float2 a2 = make_float2(__shfl_sync(0xffffffffu, alpha, 8 * t4),
                                              __shfl_sync(0xffffffffu, alpha, 8 * t4 + 4));
#pragma unroll
                for (int mt = 0; mt < Cfg::MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        o[mt][r].x *= a2.x;
                        o[mt][r].y *= a2.y;
                    }
            }
            const float off = 7.0f - m_run;
            float pw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) pw[e] = ex2_approx(sc[e] + off);   // of rows past G too: never read
            const uint32_t pb0 = pack_f16x2(pw[0], pw[1]), pb1 = pack_f16x2(pw[2], pw[3]);
            {
                const float2 l0 = f16x2_to_f32x2(pb0), l1 = f16x2_to_f32x2(pb1);
                l_run += (l0.x + l0.y) + (l1.x + l1.y);
            }
            // V: this lane's 4 keys (2 t4 + {0, 1, 8, 9}), codes d = hr * 2 MT .. + 2 MT - 1
            uint32_t vw[4][Cfg::MT / 2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (D == 128) {
                    const uint4 w4 = lds128(voff[e] + at);
                    vw[e][0] = w4.x;
                    vw[e][1] = w4.y;
                    vw[e][Cfg::MT / 2 - 2] = w4.z;
                    vw[e][Cfg::MT / 2 - 1] = w4.w;
                } else {
                    const uint2 w2 = lds64(voff[e] + at);
                    vw[e][0] = w2.x;
                    vw[e][1] = w2.y;
                }
            }
            if (tail) {
                // a slot behind the last key may hold anything; its weight of 0 has
                // to meet a 0
                asm volatile("" ::: "memory");
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key0 + 2 * t4 + (e & 1) + (e >> 1) * 8 >= end) {
#pragma unroll
                        for (int w = 0; w < Cfg::MT / 2; ++w) vw[e][w] = 0u;
                    }
            }
#pragma unroll
            for (int mt = 0; mt < Cfg::MT; ++mt) {   // byte columns 2 mt, 2 mt + 1
                const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
                const uint32_t x = __byte_perm(vw[0][mt >> 1], vw[1][mt >> 1], sel);
                const uint32_t y = __byte_perm(vw[2][mt >> 1], vw[3][mt >> 1], sel);
                float t[4];
                mma_f16(t, e4m3x2_to_f16x2((uint16_t)x), e4m3x2_to_f16x2((uint16_t)(x >> 16)),
                        e4m3x2_to_f16x2((uint16_t)y), e4m3x2_to_f16x2((uint16_t)(y >> 16)), pb0, pb1);
                o[mt][0] = ffma2(vs2[h], make_float2(t[0], t[1]), o[mt][0]);
                o[mt][1] = ffma2(vs2[h], make_float2(t[2], t[3]), o[mt][1]);
            }
        }
        __syncwarp();                                // every lane has read the stage
        if (lane == 0 && i + Cfg::STAGES < mine) issue(slot);
        stage0 += kQ8Warps * kQ8Stage;
        if (++slot == Cfg::STAGES) {
            slot = 0;
            phase ^= 1;
        }
    }
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
    if (vfac != 1.f) {                              // {m, l, o} and {m + x, 2^-x l, 2^-x o} are the same
        l_run *= kQ8Down;
        m_run += kQ8DownLog2;
    }

    __syncthreads();
    float *mg = reinterpret_cast<float *>(smem);    // [warp][G][D+2]
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int h = 2 * t4 + hh;
        if (h >= G) break;
        float *dst = mg + (warp * G + h) * (D + 2) + hr * 2 * Cfg::MT;
#pragma unroll
        for (int mt = 0; mt < Cfg::MT; ++mt) {
            dst[2 * mt] = hh ? o[mt][0].y : o[mt][0].x;
            dst[2 * mt + 1] = hh ? o[mt][1].y : o[mt][1].x;
        }
    }
    if (head_ok && t4 == 0) {
        mg[(warp * G + hr) * (D + 2) + D] = m_run;
        mg[(warp * G + hr) * (D + 2) + D + 1] = l_run;
    }
    decode_merge<D, G, CLUSTER, kQ8Warps>(mg, b, b, (long long)gridDim.z, g, Hkv, split, nsplit, nsplit_max, out, ws_ml,
                                          ws_o);
}

}  // namespace swa
