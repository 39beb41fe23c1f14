// quantize_device.cuh -- device code of the token-wise INT4 quantizer (Hadamard butterfly, min / max,
// codes, store), shared by the kernels that write the cache.  Its arithmetic is described in
// rotate_quantize.cu; every including file is compiled with -fmad=false.
#pragma once

#include <cfloat>

#include "saw_device.cuh"
#include "saw_internal.h"

namespace saw {
namespace {

constexpr float kHadamardC = 0.0883883461356163f;   // fp32(1/sqrt(128)) = 0x3DB504F3
constexpr float kHadamardC64 = 0.125f;               // 1/sqrt(64), exact
constexpr float kInv15 = 1.0f / 15.0f;               // RN(1/15)
// Codes are read off t = RN(d * 2^16 / s + kGridMagic): t lies in [2^23, 2^24), where the fp32
// spacing is 1, so t = 2^23 + 2^15 + N with N = rint(d * 2^16 / s) (the 2^-16 grid value of the
// quotient) and bits 16..19 of t hold floor(grid + 1/2).
constexpr float kGridMagic = 8421376.0f;             // 2^23 + 2^15
constexpr float kFastScaleMin = 0x1p-100f;           // scales outside [2^-100, 2^100] divide
constexpr float kFastScaleMax = 0x1p100f;
constexpr uint64_t kRqWaitLimitNs = 1000000000ull;

// Head dimension D = 64 (the 64-point transform: no 128-point block fits), 128, or 256 (two
// independent 128-point rotation blocks).  A thread holds one 64-element row (kN = 32 packed pairs);
// a vector is kThreadsPerVec rows; a warp tile is 16 rows of K and the same 16 rows of V.
template <int kD>
struct RqDims {
    static_assert(kD == 64 || kD == 128 || kD == 256, "head dimension");
    static constexpr int kN = 32;                              // packed registers per thread
    static constexpr int kThreadsPerVec = kD / 64;             // 1, 2 or 4
    static constexpr int kTileVecs = 16 / kThreadsPerVec;      // 16, 8 or 4
    static constexpr int kHalfBytes = 2048;                    // K (or V) bytes of one tile
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kCodeBytes = kD / 2;                  // packed codes per vector
};
constexpr int kRqStages = 3;
constexpr int kRqWarps = 4;
constexpr int kRqThreads = 32 * kRqWarps;
template <int kD>
__host__ __device__ constexpr size_t rq_smem_bytes()
{
    return 1024 + size_t(kRqWarps) * kRqStages * RqDims<kD>::kStageBytes + kRqWarps * kRqStages * 8;
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(__byte_perm(u, 0, 0x1044)); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Packed pairs X[8 c .. 8 c + 7] of one block from 16-byte chunk c of its elements 0 .. kN - 1
// (`lo`) and of its elements kN .. 2 kN - 1 (`hi`): X[m] = (x[m], x[m + kN]).
__device__ __forceinline__ void pairs_from_chunk(uint4 lo, uint4 hi, uint64_t X[8])
{
    const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w};
    const uint32_t b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
        X[2 * k] = f2_pack(bf16_lo(a[k]), bf16_lo(b[k]));
        X[2 * k + 1] = f2_pack(bf16_hi(a[k]), bf16_hi(b[k]));
    }
}

// The butterfly stages of the 2 kN elements one thread holds: stages h = 1 .. kN / 2 pair
// registers m and m + h (packed, two IEEE operations per instruction), stage h = kN pairs the two
// halves of each register.  Stages run in ascending h; low index gets a + b, high index a - b.
template <int kN>
__device__ __forceinline__ void fwht_stages(uint64_t X[kN])
{
#pragma unroll
    for (int hb = 1; hb < kN; hb <<= 1) {
#pragma unroll
        for (int i = 0; i < kN; i++) {
            if ((i & hb) == 0) {
                const uint64_t lo = X[i], hi = X[i + hb];
                X[i] = f2_add(lo, hi);
                X[i + hb] = f2_sub(lo, hi);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kN; i++) {
        float lo, hi;
        f2_unpack(X[i], lo, hi);
        X[i] = f2_pack(__fadd_rn(lo, hi), __fsub_rn(lo, hi));
    }
}

template <int kN>
__device__ __forceinline__ void scale_all(uint64_t X[kN], float c)
{
    const uint64_t cc = f2_pack(c, c);
#pragma unroll
    for (int i = 0; i < kN; i++)
        X[i] = f2_mul(X[i], cc);
}

// Stage h = 64 of a 128-point block split over lanes L (elements 0..63, b = 0) and L ^ 1 (elements
// 64..127, b = 1): each lane takes its partner's 64 values by shuffles and forms its own half of the
// stage's outputs: x + partner (lower lane) or partner - x = fma(x, -1, partner) (upper lane).  The
// product is exact, so either is one IEEE rounding of the stage's sum or difference.
__device__ __forceinline__ void exchange_stage64(uint64_t X[32], int b)
{
    const float sg = b ? -1.0f : 1.0f;
    const uint64_t sgn = f2_pack(sg, sg);
#pragma unroll
    for (int i = 0; i < 32; i++) {
        float lo, hi;
        f2_unpack(X[i], lo, hi);
        const uint64_t other = f2_pack(__shfl_xor_sync(0xFFFFFFFFu, lo, 1),
                                       __shfl_xor_sync(0xFFFFFFFFu, hi, 1));
        X[i] = f2_fma(X[i], sgn, other);
    }
}

// min / max over the thread's elements (4 independent chains of three-input min / max)
template <int kN>
__device__ __forceinline__ void block_min_max(const uint64_t X[kN], float &mn, float &mx)
{
    float mns[4], mxs[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float lo, hi;
        f2_unpack(X[i], lo, hi);
        mns[i] = fminf(lo, hi);
        mxs[i] = fmaxf(lo, hi);
    }
#pragma unroll
    for (int i = 4; i < kN; i++) {
        float lo, hi;
        f2_unpack(X[i], lo, hi);
        mns[i & 3] = fmin3(mns[i & 3], lo, hi);
        mxs[i & 3] = fmax3(mxs[i & 3], lo, hi);
    }
    mn = fmin3(mns[0], mns[1], fminf(mns[2], mns[3]));
    mx = fmax3(mxs[0], mxs[1], fmaxf(mxs[2], mxs[3]));
}

// RN(x / 15) for x >= 0: q0 = RN(x c), e = x - 15 q0 (exact in one fma), q1 = RN(q0 + e c) with
// c = RN(1/15) -- the correction step of P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor" (IBM J. Res. Dev. 34(1), 1990).  Checked exhaustively on the
// host: q1 equals the IEEE quotient for all 2^31 - 2^23 non-negative finite fp32 x.
__device__ __forceinline__ float div15(float x)
{
    const float q0 = __fmul_rn(x, kInv15);
    const float e = __fmaf_rn(-q0, 15.0f, x);
    return __fmaf_rn(e, kInv15, q0);
}

// 2^16 / s with relative error below 2^-23, for 2^-100 <= s <= 2^100: the hardware reciprocal
// (max error 1 ulp) refined by one Newton-Raphson step, scaled by 2^16 exactly.
__device__ __forceinline__ float recip_2p16(float s)
{
    float r0;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(s));
    const float e = __fmaf_rn(-s, r0, 1.0f);
    const float r0s = __fmul_rn(r0, 65536.0f);
    return __fmaf_rn(r0s, e, r0s);
}

// Codes from grid values.  With Q = d / s (exact), r16 = (2^16 / s)(1 + e),
// |e| < 2^-23, and t = RN(d r16 + 2^23 + 2^15) = 2^23 + 2^15 + N, N = rint(d r16):
//   |N / 2^16 - Q| <= 2^-17 + 15.0001 * 2^-23 < 0.65 * 2^-16, and |RN(Q) - Q| <= 2^-21 (Q < 16),
// so the grid value g = N / 2^16 lies within 2^-16 of RN(Q).  g + 1/2 is a multiple of 2^-16: if
// it is not an integer it is at least 2^-16 from every integer, RN(Q) + 1/2 lies strictly between
// the same two integers, and rint(RN(Q)) = floor(g + 1/2) = bits 16..19 of t (never more than
// 15).  If it is an integer K (the low 16 bits of t are 0), m = K - 1/2 is the half-integer next
// to Q (0.5 <= m <= 14.5) and the code follows from the sign of one exact remainder: let
// E = d - m s; RN(Q) = m exactly when |Q - m| <= ulp(m) / 2 (m has an even last mantissa bit, so a
// tie also rounds to m), i.e. when |E| <= T = s ulp(m) / 2, and then the code is rint(m) (ties to
// even); otherwise RN(Q) lies on the same side of m as Q and the code is m + sign(E) / 2.  E is a
// multiple of ulp(s) / 4 (d and m s both are), and where |E| <= 2 T it has at most 7 significant
// bits, so RN(E) = fma(-m, s, d) is E itself; where |E| > 2 T, |RN(E)| >= 2 T.  The test
// |RN(E)| <= T is therefore exact, as are T (a power-of-two multiple of s) and the sign, for
// s >= 2^-100.  code_at_half() returns the code of element value y (d = y - min) whose t has zero
// low bits.
__device__ __noinline__ uint32_t code_at_half(float y, float mn, float s, uint32_t t_bits)
{
    const uint32_t cand = (t_bits >> 16) & 15u;
    const float d = __fsub_rn(y, mn);
    const float m = __fsub_rn(static_cast<float>(cand), 0.5f);
    const float e = __fmaf_rn(-m, s, d);
    const float half_ulp = __int_as_float((__float_as_int(m) & 0x7F800000) - (24 << 23));
    const float code = fabsf(e) <= __fmul_rn(s, half_ulp) ? rintf(m) : __fadd_rn(m, copysignf(0.5f, e));
    return static_cast<uint32_t>(code);
}

// The IEEE-divide code (scales outside [2^-100, 2^100]).
__device__ __noinline__ uint32_t code_by_divide(float y, float mn, float s)
{
    const float q = rintf(__fdiv_rn(__fsub_rn(y, mn), s));
    return static_cast<uint32_t>(fminf(fmaxf(q, 0.0f), 15.0f));
}

// Gather byte 2 of t_0..t_7 (the codes of elements e = 0..7) into one word, element e at bits
// 4e: bytes are [k0 | k1 << 4, k2 | k3 << 4, ...] (even index in the low nibble).
__device__ __forceinline__ uint32_t pack8_b2(const uint32_t tt[8])
{
    const uint32_t e01 = __byte_perm(tt[0], tt[2], 0x0062);
    const uint32_t e23 = __byte_perm(tt[4], tt[6], 0x0062);
    const uint32_t even = __byte_perm(e01, e23, 0x5410);   // [k0, k2, k4, k6]
    const uint32_t o01 = __byte_perm(tt[1], tt[3], 0x0062);
    const uint32_t o23 = __byte_perm(tt[5], tt[7], 0x0062);
    const uint32_t odd = __byte_perm(o01, o23, 0x5410);    // [k1, k3, k5, k7]
    return even | (odd << 4);
}

// Unsigned 16-bit minimum of three packed pairs.
__device__ __forceinline__ uint32_t vmin3_u16x2(uint32_t a, uint32_t b, uint32_t c)
{
    return __vimin3_u16x2(a, b, c);
}

// Codes of one thread's elements (held rotated, or raw for the plain INT4 cache, in X) and the
// vector's fp32 scale and zero point, given the vector's min and max.  words[g] (g < kN / 8) holds
// the codes of elements 8 g .. 8 g + 7 and words[kN / 8 + g] those of elements kN + 8 g .. (low
// halves, then high halves of the registers).  Groups of 8 registers are finished one after
// another (the rare exactly half-way elements inside the group), so each group's registers are
// free once its two words exist; scales outside [2^-100, 2^100] take the IEEE divide throughout.
template <int kN>
__device__ __forceinline__ void quantize_block(const uint64_t X[kN], float mn, float mx,
                                               uint32_t words[kN / 4], float &scale_out,
                                               float &zero_out)
{
    float scale = div15(__fsub_rn(mx, mn));
    const bool degenerate = !(scale != 0.0f);
    if (degenerate)
        scale = 0.0f;                               // canonical +0
    zero_out = __fadd_rn(mn, 0.0f);                 // a zero minimum is stored as +0
    scale_out = scale;
    const bool fast = scale >= kFastScaleMin && scale <= kFastScaleMax;
    const bool divide = !fast && !degenerate;       // scales outside [2^-100, 2^100]
    // a degenerate block gets r16 = 0: every t is the magic, code 0, and never flagged
    const float r16 = fast ? recip_2p16(scale) : 0.0f;
    const uint64_t nmn2 = f2_pack(-mn, -mn), r2 = f2_pack(r16, r16);
    const uint64_t m2 = f2_pack(kGridMagic, kGridMagic);

    if (divide) {
        // scales outside [2^-100, 2^100] (rare): every element by the IEEE divide
#pragma unroll
        for (int g = 0; g < kN / 8; g++) {
            uint32_t wl = 0, wh = 0;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float a, b;
                f2_unpack(X[8 * g + e], a, b);
                wl |= code_by_divide(a, mn, scale) << (4 * e);
                wh |= code_by_divide(b, mn, scale) << (4 * e);
            }
            words[g] = wl;
            words[kN / 8 + g] = wh;
        }
        return;
    }
#pragma unroll
    for (int g = 0; g < kN / 8; g++) {
        uint32_t tlo[8], thi[8];
        // the low 16 bits of a t are 0 only at an exactly half-way grid value: f collects the
        // smallest low half (its high half is never 0: bits 16..31 of t hold 0x4B00 | code)
        uint32_t f = 0xFFFFFFFFu;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint64_t d = f2_add(X[8 * g + e], nmn2);   // y - min, one rounding
            const uint64_t t = f2_fma(d, r2, m2);
            float a, b;
            f2_unpack(t, a, b);
            tlo[e] = __float_as_uint(a);
            thi[e] = __float_as_uint(b);
            f = vmin3_u16x2(f, tlo[e], thi[e]);
        }
        if ((f & 0xFFFFu) == 0) {
            // rare: settle each exactly half-way element by the remainder test
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float a, b;
                f2_unpack(X[8 * g + e], a, b);
                if ((tlo[e] & 0xFFFFu) == 0)
                    tlo[e] = code_at_half(a, mn, scale, tlo[e]) << 16;
                if ((thi[e] & 0xFFFFu) == 0)
                    thi[e] = code_at_half(b, mn, scale, thi[e]) << 16;
            }
        }
        words[g] = pack8_b2(tlo);
        words[kN / 8 + g] = pack8_b2(thi);
    }
}

// Store one block's codes (two runs of kN / 2 bytes: low halves, then high halves) and, from the
// vector's first block, its fp16 (scale, zero); flag scales or zero points past fp16's range.
template <int kN>
__device__ __forceinline__ void store_block(uint8_t *dst, const uint32_t words[kN / 4], bool scale_here,
                                            float scale, float zero, uint32_t *scale_dst,
                                            uint32_t *status)
{
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int q = 0; q < kN / 32; q++)
            *reinterpret_cast<uint4 *>(dst + h * (kN / 2) + 16 * q) =
                make_uint4(words[h * (kN / 8) + 4 * q], words[h * (kN / 8) + 4 * q + 1],
                           words[h * (kN / 8) + 4 * q + 2], words[h * (kN / 8) + 4 * q + 3]);
    if (scale_here) {
        const __half2 sz = __halves2half2(__float2half_rn(scale), __float2half_rn(zero));
        *scale_dst = half2_as_u32(sz);
        // fp16 holds magnitudes below 65520: beyond, the stored value is infinite (as the
        // definition's round-to-nearest conversion gives), which the read side cannot use
        if (!(fabsf(scale) < 65520.0f) || !(fabsf(zero) < 65520.0f))
            set_status(status, SAW_DEV_RANGE);
    }
}

// A vector's row of the cache: (page * Hkv + h) * 2 + K/V, times 16, plus the offset in the page.
__device__ __forceinline__ int64_t cache_row(int64_t slot, uint32_t h, int half, int64_t hkv)
{
    return ((((slot >> 4) * hkv + h) * 2 + half) << 4) + (slot & 15);
}

}  // namespace
}  // namespace saw
