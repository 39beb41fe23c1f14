// rope_append.cu -- rotary positions, applied where new tokens enter the INT4 paged cache.
//
// Rotary embedding of a head vector x at position p, over its first R elements (pairs (a, b) =
// (x[i], x[i + R/2]) in the halves layout, (x[2i], x[2i + 1]) in the interleaved one, i < R/2):
//     a' = a cos(p f_i) - b sin(p f_i),   b' = b cos(p f_i) + a sin(p f_i).
// The cosines and sines come from a table, fp32 [positions][R] (R/2 cosines, then R/2 sines), filled
// once by rope_table_kernel from the frequencies f_i, which carry the scaling for long contexts.
//
// rope_append_kernel takes one step's q, k and v: q rows are rotated and written as bf16; k rows are
// rotated, rounded to bf16 (the type a model holds its keys in: the cache then has exactly the bits
// of rotating first and appending with saw_rotate_quantize_paged), and then, like v rows, Hadamard
// transformed, quantized and scattered (quantize_device.cuh).  Every product and sum of the rotary
// step is one IEEE fp32 operation (this file is compiled with -fmad=false), so codes are defined
// bit for bit.
//
// The two halves of the work are bound by different things: the q rows by memory (2/3 of all bytes
// at 4 query heads per kv head), the quantizer by its arithmetic.  One launch holds both: some CTAs
// of the grid stream q rows, the others quantize tiles, side by side on every SM.
#include <algorithm>

#include "quantize_device.cuh"

namespace saw {
namespace {

struct RopeTableParams {
    float *table;
    int64_t first, count;
    int32_t half;              // R / 2
    float amplitude;
    double turns[128];         // f_i / (2 pi): turns per position
};

// One thread per (position, pair).  The angle in turns is formed in fp64 (position 2^20 at one
// radian per position keeps 33 bits below the point), reduced to [-1/2, 1/2] exactly and only then
// rounded to fp32.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p)
{
    const int64_t n = p.count * p.half;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / p.half;
        const int col = static_cast<int>(i - row * p.half);
        const double x = static_cast<double>(p.first + row) * p.turns[col];
        const float r = static_cast<float>(x - rint(x));
        float s, c;
        sincospif(2.0f * r, &s, &c);
        p.table[row * 2 * p.half + col] = c * p.amplitude;
        p.table[row * 2 * p.half + p.half + col] = s * p.amplitude;
    }
}

struct RopeParams {
    const int64_t *slots;
    const int64_t *positions;
    const float *table;
    int64_t num_positions;
    int64_t num_slots;         // num_pages * 16
    int64_t num_vecs;          // T * Hkv
    int64_t num_tokens;
    uint32_t num_tiles;        // of 32 rows of 64 elements, K tiles and V tiles in turn
    int32_t hkv, hq;
    int32_t rotary;            // R, a multiple of 16
    int32_t interleaved;
    int32_t strided;
    int32_t kv_ctas;           // CTAs [0, kv_ctas) quantize, the others rotate q rows
    int32_t q_slices;          // a q item is one token's heads [slice * slice_heads, + slice_heads)
    int32_t slice_heads;
    int64_t q_stride;          // bf16 elements between tokens of q
    const uint16_t *q;
    uint16_t *q_out;
    uint8_t *kv_pages;
    uint32_t *scales;
    float *mass;
    uint32_t *status;
    float neg_zero;            // -0 (rotate_word)
};

// Where token `tok` goes: its slot, or -1 for a token that is skipped (a negative slot, or a slot or
// position out of range, which `report` flags).
__device__ __forceinline__ int64_t token_slot(const RopeParams &p, int64_t slot, int64_t pos, bool report)
{
    if (slot < 0)
        return -1;
    const uint32_t bad = (slot >= p.num_slots ? SAW_DEV_BAD_SLOT : 0u) |
                         (pos < 0 || pos >= p.num_positions ? SAW_DEV_BAD_POSITION : 0u);
    if (bad != 0) {
        if (report)
            set_status(p.status, bad);
        return -1;
    }
    return slot;
}

// a c + b s' for a pair of bf16 elements, rounded to bf16 (s' carries the sign).  The products are
// fused multiply-adds with -0, exactly the rounded product, whose -0 the compiler cannot see: as
// packed multiplies, one of them was contracted into the packed addition in spite of its rounding
// modifier, and the sum then differed in its last bit.
__device__ __forceinline__ uint32_t rotate_word(uint32_t own, uint32_t other, uint64_t c, uint64_t s, uint64_t neg0)
{
    const uint64_t a = f2_pack(bf16_lo(own), bf16_hi(own)), b = f2_pack(bf16_lo(other), bf16_hi(other));
    float lo, hi;
    f2_unpack(f2_add(f2_fma(a, c, neg0), f2_fma(b, s, neg0)), lo, hi);
    return bf16x2_as_u32(lo, hi);
}

// Halves layout: 8 elements `own` of a head vector and the 8 of their partners; cos / sin at the
// chunk's 8 pairs, the sine's sign flipped for the first half.
__device__ __forceinline__ uint4 rotate_halves(uint4 own, uint4 other, const float *cos, const float *sin, bool first,
                                               uint64_t neg0)
{
    const float4 c0 = __ldg(reinterpret_cast<const float4 *>(cos)), c1 = __ldg(reinterpret_cast<const float4 *>(cos) + 1);
    const float4 s0 = __ldg(reinterpret_cast<const float4 *>(sin)), s1 = __ldg(reinterpret_cast<const float4 *>(sin) + 1);
    const uint64_t flip = first ? 0x8000000080000000ull : 0ull;
    return make_uint4(rotate_word(own.x, other.x, f2_pack(c0.x, c0.y), f2_pack(s0.x, s0.y) ^ flip, neg0),
                      rotate_word(own.y, other.y, f2_pack(c0.z, c0.w), f2_pack(s0.z, s0.w) ^ flip, neg0),
                      rotate_word(own.z, other.z, f2_pack(c1.x, c1.y), f2_pack(s1.x, s1.y) ^ flip, neg0),
                      rotate_word(own.w, other.w, f2_pack(c1.z, c1.w), f2_pack(s1.z, s1.w) ^ flip, neg0));
}

__device__ __forceinline__ uint32_t swap_halves(uint32_t w) { return __byte_perm(w, 0, 0x1032); }

// Interleaved layout: 8 elements, their 4 pairs' cos / sin.
__device__ __forceinline__ uint4 rotate_pairs(uint4 own, const float *cos, const float *sin, uint64_t neg0)
{
    const float4 c = __ldg(reinterpret_cast<const float4 *>(cos)), s = __ldg(reinterpret_cast<const float4 *>(sin));
    return make_uint4(rotate_word(own.x, swap_halves(own.x), f2_pack(c.x, c.x), f2_pack(-s.x, s.x), neg0),
                      rotate_word(own.y, swap_halves(own.y), f2_pack(c.y, c.y), f2_pack(-s.y, s.y), neg0),
                      rotate_word(own.z, swap_halves(own.z), f2_pack(c.z, c.z), f2_pack(-s.z, s.z), neg0),
                      rotate_word(own.w, swap_halves(own.w), f2_pack(c.w, c.w), f2_pack(-s.w, s.w), neg0));
}

// The q rows: a warp takes one token's heads (or a slice of them), each lane one 16-byte chunk of a
// head and the same chunk of every 32 / (D / 8)-th head after it.  The partner's chunk comes from
// its lane by shuffles.
template <int kD>
__device__ __forceinline__ void rotate_queries(const RopeParams &p)
{
    constexpr int kChunks = kD / 8;                // 16-byte chunks of a head
    constexpr int kHeads = 32 / kChunks;           // heads a warp holds at once
    const int lane = threadIdx.x & 31;
    const int chunk = lane % kChunks, sub = lane / kChunks;
    const int hc = p.rotary / 16;                  // chunks of half the rotary part
    const bool turned = chunk < 2 * hc, first = chunk < hc;
    const int partner = (lane - chunk) + (first ? chunk + hc : chunk - hc);
    const uint64_t neg0 = f2_pack(p.neg_zero, p.neg_zero);
    const int64_t items = p.num_tokens * p.q_slices;
    const int64_t step = static_cast<int64_t>(gridDim.x - p.kv_ctas) * kRqWarps;
    for (int64_t it = static_cast<int64_t>(blockIdx.x - p.kv_ctas) * kRqWarps + (threadIdx.x >> 5); it < items; it += step) {
        const int64_t tok = it / p.q_slices;
        const int h0 = static_cast<int>(it - tok * p.q_slices) * p.slice_heads, h1 = min(p.hq, h0 + p.slice_heads);
        const int64_t pos = p.positions[tok];
        if (token_slot(p, p.slots[tok], pos, lane == 0 && h0 == 0) < 0)
            continue;
        const float *row = p.table + pos * p.rotary;
        const float *cos = row + (p.interleaved ? 4 * chunk : 8 * (first ? chunk : chunk - hc));
        const float *sin = cos + p.rotary / 2;
        const uint16_t *src = p.q + tok * p.q_stride + 8 * chunk;
        uint16_t *dst = p.q_out + tok * p.hq * kD + 8 * chunk;
#pragma unroll 4
        for (int h = h0 + sub; h - sub < h1; h += kHeads) {
            const bool in = h < h1;
            uint4 x = in ? *reinterpret_cast<const uint4 *>(src + h * kD) : make_uint4(0u, 0u, 0u, 0u);
            if (p.interleaved) {
                if (turned)
                    x = rotate_pairs(x, cos, sin, neg0);
            } else {
                uint4 y;
                y.x = __shfl_sync(0xFFFFFFFFu, x.x, partner);
                y.y = __shfl_sync(0xFFFFFFFFu, x.y, partner);
                y.z = __shfl_sync(0xFFFFFFFFu, x.z, partner);
                y.w = __shfl_sync(0xFFFFFFFFu, x.w, partner);
                if (turned)
                    x = rotate_halves(x, y, cos, sin, first, neg0);
            }
            if (in)
                *reinterpret_cast<uint4 *>(dst + h * kD) = x;
        }
    }
}

// The k and v rows: tiles of 32 rows of 64 elements, K and V tiles in turn, through a warp's ring of
// tensor copies; lane = row.  (The quantizer's own kernel gives half its lanes to K and half to V;
// here a tile is one of them, so that the rotary step never runs with half the lanes idle.)
template <bool kRotate, int kD>
__device__ __forceinline__ void quantize_tiles(const CUtensorMap &tk, const CUtensorMap &tv, const RopeParams &p,
                                               uint8_t *smem)
{
    using Dims = RqDims<kD>;
    constexpr int kN = Dims::kN;
    constexpr int kTpv = Dims::kThreadsPerVec;
    constexpr int kTileVecs = 32 / kTpv;
    constexpr int kStageBytes = 4096;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t W = p.kv_ctas * kRqWarps, wg = blockIdx.x * kRqWarps + warp;
    if (wg >= p.num_tiles)
        return;
    const int n = static_cast<int>((p.num_tiles - wg + W - 1) / W);   // this warp's tiles: wg + i W
    const uint32_t ring = smem_u32(smem) + warp * kRqStages * kStageBytes;
    const uint32_t bar0 = smem_u32(smem + kRqWarps * kRqStages * kStageBytes) + warp * kRqStages * 8;
    if (lane == 0)
        for (int i = 0; i < kRqStages; i++)
            mbar_init(bar0 + 8 * i, 1);
    mbar_init_fence();
    __syncwarp();

    int issued = 0;
    // queue tile wg + issued W: two boxes of 16 rows (of one token's rows, or of whole tokens)
    auto issue = [&]() {
        if (issued < n && lane == 0) {
            const uint32_t tile = wg + issued * W;
            const uint32_t dst = ring + (issued % kRqStages) * kStageBytes, bar = bar0 + 8 * (issued % kRqStages);
            const CUtensorMap *map = (tile & 1) ? &tv : &tk;
            mbar_arrive_expect_tx(bar, kStageBytes);
#pragma unroll
            for (int b = 0; b < 2; b++) {
                const uint32_t row = (tile >> 1) * 32 + 16 * b;
                if (p.strided) {
                    const uint32_t per = static_cast<uint32_t>(p.hkv) * kTpv;   // rows of a token
                    const uint32_t tok = row / per;
                    tma_load_3d(dst + 2048 * b, map, 0, static_cast<int32_t>(row - tok * per), static_cast<int32_t>(tok), bar);
                } else {
                    tma_load_2d(dst + 2048 * b, map, 0, static_cast<int32_t>(row), bar);
                }
            }
        }
        issued++;
    };
    for (int k = 0; k < kRqStages - 1; k++)
        issue();

    const int part = lane % kTpv, vt = lane / kTpv;
    const uint32_t num_vecs = static_cast<uint32_t>(p.num_vecs), hkv = static_cast<uint32_t>(p.hkv);
    const int hc = p.rotary / 16;
    const uint64_t neg0 = f2_pack(p.neg_zero, p.neg_zero);
    int i = 0;
    for (; i < n; i++) {
        issue();
        const uint32_t tile = wg + i * W;
        const int half = tile & 1;
        const uint32_t vec_raw = (tile >> 1) * kTileVecs + vt;
        const uint32_t vec = min(vec_raw, num_vecs - 1);
        const uint32_t tok = vec / hkv, h = vec - tok * hkv;
        const int64_t pos = p.positions[tok];
        const int64_t slot = vec_raw < num_vecs ? token_slot(p, p.slots[tok], pos, part == 0 && half == 0) : -1;
        const int stg = i % kRqStages;
        const bool ok = mbar_wait_bounded(bar0 + 8 * stg, (i / kRqStages) & 1, kRqWaitLimitNs);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
            if (lane == 0)
                set_status(p.status, SAW_DEV_WAIT_TIMEOUT);
            break;
        }
        // 16-byte chunk c of row r sits at chunk c ^ (r & 7) under the 128-byte swizzle
        const uint32_t stage = ring + stg * kStageBytes;
        auto chunk_at = [&](int r, int c) { return lds128(stage + r * 128 + ((c ^ (r & 7)) << 4)); };
        // a skipped token's position may be anything: rotate it by the table's first row
        const float *cos = p.table + (slot >= 0 ? pos : 0) * p.rotary, *sin = cos + p.rotary / 2;
        auto load = [&](int c) -> uint4 {
            const uint4 own = chunk_at(lane, c);
            const int vc = 8 * part + c;   // chunk of the head vector
            if (half != 0 || vc >= 2 * hc)
                return own;
            if (p.interleaved)
                return rotate_pairs(own, cos + 4 * vc, sin + 4 * vc, neg0);
            const bool first = vc < hc;
            const int pc = first ? vc + hc : vc - hc;
            const uint4 other = chunk_at(vt * kTpv + (pc >> 3), pc & 7);
            const int at = 8 * (first ? vc : pc);
            return rotate_halves(own, other, cos + at, sin + at, first, neg0);
        };
        uint64_t X[kN];
#pragma unroll
        for (int c = 0; c < 4; c++)
            pairs_from_chunk(load(c), load(c + 4), X + 8 * c);
        __syncwarp();   // every lane has read the stage
        if constexpr (kRotate) {
            fwht_stages<kN>(X);
            if constexpr (kD == 64) {
                scale_all<kN>(X, kHadamardC64);
            } else {
                exchange_stage64(X, part & 1);
                scale_all<kN>(X, kHadamardC);
            }
        }
        float mn, mx;
        block_min_max<kN>(X, mn, mx);
#pragma unroll
        for (int d = 1; d < kTpv; d <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, d));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
        }
        uint32_t words[kN / 4];
        float scale, zero;
        quantize_block<kN>(X, mn, mx, words, scale, zero);
        if (slot >= 0) {
            const int64_t crow = cache_row(slot, h, half, p.hkv);
            store_block<kN>(p.kv_pages + crow * Dims::kCodeBytes + 32 * part, words, part == 0, scale, zero,
                            p.scales + crow, p.status);
            if (p.mass != nullptr && half == 0 && part == 0)
                p.mass[((slot >> 4) * p.hkv + h) * kPageSize + (slot & 15)] = 0.0f;
        }
    }
    if (i < n)   // a wait gave up: let every queued copy land before the shared memory is released
        for (int k = i; k < min(issued, n); k++)
            mbar_wait_bounded(bar0 + 8 * (k % kRqStages), (k / kRqStages) & 1, kRqWaitLimitNs / 10);
}

template <bool kRotate, int kD>
__global__ void __launch_bounds__(kRqThreads, 4)
    rope_append_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                       const RopeParams p)
{
    extern __shared__ uint8_t smem_raw[];
    pdl_launch_dependents();
    if (static_cast<int>(blockIdx.x) >= p.kv_ctas) {
        rotate_queries<kD>(p);
        return;
    }
    quantize_tiles<kRotate, kD>(
        tk, tv, p, reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)));
}

// Tensor map of k or v: [rows][128 B] for contiguous tokens (stride 0), else [tokens][rows of a
// token][128 B]; the box is 16 rows.
bool encode_rows(CUtensorMap *map, const void *base, int64_t tokens, int64_t rows_per_token, int64_t stride)
{
    auto encode = tensor_map_encoder();
    if (encode == nullptr)
        return false;
    const cuuint32_t estr[3] = {1, 1, 1};
    const cuuint64_t dims2[2] = {128, static_cast<cuuint64_t>(tokens * rows_per_token)}, strides2[1] = {128};
    const cuuint32_t box2[2] = {128, 16};
    const cuuint64_t dims3[3] = {128, static_cast<cuuint64_t>(rows_per_token), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides3[2] = {128, static_cast<cuuint64_t>(2 * stride)};
    const cuuint32_t box3[3] = {128, static_cast<cuuint32_t>(std::min<int64_t>(rows_per_token, 16)),
                                static_cast<cuuint32_t>(std::max<int64_t>(1, 16 / rows_per_token))};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, stride ? 3 : 2, const_cast<void *>(base),
                  stride ? dims3 : dims2, stride ? strides3 : strides2, stride ? box3 : box2, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kRotate, int kD>
cudaError_t launch(const RopeAppendArgs &a, RopeParams &p, const CUtensorMap &tk, const CUtensorMap &tv,
                   cudaStream_t stream)
{
    constexpr size_t kSmem = rq_smem_bytes<kD>();
    static_assert(RqDims<kD>::kStageBytes == 4096, "the ring's stages hold a 32-row tile");
    auto *kernel = rope_append_kernel<kRotate, kD>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess)
        return e;
    // 4 CTAs per SM in all; the q rows get half of them where there is enough work
    const int64_t q_items = p.num_tokens * p.q_slices;
    const int64_t kv_need = (p.num_tiles + kRqWarps - 1) / kRqWarps, q_need = p.hq > 0 ? (q_items + kRqWarps - 1) / kRqWarps : 0;
    const int64_t room = 4 * static_cast<int64_t>(sms);
    p.kv_ctas = static_cast<int32_t>(std::min(kv_need, p.hq > 0 ? room / 2 : room));
    const int64_t q_ctas = std::min(q_need, room - p.kv_ctas);
    kernel<<<static_cast<unsigned>(p.kv_ctas + q_ctas), kRqThreads, kSmem, stream>>>(tk, tv, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs &a, cudaStream_t stream)
{
    RopeTableParams p;
    p.table = a.table;
    p.first = a.first_position;
    p.count = a.num_positions;
    p.half = a.rotary_dim / 2;
    p.amplitude = static_cast<float>(a.amplitude);
    for (int i = 0; i < p.half; i++)
        p.turns[i] = a.turns[i];
    const int64_t n = p.count * p.half;
    rope_table_kernel<<<static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 148 * 16)), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_rope_append(const RopeAppendArgs &a, cudaStream_t stream)
{
    const RotateQuantizeArgs &kv = a.kv;
    const int64_t rows_per_vec = kv.head_dim / 64, num_vecs = kv.num_tokens * kv.num_kv_heads;
    if (num_vecs * rows_per_vec > (int64_t(1) << 29))
        return cudaErrorInvalidValue;       // tensor-map rows and tile indices fit in int32
    const bool strided = kv.k_stride != 0;
    const int64_t rows_per_token = kv.num_kv_heads * rows_per_vec;
    CUtensorMap tk, tv;
    if (!encode_rows(&tk, kv.k, kv.num_tokens, rows_per_token, kv.k_stride) ||
        !encode_rows(&tv, kv.v, kv.num_tokens, rows_per_token, kv.v_stride))
        return cudaErrorInvalidValue;
    RopeParams p;
    p.slots = kv.slot_mapping;
    p.positions = a.positions;
    p.table = a.table;
    p.num_positions = a.num_positions;
    p.num_slots = kv.num_pages * kPageSize;
    p.num_vecs = num_vecs;
    p.num_tokens = kv.num_tokens;
    p.num_tiles = static_cast<uint32_t>(2 * ((num_vecs * rows_per_vec + 31) / 32));
    p.hkv = kv.num_kv_heads;
    p.hq = a.num_q_heads;
    p.rotary = a.rotary_dim;
    p.interleaved = a.interleaved ? 1 : 0;
    p.strided = strided ? 1 : 0;
    p.q = static_cast<const uint16_t *>(a.q);
    p.q_out = static_cast<uint16_t *>(a.q_out);
    p.q_stride = a.q_stride != 0 ? a.q_stride : static_cast<int64_t>(a.num_q_heads) * kv.head_dim;
    p.kv_pages = kv.kv_pages;
    p.scales = static_cast<uint32_t *>(kv.scales);
    p.mass = a.mass;
    p.status = kv.status;
    p.neg_zero = -0.0f;
    // few tokens: a warp takes 2 passes over the heads it holds, so that the call spreads over the SMs
    const int heads = 32 / (kv.head_dim / 8);
    p.slice_heads = kv.num_tokens >= 4096 ? std::max(1, a.num_q_heads) : 2 * heads;
    p.q_slices = a.num_q_heads > 0 ? (a.num_q_heads + p.slice_heads - 1) / p.slice_heads : 1;
    switch (kv.head_dim) {
    case 64:
        return kv.rotate ? launch<true, 64>(a, p, tk, tv, stream) : launch<false, 64>(a, p, tk, tv, stream);
    case 128:
        return kv.rotate ? launch<true, 128>(a, p, tk, tv, stream) : launch<false, 128>(a, p, tk, tv, stream);
    case 256:
        return kv.rotate ? launch<true, 256>(a, p, tk, tv, stream) : launch<false, 256>(a, p, tk, tv, stream);
    default:
        return cudaErrorInvalidValue;
    }
}

}  // namespace saw
