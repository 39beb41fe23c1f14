// rotate_quantize.cu -- fused Hadamard rotation + token-wise INT4 quantization + paged scatter.
//
// Implements the fused rotation-quantization kernel of "SAW-INT4: System-Aware 4-Bit KV-Cache
// Quantization for Real-World LLM Serving" (Research Findings): every new key and value head
// vector is rotated by the normalised 128-point Hadamard transform (per 128-element block; a
// 64-element head vector by the 64-point transform), quantized token-wise to
// asymmetric INT4 and written straight into its page of the paged KV cache.
//
// Results are bit-identical to the definition in saw.h:
//   * the butterfly performs exactly the IEEE fp32 adds/subtracts of the natural-order
//     Sylvester transform, stage h = 1, 2, ..., 64 in that order, then one multiply by
//     fp32(1/sqrt(128)); two fp32 operations are issued per packed f32x2 instruction, each
//     individually rounded, so the register layout does not change any result;
//   * scale = (max - min) / 15 is the IEEE quotient (computed by a three-operation sequence
//     checked against the IEEE divide for every non-negative fp32 dividend, below); each code is
//     read off one fused multiply-add on a 2^-16 grid, which is provably the IEEE-divide code
//     except where the grid value is exactly half-way between two codes; those rare elements
//     are settled by an exact remainder test (note above code_at_half()).
// This translation unit is compiled with -fmad=false as a second guard against contraction.
//
// Data movement: every warp streams its own tiles of 16 rows of 128 bytes (64 bf16 elements) of K
// and the same 16 rows of V into a private 3-stage shared-memory ring with tensor copies (TMA,
// 128-byte swizzle) completing on mbarriers, so warps never wait for each other.  The warps of the
// persistent grid take tiles round-robin.
//
// Thread layout: one thread per 64-element row; lanes 0-15 take the tile's K rows and lanes 16-31
// its V rows.  A thread keeps its row as packed pairs X[m] = (x[m], x[m + 32]), so butterfly
// stages h = 1 .. 16 of its 64 elements run on packed f32x2 instructions and stage h = 32 pairs the
// two halves of each register.  D = 64: that is the whole transform.  D = 128 and 256: a row is half
// of a 128-point block and stage h = 64 pairs lane r with lane r ^ 1; the two lanes swap their 64
// values by shuffles and each forms its own half of the stage's outputs: x + partner (lower row) or
// partner - x = fma(x, -1, partner), one IEEE rounding either way.  min / max combine over the
// vector's lanes by shuffles.
#include <algorithm>

#include "quantize_device.cuh"

namespace saw {
namespace {

struct RqParams {
    const int64_t *slot_mapping;
    int64_t num_vecs;        // T * Hkv
    int64_t num_tiles;
    int32_t hkv;
    int64_t num_slots;       // num_pages * 16
    uint8_t *kv_pages;
    uint32_t *scales;        // fp16x2 (scale, zero) per row
    uint32_t *status;
    int32_t strided;         // k / v through 3-D tensor maps with a token stride
    uint32_t hkv_mul;        // vec / hkv by multiply and shift (div_hkv)
    uint32_t hkv_shift;
};

// vec / hkv without a divide (T. Granlund, P. Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994, with a 33-bit multiplier): with s = ceil(log2 hkv) and
// m' = ceil(2^(32 + s) / hkv), floor(vec m' / 2^(32 + s)) = floor(vec / hkv) for every vec < 2^32;
// m' = 2^32 + hkv_mul, so vec m' / 2^32 = umulhi(vec, hkv_mul) + vec (no overflow for vec < 2^31).
__device__ __forceinline__ uint32_t div_hkv(uint32_t vec, const RqParams &p)
{
    return (__umulhi(vec, p.hkv_mul) + vec) >> p.hkv_shift;
}

template <bool kRotate, int kD>
__global__ void __launch_bounds__(kRqThreads, 4)
    rotate_quantize_kernel(const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv, const RqParams p)
{
    using Dims = RqDims<kD>;
    constexpr int kN = Dims::kN;
    constexpr int kStageBytes = Dims::kStageBytes;
    constexpr int kTpv = Dims::kThreadsPerVec;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    // all indices below fit in 32 bits: the host limits the rows to 2^29
    const uint32_t W = gridDim.x * kRqWarps;
    const uint32_t wg = blockIdx.x * kRqWarps + warp;
    const uint32_t num_tiles = static_cast<uint32_t>(p.num_tiles);
    if (wg >= num_tiles)
        return;
    const int n = static_cast<int>((num_tiles - wg + W - 1) / W);   // this warp's tiles: wg + i W
    const uint32_t ring = smem_u32(smem) + warp * kRqStages * kStageBytes;
    const uint32_t bar0 = smem_u32(smem + kRqWarps * kRqStages * kStageBytes) + warp * kRqStages * 8;
    if (lane == 0)
        for (int i = 0; i < kRqStages; i++)
            mbar_init(bar0 + 8 * i, 1);
    mbar_init_fence();
    __syncwarp();

    int issued = 0, istg = 0;
    uint32_t itile = wg;
    // queue tile `itile` (16 rows of K and of V) into stage istg
    auto issue = [&]() {
        if (issued < n) {
            if (lane == 0) {
                const uint32_t dst = ring + istg * kStageBytes;
                const uint32_t bar = bar0 + 8 * istg;
                mbar_arrive_expect_tx(bar, kStageBytes);
                if (p.strided) {
                    // the tile's first vector: token and head (the box spans whole tiles)
                    const uint32_t v0 = itile * Dims::kTileVecs;
                    const int32_t tok = static_cast<int32_t>(div_hkv(v0, p));
                    const int32_t row = static_cast<int32_t>(kTpv * (v0 - tok * static_cast<uint32_t>(p.hkv)));
                    tma_load_3d(dst, &tk, 0, row, tok, bar);
                    tma_load_3d(dst + Dims::kHalfBytes, &tv, 0, row, tok, bar);
                } else {
                    const int32_t y = static_cast<int32_t>(itile * 16);
                    tma_load_2d(dst, &tk, 0, y, bar);
                    tma_load_2d(dst + Dims::kHalfBytes, &tv, 0, y, bar);
                }
            }
            issued++;
            itile += W;
            if (++istg == kRqStages)
                istg = 0;
        }
    };
    for (int k = 0; k < kRqStages - 1; k++)
        issue();

    const int half = lane >> 4;                     // 0: K, 1: V
    const int r = lane & 15;                        // row of the tile
    const int part = r % kTpv;                      // row of the vector (64 elements each)
    const int vt = r / kTpv;                        // vector of the tile
    const uint32_t num_vecs = static_cast<uint32_t>(p.num_vecs);
    const uint32_t hkv = static_cast<uint32_t>(p.hkv);
    uint32_t tile = wg;
    // slot of this thread's vector in the tile (prefetched one tile ahead)
    auto slot_of = [&](uint32_t t, uint32_t &vec) -> int64_t {
        const uint32_t vec_raw = t * Dims::kTileVecs + vt;
        vec = vec_raw < num_vecs ? vec_raw : num_vecs - 1;
        return p.slot_mapping[div_hkv(vec, p)];
    };
    uint32_t vec_next;
    int64_t slot_next = slot_of(tile, vec_next);
    int cstg = 0;
    uint32_t cphase = 0;
    int i = 0;
    for (; i < n; i++, tile += W) {
        issue();
        const uint32_t vec = vec_next;
        const bool in_range = tile * Dims::kTileVecs + vt < num_vecs;
        const int64_t slot = slot_next;
        if (i + 1 < n)
            slot_next = slot_of(tile + W, vec_next);
        const int stg = cstg;
        const bool ok = mbar_wait_bounded(bar0 + 8 * stg, cphase, kRqWaitLimitNs);
        if (++cstg == kRqStages) {
            cstg = 0;
            cphase ^= 1;
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) {
            if (lane == 0)
                set_status(p.status, SAW_DEV_WAIT_TIMEOUT);
            break;
        }
        const uint32_t tok = div_hkv(vec, p);
        const uint32_t h = vec - tok * hkv;
        bool store = in_range && slot >= 0;
        if (store && slot >= p.num_slots) {
            if (part == 0 && half == 0)
                set_status(p.status, SAW_DEV_BAD_SLOT);
            store = false;
        }

        // this thread's row r of the stage's K or V half; the 16-byte chunk c of a row sits at
        // chunk c ^ (r & 7) under the 128-byte swizzle: X[m] = (x[m], x[m + 32])
        const uint32_t stage = ring + stg * kStageBytes;
        const uint32_t row = stage + half * Dims::kHalfBytes + r * 128;
        uint64_t X[kN];
#pragma unroll
        for (int c = 0; c < 4; c++)
            pairs_from_chunk(lds128(row + ((c ^ (r & 7)) << 4)),
                             lds128(row + (((c + 4) ^ (r & 7)) << 4)), X + 8 * c);
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
        if (store) {
            const int64_t crow = cache_row(slot, h, half, p.hkv);
            store_block<kN>(p.kv_pages + crow * Dims::kCodeBytes + 32 * part, words, part == 0, scale,
                            zero, p.scales + crow, p.status);
        }
    }
    if (i < n) {
        // a wait gave up: let every queued copy land before the shared memory is released
        for (int k = i; k < issued; k++)
            mbar_wait_bounded(bar0 + 8 * (k % kRqStages), (k / kRqStages) & 1, kRqWaitLimitNs / 10);
    }
}

// ---- the full-precision window beside the INT4 cache: one serving step ----------------------
//
// "InnerQ: Hardware-Aware Tuning-Free Quantization of KV Cache for Large Language Models",
// Abstract and Figure 2: a small bf16 window of sink and recent tokens stays beside the quantized
// cache.  Sequence s's new token sits at position p = seq_lens[s] - 1: a sink (p < w_sink) takes
// window slot p; otherwise its slot in the recent ring is w_sink + (p - w_sink) mod w_recent, and
// the token it displaces (position p - w_recent, when that is not a sink) is rotated, quantized
// and scattered into the INT4 pages at quantized index p - w_recent - w_sink, bit-identically to
// the rotate+quantize kernel (same device code).  With w_recent = 0 the new token itself is
// quantized.  Window slot i lives in bf16 page win_table[s][i / 16] at offset i mod 16.
//
// Lanes as in the rotate+quantize kernel at D = 128: a warp takes 8 (sequence, kv head) pairs,
// lanes 0-15 their K vectors and lanes 16-31 their V vectors, two lanes per vector (lane 2 i + b
// holds elements 64 b .. 64 b + 63 of pair i; stage h = 64 is the shuffle exchange).  Each thread
// reads exactly the 128 bytes of the displaced vector that it later overwrites with the new
// token, so the read and the write of those bytes are ordered within one thread.
struct WinAppendParams {
    const uint16_t *k, *v;
    const int32_t *seq_lens;
    int32_t num_seqs, hkv, w_sink, w_recent;
    uint16_t *win_kv;
    const int32_t *win_table;
    int32_t win_blocks;
    int64_t num_win_pages;
    const int32_t *block_table;
    int32_t max_blocks;
    int64_t num_pages;
    uint8_t *kv_pages;
    uint32_t *scales;
    uint32_t *status;
};

template <bool kRotate>
__global__ void __launch_bounds__(kRqThreads)
    window_append_kernel(const WinAppendParams p)
{
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = lane >> 4;
    const int part = lane & 1;
    const int64_t pair = (static_cast<int64_t>(blockIdx.x) * kRqWarps + warp) * 8 + ((lane & 15) >> 1);
    const bool live = pair < static_cast<int64_t>(p.num_seqs) * p.hkv;
    const int s = live ? static_cast<int>(pair / p.hkv) : 0;
    const int h = live ? static_cast<int>(pair - static_cast<int64_t>(s) * p.hkv) : 0;
    const int L = live ? p.seq_lens[s] : 0;
    const bool report = half == 0 && part == 0;
    // this thread's 64 elements of the new token, loaded now: nothing below depends on them, so
    // their latency overlaps the table lookups instead of following the quantization
    const uint16_t *src = (half ? p.v : p.k) + (static_cast<int64_t>(s) * p.hkv + h) * 128 + 64 * part;
    uint4 fresh[8];
    if (live) {
#pragma unroll
        for (int c = 0; c < 8; c++)
            fresh[c] = *reinterpret_cast<const uint4 *>(src + 8 * c);
    }

    // where the new token goes and which token is quantized
    bool to_win = false, quant = false, from_win = false;
    int slot = 0, j = 0;
    if (L > 0) {
        const int pos = L - 1;
        if (pos < p.w_sink) {
            to_win = true;
            slot = pos;
        } else if (p.w_recent == 0) {
            quant = true;
            j = pos - p.w_sink;
        } else {
            to_win = true;
            slot = p.w_sink + (pos - p.w_sink) % p.w_recent;
            if (pos - p.w_recent >= p.w_sink) {
                quant = from_win = true;
                j = pos - p.w_recent - p.w_sink;
            }
        }
    } else if (L < 0 && report) {
        set_status(p.status, SAW_DEV_BAD_SEQ_LEN);
    }
    // both table lookups depend only on the length: issue them together
    const bool q_in_table = j / kPageSize < p.max_blocks;
    const int32_t wpage = to_win ? p.win_table[static_cast<int64_t>(s) * p.win_blocks + slot / 16] : 0;
    const int32_t qpage = quant && q_in_table
                              ? p.block_table[static_cast<int64_t>(s) * p.max_blocks + j / kPageSize]
                              : -1;
    uint16_t *win = nullptr;   // this thread's 64 elements of the window slot
    if (to_win) {
        const int32_t page = wpage;
        if (page < 0 || page >= p.num_win_pages) {
            if (report)
                set_status(p.status, SAW_DEV_BAD_PAGE);
            to_win = quant = false;   // the displaced token cannot be read: leave the pair
        } else {
            win = p.win_kv + ((((static_cast<int64_t>(page) * p.hkv + h) * 2 + half) * kPageSize) +
                              slot % kPageSize) * 128 + 64 * part;
        }
    }
    int64_t row = 0;
    if (quant) {
        const int32_t page = qpage;
        if (page < 0 || page >= p.num_pages) {
            if (report)
                set_status(p.status, q_in_table ? SAW_DEV_BAD_PAGE : SAW_DEV_BAD_SEQ_LEN);
            to_win = quant = false;   // keep the displaced token where it is
        } else {
            row = ((static_cast<int64_t>(page) * p.hkv + h) * 2 + half) * kPageSize + j % kPageSize;
        }
    }

    // the vector to quantize (the displaced window token, or the new token itself when there is
    // no recent ring); both lanes of a vector decide alike, and every lane runs the transform
    // (its stage h = 64 pairs lanes 2 i and 2 i + 1): lanes with nothing to quantize run it on
    // zeros and store nothing
    uint64_t X[32];
    if (quant) {
        const uint16_t *qsrc = from_win ? win : src;
#pragma unroll
        for (int c = 0; c < 4; c++)
            pairs_from_chunk(*reinterpret_cast<const uint4 *>(qsrc + 8 * c),
                             *reinterpret_cast<const uint4 *>(qsrc + 32 + 8 * c), X + 8 * c);
    } else {
#pragma unroll
        for (int i = 0; i < 32; i++)
            X[i] = 0;
    }
    if constexpr (kRotate) {
        fwht_stages<32>(X);
        exchange_stage64(X, part);
        scale_all<32>(X, kHadamardC);
    }
    float mn, mx;
    block_min_max<32>(X, mn, mx);
    mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    uint32_t words[8];
    float scale, zero;
    quantize_block<32>(X, mn, mx, words, scale, zero);
    if (quant)
        store_block<32>(p.kv_pages + row * 64 + 32 * part, words, part == 0, scale, zero, p.scales + row,
                        p.status);
    // then the new token takes the slot (after this thread's own read of these bytes)
    if (to_win) {
#pragma unroll
        for (int c = 0; c < 8; c++)
            *reinterpret_cast<uint4 *>(win + 8 * c) = fresh[c];
    }
}

}  // namespace

cudaError_t launch_window_append(const WindowAppendArgs &a, cudaStream_t stream)
{
    const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
    if (pairs == 0)
        return cudaSuccess;
    WinAppendParams p;
    p.k = static_cast<const uint16_t *>(a.k);
    p.v = static_cast<const uint16_t *>(a.v);
    p.seq_lens = a.seq_lens;
    p.num_seqs = a.num_seqs;
    p.hkv = a.num_kv_heads;
    p.w_sink = a.w_sink;
    p.w_recent = a.w_recent;
    p.win_kv = static_cast<uint16_t *>(a.win_kv);
    p.win_table = a.win_table;
    p.win_blocks = a.win_blocks;
    p.num_win_pages = a.num_win_pages;
    p.block_table = a.block_table;
    p.max_blocks = a.max_blocks;
    p.num_pages = a.num_pages;
    p.kv_pages = a.kv_pages;
    p.scales = static_cast<uint32_t *>(a.scales);
    p.status = a.status;
    const int64_t grid = (pairs + 8 * kRqWarps - 1) / (8 * kRqWarps);
    window_append_kernel<true><<<static_cast<unsigned>(grid), kRqThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_rotate_quantize(const RotateQuantizeArgs &a, cudaStream_t stream,
                                   bool trigger_dependents)
{
    (void)trigger_dependents;   // the kernel always releases dependents at its start
    const int64_t num_vecs = a.num_tokens * a.num_kv_heads;
    if (num_vecs == 0)
        return cudaSuccess;
    if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256)
        return cudaErrorInvalidValue;
    const int64_t rows_per_vec = a.head_dim / 64;   // 128-byte rows (64 elements) per vector
    const int64_t tile_vecs = 16 / rows_per_vec;
    if (num_vecs * rows_per_vec > (int64_t(1) << 29))
        return cudaErrorInvalidValue;       // tensor-map rows and tile indices fit in int32

    // k / v: contiguous [T][Hkv][D] (k_stride = v_stride = 0) through a 2-D map of 128-byte
    // rows whose box is one warp tile (16 rows), or with a token stride through 3-D maps (row,
    // row within the token, token) whose box is also one whole tile: 16 rows of one token (rows
    // per token a multiple of 16) or 16 / R whole tokens of R rows (R dividing 16).  Every copy
    // lands on a 1024-byte aligned stage.
    const bool strided = a.k_stride != 0 || a.v_stride != 0;
    const int64_t rows_per_token = a.num_kv_heads * rows_per_vec;
    static thread_local struct {
        const void *k = nullptr, *v = nullptr;
        int64_t num_vecs = 0, k_stride = -1, v_stride = -1;
        int32_t hkv = 0, head_dim = 0;
        CUtensorMap mk, mv;
    } cache;
    if (cache.k != a.k || cache.v != a.v || cache.num_vecs != num_vecs || cache.hkv != a.num_kv_heads ||
        cache.k_stride != a.k_stride || cache.v_stride != a.v_stride || cache.head_dim != a.head_dim) {
        auto encode = tensor_map_encoder();
        if (encode == nullptr)
            return cudaErrorNotSupported;
        if (strided && rows_per_token % 16 != 0 && 16 % rows_per_token != 0)
            return cudaErrorInvalidValue;
        const cuuint32_t estr[3] = {1, 1, 1};
        for (int which = 0; which < 2; which++) {
            CUresult r;
            void *base = const_cast<void *>(which ? a.v : a.k);
            if (!strided) {
                const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(rows_per_vec * num_vecs)};
                const cuuint64_t strides[1] = {128};
                const cuuint32_t box[2] = {128, 16};
                r = encode(which ? &cache.mv : &cache.mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base,
                           dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            } else {
                const int64_t stride = which ? a.v_stride : a.k_stride;   // bf16 elements
                const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(rows_per_token),
                                            static_cast<cuuint64_t>(a.num_tokens)};
                const cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(stride * 2)};
                const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(std::min<int64_t>(rows_per_token, 16)),
                                           static_cast<cuuint32_t>(std::max<int64_t>(1, 16 / rows_per_token))};
                r = encode(which ? &cache.mv : &cache.mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base,
                           dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            }
            if (r != CUDA_SUCCESS) {
                cache.k = nullptr;
                return cudaErrorInvalidValue;
            }
        }
        cache.k = a.k;
        cache.v = a.v;
        cache.num_vecs = num_vecs;
        cache.hkv = a.num_kv_heads;
        cache.head_dim = a.head_dim;
        cache.k_stride = a.k_stride;
        cache.v_stride = a.v_stride;
    }

    RqParams p;
    p.slot_mapping = a.slot_mapping;
    p.num_vecs = num_vecs;
    p.num_tiles = (num_vecs + tile_vecs - 1) / tile_vecs;
    p.hkv = a.num_kv_heads;
    p.num_slots = a.num_pages * kPageSize;
    p.kv_pages = a.kv_pages;
    p.scales = static_cast<uint32_t *>(a.scales);
    p.status = a.status;
    p.strided = strided ? 1 : 0;
    {
        uint32_t sh = 0;
        while ((int64_t(1) << sh) < a.num_kv_heads)
            sh++;
        const uint64_t d = static_cast<uint64_t>(a.num_kv_heads);
        p.hkv_shift = sh;
        p.hkv_mul = static_cast<uint32_t>(((uint64_t(1) << (32 + sh)) + d - 1) / d - (uint64_t(1) << 32));
    }

    // per device and kernel: multiprocessor count, the shared-memory attribute and occupancy
    constexpr int kMaxDevices = 64;
    constexpr int kVariants = 6;
    static int sms_of[kMaxDevices] = {}, occ_of[kMaxDevices][kVariants] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    using KernelFn = void (*)(CUtensorMap, CUtensorMap, RqParams);
    static const KernelFn kernels[kVariants] = {
        rotate_quantize_kernel<true, 128>, rotate_quantize_kernel<false, 128>,
        rotate_quantize_kernel<true, 256>, rotate_quantize_kernel<false, 256>,
        rotate_quantize_kernel<true, 64>, rotate_quantize_kernel<false, 64>};
    static const size_t smem_of[kVariants] = {rq_smem_bytes<128>(), rq_smem_bytes<128>(),
                                              rq_smem_bytes<256>(), rq_smem_bytes<256>(),
                                              rq_smem_bytes<64>(), rq_smem_bytes<64>()};
    const int which = (a.head_dim == 128 ? 0 : a.head_dim == 256 ? 2 : 4) + (a.rotate ? 0 : 1);
    if (sms_of[dev] == 0) {
        int sms = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        for (int r = 0; r < kVariants && e == cudaSuccess; r++) {
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernels[r]),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(smem_of[r]));
            int occ = 0;
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                    &occ, reinterpret_cast<const void *>(kernels[r]), kRqThreads, smem_of[r]);
            if (e == cudaSuccess && occ <= 0)
                e = cudaErrorInvalidConfiguration;
            occ_of[dev][r] = occ;
        }
        if (e != cudaSuccess)
            return e;
        sms_of[dev] = sms;
    }
    const int64_t grid = std::min<int64_t>((p.num_tiles + kRqWarps - 1) / kRqWarps,
                                           static_cast<int64_t>(sms_of[dev]) * occ_of[dev][which]);
    kernels[which]<<<static_cast<unsigned>(grid), kRqThreads, smem_of[which], stream>>>(cache.mk, cache.mv, p);
    return cudaGetLastError();
}

}  // namespace saw
