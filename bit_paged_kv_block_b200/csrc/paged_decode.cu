// paged_decode.cu -- decode attention over the INT4 paged KV cache (split-K, GQA-stacked).
//
// The read side of "SAW-INT4: System-Aware 4-Bit KV-Cache Quantization for Real-World LLM
// Serving" (Research Findings: the quantized cache must keep fused attention execution over
// paged memory with regular access), with the query heads of one kv head stacked into one
// tensor-core tile as in "BitDecoding-FP4" (abstract: stacked query MMA on paged KV caches).
// Because H is orthogonal and symmetric, <q, k> = <Hq, Hk> and sum p_t v_t = H sum p_t (H v_t):
// the kernel rotates q once, attends over the rotated codes and rotates the output back.
//
// Work split.  A (sequence s, kv head h) pair is a segment of n = ceil(len_s / 16) pages.  All
// segments are laid end to end (seq-major, then kv head) in a cost space where a segment costs
// n + kKappa (kKappa pages' worth of per-segment work: query rotation and output rotation), and
// that cost range is cut into W equal slices, one per warp of a persistent grid.  Each warp
// owns the contiguous run of pages whose cost positions fall in its slice and works on it
// independently: no barrier, atomic or fence between warps.  A segment that lies entirely in one
// warp's run is finished by that warp; the pieces of a segment split across warps are written to
// the workspace (slot segment + warp, unique because both orders are monotone) and combined by
// a second kernel (paged_decode_merge_kernel), launched as a programmatic dependent.
//
// Per page (16 tokens x one kv head, 2 KiB of codes + 128 B of scales), per warp:
//   * one elected lane queues a 2-D tensor copy of the 32 code rows (64B swizzle, so the K
//     reads and the transposed V reads below are bank-conflict free) and a 1-D bulk copy of the
//     scales into a 4-stage ring, completion on an mbarrier (bounded wait), three pages ahead;
//   * S^T[16 tok x 8 heads] = K_codes[16 x 128] . Q^T with mma.m16n8k16 (fp16 in, fp32 acc):
//     the codes are exact fp16 subnormals, and s = scale * acc + zero * sum(q) in fp32;
//   * online softmax in the log2 domain (q carries sm_scale * log2 e);
//   * O^T[128 d x 8 heads] += V_codes^T . P'^T with P' = p * scale_V in fp16 and the zero
//     point added in fp32 through sum_t p_t zero_t.
// The work split, the piece loop, the split-K slots and the merge kernel are generic over the
// page format and live in decode_common.cuh; the INT4 page format (Int4Format) is int4_format.cuh.
// The query of the next segment is bulk-copied into a per-warp buffer while the current one is
// processed.  The query dimension d of QK and the value dimension of PV are consumed in a
// permuted order (both sides permuted alike), which lets every thread unpack whole 32-bit code
// words; the final inverse rotation undoes it.
#include "int4_format.cuh"

namespace saw {
namespace {

// Multiprocessor count and decode-kernel occupancy on the current device for head dimension kD
// (see decode::launch_shape).
template <int kD>
cudaError_t launch_shape(size_t smem, size_t merge_smem, LaunchShape &out)
{
    static ShapeCache shapes;
    static const void *const decode_kernels[kShapeVariants] = {
        reinterpret_cast<const void *>(paged_decode_kernel<Int4Format<true, kD>, false>),
        reinterpret_cast<const void *>(paged_decode_kernel<Int4Format<false, kD>, false>),
        reinterpret_cast<const void *>(paged_decode_kernel<Int4Format<true, kD>, true>),
        reinterpret_cast<const void *>(paged_decode_kernel<Int4Format<false, kD>, true>)};
    static const void *const merge_kernels[kShapeVariants] = {
        reinterpret_cast<const void *>(paged_decode_merge_kernel<Int4Format<true, kD>, false>),
        reinterpret_cast<const void *>(paged_decode_merge_kernel<Int4Format<false, kD>, false>),
        reinterpret_cast<const void *>(paged_decode_merge_kernel<Int4Format<true, kD>, true>),
        reinterpret_cast<const void *>(paged_decode_merge_kernel<Int4Format<false, kD>, true>)};
    return decode::launch_shape(shapes, decode_kernels, merge_kernels,
                                32 * Int4Format<true, kD>::kWarps, smem, merge_smem, out);
}

// The windowed decode's quantized part (rotated, decode, head_dim 128): only the shared-memory
// attributes are set here; its grid is the plain family's (same layout and launch bounds), which
// the workspace is sized for.
cudaError_t set_window_merge_attributes(size_t smem, size_t merge_smem)
{
    static ShapeCache shapes;
    using W = Int4Format<true, 128, kRoleWindow>;
    static const void *const decode_kernels[kShapeVariants] = {
        reinterpret_cast<const void *>(paged_decode_kernel<W, false>),
        reinterpret_cast<const void *>(paged_decode_kernel<W, false>),
        reinterpret_cast<const void *>(paged_decode_kernel<W, false>),
        reinterpret_cast<const void *>(paged_decode_kernel<W, false>)};
    static const void *const merge_kernels[kShapeVariants] = {
        reinterpret_cast<const void *>(paged_decode_merge_kernel<W, false>),
        reinterpret_cast<const void *>(paged_decode_merge_kernel<W, false>),
        reinterpret_cast<const void *>(paged_decode_merge_kernel<W, false>),
        reinterpret_cast<const void *>(paged_decode_merge_kernel<W, false>)};
    LaunchShape unused;
    return decode::launch_shape(shapes, decode_kernels, merge_kernels, 32 * W::kWarps, smem,
                                merge_smem, unused);
}

template <int kD>
size_t workspace_bytes(int32_t num_kv_heads, int32_t num_q_heads, int32_t num_seqs, int64_t total_q)
{
    using Fmt = Int4Format<true, kD>;
    const bool prefill = total_q >= 0;
    LaunchShape ls;
    if (launch_shape<kD>(decode_smem_bytes<Fmt>(num_seqs, query_rows(num_kv_heads, num_q_heads, prefill)),
                         merge_smem_bytes<Fmt::kTiles>(num_seqs), ls) != cudaSuccess)
        return 0;
    return workspace_bytes_for<Fmt::kTiles>(static_cast<size_t>(ls.sms) * ls.occ * Fmt::kWarps,
                                            max_segments(num_kv_heads, num_q_heads, num_seqs,
                                                         total_q, prefill));
}

template <int kD>
cudaError_t launch(const DecodeArgs &a, cudaStream_t stream, bool programmatic)
{
    // Chunked prefill whose chunks average at least half a 128-row tile per sequence runs on the
    // tensor cores (prefill_tc.cu); shorter chunks keep this kernel's split-K work split, which
    // spreads a few long rows over every SM.
    if (kD == 128 && a.q_start != nullptr && a.win_part == 0 &&
        a.total_q * (a.num_q_heads / a.num_kv_heads) >= 64 * static_cast<int64_t>(a.num_seqs))
        return launch_prefill_tc(a, stream, programmatic);
    const CUtensorMap *map = code_tensor_map<kD>(a.kv_pages, a.num_pages * a.num_kv_heads * 32);
    if (map == nullptr)
        return cudaErrorInvalidValue;

    using Fmt = Int4Format<true, kD>;   // the layout is the same for both variants
    const bool prefill = a.q_start != nullptr;
    const int32_t qrows = query_rows(a.num_kv_heads, a.num_q_heads, prefill);
    const size_t smem = decode_smem_bytes<Fmt>(a.num_seqs, qrows);
    const size_t msmem = merge_smem_bytes<Fmt::kTiles>(a.num_seqs);
    LaunchShape ls;
    cudaError_t e = launch_shape<kD>(smem, msmem, ls);
    if (e != cudaSuccess)
        return e;

    DecodeParams p;
    p.q = static_cast<const uint16_t *>(a.q);
    p.q_start = a.q_start;
    p.scales = static_cast<const uint8_t *>(a.scales);
    p.block_table = a.block_table;
    p.seq_lens = a.seq_lens;
    p.out = a.out;
    p.partials = static_cast<float *>(a.workspace);
    p.status = a.status;
    p.num_pages = a.num_pages;
    p.max_blocks = a.max_blocks;
    p.num_seqs = a.num_seqs;
    p.hq = a.num_q_heads;
    p.hkv = a.num_kv_heads;
    p.group = a.num_q_heads / a.num_kv_heads;
    p.qrows = qrows;
    p.lse = a.lse;
    p.win_part = a.win_part;
    p.win_sink = a.win_sink;
    p.win_recent = a.win_recent;
    p.max_segments = max_segments(a.num_kv_heads, a.num_q_heads, a.num_seqs, a.total_q, prefill);
    p.total_warps = ls.sms * ls.occ * Fmt::kWarps;
    // q carries sm_scale * log2(e), and 1/sqrt(B) of the (unnormalised) query butterfly
    p.q_mult = static_cast<float>((a.rotate ? static_cast<double>(hadamard_c(kD)) : 1.0) * a.sm_scale *
                                  1.4426950408889634);

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ls.sms * ls.occ));
    cfg.blockDim = dim3(32 * Fmt::kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = programmatic ? 1 : 0;
    const bool window_merge = a.win_part == 2;
    if (window_merge && (kD != 128 || prefill || !a.rotate))
        return cudaErrorInvalidValue;
    if (window_merge && (e = set_window_merge_attributes(smem, msmem)) != cudaSuccess)
        return e;
    auto *kernel = window_merge ? paged_decode_kernel<Int4Format<true, kD, kRoleWindow>, false>
                   : a.rotate   ? (prefill ? paged_decode_kernel<Int4Format<true, kD>, true>
                                           : paged_decode_kernel<Int4Format<true, kD>, false>)
                                : (prefill ? paged_decode_kernel<Int4Format<false, kD>, true>
                                           : paged_decode_kernel<Int4Format<false, kD>, false>);
    e = cudaLaunchKernelEx(&cfg, kernel, *map, p);
    if (e != cudaSuccess)
        return e;

    const int64_t segs = p.max_segments;
    cudaLaunchConfig_t mcfg = cfg;
    mcfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(segs, 8 * ls.sms))));
    mcfg.blockDim = dim3(kMergeThreads);
    mcfg.dynamicSmemBytes = msmem;
    mcfg.numAttrs = 1;
    // at most one segment per SM: every segment is split over tens of warps, whose partials the
    // wider merge folds in fewer rounds (its shared memory stays below the default 48 KiB)
    // (the chunked prefill on this kernel takes the same choice from the same count, the decode's
    // segments, so that a one-token chunk stays bit-identical to the decode)
    const int64_t decode_segs = max_segments(a.num_kv_heads, a.num_q_heads, a.num_seqs, 0, false);
    if (kD <= 128 && !window_merge && decode_segs <= ls.sms) {
        constexpr int kW = kMergeWarpsWide;
        mcfg.blockDim = dim3(32 * kW);
        mcfg.dynamicSmemBytes = merge_smem_bytes<Fmt::kTiles, kW>(a.num_seqs);
        e = cudaLaunchKernelEx(&mcfg, a.rotate ? (prefill ? paged_decode_merge_kernel<Int4Format<true, kD>, true, kW>
                                                          : paged_decode_merge_kernel<Int4Format<true, kD>, false, kW>)
                                               : (prefill ? paged_decode_merge_kernel<Int4Format<false, kD>, true, kW>
                                                          : paged_decode_merge_kernel<Int4Format<false, kD>, false, kW>),
                               p);
        if (e != cudaSuccess)
            return e;
        return cudaGetLastError();
    }
    // many short segments (more than 4 per SM, each split over one or two warps): fewer warps per
    // segment, and enough CTAs for one wave over them
    if (kD <= 128 && !window_merge && decode_segs > 4 * static_cast<int64_t>(ls.sms)) {
        constexpr int kW = kMergeWarpsNarrow;
        mcfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(segs, (32 / kW) * ls.sms)));
        mcfg.blockDim = dim3(32 * kW);
        mcfg.dynamicSmemBytes = merge_smem_bytes<Fmt::kTiles, kW>(a.num_seqs);
        e = cudaLaunchKernelEx(&mcfg, a.rotate ? (prefill ? paged_decode_merge_kernel<Int4Format<true, kD>, true, kW>
                                                          : paged_decode_merge_kernel<Int4Format<true, kD>, false, kW>)
                                               : (prefill ? paged_decode_merge_kernel<Int4Format<false, kD>, true, kW>
                                                          : paged_decode_merge_kernel<Int4Format<false, kD>, false, kW>),
                               p);
        if (e != cudaSuccess)
            return e;
        return cudaGetLastError();
    }
    auto *merge = window_merge ? paged_decode_merge_kernel<Int4Format<true, kD, kRoleWindow>, false>
                  : a.rotate   ? (prefill ? paged_decode_merge_kernel<Int4Format<true, kD>, true>
                                          : paged_decode_merge_kernel<Int4Format<true, kD>, false>)
                               : (prefill ? paged_decode_merge_kernel<Int4Format<false, kD>, true>
                                          : paged_decode_merge_kernel<Int4Format<false, kD>, false>);
    e = cudaLaunchKernelEx(&mcfg, merge, p);
    if (e != cudaSuccess)
        return e;
    return cudaGetLastError();
}

}  // namespace

size_t decode_workspace_bytes(int32_t num_kv_heads, int32_t num_q_heads, int32_t num_seqs,
                              int64_t total_q, int32_t head_dim)
{
    if (num_kv_heads <= 0 || num_q_heads <= 0 || num_seqs < 0 || num_q_heads % num_kv_heads)
        return 0;
    if (head_dim == 128)
        return workspace_bytes<128>(num_kv_heads, num_q_heads, num_seqs, total_q);
    if (head_dim == 256)
        return workspace_bytes<256>(num_kv_heads, num_q_heads, num_seqs, total_q);
    if (head_dim == 64)
        return workspace_bytes<64>(num_kv_heads, num_q_heads, num_seqs, total_q);
    return 0;
}

cudaError_t launch_paged_decode(const DecodeArgs &a, cudaStream_t stream, bool programmatic)
{
    if (a.head_dim == 128)
        return launch<128>(a, stream, programmatic);
    if (a.head_dim == 256)
        return launch<256>(a, stream, programmatic);
    if (a.head_dim == 64)
        return launch<64>(a, stream, programmatic);
    return cudaErrorInvalidValue;
}

}  // namespace saw
