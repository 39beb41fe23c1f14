// paged_decode_prefix.cu -- decode attention for a batch that shares a prefix, over the INT4 paged
// cache: the prefix's pages are read for all sequences together.
//
// Every sequence s attends over the P prefix tokens (pages of prefix_table) and then over its own
// seq_lens[s] tokens (its row of block_table), one softmax over both.  With m, l, o the maximum,
// sum and weighted values of a part, two parts join as
//     M = max(m1, m2),  l = l1 2^(m1 - M) + l2 2^(m2 - M),  o = o1 2^(m1 - M) + o2 2^(m2 - M),
// so the prefix is one more sequence whose query rows are those of the whole batch, and the merge
// kernel, which joins a segment's split pieces anyway, joins the prefix's pieces too.
//
// The decode kernel (decode_common.cuh, kModePrefix) takes the batch's own tokens and the prefix in
// one plan: kv head h of the prefix has S G query rows in blocks of 8, each block a segment over the
// prefix's pages.  All pieces go to workspace slots as rows ([8][D] fp32, then m[8] and l[8]), since
// the rows of an output segment (sequence, kv head, up to 8 heads) may lie in two blocks of the prefix.
//
// At D = 128 and from kTensorRows query rows per kv head on, the prefix is instead a kernel of its own on
// the 5th-generation tensor cores (prefix_tc.cu), which the decode kernel over the own tokens runs
// beside as its programmatic dependent, and the merge joins both kernels' pieces.
#include <algorithm>

#include "int4_format.cuh"
#include "prefix_tc.h"

namespace saw {
namespace {

template <bool kRotate, int kD>
using PrefixFormat = Int4Format<kRotate, kD, kRolePrefix>;

// Row blocks of the prefix's kv heads: S G query rows in blocks of 8.
inline int64_t prefix_blocks(int32_t num_q_heads, int32_t num_kv_heads, int32_t num_seqs)
{
    return (static_cast<int64_t>(num_seqs) * (num_q_heads / num_kv_heads) + kRowsPerBlock - 1) / kRowsPerBlock;
}

// The prefix's pieces where a kernel of its own wrote them: [Hkv][row_blocks][splits] (splits = 0: the
// prefix is in the decode kernel's plan).
struct PrefixPieces {
    const float *slots;
    int32_t row_blocks, splits;
};

constexpr int kRowWarps = 4;

// One output row's elements of a lane: D / 32 of them, in runs of at most 4 (d = 4 lane + j in each
// 128-block; for D = 64 d = 2 lane + j).
template <int kD>
struct RowVec {
    static constexpr int kRuns = kD == 256 ? 2 : 1, kRun = kD == 64 ? 2 : 4;
    float v[kRuns][kRun];

    __device__ void fma_row(const float *row, int lane, float w)
    {
#pragma unroll
        for (int b = 0; b < kRuns; b++) {
            if constexpr (kRun == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(row + 128 * b + 4 * lane);
                v[b][0] = fmaf(w, x.x, v[b][0]);
                v[b][1] = fmaf(w, x.y, v[b][1]);
                v[b][2] = fmaf(w, x.z, v[b][2]);
                v[b][3] = fmaf(w, x.w, v[b][3]);
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(row + 2 * lane);
                v[b][0] = fmaf(w, x.x, v[b][0]);
                v[b][1] = fmaf(w, x.y, v[b][1]);
            }
        }
    }
    // the unnormalised Hadamard transform of each block: the run in registers, the rest across lanes
    __device__ void hadamard(int lane)
    {
#pragma unroll
        for (int b = 0; b < kRuns; b++) {
#pragma unroll
            for (int hb = 1; hb < kRun; hb <<= 1)
#pragma unroll
                for (int j = 0; j < kRun; j++)
                    if ((j & hb) == 0) {
                        const float x = v[b][j], y = v[b][j + hb];
                        v[b][j] = x + y;
                        v[b][j + hb] = x - y;
                    }
#pragma unroll
            for (int lb = 1; lb < 32; lb <<= 1) {
#pragma unroll
                for (int j = 0; j < kRun; j++) {
                    const float o = __shfl_xor_sync(0xFFFFFFFFu, v[b][j], lb);
                    v[b][j] = (lane & lb) ? o - v[b][j] : v[b][j] + o;
                }
            }
        }
    }
    __device__ void store(uint16_t *row, int lane, float f) const
    {
#pragma unroll
        for (int b = 0; b < kRuns; b++) {
            if constexpr (kRun == 4)
                *reinterpret_cast<uint2 *>(row + 128 * b + 4 * lane) =
                    make_uint2(bf16x2_as_u32(v[b][0] * f, v[b][1] * f), bf16x2_as_u32(v[b][2] * f, v[b][3] * f));
            else
                *reinterpret_cast<uint32_t *>(row + 2 * lane) = bf16x2_as_u32(v[b][0] * f, v[b][1] * f);
        }
    }
};

// The rows of a piece: slot k of a row's list is base + k slots, at row `row` of 8.
struct RowPieces {
    const float *base;
    int count, row;
};

// One CTA per output segment (sequence s, kv head h, block of up to 8 of its heads), one warp per row:
// the row's pieces (those of its own tokens, then the prefix's) are joined with weights 2^(m_k - M),
// which the lanes form for 32 pieces at once, so that the loads of the pieces' rows depend on nothing
// but the list.  Pieces are taken in a fixed order: the result does not depend on timing.  (Folding one
// piece after another, each waiting for the one before, took 16 us for 17 splits.)
template <bool kRotate, int kD>
__global__ void __launch_bounds__(32 * kRowWarps) prefix_merge_kernel(const DecodeParams p, const PrefixPieces pre)
{
    constexpr int kSlot = slot_floats<kD / 16>();
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int64_t *flags = reinterpret_cast<volatile int64_t *>(smem);
    SeqTables tb;
    tb.bind(smem + 16 * kRowWarps, p.num_seqs);
    scan_sequences<kModePrefix>(p, tb, flags, false);
    Plan plan;
    plan.init(tb, p.num_seqs, p.total_warps, kMinSlice);
    // the pieces of segment j of sequence s in the plan
    auto planned = [&](int s, int j, int row) -> RowPieces {
        const int64_t u_lo = plan.warp_of_cost(plan.page_cost(s, j, 0));
        const int64_t u_hi = plan.warp_of_cost(plan.page_cost(s, j, tb.npg[s] - 1));
        return {p.partials + (tb.spre[s] + j + u_lo) * kSlot, static_cast<int>(u_hi - u_lo) + 1, row};
    };
    pdl_wait();
    const int nb = (p.group + kRowsPerBlock - 1) / kRowsPerBlock;
    for (int o = blockIdx.x; o < p.batch * p.hkv * nb; o += gridDim.x) {
        const int s = o / (p.hkv * nb), j = o - s * (p.hkv * nb);
        const int h = j / nb, row0 = kRowsPerBlock * (j - h * nb), nrows = min(kRowsPerBlock, p.group - row0);
        const int len = p.seq_lens[s];
        const bool valid = len >= 0 && len <= p.max_blocks * kPageSize;
        RowPieces own = {nullptr, 0, 0};
        if (valid && tb.npg[s] > 0)
            own = planned(s, j, 0);
        for (int e = warp; e < nrows; e += kRowWarps) {
            RowPieces part[2] = {own, {nullptr, 0, 0}};
            part[0].row = e;
            const int row = s * p.group + row0 + e;   // the prefix's row of this head
            if (valid && pre.splits > 0)
                part[1] = {pre.slots + (static_cast<int64_t>(h) * pre.row_blocks + row / kRowsPerBlock) * pre.splits * kSlot,
                           pre.splits, row % kRowsPerBlock};
            else if (valid && p.prefix_seq >= 0)
                part[1] = planned(p.prefix_seq, h * tb.nbk[p.prefix_seq] + row / kRowsPerBlock, row % kRowsPerBlock);
            RowVec<kD> acc = {};
            float M = -INFINITY, l = 0.0f;   // l: this lane's share
#pragma unroll
            for (int q = 0; q < 2; q++) {
                for (int k0 = 0; k0 < part[q].count; k0 += 32) {
                    const int n = min(32, part[q].count - k0);
                    const float *slot = part[q].base + static_cast<int64_t>(k0) * kSlot;
                    const float mk = lane < n ? slot[static_cast<int64_t>(lane) * kSlot + 8 * kD + part[q].row] : -INFINITY;
                    const float lk = lane < n ? slot[static_cast<int64_t>(lane) * kSlot + 8 * kD + 8 + part[q].row] : 0.0f;
                    float top = mk;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                    top = fmaxf(top, M);
                    const float old = M == -INFINITY ? 0.0f : ex2_approx(M - top);
                    const float w = mk == -INFINITY ? 0.0f : ex2_approx(mk - top);
                    M = top;
                    l = l * old + lk * w;
#pragma unroll
                    for (int b = 0; b < RowVec<kD>::kRuns; b++)
#pragma unroll
                        for (int i = 0; i < RowVec<kD>::kRun; i++)
                            acc.v[b][i] *= old;
                    const float *r = slot + part[q].row * kD;
#pragma unroll 8
                    for (int k = 0; k < n; k++)
                        acc.fma_row(r + static_cast<int64_t>(k) * kSlot, lane, __shfl_sync(0xFFFFFFFFu, w, k));
                }
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1)
                l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
            if (kRotate)
                acc.hadamard(lane);
            // a row that attended over nothing is zero
            const float f = l == 0.0f ? 0.0f : (kRotate ? hadamard_c(kD) : 1.0f) / l;
            acc.store(p.out_bf16 + (static_cast<int64_t>(s) * p.hq + h * p.group + row0 + e) * kD, lane, f);
        }
    }
}

inline size_t row_merge_smem(int32_t num_seqs) { return 16 * kRowWarps + seq_table_bytes(num_seqs); }

template <int kD>
cudaError_t prefix_shape(size_t smem, size_t merge_smem, LaunchShape &out)
{
    static ShapeCache shapes;
    static const void *const decode_kernels[kShapeVariants] = {
        reinterpret_cast<const void *>(paged_decode_kernel<PrefixFormat<true, kD>, kModePrefix>),
        reinterpret_cast<const void *>(paged_decode_kernel<PrefixFormat<false, kD>, kModePrefix>),
        reinterpret_cast<const void *>(paged_decode_kernel<PrefixFormat<true, kD>, kModePrefix>),
        reinterpret_cast<const void *>(paged_decode_kernel<PrefixFormat<false, kD>, kModePrefix>)};
    static const void *const merge_kernels[kShapeVariants] = {
        reinterpret_cast<const void *>(prefix_merge_kernel<true, kD>),
        reinterpret_cast<const void *>(prefix_merge_kernel<false, kD>),
        reinterpret_cast<const void *>(prefix_merge_kernel<true, kD>),
        reinterpret_cast<const void *>(prefix_merge_kernel<false, kD>)};
    return decode::launch_shape(shapes, decode_kernels, merge_kernels, 32 * PrefixFormat<true, kD>::kWarps,
                                smem, merge_smem, out);
}

// The fewest query rows per kv head (S G) that take the prefix to the tensor cores.
constexpr int64_t kTensorRows = 24;

// What a call launches, from its sizes alone (the workspace is sized by the same function).
struct PrefixPlan {
    LaunchShape ls;
    size_t smem, merge_smem;
    size_t tc_slots;         // byte offset of the tensor-core kernel's pieces in the workspace
    size_t workspace;
    int64_t segments;
    int32_t plan_seqs;       // sequences of the decode kernel's plan
    bool tensor;             // the prefix on the tensor cores (else in the plan)
    PrefixTcShape tc;
};

template <int kD>
cudaError_t prefix_plan(int32_t hkv, int32_t hq, int32_t num_seqs, int32_t prefix_len, PrefixPlan &pl)
{
    using Fmt = PrefixFormat<true, kD>;
    const int64_t rows = static_cast<int64_t>(num_seqs) * (hq / hkv);
    pl.tensor = kD == 128 && prefix_len > 0 && rows >= kTensorRows;
    pl.plan_seqs = num_seqs + (prefix_len > 0 && !pl.tensor ? 1 : 0);
    pl.smem = decode_smem_bytes<Fmt>(pl.plan_seqs, kRowsPerBlock);
    pl.merge_smem = row_merge_smem(pl.plan_seqs);
    const cudaError_t e = prefix_shape<kD>(pl.smem, pl.merge_smem, pl.ls);
    if (e != cudaSuccess)
        return e;
    const int64_t own = max_segments(hkv, hq, num_seqs, 0, false), blocks = hkv * prefix_blocks(hq, hkv, num_seqs);
    pl.segments = own + (pl.plan_seqs > num_seqs ? blocks : 0);
    // slots of the plan's pieces (either with or without the prefix), then those of the tensor-core
    // kernel: splits > 1 only while splits * hkv * row_pairs <= SMs, and a pair holds 32 row blocks
    pl.tc_slots = workspace_bytes_for<Fmt::kTiles>(static_cast<size_t>(pl.ls.sms) * pl.ls.occ * Fmt::kWarps, own);
    pl.workspace = pl.tc_slots + (blocks + (kD == 128 ? 32 * static_cast<int64_t>(pl.ls.sms) : 0)) *
                                     slot_floats<Fmt::kTiles>() * sizeof(float);
    if (pl.tensor)
        pl.tc = prefix_tc_shape(hkv, rows, prefix_len, pl.ls.sms);
    return cudaSuccess;
}

template <bool kRotate, int kD>
cudaError_t launch(const DecodeArgs &a, const int32_t *prefix_table, int32_t prefix_len, cudaStream_t stream)
{
    using Fmt = PrefixFormat<kRotate, kD>;
    const CUtensorMap *map = code_tensor_map<kD>(a.kv_pages, a.num_pages * a.num_kv_heads * 32);
    if (map == nullptr)
        return cudaErrorInvalidValue;
    PrefixPlan pl;
    cudaError_t e = prefix_plan<kD>(a.num_kv_heads, a.num_q_heads, a.num_seqs, prefix_len, pl);
    if (e != cudaSuccess)
        return e;
    DecodeParams p;
    fill_decode_params<kD>(a, p);
    p.num_seqs = pl.plan_seqs;
    p.qrows = kRowsPerBlock;
    p.max_segments = pl.segments;
    p.total_warps = pl.ls.sms * pl.ls.occ * Fmt::kWarps;
    p.prefix_seq = pl.plan_seqs > a.num_seqs ? a.num_seqs : -1;
    p.prefix_len = prefix_len;
    p.prefix_table = prefix_table;

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pl.ls.sms * pl.ls.occ));
    cfg.blockDim = dim3(32 * Fmt::kWarps);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    PrefixPieces pre = {nullptr, 0, 0};
    if (pl.tensor) {
        float *slots = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + pl.tc_slots);
        e = launch_prefix_tc(a, prefix_table, prefix_len, pl.tc, slots, stream);
        if (e != cudaSuccess)
            return e;
        pre = {slots, pl.tc.row_blocks, pl.tc.splits};
    }
    cfg.numAttrs = pl.tensor ? 1 : 0;   // the own tokens run beside the prefix
    e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<Fmt, kModePrefix>, *map, p);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(max_segments(a.num_kv_heads, a.num_q_heads, a.num_seqs, 0, false),
                                                               16 * pl.ls.sms)));
    cfg.blockDim = dim3(32 * kRowWarps);
    cfg.dynamicSmemBytes = pl.merge_smem;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, prefix_merge_kernel<kRotate, kD>, p, pre);
    if (e != cudaSuccess)
        return e;
    return cudaGetLastError();
}

}  // namespace

size_t decode_prefix_workspace_bytes(int32_t num_kv_heads, int32_t num_q_heads, int32_t num_seqs,
                                     int32_t prefix_len, int32_t head_dim)
{
    PrefixPlan pl;
    const cudaError_t e =
        head_dim == 64    ? prefix_plan<64>(num_kv_heads, num_q_heads, num_seqs, prefix_len, pl)
        : head_dim == 128 ? prefix_plan<128>(num_kv_heads, num_q_heads, num_seqs, prefix_len, pl)
        : head_dim == 256 ? prefix_plan<256>(num_kv_heads, num_q_heads, num_seqs, prefix_len, pl)
                          : cudaErrorInvalidValue;
    return e == cudaSuccess ? pl.workspace : 0;
}

cudaError_t launch_paged_decode_prefix(const DecodeArgs &a, const int32_t *prefix_table, int32_t prefix_len,
                                       cudaStream_t stream)
{
    switch (a.head_dim) {
    case 64:
        return a.rotate ? launch<true, 64>(a, prefix_table, prefix_len, stream)
                        : launch<false, 64>(a, prefix_table, prefix_len, stream);
    case 128:
        return a.rotate ? launch<true, 128>(a, prefix_table, prefix_len, stream)
                        : launch<false, 128>(a, prefix_table, prefix_len, stream);
    case 256:
        return a.rotate ? launch<true, 256>(a, prefix_table, prefix_len, stream)
                        : launch<false, 256>(a, prefix_table, prefix_len, stream);
    default:
        return cudaErrorInvalidValue;
    }
}

}  // namespace saw
