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
// prefix's pages.  All pieces go to workspace slots; the prefix's are stored as rows, since the rows
// of an output segment (sequence, kv head, up to 8 heads) may lie in two of its blocks.
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

// One CTA per output segment (sequence s, kv head h, block of up to 8 of its heads): fold the pieces
// of the sequence's own tokens, then those of the prefix for the same query rows, and write the rows.
// The warps take pieces in turn and warp 0 folds the warps' results in order, so the result does not
// depend on timing.
template <bool kRotate, int kD>
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const DecodeParams p, const PrefixPieces pre)
{
    using Fmt = PrefixFormat<kRotate, kD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 15) & ~uintptr_t(15));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kTiles = Fmt::kTiles;
    constexpr int kSlot = slot_floats<kTiles>();
    SeqTables tb;
    tb.bind(smem + merge_smem_tables<kTiles>(), p.num_seqs);
    volatile int64_t *flags = reinterpret_cast<volatile int64_t *>(smem + merge_smem_flags<kTiles>());
    float *slots = reinterpret_cast<float *>(smem);

    scan_sequences<kModePrefix>(p, tb, flags, false);
    Plan plan;
    plan.init(tb, p.num_seqs, p.total_warps);
    pdl_wait();   // the pieces
    const int nb = (p.group + kRowsPerBlock - 1) / kRowsPerBlock;
    const int g = lane >> 2, t = lane & 3;
    for (int o = blockIdx.x; o < p.batch * p.hkv * nb; o += gridDim.x) {
        const int s = o / (p.hkv * nb), j = o - s * (p.hkv * nb);
        const int len = p.seq_lens[s];
        const bool valid = len >= 0 && len <= p.max_blocks * kPageSize;
        WarpState<kTiles> st;
        state_reset(st);
        if (valid && tb.npg[s] > 0) {
            const int64_t gseg = tb.spre[s] + j;
            const int64_t u_hi = plan.warp_of_cost(plan.page_cost(s, j, tb.npg[s] - 1));
            for (int64_t u = plan.warp_of_cost(plan.page_cost(s, j, 0)) + warp; u <= u_hi; u += kMergeWarps) {
                float bm[2], bl[2];
                float4 bo[kTiles];
                load_partial(p.partials + (gseg + u) * kSlot, lane, bm, bl, bo);
                merge_into(st.m, st.l, st.o, bm, bl, bo);
            }
        }
        Segment<kModePrefix> sg;
        sg.s = s;
        sg.j = j;
        sg.h = j / nb;
        sg.b = j - sg.h * nb;
        sg.row0 = kRowsPerBlock * sg.b;
        sg.nrows = min(kRowsPerBlock, p.group - sg.row0);
        sg.qrow0 = s;
        if (valid && (p.prefix_seq >= 0 || pre.splits > 0)) {
            const int ps = p.prefix_seq;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                if (2 * t + e >= sg.nrows)
                    continue;
                const int row = s * p.group + sg.row0 + 2 * t + e;
                const int pr = row % kRowsPerBlock;
                const float *slot0;
                int pieces;
                if (pre.splits > 0) {
                    slot0 = pre.slots + (static_cast<int64_t>(sg.h) * pre.row_blocks + row / kRowsPerBlock) * pre.splits * kSlot;
                    pieces = pre.splits;
                } else {
                    const int pj = sg.h * tb.nbk[ps] + row / kRowsPerBlock;
                    const int64_t u_lo = plan.warp_of_cost(plan.page_cost(ps, pj, 0));
                    slot0 = p.partials + (tb.spre[ps] + pj + u_lo) * kSlot;
                    pieces = static_cast<int>(plan.warp_of_cost(plan.page_cost(ps, pj, tb.npg[ps] - 1)) - u_lo) + 1;
                }
                for (int k = warp; k < pieces; k += kMergeWarps) {
                    const float *slot = slot0 + static_cast<int64_t>(k) * kSlot;
                    const float bm = slot[8 * kD + pr], bl = slot[8 * kD + 8 + pr];
                    const float4 *o4 = reinterpret_cast<const float4 *>(slot + pr * kD) + g;
                    const float mn = fmaxf(st.m[e], bm);
                    const float fa = mn == -INFINITY ? 0.0f : ex2_approx(st.m[e] - mn);
                    const float fb = mn == -INFINITY ? 0.0f : ex2_approx(bm - mn);
                    st.m[e] = mn;
                    st.l[e] = st.l[e] * fa + bl * fb;
#pragma unroll
                    for (int c = 0; c < kTiles / 2; c++) {
                        const float4 v = o4[8 * c];
                        st.o[2 * c][e] = st.o[2 * c][e] * fa + v.x * fb;
                        st.o[2 * c][2 + e] = st.o[2 * c][2 + e] * fa + v.y * fb;
                        st.o[2 * c + 1][e] = st.o[2 * c + 1][e] * fa + v.z * fb;
                        st.o[2 * c + 1][2 + e] = st.o[2 * c + 1][2 + e] * fa + v.w * fb;
                    }
                }
            }
        }
        if (warp > 0)
            store_partial(slots + (warp - 1) * kSlot, lane, st);
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kMergeWarps; w++) {
                float bm[2], bl[2];
                float4 bo[kTiles];
                load_partial(slots + (w - 1) * kSlot, lane, bm, bl, bo);
                merge_into(st.m, st.l, st.o, bm, bl, bo);
            }
            Fmt::finalize(p, sg, lane, st.o, st.m, st.l);
        }
        __syncthreads();
    }
}

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
    pl.merge_smem = merge_smem_bytes<Fmt::kTiles>(pl.plan_seqs);
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
                                                               8 * pl.ls.sms)));
    cfg.blockDim = dim3(kMergeThreads);
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
