// evict.cu -- eviction from the INT4 paged cache by accumulated attention weight.
//
// Of a sequence of L tokens, n = min(L, keep) survive, per kv head: the first `sink` tokens, the last
// `recent` ones, and of those between them the keep - sink - recent with the largest mass (ties to the
// earlier token).  They move, in order, into the pages of new_table: codes, scales and masses as they
// are.  Each kv head keeps its own tokens; the page layout keeps heads apart, so a page simply holds
// other tokens for other heads.  The old pages are only read: they may be shared with other
// sequences, and go back to the allocator afterwards.
//
// Two kernels.  The selection (a CTA per sequence and kv head) finds the need-th largest mass by a
// radix select over the masses' bits (non-negative floats order as their bits) and writes the kept
// tokens' indices; the move (a warp per new page and kv head) gathers the rows.  Both are bound by
// the bytes of the masses and of the kept rows.
#include <algorithm>

#include "saw_device.cuh"
#include "saw_internal.h"

namespace saw {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelSmemKeys = 49152;   // masses held in shared memory (192 KiB); more are read again

struct EvictParams {
    uint8_t *kv_pages;
    uint8_t *scales;
    float *mass;
    int32_t hkv;
    int64_t num_pages;
    const int32_t *block_table;
    int32_t max_blocks;
    const int32_t *seq_lens;
    int32_t num_seqs;
    const int32_t *new_table;
    int32_t new_blocks;
    int32_t *new_lens;
    int32_t *kept;
    int32_t keep, sink, recent;
    int32_t smem_keys;
    uint32_t *status;
};

// Inclusive sum over the CTA of (a, b) packed in 64 bits; every thread gets its own prefix and the total.
__device__ __forceinline__ uint64_t cta_scan(uint64_t v, uint64_t *warp_sums, uint64_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d)
            x += y;
    }
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    uint64_t w = lane < kSelWarps ? warp_sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, w, d);
        if (lane >= d)
            w += y;
    }
    const uint64_t before = __shfl_sync(0xFFFFFFFFu, w, max(warp - 1, 0));
    total = __shfl_sync(0xFFFFFFFFu, w, 31);
    __syncthreads();
    return x + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p)
{
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t hist[256];
    __shared__ uint64_t warp_sums[kSelWarps];
    __shared__ uint32_t sh_digit, sh_need;
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int s = blockIdx.x / p.hkv, h = blockIdx.x - s * p.hkv;
    int32_t *kept = p.kept + static_cast<int64_t>(blockIdx.x) * p.keep;
    int L = p.seq_lens[s];
    // a length out of range, or more kept tokens than the new pages hold: left out
    const bool valid = L >= 0 && L <= p.max_blocks * kPageSize && min(L, p.keep) <= p.new_blocks * kPageSize;
    if (!valid) {
        if (tid == 0 && h == 0)
            set_status(p.status, SAW_DEV_BAD_SEQ_LEN);
        L = 0;
    }
    const int n = min(L, p.keep);
    if (tid == 0 && h == 0)
        p.new_lens[s] = n;
    for (int j = n + tid; j < p.keep; j += kSelThreads)
        kept[j] = -1;
    if (L <= p.keep) {
        for (int j = tid; j < n; j += kSelThreads)
            kept[j] = j;
        return;
    }
    // the middle tokens [sink, sink + M): keep `need` of them
    const int M = L - p.sink - p.recent;
    const uint32_t want = static_cast<uint32_t>(p.keep - p.sink - p.recent);
    const int32_t *table = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
    const bool in_smem = M <= p.smem_keys;
    // order-preserving key of middle token i; a NaN or negative mass counts as 0
    auto read_key = [&](int i) -> uint32_t {
        const int t = p.sink + i;
        const int32_t page = table[t / kPageSize];
        if (page < 0 || page >= p.num_pages) {
            set_status(p.status, SAW_DEV_BAD_PAGE);
            return 0;
        }
        const float m = p.mass[(static_cast<int64_t>(page) * p.hkv + h) * kPageSize + t % kPageSize];
        return m > 0.0f ? __float_as_uint(m) : 0u;
    };
    if (in_smem) {
        for (int i = tid; i < M; i += kSelThreads)
            keys[i] = read_key(i);
        __syncthreads();
    }
    auto key = [&](int i) { return in_smem ? keys[i] : read_key(i); };

    // radix select, 8 bits at a time: `prefix` holds the digits found so far of the want-th largest key
    uint32_t prefix = 0, need = want;
    if (want > 0)
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads)
                hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < M; i += kSelThreads) {
                const uint32_t k = key(i);
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                    atomicAdd(&hist[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid < 32) {
                // lane holds 8 digits, highest first over the warp: the digit where the running count
                // from above reaches `need`
                uint32_t c[8], sum = 0;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    c[e] = hist[255 - (8 * tid + e)];
                    sum += c[e];
                }
                uint32_t x = sum;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                    if (tid >= d)
                        x += y;
                }
                uint32_t above = x - sum;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    if (above < need && above + c[e] >= need) {
                        sh_digit = 255 - (8 * tid + e);
                        sh_need = need - above;
                    }
                    above += c[e];
                }
            }
            __syncthreads();
            prefix |= sh_digit << shift;
            need = sh_need;   // of the keys that share the digits so far
            __syncthreads();
        }
    // keys above `prefix` stay, and the first `need` that equal it
    for (int j = tid; j < p.sink; j += kSelThreads)
        kept[j] = j;
    for (int j = tid; j < p.recent; j += kSelThreads)
        kept[p.keep - p.recent + j] = L - p.recent + j;
    if (want == 0)
        return;
    const int per = ((M + kSelThreads - 1) / kSelThreads) | 1;   // odd: no bank conflicts between threads
    const int i0 = min(M, tid * per), i1 = min(M, i0 + per);
    uint64_t mine = 0;   // (above, equal) of this thread's run
    for (int i = i0; i < i1; i++) {
        const uint32_t k = key(i);
        mine += (static_cast<uint64_t>(k > prefix) << 32) | (k == prefix);
    }
    uint64_t total;
    const uint64_t incl = cta_scan(mine, warp_sums, total);
    uint32_t above = static_cast<uint32_t>((incl - mine) >> 32), equal = static_cast<uint32_t>(incl - mine);
    for (int i = i0; i < i1; i++) {
        const uint32_t k = key(i);
        if (k > prefix || (k == prefix && equal < need))
            kept[p.sink + above + min(equal, need)] = p.sink + i;
        above += k > prefix;
        equal += k == prefix;
    }
}

// A warp per (sequence, kv head, new page).
template <int kD>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictParams p)
{
    constexpr int kRowBytes_ = kD / 2;
    constexpr int kLanes = kRowBytes_ / 16;            // lanes of a code row
    constexpr int kRowsPerStep = 32 / kLanes;
    constexpr int kSteps = 32 / kRowsPerStep;          // 16 K rows, then 16 V rows
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int pages_per = (p.keep + kPageSize - 1) / kPageSize;
    const int64_t units = static_cast<int64_t>(p.num_seqs) * p.hkv * pages_per;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units; u += step) {
        const int64_t sh = u / pages_per;
        const int jp = static_cast<int>(u - sh * pages_per);
        const int s = static_cast<int>(sh / p.hkv), h = static_cast<int>(sh - static_cast<int64_t>(s) * p.hkv);
        const int n = min(kPageSize, p.new_lens[s] - kPageSize * jp);
        if (n <= 0)
            continue;
        const int32_t to = p.new_table[static_cast<int64_t>(s) * p.new_blocks + jp];
        // lane r (and r + 16): kept token r of the page, as its row within one (page, kv head, half)
        int64_t src = -1;
        const int r16 = lane & 15;
        if (r16 < n) {
            const int32_t t = p.kept[sh * p.keep + kPageSize * jp + r16];
            const int32_t page = p.block_table[static_cast<int64_t>(s) * p.max_blocks + t / kPageSize];
            if (page >= 0 && page < p.num_pages)
                src = (static_cast<int64_t>(page) * p.hkv + h) * (2 * kPageSize) + t % kPageSize;
            else
                set_status(p.status, SAW_DEV_BAD_PAGE);
        }
        if (to < 0 || to >= p.num_pages) {
            if (lane == 0)
                set_status(p.status, SAW_DEV_BAD_PAGE);
            continue;
        }
        const int64_t dst = (static_cast<int64_t>(to) * p.hkv + h) * (2 * kPageSize);
        uint4 w[kSteps];
        bool live[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
            const int row = i * kRowsPerStep + lane / kLanes, half = row >> 4;
            const int64_t from = __shfl_sync(0xFFFFFFFFu, src, row & 15);
            live[i] = from >= 0;
            if (live[i])
                w[i] = ldg_stream16(p.kv_pages + (from + half * kPageSize) * kRowBytes_ + 16 * (lane % kLanes));
        }
        const uint32_t *sc = reinterpret_cast<const uint32_t *>(p.scales);
        uint32_t pair = 0;
        float m = 0.0f;
        if (src >= 0) {
            pair = sc[src + (lane >> 4) * kPageSize];
            if (lane < 16)
                m = p.mass[(src / (2 * kPageSize)) * kPageSize + src % (2 * kPageSize)];
        }
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
            const int row = i * kRowsPerStep + lane / kLanes;
            if (live[i])
                *reinterpret_cast<uint4 *>(p.kv_pages + (dst + row) * kRowBytes_ + 16 * (lane % kLanes)) = w[i];
        }
        if (src >= 0) {
            reinterpret_cast<uint32_t *>(p.scales)[dst + lane] = pair;
            if (lane < 16)
                p.mass[(dst / (2 * kPageSize)) * kPageSize + lane] = m;
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t stream)
{
    EvictParams p;
    p.kv_pages = a.kv_pages;
    p.scales = static_cast<uint8_t *>(a.scales);
    p.mass = a.mass;
    p.hkv = a.num_kv_heads;
    p.num_pages = a.num_pages;
    p.block_table = a.block_table;
    p.max_blocks = a.max_blocks;
    p.seq_lens = a.seq_lens;
    p.num_seqs = a.num_seqs;
    p.new_table = a.new_table;
    p.new_blocks = a.new_blocks;
    p.new_lens = a.new_lens;
    p.kept = a.kept;
    p.keep = a.keep;
    p.sink = a.sink;
    p.recent = a.recent;
    p.status = a.status;
    const int64_t most = static_cast<int64_t>(a.max_blocks) * kPageSize;
    p.smem_keys = static_cast<int32_t>(std::min<int64_t>(most, kSelSmemKeys));

    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const size_t smem = static_cast<size_t>(p.smem_keys) * 4;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSelSmemKeys * 4);
    if (e != cudaSuccess)
        return e;
    evict_select_kernel<<<static_cast<unsigned>(a.num_seqs * a.num_kv_heads), kSelThreads, smem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * ((a.keep + kPageSize - 1) / kPageSize);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((units + 7) / 8, 8 * sms)));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = a.head_dim == 64    ? cudaLaunchKernelEx(&cfg, evict_move_kernel<64>, p)
        : a.head_dim == 128 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<128>, p)
                            : cudaLaunchKernelEx(&cfg, evict_move_kernel<256>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace saw
