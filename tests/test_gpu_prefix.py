"""Decode for a batch that shares a prefix, on the GPU against the fp64 oracle over each sequence's
concatenated tokens.  Tolerance: that of the decode (max abs 1e-2, mean abs 1e-3) and one rounding of
the output to bf16 (2^-8 relative)."""
import numpy as np
import pytest
import torch

from oracle import serving
from bit_paged_kv_block_b200 import synth
from helpers import MAX_ABS_TOL, MEAN_ABS_TOL, device_cache_from, oracle_cache, u16

pytestmark = pytest.mark.gpu

BF16_STEP = 2.0 ** -8


def assert_bf16_close(got, want, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    d = np.abs(got - want)
    over = d - BF16_STEP * np.abs(want)
    assert over.max() <= MAX_ABS_TOL, f"{what}: max {d.max():.3e}"
    assert d.mean() <= MEAN_ABS_TOL + BF16_STEP * np.abs(want).mean(), f"{what}: mean {d.mean():.3e}"


def _case(prefix, lens, hq, hkv, d, seed, rotate=True):
    """A cache whose sequence 0 is the prefix and whose others are the batch's own tokens."""
    wl = synth.custom(f"px{seed}", [prefix] + list(lens), num_q_heads=hq, num_kv_heads=hkv, seed=seed,
                      outlier_range=(10.0, 30.0), head_dim=d, num_pages=None)
    pages, scales = oracle_cache(wl, rotate=rotate)
    q = torch.randn(len(lens), hq, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    return wl, pages, scales, q


def _want(wl, pages, scales, q, prefix, lens, rotate=True):
    parts = [[(wl.block_table[0], prefix), (wl.block_table[1 + s], n)] for s, n in enumerate(lens)]
    return serving.decode_rows_fp64(u16(q), pages, scales, parts, rotate=rotate)[0]


def _run(saw, wl, pages, scales, q, prefix, lens, device, rotate=True, status=None, ws=None, out=None):
    kv, sc = device_cache_from(pages, scales, device)
    table = torch.from_numpy(wl.block_table).to(device)
    S, hq, d = q.shape
    hkv = pages.shape[1]
    if out is None:
        out = torch.full((S, hq, d), float("nan"), dtype=torch.bfloat16, device=device)
    if ws is None:
        ws = saw.allocate_prefix_workspace(hkv, hq, S, prefix, device, head_dim=d)
        ws.fill_(0x5A)
    saw.saw_paged_decode_attn_prefix(
        q.to(device), kv, sc, table[0].contiguous() if prefix else None, prefix,
        table[1:].contiguous(), torch.tensor(lens, dtype=torch.int32, device=device), out, ws,
        dev_status=status, rotate=rotate)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 128), (16, 1, 128), (6, 2, 128), (14, 2, 128),
                                      (10, 1, 64), (16, 4, 64), (8, 1, 256), (12, 4, 256)])
@pytest.mark.parametrize("prefix", [1, 15, 16, 37, 300])
def test_prefix_decode_matches_oracle(cuda_device, hq, hkv, d, prefix):
    """Prefixes of one token, ending inside and at the end of a page; own parts of 0, 1, page edges and
    a long one; 1 to 16 query heads per kv head, groups that straddle the prefix's row blocks."""
    from bit_paged_kv_block_b200 import saw
    lens = [0, 1, 16, 17, 200]
    wl, pages, scales, q = _case(prefix, lens, hq, hkv, d, seed=prefix + hq)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    got = _run(saw, wl, pages, scales, q, prefix, lens, cuda_device, status=status)
    assert int(status.item()) == 0
    assert_bf16_close(got, _want(wl, pages, scales, q, prefix, lens), f"{hq}/{hkv}/{d} prefix {prefix}")


@pytest.mark.parametrize("S", [1, 2, 31, 32, 33, 64, 100])
@pytest.mark.parametrize("rotate", [True, False])
def test_prefix_decode_batches(cuda_device, S, rotate):
    """Batches around the row counts of the prefix's tiles (4 query heads per kv head)."""
    from bit_paged_kv_block_b200 import saw
    lens = [(7 * s) % 40 for s in range(S)]
    prefix = 530
    wl, pages, scales, q = _case(prefix, lens, 8, 2, 128, seed=S, rotate=rotate)
    got = _run(saw, wl, pages, scales, q, prefix, lens, cuda_device, rotate=rotate)
    assert_bf16_close(got, _want(wl, pages, scales, q, prefix, lens, rotate), f"S={S}")


def test_prefix_decode_long_prefix(cuda_device):
    """A prefix long enough to be split over many warps and tiles, one sequence without tokens."""
    from bit_paged_kv_block_b200 import saw
    for lens, hq, hkv in (([0], 4, 1), ([3, 0, 50] * 14, 8, 1)):
        prefix = 6001
        wl, pages, scales, q = _case(prefix, lens, hq, hkv, 128, seed=len(lens))
        got = _run(saw, wl, pages, scales, q, prefix, lens, cuda_device)
        assert_bf16_close(got, _want(wl, pages, scales, q, prefix, lens), f"long, {len(lens)} sequences")


def test_no_prefix_is_the_decode(cuda_device):
    """prefix_len = 0: a plain decode; a sequence of no tokens is zero."""
    from bit_paged_kv_block_b200 import saw
    lens = [0, 5, 100, 0]
    wl, pages, scales, q = _case(1, lens, 8, 2, 128, seed=5)
    got = _run(saw, wl, pages, scales, q, 0, lens, cuda_device)
    want = _want(wl, pages, scales, q, 0, lens)
    assert_bf16_close(got, want, "no prefix")
    assert bool((got[0] == 0).all()) and bool((got[3] == 0).all())


@pytest.mark.parametrize("S", [3, 64])
def test_prefix_decode_flags_bad_lengths_and_pages(cuda_device, S):
    """A length out of range zeroes its rows and is flagged, the others are right; a page id out of
    range is flagged."""
    from bit_paged_kv_block_b200 import saw
    lens = [5 + s for s in range(S)]
    wl, pages, scales, q = _case(200, lens, 8, 2, 128, seed=21)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    bad = list(lens)
    bad[1], bad[2] = -3, 16 * wl.block_table.shape[1] + 1
    got = _run(saw, wl, pages, scales, q, 200, bad, cuda_device, status=status)
    assert int(status.item()) == saw.SAW_DEV_BAD_SEQ_LEN
    want = _want(wl, pages, scales, q, 200, lens)
    want[1:3] = 0.0
    assert_bf16_close(got, want, "bad lengths")
    for row, bit in ((0, 10 ** 6), (1, -7)):
        status.zero_()
        broken = synth.Workload(**{**wl.__dict__})
        broken.block_table = wl.block_table.copy()
        broken.block_table[row, 0] = bit
        _run(saw, broken, pages, scales, q, 200, lens, cuda_device, status=status)
        assert int(status.item()) == saw.SAW_DEV_BAD_PAGE


@pytest.mark.parametrize("S", [4, 64])
def test_prefix_decode_repeats_and_replays(cuda_device, S):
    """The same bits on every call, from a captured graph, on another stream, and with a workspace
    sized for more sequences and a longer prefix."""
    from bit_paged_kv_block_b200 import saw
    lens = [(13 * s) % 90 for s in range(S)]
    prefix = 900
    wl, pages, scales, q = _case(prefix, lens, 8, 2, 128, seed=33)
    kv, sc = device_cache_from(pages, scales, cuda_device)
    table = torch.from_numpy(wl.block_table).to(cuda_device)
    args = (q.to(cuda_device), kv, sc, table[0].contiguous(), prefix, table[1:].contiguous(),
            torch.tensor(lens, dtype=torch.int32, device=cuda_device))
    first = torch.empty(S, 8, 128, dtype=torch.bfloat16, device=cuda_device)
    ws = saw.allocate_prefix_workspace(2, 8, S + 40, 2 * prefix, cuda_device)
    saw.saw_paged_decode_attn_prefix(*args, first, ws)
    torch.cuda.synchronize()
    out = torch.empty_like(first)
    ws2 = saw.allocate_prefix_workspace(2, 8, S, prefix, cuda_device)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        saw.saw_paged_decode_attn_prefix(*args, out, ws2)
    stream.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saw.saw_paged_decode_attn_prefix(*args, out, ws2)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


# ---- the prefix on the tensor cores (64 query rows per kv head and 2^20 row-token pairs on) -------

@pytest.mark.parametrize("G,S,prefix", [
    (16, 64, 1024), (16, 64, 1025), (16, 64, 1087), (16, 64, 1088), (16, 64, 1151), (16, 65, 1152),
    (4, 18, 14600), (16, 9, 7300), (3, 43, 8192), (1, 100, 10500)])
def test_prefix_tensor_cores_match_oracle(cuda_device, G, S, prefix):
    """Row counts of one tile, two, and several pairs, whole and ragged (odd groups, rows past the last
    block of 8); prefixes that end at, just past and just before the edges of a 128-token block and of
    its halves; own parts from none on."""
    from bit_paged_kv_block_b200 import saw
    lens = [(11 * s) % 50 for s in range(S)]
    wl, pages, scales, q = _case(prefix, lens, G, 1, 128, seed=prefix + G)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    got = _run(saw, wl, pages, scales, q, prefix, lens, cuda_device, status=status)
    assert int(status.item()) == 0
    assert_bf16_close(got, _want(wl, pages, scales, q, prefix, lens), f"G={G} S={S} prefix {prefix}")


def test_prefix_tensor_cores_plain_cache_and_heads(cuda_device):
    from bit_paged_kv_block_b200 import saw
    lens = [(5 * s) % 30 for s in range(40)]
    wl, pages, scales, q = _case(2200, lens, 24, 3, 128, seed=3, rotate=False)
    got = _run(saw, wl, pages, scales, q, 2200, lens, cuda_device, rotate=False)
    assert_bf16_close(got, _want(wl, pages, scales, q, 2200, lens, rotate=False), "plain, 3 kv heads")


def test_prefix_tensor_cores_repeat_flag_and_replay(cuda_device):
    """The same bits eagerly and replayed; bad lengths zero their rows; a bad prefix page is flagged."""
    from bit_paged_kv_block_b200 import saw
    S, prefix = 64, 1100
    lens = [(13 * s) % 90 for s in range(S)]
    wl, pages, scales, q = _case(prefix, lens, 16, 1, 128, seed=34)
    want = _want(wl, pages, scales, q, prefix, lens)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    bad = list(lens)
    bad[1], bad[2] = -3, 16 * wl.block_table.shape[1] + 1
    got = _run(saw, wl, pages, scales, q, prefix, bad, cuda_device, status=status)
    assert int(status.item()) == saw.SAW_DEV_BAD_SEQ_LEN
    zeroed = want.copy()
    zeroed[1:3] = 0.0
    assert_bf16_close(got, zeroed, "bad lengths")
    status.zero_()
    broken = synth.Workload(**{**wl.__dict__})
    broken.block_table = wl.block_table.copy()
    broken.block_table[0, 3] = pages.shape[0]
    _run(saw, broken, pages, scales, q, prefix, lens, cuda_device, status=status)
    assert int(status.item()) == saw.SAW_DEV_BAD_PAGE
    kv, sc = device_cache_from(pages, scales, cuda_device)
    table = torch.from_numpy(wl.block_table).to(cuda_device)
    args = (q.to(cuda_device), kv, sc, table[0].contiguous(), prefix, table[1:].contiguous(),
            torch.tensor(lens, dtype=torch.int32, device=cuda_device))
    ws = saw.allocate_prefix_workspace(1, 16, S, prefix, cuda_device)
    first, out = (torch.empty(S, 16, 128, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    saw.saw_paged_decode_attn_prefix(*args, first, ws)
    torch.cuda.synchronize()
    assert_bf16_close(first, want, "eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saw.saw_paged_decode_attn_prefix(*args, out, ws)
    for _ in range(3):
        out.fill_(float("nan"))
        ws.fill_(0xFF)                     # NaN bits: nothing of the last call is read
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_prefix_few_rows_many_pieces(cuda_device):
    """One sequence behind a long prefix: each row joined from hundreds of pieces by a CTA of its own;
    also at D = 64 and 256, and the decode with weights over one long sequence."""
    from bit_paged_kv_block_b200 import saw
    for hq, hkv, d, prefix in ((4, 1, 128, 9000), (16, 1, 64, 5000), (6, 2, 256, 4001)):
        wl, pages, scales, q = _case(prefix, [9], hq, hkv, d, seed=d)
        got = _run(saw, wl, pages, scales, q, prefix, [9], cuda_device)
        assert_bf16_close(got, _want(wl, pages, scales, q, prefix, [9]), f"{hq}/{hkv}/{d}")


def test_prefix_batches_in_turn(cuda_device):
    """Tables past 48 KB of shared memory, with the prefix in the plan and on the tensor cores, and small
    calls between."""
    from bit_paged_kv_block_b200 import saw
    for S, hq, prefix in ((2600, 2, 40), (3, 2, 40), (2600, 2, 300), (2, 4, 33), (2600, 2, 40)):
        lens = [(7 * s) % 19 % 4 for s in range(S)]
        wl, pages, scales, q = _case(prefix, lens, hq, 1, 128, seed=S)
        got = _run(saw, wl, pages, scales, q, prefix, lens, cuda_device)
        assert_bf16_close(got, _want(wl, pages, scales, q, prefix, lens), f"{S} sequences")


@pytest.mark.parametrize("big", [2.0 ** 20, 2.0 ** -12])
def test_prefix_tensor_cores_query_magnitudes(cuda_device, big):
    """Queries far outside fp16's range once scaled: one element, on a channel whose largest key leads the
    next by 2% of it or more (logits are off by 2^-10 of themselves at most), so that a huge query takes
    that token's value; a tiny one the mean."""
    from bit_paged_kv_block_b200 import saw
    S, prefix, hq = 64, 1100, 16
    wl, pages, scales, q = _case(prefix, [0] * S, hq, 1, 128, seed=81, rotate=False)
    K = serving.rows_fp64(pages, scales, wl.block_table[0], prefix, 0, 0)
    top = np.sort(K, axis=0)
    clear = [c for c in range(128) if top[-1, c] - top[-2, c] >= 0.02 * top[-1, c] > 0.02]
    assert len(clear) >= 4
    q.zero_()
    for s in range(S):
        for h in range(hq):
            q[s, h, clear[(s + h) % len(clear)]] = big
    got = _run(saw, wl, pages, scales, q, prefix, [0] * S, cuda_device, rotate=False)
    assert_bf16_close(got, _want(wl, pages, scales, q, prefix, [0] * S, rotate=False), f"{big}")
