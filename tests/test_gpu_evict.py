"""Decode with accumulated attention weights, eviction by them, and a run of the serving operators
together, on the GPU against the oracle.  The eviction is exact.  A weight w is off by at most
w (e^(2 d) - 1), d the error of a logit: fp32 sums of D + 16 terms whose magnitudes the oracle bounds
(each addition and product off by at most 2^-24 of the magnitudes' sum), plus 2^-22 of it for the two
fp16 parts of the query; and exp2 and the sums over heads and tokens add a few 2^-22 relative."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving
from bit_paged_kv_block_b200 import synth
from helpers import NTHREADS, device_cache_from, oracle_cache, u16
from test_gpu_prefix import assert_bf16_close

pytestmark = pytest.mark.gpu


def _case(lens, hq, hkv, d, seed, rotate=True):
    wl = synth.custom(f"ev{seed}", lens, num_q_heads=hq, num_kv_heads=hkv, seed=seed,
                      outlier_range=(10.0, 30.0), head_dim=d)
    pages, scales = oracle_cache(wl, rotate=rotate)
    q = torch.randn(len(lens), hq, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    mass = np.random.default_rng(seed).random((pages.shape[0], hkv, 16)).astype(np.float32)
    return wl, pages, scales, q, mass


def _assert_mass(got, before, wl, lens, weights, terms, d):
    want = before.astype(np.float64)
    tol = np.zeros_like(want)
    for s, n in enumerate(lens):
        for h in range(before.shape[1]):
            err = terms[s, h] * ((d + 16) * 2.0 ** -24 + 2.0 ** -22)
            for t in range(n):
                at = wl.block_table[s, t // 16], h, t % 16
                w = weights[s][h][t]
                want[at] += w
                tol[at] += w * np.expm1(2 * err + 2.0 ** -19) + 2.0 ** -23 * want[at]
    off = np.abs(got.astype(np.float64) - want) - tol
    assert off.max() <= 0, f"mass off by {np.abs(got - want).max():.3e}"
    untouched = tol == 0
    assert np.array_equal(got[untouched], before[untouched])      # slots past the lengths


def _decode(saw, device, wl, pages, scales, q, mass, lens, rotate=True, status=None, sm_scale=None):
    kv, sc = device_cache_from(pages, scales, device)
    S, hq, d = q.shape
    hkv = pages.shape[1]
    out = torch.full((S, hq, d), float("nan"), dtype=torch.bfloat16, device=device)
    ws = saw.allocate_mass_workspace(hkv, hq, S, wl.block_table.shape[1], device, head_dim=d)
    ws.fill_(0x5A)
    dmass = torch.from_numpy(mass.copy()).to(device)
    saw.saw_paged_decode_attn_mass(q.to(device), kv, sc, dmass, torch.from_numpy(wl.block_table).to(device),
                                   torch.tensor(lens, dtype=torch.int32, device=device), out, ws,
                                   dev_status=status, rotate=rotate, sm_scale=sm_scale)
    torch.cuda.synchronize()
    return out, dmass.cpu().numpy()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 128), (16, 1, 128), (6, 2, 128), (10, 1, 128),
                                      (14, 2, 64), (16, 4, 64), (8, 1, 256), (12, 1, 256)])
@pytest.mark.parametrize("rotate", [True, False])
def test_decode_mass_matches_oracle(cuda_device, hq, hkv, d, rotate):
    """Lengths 0, 1, page edges and long enough to be split; odd and even groups up to 16."""
    from bit_paged_kv_block_b200 import saw
    lens = [0, 1, 15, 16, 33, 700]
    wl, pages, scales, q, mass = _case(lens, hq, hkv, d, seed=hq + d, rotate=rotate)
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out, got = _decode(saw, cuda_device, wl, pages, scales, q, mass, lens, rotate, status)
    assert int(status.item()) == 0
    parts = [[(wl.block_table[s], n)] for s, n in enumerate(lens)]
    want, weights, terms = serving.decode_rows_fp64(u16(q), pages, scales, parts, rotate=rotate)
    assert_bf16_close(out, want, f"{hq}/{hkv}/{d}")
    _assert_mass(got, mass, wl, lens, weights, terms, d)


def test_decode_mass_many_and_few_segments(cuda_device):
    """One long sequence on one kv head (split over every warp), and many short ones."""
    from bit_paged_kv_block_b200 import saw
    for lens, hq, hkv in (([4000], 2, 1), ([9001], 6, 1), ([(5 * s) % 37 for s in range(200)], 8, 4)):
        wl, pages, scales, q, mass = _case(lens, hq, hkv, 128, seed=len(lens))
        out, got = _decode(saw, cuda_device, wl, pages, scales, q, mass, lens)
        parts = [[(wl.block_table[s], n)] for s, n in enumerate(lens)]
        want, weights, terms = serving.decode_rows_fp64(u16(q), pages, scales, parts)
        assert_bf16_close(out, want, f"{len(lens)} sequences")
        _assert_mass(got, mass, wl, lens, weights, terms, 128)


def test_decode_mass_batches_and_groups_in_turn(cuda_device):
    """Many sequences (tables past 48 KB of shared memory), then few with the other group size, then many
    again: what a call may use does not depend on the calls before it."""
    from bit_paged_kv_block_b200 import saw
    cases = []
    for S, hq in ((2600, 2), (3, 8), (2600, 2), (2500, 8), (200, 2), (2500, 8)):
        lens = [(7 * s) % 19 % 4 for s in range(S)]
        wl, pages, scales, q, mass = _case(lens, hq, 1, 128, seed=hq)
        cases.append((wl, q, mass, lens, pages, scales, *_decode(saw, cuda_device, wl, pages, scales, q, mass, lens)))
    for wl, q, mass, lens, pages, scales, out, got in cases:
        parts = [[(wl.block_table[s], n)] for s, n in enumerate(lens)]
        want, weights, terms = serving.decode_rows_fp64(u16(q), pages, scales, parts)
        assert_bf16_close(out, want, f"{len(lens)} sequences")
        _assert_mass(got, mass, wl, lens, weights, terms, 128)


def test_decode_mass_shared_pages_and_flags(cuda_device):
    """Two sequences over the same pages both add; bad lengths and page ids are flagged, add nothing,
    and leave the others right."""
    from bit_paged_kv_block_b200 import saw
    lens = [40, 40, 20, 20, 30]
    wl, pages, scales, q, mass = _case(lens, 8, 2, 128, seed=2)
    wl.block_table[1] = wl.block_table[0]
    status = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out, got = _decode(saw, cuda_device, wl, pages, scales, q, mass, lens, status=status)
    assert int(status.item()) == 0
    parts = [[(wl.block_table[s], n)] for s, n in enumerate(lens)]
    want, weights, terms = serving.decode_rows_fp64(u16(q), pages, scales, parts)
    assert_bf16_close(out, want, "shared")
    _assert_mass(got, mass, wl, lens, weights, terms, 128)
    bad = [40, 0, -1, 16 * wl.block_table.shape[1] + 1, 30]
    out, got = _decode(saw, cuda_device, wl, pages, scales, q, mass, bad, status=status)
    assert int(status.item()) == saw.SAW_DEV_BAD_SEQ_LEN
    assert bool((out[1:4] == 0).all())
    _assert_mass(got, mass, wl, [40, 0, 0, 0, 30], weights, terms, 128)
    status.zero_()
    wl.block_table[4, 1] = pages.shape[0]
    out, got = _decode(saw, cuda_device, wl, pages, scales, q, mass, lens, status=status)
    assert int(status.item()) == saw.SAW_DEV_BAD_PAGE
    assert np.isfinite(got).all()


def test_decode_mass_extreme_logits(cuda_device):
    """A softmax scale that makes one token take everything: weights 1 and 0, no NaN."""
    from bit_paged_kv_block_b200 import saw
    lens = [300, 17]
    wl, pages, scales, q, mass = _case(lens, 4, 2, 128, seed=4)
    out, got = _decode(saw, cuda_device, wl, pages, scales, q, mass, lens, sm_scale=40.0)
    assert np.isfinite(got).all() and bool(torch.isfinite(out).all())
    total = (got.astype(np.float64) - mass).sum(axis=(0, 2))
    assert np.abs(total - 2 * len(lens)).max() < 1e-3      # G weights of 1 per sequence and kv head


def _masses(rng, kind, shape):
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, np.float32)
    if kind == "zero":
        return np.zeros(shape, np.float32)
    if kind == "wide":
        return (10.0 ** rng.uniform(-40, 30, shape)).astype(np.float32)
    if kind == "odd":
        m = rng.random(shape).astype(np.float32)
        m[rng.random(shape) < 0.1] = np.nan
        m[rng.random(shape) < 0.1] = -1.0
        m[rng.random(shape) < 0.05] = np.inf
        return m
    return rng.random(shape).astype(np.float32)


def _evict(saw, device, lens, hkv, d, keep, sink, recent, kind, seed, max_len=None):
    rng = np.random.default_rng(seed)
    S = len(lens)
    blocks = max(1, max((n + 15) // 16 for n in lens)) + 1
    new_blocks = max(1, max((min(n, keep) + 15) // 16 for n in lens))
    total = S * (blocks + new_blocks) + 2
    ids = rng.permutation(total).astype(np.int32)
    table, new_table = ids[:S * blocks].reshape(S, blocks), ids[S * blocks:S * (blocks + new_blocks)].reshape(S, new_blocks)
    pages = rng.integers(0, 256, (total, hkv, 2, 16, d // 2)).astype(np.uint8)
    scales = rng.integers(0, 1 << 16, (total, hkv, 2, 16, 2)).astype(np.uint16)
    mass = _masses(rng, kind, (total, hkv, 16))
    kv, sc = device_cache_from(pages, scales, device)
    dmass = torch.from_numpy(mass.copy()).to(device)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
    new_lens = torch.full((S,), -9, dtype=torch.int32, device=device)
    kept = torch.full((S, hkv, keep), -9, dtype=torch.int32, device=device)
    status = torch.zeros(1, dtype=torch.int32, device=device)
    lens = np.array(lens, np.int32)
    saw.saw_evict_paged(kv, sc, dmass, dev(table), dev(lens), dev(new_table), new_lens, kept, sink=sink,
                        recent=recent, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want_lens, want_kept = serving.evict(pages, scales, mass, table, lens, new_table, keep, sink, recent)
    assert np.array_equal(new_lens.cpu().numpy(), want_lens)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(kv.cpu().numpy(), pages) and np.array_equal(u16(sc), scales)
    assert np.array_equal(dmass.cpu().numpy().view(np.int32), mass.view(np.int32))


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "zero", "wide", "odd"])
@pytest.mark.parametrize("keep,sink,recent", [(64, 4, 16), (40, 0, 0), (40, 40, 0), (33, 0, 33), (1, 0, 0),
                                              (50, 20, 29)])
def test_evict_matches_oracle(cuda_device, kind, keep, sink, recent):
    """Lengths of 0, 1, at and around `keep`, and longer; ties, constants, wide ranges, NaN, negative
    and infinite masses; every slot that is not written keeps its bits."""
    from bit_paged_kv_block_b200 import saw
    _evict(saw, cuda_device, [0, 1, keep, keep + 1, 300, 97], 2, 128, keep, sink, recent, kind, seed=keep)


@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 1), (256, 2)])
def test_evict_long_sequences(cuda_device, d, hkv):
    from bit_paged_kv_block_b200 import saw
    _evict(saw, cuda_device, [5000, 1234], hkv, d, 1111, 4, 100, "random", seed=d)
    _evict(saw, cuda_device, [5000], hkv, d, 4990, 4, 100, "ties", seed=d + 1)


def test_evict_more_masses_than_shared_memory(cuda_device):
    """A sequence whose masses do not fit the selection's shared memory."""
    from bit_paged_kv_block_b200 import saw
    _evict(saw, cuda_device, [60000], 1, 64, 700, 4, 300, "ties", seed=6)


def test_evict_flags_bad_sequences(cuda_device):
    """Lengths out of range and too few new pages leave the sequence out; a page id out of range skips
    its tokens; the others move."""
    from bit_paged_kv_block_b200 import saw
    dev = cuda_device
    kv = torch.randint(0, 256, (30, 1, 2, 16, 64), dtype=torch.uint8, device=dev)
    sc = torch.rand(30, 1, 2, 16, 2, device=dev).half()
    mass = torch.rand(30, 1, 16, device=dev)
    before = kv.clone()
    table = torch.arange(15, dtype=torch.int32, device=dev).view(5, 3)
    new = torch.arange(15, 25, dtype=torch.int32, device=dev).view(5, 2)
    lens = torch.tensor([-1, 49, 48, 48, 20], dtype=torch.int32, device=dev)
    new_lens = torch.full((5,), -9, dtype=torch.int32, device=dev)
    kept = torch.full((5, 1, 33), -9, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    saw.saw_evict_paged(kv, sc, mass, table, lens, new, new_lens, kept, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == saw.SAW_DEV_BAD_SEQ_LEN         # 33 kept tokens need 3 pages
    assert new_lens.tolist() == [0, 0, 0, 0, 20]
    assert bool((kept[:4] == -1).all()) and kept[4, 0, :20].tolist() == list(range(20))
    assert torch.equal(kv[23, 0], before[12, 0]) and torch.equal(kv[:15], before[:15])
    assert torch.equal(kv[15:23], before[15:23])
    status.zero_()
    table[4, 1] = 10 ** 6
    new[3, 0] = -2
    saw.saw_evict_paged(kv, sc, mass, table, torch.tensor([0, 0, 0, 10, 20], dtype=torch.int32, device=dev),
                        new, new_lens, kept, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == saw.SAW_DEV_BAD_PAGE
    assert new_lens.tolist() == [0, 0, 0, 10, 20] and torch.equal(kv[23, 0], before[12, 0])


def test_evict_replays(cuda_device):
    """A captured eviction and decode, replayed, give the eager calls' bits."""
    from bit_paged_kv_block_b200 import saw
    lens = [200, 90, 33]
    wl, pages, scales, q, mass = _case(lens, 8, 2, 128, seed=14)
    kv, sc = device_cache_from(np.concatenate([pages, pages]), np.concatenate([scales, scales]), cuda_device)
    n0 = pages.shape[0]
    assert n0 >= 6
    dmass = torch.from_numpy(np.concatenate([mass, mass])).to(cuda_device)
    table = torch.from_numpy(wl.block_table).to(cuda_device)
    new = torch.arange(n0, n0 + 6, dtype=torch.int32, device=cuda_device).view(3, 2)
    dlens = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    new_lens = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    kept = torch.zeros(3, 2, 32, dtype=torch.int32, device=cuda_device)
    out = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device=cuda_device)
    ws = saw.allocate_mass_workspace(2, 8, 3, 2, cuda_device)
    dq = q.to(cuda_device)

    def step():
        saw.saw_evict_paged(kv, sc, dmass, table, dlens, new, new_lens, kept, sink=2, recent=8)
        saw.saw_paged_decode_attn_mass(dq, kv, sc, dmass, new, new_lens, out, ws)

    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in (kv, sc, dmass, new_lens, kept, out)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (new_lens, kept, out):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, (kv, sc, dmass, new_lens, kept, out)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("d", [64, 128])
def test_serving_run(cuda_device, d):
    """The operators as they are used together: prompts appended with rotary positions, decode steps
    that accumulate weights, an eviction, further steps on the shorter cache at their true positions,
    and a decode of the same sequences behind a shared prefix; cache bits against the oracle throughout."""
    from bit_paged_kv_block_b200 import saw
    dev = cuda_device
    S, hq, hkv, keep, sink, recent, prefix = 3, 8, 2, 24, 2, 8, 35
    prompts, steps = [40, 21, 60], 3
    g = torch.Generator().manual_seed(d)
    draw = lambda n, h: torch.randn(n, h, d, generator=g).to(torch.bfloat16)
    table = torch.zeros(256, d, device=dev)
    saw.saw_rope_table(table, saw.rope_scaling("banded", base=500000.0, factor=8.0, original_positions=64))
    rope, host_table = (table, False), table.cpu().numpy()
    P, blocks = 40, 5
    pages, scales = oracle.empty_cache(P, hkv, d)
    pages[:], scales[:] = 0xA5, 0x7E00
    mass = np.zeros((P, hkv, 16), np.float32)
    kv, sc = device_cache_from(pages, scales, dev)
    dmass = saw.allocate_mass(P, hkv, dev)
    ids = np.random.default_rng(d).permutation(P).astype(np.int32)
    bt, new_bt, pt = ids[:15].reshape(S, blocks), ids[15:30].reshape(S, blocks), ids[30:33]

    def append(q, k, v, pos, slots):
        pos, slots = np.array(pos, np.int64), np.array(slots, np.int64)
        q_out = torch.empty_like(q, device=dev)
        saw.saw_rope_rotate_quantize_paged(q.to(dev), k.to(dev), v.to(dev), torch.from_numpy(pos).to(dev),
                                           torch.from_numpy(slots).to(dev), rope, q_out, kv, sc, mass=dmass)
        oracle.rotate_quantize_paged(serving.rope_bf16(synth.bf16_bits(k), pos, host_table, False),
                                     synth.bf16_bits(v), slots, pages, scales, nthreads=NTHREADS)

    # the prefix, then each sequence's prompt at the positions after it
    append(draw(prefix, hq), draw(prefix, hkv), draw(prefix, hkv), range(prefix),
           [int(pt[t // 16]) * 16 + t % 16 for t in range(prefix)])
    for s, n in enumerate(prompts):
        append(draw(n, hq), draw(n, hkv), draw(n, hkv), range(prefix, prefix + n),
               [int(bt[s, t // 16]) * 16 + t % 16 for t in range(n)])
    cur_table, lens, pos = bt, list(prompts), [prefix + n for n in prompts]
    q_rot = torch.empty(S, hq, d, dtype=torch.bfloat16, device=dev)
    out = torch.empty(S, hq, d, dtype=torch.bfloat16, device=dev)
    ws = saw.allocate_mass_workspace(hkv, hq, S, blocks, dev, head_dim=d)

    def step():
        q, k, v = draw(S, hq), draw(S, hkv), draw(S, hkv)
        slots = np.array([int(cur_table[s, lens[s] // 16]) * 16 + lens[s] % 16 for s in range(S)], np.int64)
        at = np.array(pos, np.int64)
        for s in range(S):
            lens[s] += 1
            pos[s] += 1
        dlens = torch.tensor(lens, dtype=torch.int32, device=dev)
        before = dmass.clone()
        saw.saw_decode_step_rope(q.to(dev), k.to(dev), v.to(dev), torch.from_numpy(at).to(dev),
                                 torch.from_numpy(slots).to(dev), rope, q_rot, kv, sc,
                                 torch.from_numpy(cur_table).to(dev), dlens, out, ws, mass=dmass)
        qr = serving.rope_bf16(synth.bf16_bits(q), at, host_table, False)
        oracle.rotate_quantize_paged(serving.rope_bf16(synth.bf16_bits(k), at, host_table, False),
                                     synth.bf16_bits(v), slots, pages, scales)
        assert np.array_equal(u16(q_rot), qr)
        assert np.array_equal(kv.cpu().numpy(), pages) and np.array_equal(u16(sc), scales)
        want, weights, terms = serving.decode_rows_fp64(qr, pages, scales,
                                                        [[(cur_table[s], lens[s])] for s in range(S)])
        assert_bf16_close(out, want, "step")
        start = before.cpu().numpy()
        for s in slots:
            start[s // 16, :, s % 16] = 0.0
        wl = synth.Workload(**{**synth.custom("x", [1], num_q_heads=1, num_kv_heads=1).__dict__})
        wl.block_table = cur_table
        _assert_mass(dmass.cpu().numpy(), start, wl, lens, weights, terms, d)
        return qr

    for _ in range(steps):
        step()
    new_lens = torch.zeros(S, dtype=torch.int32, device=dev)
    kept = torch.zeros(S, hkv, keep, dtype=torch.int32, device=dev)
    mass[:] = dmass.cpu().numpy()
    saw.saw_evict_paged(kv, sc, dmass, torch.from_numpy(bt).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                        torch.from_numpy(new_bt).to(dev), new_lens, kept, sink=sink, recent=recent)
    want_lens, want_kept = serving.evict(pages, scales, mass, bt, lens, new_bt, keep, sink, recent)
    assert np.array_equal(kept.cpu().numpy(), want_kept) and new_lens.tolist() == want_lens.tolist()
    assert np.array_equal(dmass.cpu().numpy(), mass)
    cur_table, lens = new_bt, want_lens.tolist()
    for _ in range(steps):
        qr = step()
    # the last queries again, behind the shared prefix
    pws = saw.allocate_prefix_workspace(hkv, hq, S, prefix, dev, head_dim=d)
    saw.saw_paged_decode_attn_prefix(q_rot, kv, sc, torch.from_numpy(pt).to(dev), prefix,
                                     torch.from_numpy(cur_table).to(dev),
                                     torch.tensor(lens, dtype=torch.int32, device=dev), out, pws)
    want = serving.decode_rows_fp64(qr, pages, scales, [[(pt, prefix), (cur_table[s], lens[s])] for s in range(S)])[0]
    assert_bf16_close(out, want, "behind the prefix")


def test_step_rope_matches_append_then_decode(cuda_device):
    """saw_decode_step_rope without masses: the ordinary decode's bits after the append."""
    from bit_paged_kv_block_b200 import saw
    dev = cuda_device
    lens = [30, 1, 500]
    wl, pages, scales, q, _ = _case(lens, 8, 2, 128, seed=41)
    kv, sc = device_cache_from(pages, scales, dev)
    kv2, sc2 = kv.clone(), sc.clone()
    table = torch.zeros(600, 64, device=dev)
    saw.saw_rope_table(table, saw.rope_scaling())
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(3, 2, 128, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    pos = torch.tensor([n - 1 for n in lens], device=dev)
    bt = torch.from_numpy(wl.block_table).to(dev)
    slots = bt[torch.arange(3, device=dev), pos // 16].long() * 16 + pos % 16
    dlens = torch.tensor(lens, dtype=torch.int32, device=dev)
    ws = saw.allocate_workspace(2, 8, 3, dev)
    out, out2 = (torch.empty(3, 8, 128, device=dev) for _ in range(2))
    q_rot, q_rot2 = (torch.empty(3, 8, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
    saw.saw_decode_step_rope(q.to(dev), k, v, pos, slots, (table, True), q_rot, kv, sc, bt, dlens, out, ws)
    saw.saw_rope_rotate_quantize_paged(q.to(dev), k, v, pos, slots, (table, True), q_rot2, kv2, sc2)
    saw.saw_paged_decode_attn(q_rot2, kv2, sc2, bt, dlens, out2, ws)
    torch.cuda.synchronize()
    assert torch.equal(q_rot.view(torch.int16), q_rot2.view(torch.int16))
    assert torch.equal(kv, kv2) and torch.equal(out, out2)


@pytest.mark.parametrize("with_mass", [False, True])
def test_step_rope_appends_behind_empty_lengths(cuda_device, with_mass):
    """Lengths of zero: nothing to decode, but the step is over only once the tokens are in the cache."""
    from bit_paged_kv_block_b200 import saw
    dev = cuda_device
    S = 300
    kv = torch.zeros(S, 2, 2, 16, 64, dtype=torch.uint8, device=dev)
    sc = torch.zeros(S, 2, 2, 16, 2, dtype=torch.float16, device=dev)
    kv2, sc2 = kv.clone(), sc.clone()
    table = torch.zeros(64, 128, device=dev)
    saw.saw_rope_table(table, saw.rope_scaling())
    g = torch.Generator().manual_seed(2)
    q = torch.randn(S, 8, 128, generator=g).to(torch.bfloat16).to(dev)
    k, v = (torch.randn(S, 2, 128, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    pos = torch.arange(S, device=dev) % 64
    slots = torch.arange(S, device=dev) * 16 + 3
    bt = torch.arange(S, dtype=torch.int32, device=dev).view(S, 1)
    lens = torch.zeros(S, dtype=torch.int32, device=dev)
    q_rot = torch.empty_like(q)
    if with_mass:
        mass = torch.ones(S, 2, 16, device=dev)
        out = torch.full((S, 8, 128), float("nan"), dtype=torch.bfloat16, device=dev)
        ws = saw.allocate_mass_workspace(2, 8, S, 1, dev)
        saw.saw_decode_step_rope(q, k, v, pos, slots, (table, False), q_rot, kv, sc, bt, lens, out, ws, mass=mass)
    else:
        out = torch.full((S, 8, 128), float("nan"), device=dev)
        ws = saw.allocate_workspace(2, 8, S, dev)
        saw.saw_decode_step_rope(q, k, v, pos, slots, (table, False), q_rot, kv, sc, bt, lens, out, ws)
    got, got_q = kv.clone(), q_rot.clone()          # queued right behind the step
    q_rot2 = torch.empty_like(q)
    saw.saw_rope_rotate_quantize_paged(q, k, v, pos, slots, (table, False), q_rot2, kv2, sc2)
    torch.cuda.synchronize()
    assert torch.equal(got, kv2) and torch.equal(got_q, q_rot2)
    assert bool((out == 0).all())
    if with_mass:
        want = torch.ones(S, 2, 16)
        want[:, :, 3] = 0.0
        assert torch.equal(mass.cpu(), want)


def test_calls_on_two_streams_at_once(cuda_device):
    """Prefix decodes (tensor cores and plan) and decodes with weights in flight together, each stream with
    its own workspaces, outputs and masses: the bits of one call at a time."""
    from bit_paged_kv_block_b200 import saw
    dev = cuda_device
    lens = [(29 * s) % 120 for s in range(64)]
    wl, pages, scales, q, mass = _case([1100] + lens, 16, 1, 128, seed=91)
    kv, sc = device_cache_from(pages, scales, dev)
    table = torch.from_numpy(wl.block_table).to(dev)
    own, prefix = table[1:].contiguous(), table[0].contiguous()
    dlens, dq = torch.tensor(lens, dtype=torch.int32, device=dev), q[1:].contiguous().to(dev)

    def buffers():
        return ([torch.full((64, 16, 128), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(3)],
                saw.allocate_prefix_workspace(1, 16, 64, 1100, dev), saw.allocate_prefix_workspace(1, 16, 64, 1100, dev),
                saw.allocate_mass_workspace(1, 16, 64, own.shape[1], dev), torch.from_numpy(mass.copy()).to(dev))

    def run(b, stream=None):
        out, ws, ws2, wm, dm = b
        saw.saw_paged_decode_attn_prefix(dq, kv, sc, prefix, 1100, own, dlens, out[0], ws, stream=stream)
        saw.saw_paged_decode_attn_prefix(dq, kv, sc, prefix, 40, own, dlens, out[1], ws2, stream=stream)
        saw.saw_paged_decode_attn_mass(dq, kv, sc, dm, own, dlens, out[2], wm, stream=stream)

    want = buffers()
    run(want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[buffers() for _ in range(8)] for _ in streams]
    torch.cuda.synchronize()
    for k in range(8):
        for st, b in zip(streams, got):
            run(b[k], st)
    torch.cuda.synchronize()
    for b in got[0] + got[1]:
        for x, y in zip(b[0], want[0]):
            assert torch.equal(x, y)
        assert torch.equal(b[4], want[4])


def test_two_graphs_share_a_workspace(cuda_device):
    """Two captured calls of different sizes over one workspace, replayed in turn on one stream."""
    from bit_paged_kv_block_b200 import saw
    dev = cuda_device
    lens = [300, 17, 0, 64, 1000]
    wl, pages, scales, q, mass = _case(lens, 8, 2, 128, seed=92)
    kv, sc = device_cache_from(pages, scales, dev)
    table = torch.from_numpy(wl.block_table).to(dev)
    dlens, dq = torch.tensor(lens, dtype=torch.int32, device=dev), q.to(dev)
    ws = saw.allocate_mass_workspace(2, 8, 5, table.shape[1], dev)
    wp = saw.allocate_prefix_workspace(2, 8, 5, 600, dev)
    dm0 = torch.from_numpy(mass.copy()).to(dev)     # outlives both graphs
    jobs = []
    for n, prefix in ((5, 600), (2, 33)):
        out = [torch.empty(n, 8, 128, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        dm = torch.from_numpy(mass.copy()).to(dev)
        args = dq[:n].contiguous(), table[:n].contiguous(), dlens[:n].contiguous()

        def call(out=out, dm=dm, args=args, prefix=prefix):
            dm.copy_(dm0)
            saw.saw_paged_decode_attn_mass(args[0], kv, sc, dm, args[1], args[2], out[0], ws)
            saw.saw_paged_decode_attn_prefix(args[0], kv, sc, table[4], prefix, args[1], args[2], out[1], wp)
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in (*out, dm)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        jobs.append((graph, (*out, dm), want))
    for _ in range(3):
        for graph, got, _ in jobs:
            for t in got:
                t.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        for _, got, want in jobs:
            for x, y in zip(got, want):
                same = torch.equal(x, y)
                assert same
    for graph, _, _ in jobs:
        graph.reset()


@pytest.mark.parametrize("bits", [0x7E00, 0x7C00, 0xFBFF])
def test_slots_past_the_ends_are_never_read_into_results(cuda_device, bits):
    """NaN, infinite and largest scales and zeros behind a sequence's last token (and a prefix's): the same
    bits as with zeros there, and no mass for them."""
    from bit_paged_kv_block_b200 import saw
    dev = cuda_device
    for hq, hkv, d, first in ((16, 1, 128, 1101), (8, 2, 128, 37), (6, 2, 64, 21), (12, 1, 256, 40)):
        lens = [first] + [(17 * s) % 90 for s in range(64 if first == 1101 else 9)]
        wl, pages, scales, q, mass = _case(lens, hq, hkv, d, seed=first)
        table = torch.from_numpy(wl.block_table).to(dev)
        dlens, dq = torch.tensor(lens, dtype=torch.int32, device=dev), q.to(dev)
        S = len(lens) - 1
        results = []
        for fill in (0, bits):
            sc_np, code = scales.copy().view(np.uint16), pages.copy()
            for s, n in enumerate(lens):
                for t in range(n, (n + 15) // 16 * 16):
                    sc_np[wl.block_table[s, t // 16], :, :, t % 16] = fill
                    code[wl.block_table[s, t // 16], :, :, t % 16] = 0xFF if fill else 0
            kv, sc = device_cache_from(code, sc_np.view(scales.dtype), dev)
            out = [torch.empty(S + 1, hq, d, dtype=torch.bfloat16, device=dev),
                   torch.empty(S, hq, d, dtype=torch.bfloat16, device=dev)]
            dm = torch.from_numpy(mass.copy()).to(dev)
            saw.saw_paged_decode_attn_mass(dq, kv, sc, dm, table, dlens, out[0],
                                           saw.allocate_mass_workspace(hkv, hq, S + 1, table.shape[1], dev, head_dim=d))
            saw.saw_paged_decode_attn_prefix(dq[1:].contiguous(), kv, sc, table[0].contiguous(), first,
                                             table[1:].contiguous(), dlens[1:].contiguous(), out[1],
                                             saw.allocate_prefix_workspace(hkv, hq, S, first, dev, head_dim=d))
            torch.cuda.synchronize()
            results.append((*out, dm))
        for x, y in zip(*results):
            same, finite = torch.equal(x, y), bool(torch.isfinite(y.float()).all())
            assert same and finite, f"{hq}/{hkv}/{d}"


def test_a_refused_batch_leaves_the_next_call_alone(cuda_device):
    """More sequences than the plan's tables hold in shared memory: an error, and the next call is right."""
    from bit_paged_kv_block_b200 import saw
    for allocate in (lambda n: saw.allocate_mass_workspace(1, 2, n, 1, cuda_device),
                     lambda n: saw.allocate_prefix_workspace(1, 2, n, 16, cuda_device)):
        with pytest.raises(saw.SawError):
            allocate(20000)
        wl, pages, scales, q, mass = _case([20, 5], 2, 1, 128, seed=93)
        out, got = _decode(saw, cuda_device, wl, pages, scales, q, mass, [20, 5])
        parts = [[(wl.block_table[s], n)] for s, n in enumerate([20, 5])]
        want, weights, terms = serving.decode_rows_fp64(u16(q), pages, scales, parts)
        assert_bf16_close(out, want, "after a refusal")
        _assert_mass(got, mass, wl, [20, 5], weights, terms, 128)
        table = torch.zeros(8, 64, device=cuda_device)
        saw.saw_rope_table(table, saw.rope_scaling())
        assert bool((table[0, :32] == 1).all())
