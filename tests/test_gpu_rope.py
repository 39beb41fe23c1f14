"""Rotary positions at the append on the GPU against the oracle.  The table agrees with fp64 within
the error of one fp32 angle and the cosine of it; q, the codes, the scales and the cleared masses are
bit-exact, since every step of the append is one IEEE operation."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving
from bit_paged_kv_block_b200 import synth
from helpers import CANARY_CODE, CANARY_SCALE, NTHREADS, u16

pytestmark = pytest.mark.gpu

SCALINGS = [dict(kind="none", base=10000.0), dict(kind="linear", base=10000.0, factor=4.0),
            dict(kind="ntk", base=10000.0, factor=8.0),
            dict(kind="banded", base=500000.0, factor=8.0, original=8192),
            dict(kind="yarn", base=10000.0, factor=32.0, original=4096),
            dict(kind="linear", base=10000.0, factor=2.0, amplitude=1.5)]


def _scaling(saw, sc):
    sc = dict(sc)
    if "original" in sc:
        sc["original_positions"] = sc.pop("original")
    return saw.rope_scaling(**sc)


def _table_tolerance(sc):
    """An entry is a cosine and sine turned by another angle's.  Each angle in turns is rounded to fp32 once
    (at most half a turn: 2^-26 turns, 9.4e-8 rad), and the two errors add: 1.9e-7.  sincospif is within
    2 ulp (2^-23 at most, 1.2e-7) of each component; of a pair of components that enter with the other
    angle's cosine and sine, at most sqrt(2) times that: 1.7e-7 for either angle.  The amplitude and its
    product are rounded once each (2^-24, on two components: 1.7e-7 in all), and so are one product and the
    sum (2^-25 each): 1.9e-7 + 3.4e-7 + 1.7e-7 + 6e-8 < 7.7e-7, times the amplitude."""
    amp = sc.get("amplitude") or (0.1 * np.log(sc["factor"]) + 1 if sc["kind"] == "yarn" else 1.0)
    return 7.7e-7 * amp


@pytest.mark.parametrize("sc", SCALINGS, ids=lambda s: s["kind"])
@pytest.mark.parametrize("rotary", [16, 48, 64, 128, 256])
def test_table_matches_fp64(cuda_device, sc, rotary):
    from bit_paged_kv_block_b200 import saw
    for first, count in ((0, 1), (0, 777), (1_000_000, 130), (5, 20_011)):
        table = torch.full((count + 1, rotary), 7.0, device=cuda_device)
        saw.saw_rope_table(table[:count], _scaling(saw, sc), first_position=first)
        torch.cuda.synchronize()
        want = serving.rope_table_fp64(first, count, rotary, **sc)
        got = table.cpu().double().numpy()
        assert np.abs(got[:count] - want).max() <= _table_tolerance(sc)
        assert (got[count] == 7.0).all()       # the row behind the last


def _inputs(T, hq, hkv, d, seed, positions=1000, rotary=None):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(T, hq, d, generator=g).to(torch.bfloat16)
    k = torch.randn(T, hkv, d, generator=g)
    k[..., 5] *= 25.0
    k, v = k.to(torch.bfloat16), torch.randn(T, hkv, d, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, positions, (T,), generator=g)
    pages = (T + 15) // 16 + 2
    slots = torch.randperm(pages * 16, generator=g)[:T]
    table = torch.from_numpy(serving.rope_table_fp64(0, positions, rotary or d)).float()
    return q, k, v, pos, slots, table, pages


def _canary(pages, hkv, d):
    kv = np.full((pages, hkv, 2, 16, d // 2), CANARY_CODE, np.uint8)
    sc = np.full((pages, hkv, 2, 16, 2), CANARY_SCALE, np.uint16)
    mass = np.full((pages, hkv, 16), 3.0, np.float32)
    return kv, sc, mass


def _dev(kv, sc, mass, device):
    return (torch.from_numpy(kv.copy()).to(device),
            torch.from_numpy(sc.copy().view(np.int16)).view(torch.float16).to(device),
            torch.from_numpy(mass.copy()).to(device))


def _expect(q, k, v, pos, slots, table, kv, sc, mass, interleaved, rotate, skip=()):
    """The oracle's append in place; returns q_out bits (NaN bits where a token is skipped)."""
    slots = slots.numpy().copy()
    safe = pos.numpy().copy()
    safe[list(skip)] = 0
    slots[list(skip)] = -1
    kr = serving.rope_bf16(synth.bf16_bits(k), safe, table.numpy(), interleaved)
    qr = serving.rope_bf16(synth.bf16_bits(q), safe, table.numpy(), interleaved)
    qr[slots < 0] = 0x7FC0
    assert oracle.rotate_quantize_paged(kr, synth.bf16_bits(v), slots, kv, sc, rotate=rotate,
                                        nthreads=NTHREADS) == 0
    for s in slots[slots >= 0]:
        mass[s // 16, :, s % 16] = 0.0
    return qr


def _check(saw, device, case, interleaved, rotate, q=None, k=None, v=None, skip=(), status_bits=0):
    qc, kc, vc, pos, slots, table, pages = case
    kv, sc, mass = _canary(pages, kc.shape[1], kc.shape[2])
    dkv, dsc, dmass = _dev(kv, sc, mass, device)
    want_q = _expect(qc, kc, vc, pos, slots, table, kv, sc, mass, interleaved, rotate, skip)
    q = qc.to(device) if q is None else q
    q_out = torch.full(qc.shape, float("nan"), dtype=torch.bfloat16, device=device)
    status = torch.zeros(1, dtype=torch.int32, device=device)
    saw.saw_rope_rotate_quantize_paged(
        q, kc.to(device) if k is None else k, vc.to(device) if v is None else v, pos.to(device),
        slots.to(device), (table.to(device), interleaved), q_out, dkv, dsc, mass=dmass,
        dev_status=status, rotate=rotate)
    torch.cuda.synchronize()
    assert int(status.item()) == status_bits
    for name, a, b in (("q", u16(q_out), want_q), ("codes", dkv.cpu().numpy(), kv),
                       ("scales", u16(dsc), sc), ("masses", dmass.cpu().numpy(), mass)):
        same = np.array_equal(a, b)
        assert same, f"{name}: {int((a != b).sum())} of {a.size} differ, first at {np.argwhere(a != b)[0]}"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112),
                                      (256, 256), (256, 64), (256, 160)])
def test_append_bit_exact(cuda_device, d, rotary, interleaved):
    """Each head dimension with the whole head, a small and an odd part of it rotated; 37 tokens x 3
    kv heads (ragged tiles), 7 query heads per kv head (an odd last pass)."""
    from bit_paged_kv_block_b200 import saw
    case = _inputs(37, 21, 3, d, seed=d + rotary, rotary=rotary)
    _check(saw, cuda_device, case, interleaved, rotate=True)


@pytest.mark.parametrize("T,hq,hkv,rotate", [(1, 8, 1, True), (1, 4, 4, False), (16, 8, 8, True),
                                             (333, 16, 2, False), (5000, 8, 2, True)])
def test_append_sizes(cuda_device, T, hq, hkv, rotate):
    """One token; whole tiles; enough tokens for several tiles per warp and one warp per token."""
    from bit_paged_kv_block_b200 import saw
    _check(saw, cuda_device, _inputs(T, hq, hkv, 128, seed=T), False, rotate)


@pytest.mark.parametrize("d,hkv", [(64, 4), (64, 16), (128, 2), (128, 8), (256, 1), (256, 4)])
def test_append_fused_projection_slices(cuda_device, d, hkv):
    """q, k and v as slices of one [T][(Hq + 2 Hkv) D] projection output."""
    from bit_paged_kv_block_b200 import saw
    case = _inputs(45, 2 * hkv, hkv, d, seed=d * hkv, rotary=d // 2)
    fused = torch.cat(case[:3], 1).to(cuda_device)
    _check(saw, cuda_device, case, True, True, q=fused[:, :2 * hkv], k=fused[:, 2 * hkv:3 * hkv],
           v=fused[:, 3 * hkv:])


def test_append_in_place_and_keys_alone(cuda_device):
    """q_out may be q; without q the keys are rotated and appended alone."""
    from bit_paged_kv_block_b200 import saw
    q, k, v, pos, slots, table, pages = _inputs(50, 8, 2, 128, seed=3)
    kv, sc, mass = _canary(pages, 2, 128)
    dkv, dsc, dmass = _dev(kv, sc, mass, cuda_device)
    want = _expect(q, k, v, pos, slots, table, kv, sc, mass, False, True)
    dev = lambda t: t.to(cuda_device)
    dq = dev(q)
    saw.saw_rope_rotate_quantize_paged(dq, dev(k), dev(v), dev(pos), dev(slots), (dev(table), False),
                                       dq, dkv, dsc, mass=dmass)
    assert np.array_equal(u16(dq), want)
    assert np.array_equal(dkv.cpu().numpy(), kv) and np.array_equal(dmass.cpu().numpy(), mass)
    kv2, sc2, mass2 = _dev(*_canary(pages, 2, 128), cuda_device)
    saw.saw_rope_rotate_quantize_paged(None, dev(k), dev(v), dev(pos), dev(slots),
                                       (dev(table), False), None, kv2, sc2)
    assert torch.equal(kv2, dkv) and np.array_equal(u16(sc2), u16(dsc))
    assert bool((mass2 == 3.0).all())


def test_append_equals_rotating_first(cuda_device):
    """The cache holds the bits that appending the already rotated keys gives."""
    from bit_paged_kv_block_b200 import saw
    q, k, v, pos, slots, table, pages = _inputs(200, 4, 4, 128, seed=8)
    dev = lambda t: t.to(cuda_device)
    kv, sc, _ = _dev(*_canary(pages, 4, 128), cuda_device)
    kv2, sc2, _ = _dev(*_canary(pages, 4, 128), cuda_device)
    k_rot = torch.empty_like(dev(k))
    # rotate the keys as queries of a call that appends elsewhere
    saw.saw_rope_rotate_quantize_paged(dev(k), dev(k), dev(v), dev(pos), dev(slots),
                                       (dev(table), False), k_rot, kv, sc)
    saw.saw_rotate_quantize_paged(k_rot, dev(v), dev(slots), kv2, sc2)
    assert torch.equal(kv, kv2) and np.array_equal(u16(sc), u16(sc2))


def test_append_skips_padding_and_flags_bad_tokens(cuda_device):
    """Padding (negative slots, whatever their position), positions past the table and slots past
    the cache: the token is skipped as a whole, the others are written."""
    from bit_paged_kv_block_b200 import saw
    case = list(_inputs(40, 8, 2, 128, seed=11))
    pos, slots, pages = case[3].clone(), case[4].clone(), case[6]
    slots[37:] = -1
    pos[38] = 1 << 40
    pos[39] = -5
    case[3], case[4] = pos, slots
    _check(saw, cuda_device, case, False, True, skip=(38, 39))
    pos, slots = pos.clone(), slots.clone()
    pos[3], pos[17], slots[20], slots[0] = 1000, -1, pages * 16, 1 << 45
    case[3], case[4] = pos, slots
    _check(saw, cuda_device, case, True, True, skip=(0, 3, 17, 20, 38, 39),
           status_bits=saw.SAW_DEV_BAD_SLOT | saw.SAW_DEV_BAD_POSITION)


def test_append_no_tokens_and_other_stream(cuda_device):
    from bit_paged_kv_block_b200 import saw
    q, k, v, pos, slots, table, pages = _inputs(64, 8, 2, 128, seed=13)
    dev = lambda t: t.to(cuda_device)
    kv, sc, mass = _canary(pages, 2, 128)
    dkv, dsc, dmass = _dev(kv, sc, mass, cuda_device)
    a = [dev(t) for t in (q, k, v, pos, slots)]
    q_out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=cuda_device)
    rope = (dev(table), False)
    saw.saw_rope_rotate_quantize_paged(*[t[:0] for t in a], rope, q_out[:0], dkv, dsc, mass=dmass)
    torch.cuda.synchronize()
    assert np.array_equal(dkv.cpu().numpy(), kv)
    want = _expect(q, k, v, pos, slots, table, kv, sc, mass, False, True)
    stream = torch.cuda.Stream()
    saw.saw_rope_rotate_quantize_paged(*a, rope, q_out, dkv, dsc, mass=dmass, stream=stream)
    stream.synchronize()
    assert np.array_equal(u16(q_out), want) and np.array_equal(dkv.cpu().numpy(), kv)
