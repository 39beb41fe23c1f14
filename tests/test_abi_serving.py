"""Host-side checks of the serving operators' entry points: bad arguments are refused with their status
before any CUDA call, and the binding refuses wrong tensors (no GPU needed)."""
import ctypes

import pytest
import torch

from bit_paged_kv_block_b200 import saw

P = ctypes.c_void_p
INVALID, UNSUPPORTED, OK = saw.SAW_ERR_INVALID_ARGUMENT, saw.SAW_ERR_UNSUPPORTED, saw.SAW_OK


def _desc(hkv=8, d=128, p=16, pages=64):
    return saw.saw_cache_desc(hkv, d, p, pages)


def _table(kind="none", rotary=128, count=16, first=0, table=16, **kw):
    sc = saw.rope_scaling(kind, **kw)
    return saw.lib.saw_rope_table(P(table), first, count, rotary, ctypes.byref(sc), None)


def test_rope_table_checks():
    assert _table(rotary=0) == INVALID
    assert _table(rotary=24) == UNSUPPORTED                    # not a multiple of 16
    assert _table(rotary=272) == UNSUPPORTED
    assert _table(first=-1) == INVALID
    assert _table(count=-1) == INVALID
    assert _table(first=1 << 31, count=1) == INVALID
    assert _table(table=0) == INVALID
    assert _table(table=8) == INVALID                          # misaligned
    assert _table(base=1.0) == INVALID
    assert _table(base=float("nan")) == INVALID
    assert _table("linear", factor=0.5) == INVALID
    assert _table("ntk", factor=float("inf")) == INVALID
    assert _table("banded", low=4.0, high=4.0) == INVALID
    assert _table("banded", original_positions=0) == INVALID
    assert _table("yarn", fast=0.0) == INVALID
    assert _table(amplitude=-1.0) == INVALID
    assert saw.lib.saw_rope_table(P(16), 0, 4, 16, None, None) == INVALID
    bad = saw.rope_scaling()
    bad.kind = 9
    assert saw.lib.saw_rope_table(P(16), 0, 4, 16, ctypes.byref(bad), None) == INVALID
    assert _table(count=0, table=0) == OK                      # nothing to do
    with pytest.raises(ValueError):
        saw.rope_scaling("quadratic")


def _rope(table=16, positions=100, rotary=128, interleaved=0):
    return saw.saw_rope(table, positions, rotary, interleaved)


def _append(desc=None, rope=None, hq=32, q=16, qs=0, k=16, ks=0, v=16, vs=0, pos=16, slots=16, T=4,
            q_out=32, pages=16, scales=16, mass=0):
    return saw.lib.saw_rope_rotate_quantize_paged(
        ctypes.byref(desc or _desc()), None if rope == 0 else ctypes.byref(rope or _rope()), hq, P(q), qs,
        P(k), ks, P(v), vs, P(pos), P(slots), T, P(q_out), P(pages), P(scales), P(mass), None, None)


def test_rope_append_checks():
    assert _append(rope=0) == INVALID
    assert _append(_desc(d=96)) == UNSUPPORTED
    assert _append(rope=_rope(rotary=40)) == UNSUPPORTED
    assert _append(_desc(d=64), _rope(rotary=128)) == UNSUPPORTED      # more than the head
    assert _append(rope=_rope(interleaved=2)) == INVALID
    assert _append(rope=_rope(table=0)) == INVALID
    assert _append(rope=_rope(table=4)) == INVALID
    assert _append(rope=_rope(positions=0)) == INVALID
    assert _append(rope=_rope(positions=-1)) == INVALID
    assert _append(hq=-1) == INVALID
    assert _append(q=0) == INVALID
    assert _append(q=8) == INVALID
    assert _append(q_out=0) == INVALID
    assert _append(q_out=8) == INVALID
    assert _append(k=0) == INVALID
    assert _append(pos=0) == INVALID
    assert _append(pos=4) == INVALID
    assert _append(slots=0) == INVALID
    assert _append(mass=8) == INVALID
    assert _append(T=-1) == INVALID
    assert _append(qs=32 * 128 - 8) == INVALID                         # less than a token's rows
    assert _append(ks=8 * 128 + 4) == INVALID                          # not a multiple of 8
    assert _append(vs=-8) == INVALID
    assert _append(_desc(hkv=3), ks=1024, vs=1024) == UNSUPPORTED      # strided, 3 kv heads
    assert _append(q=16, q_out=16, qs=8192) == INVALID                 # in place on strided rows
    assert _append(T=1 << 40) == UNSUPPORTED
    assert _append(T=0, q=0, k=0, v=0, pos=0, slots=0, q_out=0, pages=0, scales=0) == OK


def _prefix(desc=None, hq=32, S=2, q=16, table=16, prefix=40, bt=16, lens=16, out=32, ws=256, ws_bytes=16,
            max_blocks=4, sm_scale=0.1):
    return saw.lib.saw_paged_decode_attn_prefix(
        ctypes.byref(desc or _desc()), hq, P(q), P(16), P(16), P(table), prefix, P(bt), max_blocks, P(lens),
        S, sm_scale, P(out), P(ws), ws_bytes, None, None)


def _mass(desc=None, hq=32, S=2, q=16, mass=16, bt=16, lens=16, out=32, ws=256, ws_bytes=16, max_blocks=4,
          sm_scale=0.1):
    return saw.lib.saw_paged_decode_attn_mass(
        ctypes.byref(desc or _desc()), hq, P(q), P(16), P(16), P(mass), P(bt), max_blocks, P(lens), S,
        sm_scale, P(out), P(ws), ws_bytes, None, None)


@pytest.mark.parametrize("call", [_prefix, _mass])
def test_bf16_decode_checks(call):
    assert call(_desc(d=96)) == UNSUPPORTED
    assert call(_desc(p=8)) == UNSUPPORTED
    assert call(_desc(pages=0)) == INVALID
    assert call(hq=12) == INVALID                                      # Hq % Hkv
    assert call(hq=136) == UNSUPPORTED                                 # G = 17
    assert call(hq=0) == INVALID
    assert call(S=-1) == INVALID
    assert call(q=0) == INVALID
    assert call(q=8) == INVALID
    assert call(out=8) == INVALID
    assert call(out=16) == INVALID                                     # out is q
    assert call(bt=2) == INVALID
    assert call(lens=0) == INVALID
    assert call(max_blocks=0) == INVALID
    assert call(max_blocks=1 << 28) == INVALID                         # 2^32 tokens
    assert call(sm_scale=float("nan")) == INVALID
    assert call(S=1 << 26) == UNSUPPORTED                              # 2^31 query rows
    assert call(S=0, q=0, out=0) == OK


def test_prefix_and_mass_checks():
    assert _prefix(prefix=-1) == INVALID
    assert _prefix(prefix=2 ** 31 - 1) == INVALID
    assert _prefix(prefix=2 ** 30 + 1) == INVALID
    assert _prefix(table=0) == INVALID
    assert _prefix(table=2) == INVALID
    assert _mass(mass=0) == INVALID
    assert _mass(mass=4) == INVALID
    f, g = saw.lib.saw_paged_decode_prefix_workspace_bytes, saw.lib.saw_paged_decode_mass_workspace_bytes
    d = _desc()
    for call in (lambda hq, s: f(ctypes.byref(d), hq, s, 100), lambda hq, s: g(ctypes.byref(d), hq, s, 4)):
        assert call(12, 4) == 0 and call(136, 4) == 0 and call(32, -1) == 0
    assert f(ctypes.byref(d), 32, 4, -1) == 0
    assert f(ctypes.byref(d), 32, 4, 2 ** 30 + 1) == 0
    assert g(ctypes.byref(d), 32, 4, 0) == 0


def _evict(desc=None, pages=16, mass=16, bt=16, max_blocks=4, lens=16, S=2, new=16, new_blocks=2, new_lens=32,
           kept=16, keep=20, sink=2, recent=4):
    return saw.lib.saw_evict_paged(
        ctypes.byref(desc or _desc()), P(pages), P(16), P(mass), P(bt), max_blocks, P(lens), S, P(new),
        new_blocks, P(new_lens), P(kept), keep, sink, recent, None, None)


def test_evict_checks():
    assert _evict(_desc(d=32)) == UNSUPPORTED
    assert _evict(_desc(pages=0)) == INVALID
    assert _evict(S=-1) == INVALID
    assert _evict(keep=0) == INVALID
    assert _evict(sink=-1) == INVALID
    assert _evict(recent=-1) == INVALID
    assert _evict(sink=10, recent=11) == INVALID                       # more than keep
    assert _evict(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == INVALID     # the sum passes 32 bits
    assert _evict(pages=0) == INVALID
    assert _evict(mass=0) == INVALID
    assert _evict(mass=8) == INVALID
    assert _evict(new=0) == INVALID
    assert _evict(new_blocks=0) == INVALID
    assert _evict(new_lens=16) == INVALID                              # new_lens is seq_lens
    assert _evict(kept=2) == INVALID
    assert _evict(S=2 ** 30) == UNSUPPORTED
    assert _evict(keep=2 ** 30 + 1) == UNSUPPORTED
    assert _evict(max_blocks=2 ** 26 + 1) == INVALID                   # past 2^30 tokens
    assert _evict(S=0, pages=0) == OK


def test_steps_check_both_halves():
    d, r = _desc(), _rope()

    def call(fn, q=16, q_rot=32, out=48, extra=()):
        return fn(ctypes.byref(d), ctypes.byref(r), 32, P(q), P(16), P(16), P(16), P(16), P(q_rot), P(16), P(16),
                  *extra, P(16), 4, P(16), 2, 0.1, P(out), P(256), 16, None, None)
    assert call(saw.lib.saw_decode_step_rope, q=0) == INVALID
    assert call(saw.lib.saw_decode_step_rope, q_rot=8) == INVALID
    assert call(saw.lib.saw_decode_step_rope, out=0) == INVALID
    assert call(saw.lib.saw_decode_step_rope_mass, q=0, extra=(P(16),)) == INVALID
    assert call(saw.lib.saw_decode_step_rope_mass, extra=(P(0),)) == INVALID     # needs the masses
    assert call(saw.lib.saw_decode_step_rope_mass, out=8, extra=(P(16),)) == INVALID
    assert call(saw.lib.saw_decode_step_rope_mass, out=32, extra=(P(16),)) == INVALID    # out is q_rot


def test_status_bits_and_strings():
    bits = [saw.SAW_DEV_BAD_SLOT, saw.SAW_DEV_BAD_PAGE, saw.SAW_DEV_BAD_SEQ_LEN, saw.SAW_DEV_WAIT_TIMEOUT,
            saw.SAW_DEV_RANGE, saw.SAW_DEV_BAD_POSITION]
    assert bits == [1 << i for i in range(6)]


def test_binding_rejects_wrong_tensors():
    kv = torch.zeros(4, 2, 2, 16, 64, dtype=torch.uint8)
    sc = torch.zeros(4, 2, 2, 16, 2, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                    # CPU tensors
        saw.saw_paged_decode_attn_prefix(q, kv, sc, i32(1), 16, i32(3, 1), i32(3), q, kv.view(-1))
    with pytest.raises(TypeError):
        saw.saw_paged_decode_attn_mass(q, kv, sc, None, i32(3, 1), i32(3), q, kv.view(-1))
    with pytest.raises(TypeError):
        saw.saw_evict_paged(kv, sc, None, i32(3, 1), i32(3), i32(3, 1), i32(3), i32(3, 2, 8))
    with pytest.raises(ValueError):
        saw.saw_rope_table(torch.zeros(4, 32), saw.rope_scaling())
    with pytest.raises(TypeError):
        saw.saw_rope_table(torch.zeros(4, 32, dtype=torch.float64), saw.rope_scaling())
