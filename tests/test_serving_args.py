"""CPU checks of qk_norm_rope, append_paged and decode_paged_q8: refusals of the binding and of the
C ABI (both come before anything touches a GPU), and the append's page arithmetic compiled for the host."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import serving_oracle as R
from trainable_gated_block_b200 import build, sas

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)       # not 16-byte aligned


@pytest.fixture(scope="module")
def L():
    build.build()
    return sas.lib()


def _with(args, changes):
    a = list(args)
    for i, v in changes.items():
        a[i] = v
    return a


#          dtype          q     ld_q k     ld_k wq    wk    table max  pos  S   T    Hq Hkv D   eps   q_out k_out stream
NR = [sas.SAS_BF16, FAKE, 512, FAKE, 256, FAKE, FAKE, FAKE, 64, None, 64, 128, 4, 2, 128, 1e-6, FAKE, FAKE, None]


@pytest.mark.parametrize("changes,code", [
    ({0: 5}, sas.SAS_ERR_INVALID_ARG), ({1: None}, sas.SAS_ERR_INVALID_ARG), ({1: ODD}, sas.SAS_ERR_INVALID_ARG),
    ({2: 511}, sas.SAS_ERR_INVALID_ARG), ({2: 516}, sas.SAS_ERR_INVALID_ARG), ({4: 0}, sas.SAS_ERR_INVALID_ARG),
    ({5: None}, sas.SAS_ERR_INVALID_ARG), ({6: ODD}, sas.SAS_ERR_INVALID_ARG), ({7: None}, sas.SAS_ERR_INVALID_ARG),
    ({8: 0}, sas.SAS_ERR_INVALID_ARG), ({10: 0}, sas.SAS_ERR_INVALID_ARG), ({11: -1}, sas.SAS_ERR_INVALID_ARG),
    ({11: 1 << 30}, sas.SAS_ERR_UNSUPPORTED), ({12: 0}, sas.SAS_ERR_INVALID_ARG), ({14: 96}, sas.SAS_ERR_UNSUPPORTED),
    ({15: 0.0}, sas.SAS_ERR_INVALID_ARG), ({15: float("nan")}, sas.SAS_ERR_INVALID_ARG),
    ({16: None}, sas.SAS_ERR_INVALID_ARG), ({17: ODD}, sas.SAS_ERR_INVALID_ARG), ({11: 0}, sas.SAS_OK)])
def test_norm_rope_refusals(L, changes, code):
    assert L.sas_qk_norm_rope(*_with(NR, changes)) == code
    assert bool(L.sas_last_error()) == (code != sas.SAS_OK)


@pytest.mark.parametrize("changes,code", [
    ({0: None}, sas.SAS_ERR_INVALID_ARG), ({1: ODD}, sas.SAS_ERR_INVALID_ARG), ({17: None}, sas.SAS_ERR_INVALID_ARG),
    ({19: None}, sas.SAS_ERR_INVALID_ARG), ({20: None}, sas.SAS_ERR_INVALID_ARG), ({21: None}, sas.SAS_ERR_INVALID_ARG),
    ({21: ctypes.c_void_p(0x10010)}, sas.SAS_ERR_INVALID_ARG), ({22: 16}, sas.SAS_ERR_INVALID_ARG),
    ({6: None, 7: None}, sas.SAS_ERR_INVALID_ARG)])          # weight gradients without weights
def test_norm_rope_bwd_refusals(L, changes, code):
    args = [FAKE, FAKE] + NR[1:16] + [FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None]
    assert len(args) == 24
    assert L.sas_qk_norm_rope_bwd(sas.SAS_BF16, *_with(args, changes)) == code


#          q  ld   k     ld   v     ld   wq    wk    table max cu  N  new T  kv    ptab  maxp P  Hq Hkv D  psz eps  qo    ko    kc    vc   pool st
AP = [FAKE, 512, FAKE, 256, FAKE, 256, FAKE, FAKE, FAKE, 64, None, 3, 1, 3, FAKE, FAKE, 4, 9, 4, 2, 128, 64, 1e-6,
      FAKE, None, FAKE, FAKE, None, None]


@pytest.mark.parametrize("changes,code", [
    ({0: None}, sas.SAS_ERR_INVALID_ARG), ({1: 500}, sas.SAS_ERR_INVALID_ARG), ({2: None}, sas.SAS_ERR_INVALID_ARG),
    ({4: ODD}, sas.SAS_ERR_INVALID_ARG), ({7: None}, sas.SAS_ERR_INVALID_ARG), ({8: ODD}, sas.SAS_ERR_INVALID_ARG),
    ({9: 0}, sas.SAS_ERR_INVALID_ARG), ({11: 2}, sas.SAS_ERR_INVALID_ARG), ({12: 2}, sas.SAS_ERR_INVALID_ARG),
    ({12: 0, 10: FAKE}, sas.SAS_ERR_INVALID_ARG), ({13: -1, 10: FAKE}, sas.SAS_ERR_INVALID_ARG),
    ({14: None}, sas.SAS_ERR_INVALID_ARG), ({15: None}, sas.SAS_ERR_INVALID_ARG), ({16: 0}, sas.SAS_ERR_INVALID_ARG),
    ({17: 0}, sas.SAS_ERR_INVALID_ARG), ({20: 96}, sas.SAS_ERR_UNSUPPORTED), ({21: 32}, sas.SAS_ERR_UNSUPPORTED),
    ({22: -1.0}, sas.SAS_ERR_INVALID_ARG), ({23: None}, sas.SAS_ERR_INVALID_ARG), ({24: ODD}, sas.SAS_ERR_INVALID_ARG),
    ({25: None}, sas.SAS_ERR_INVALID_ARG), ({27: ODD}, sas.SAS_ERR_INVALID_ARG),
    ({10: FAKE, 13: 1 << 30}, sas.SAS_ERR_UNSUPPORTED), ({10: FAKE, 12: (1 << 30) + 1}, sas.SAS_ERR_UNSUPPORTED),
    ({10: FAKE, 11: 1 << 28}, sas.SAS_ERR_UNSUPPORTED),
    ({11: 0, 13: 0}, sas.SAS_OK), ({10: FAKE, 13: 0}, sas.SAS_OK)])
def test_append_refusals(L, changes, code):
    assert L.sas_append_paged(*_with(AP, changes)) == code
    q8 = _with(AP, changes)
    assert L.sas_append_paged_q8(*q8[:27], FAKE, FAKE, *q8[27:]) == code


def test_append_q8_needs_scales(L):
    assert L.sas_append_paged_q8(*AP[:27], None, FAKE, *AP[27:]) == sas.SAS_ERR_INVALID_ARG
    assert L.sas_append_paged_q8(*AP[:27], FAKE, None, *AP[27:]) == sas.SAS_ERR_INVALID_ARG


#      q     kc    vc    ks    vs    P  ptab maxp kv   N  Hq Hkv D    psz K  idx   cnt   gate  sm   o     lse   ws    bytes    st
DQ = [FAKE, FAKE, FAKE, FAKE, FAKE, 9, FAKE, 4, FAKE, 3, 8, 2, 128, 64, 2, FAKE, FAKE, FAKE, 0.1, FAKE, FAKE, FAKE, 1 << 30, None]


@pytest.mark.parametrize("changes,code", [
    ({0: None}, sas.SAS_ERR_INVALID_ARG), ({1: ODD}, sas.SAS_ERR_INVALID_ARG), ({3: None}, sas.SAS_ERR_INVALID_ARG),
    ({4: None}, sas.SAS_ERR_INVALID_ARG), ({5: 0}, sas.SAS_ERR_INVALID_ARG), ({7: 0}, sas.SAS_ERR_INVALID_ARG),
    ({9: 0}, sas.SAS_ERR_INVALID_ARG), ({10: 7}, sas.SAS_ERR_INVALID_ARG), ({10: 18}, sas.SAS_ERR_UNSUPPORTED),
    ({12: 64}, sas.SAS_ERR_UNSUPPORTED), ({13: 16}, sas.SAS_ERR_UNSUPPORTED), ({14: -1}, sas.SAS_ERR_INVALID_ARG),
    ({14: (1 << 24) + 1}, sas.SAS_ERR_UNSUPPORTED), ({15: None}, sas.SAS_ERR_INVALID_ARG),
    ({5: 1 << 25}, sas.SAS_ERR_UNSUPPORTED), ({18: float("inf")}, sas.SAS_ERR_INVALID_ARG),
    ({19: None}, sas.SAS_ERR_INVALID_ARG), ({21: None}, sas.SAS_ERR_INVALID_ARG),
    ({21: ctypes.c_void_p(0x10010)}, sas.SAS_ERR_INVALID_ARG), ({22: 8}, sas.SAS_ERR_INVALID_ARG)])
def test_decode_q8_refusals(L, changes, code):
    assert L.sas_decode_paged_q8(*_with(DQ, changes)) == code


def test_workspace_queries(L):
    assert L.sas_decode_q8_workspace_size(3, 8, 2, 128, 2) > 0
    assert L.sas_decode_q8_workspace_size(3, 8, 2, 64, 2) == 0
    assert L.sas_qk_norm_rope_bwd_workspace_size(0, 4, 2, 128) > 0
    assert L.sas_qk_norm_rope_bwd_workspace_size(10, 4, 2, 96) == 0
    assert L.sas_qk_norm_rope_bwd_workspace_size(-1, 4, 2, 128) == 0


# ------------------------------------------------------------------------------------------ the binding (CPU tensors)
def _nr(**kw):
    d = dict(q=torch.zeros((5, 4, 64)), k=torch.zeros((5, 2, 64)), table=torch.zeros((9, 64)),
             q_weight=torch.zeros(64), k_weight=torch.zeros(64))
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,err", [
    (dict(k=torch.zeros((4, 2, 64))), ValueError), (dict(k=torch.zeros((5, 2, 64), dtype=torch.bfloat16)), TypeError),
    (dict(table=torch.zeros((9, 32))), ValueError), (dict(table=torch.zeros((9, 64)).double()), TypeError),
    (dict(table=torch.zeros((4, 64))), ValueError), (dict(k_weight=None), ValueError),
    (dict(q_weight=torch.zeros(32)), ValueError), (dict(positions=torch.zeros(5, dtype=torch.int64)), TypeError),
    (dict(positions=torch.zeros(4, dtype=torch.int32)), ValueError),
    (dict(q=torch.zeros((5, 64, 4)).transpose(1, 2)), ValueError),
    (dict(q=torch.zeros((5, 4, 64), dtype=torch.float16), k=torch.zeros((5, 2, 64), dtype=torch.float16),
          q_weight=None, k_weight=None), TypeError),
    (dict(), ValueError)])                                     # CPU tensors
def test_norm_rope_binding_refuses(kw, err):
    with pytest.raises(err):
        sas.qk_norm_rope(**_nr(**kw))


def test_norm_rope_bwd_binding_refuses():
    a = _nr()
    with pytest.raises(ValueError):
        sas.qk_norm_rope_bwd(torch.zeros((5, 4, 32)), torch.zeros((5, 2, 64)), **a)
    with pytest.raises(ValueError):                            # upstream gradients must be contiguous
        sas.qk_norm_rope_bwd(torch.zeros((5, 8, 64))[:, :4], torch.zeros((5, 2, 64)), **a)


def _ap(q8, **kw):
    bf = torch.bfloat16
    dt = torch.float8_e4m3fn if q8 else bf
    d = dict(q=torch.zeros((3, 4, 64), dtype=bf), k=torch.zeros((3, 2, 64), dtype=bf), v=torch.zeros((3, 2, 64), dtype=bf),
             table=torch.zeros((9, 64)), k_cache=torch.zeros((5, 2, 64, 64), dtype=dt),
             v_cache=torch.zeros((5, 2, 64, 64), dtype=dt), page_table=torch.zeros((3, 2), dtype=torch.int32),
             kv_len=torch.ones(3, dtype=torch.int32))
    if q8:
        d.update(k_scale=torch.ones((5, 2)), v_scale=torch.ones((5, 2)))
    d.update(kw)
    return d


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,err", [
    (dict(v=torch.zeros((3, 2, 64))), TypeError), (dict(k=torch.zeros((4, 2, 64), dtype=torch.bfloat16)), ValueError),
    (dict(k_cache=torch.zeros((5, 2, 64, 64), dtype=torch.uint8)), TypeError),
    (dict(page_table=torch.zeros((2, 2), dtype=torch.int32)), ValueError),
    (dict(kv_len=torch.ones(3, dtype=torch.int64)), TypeError), (dict(cu_new=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(kpool=torch.zeros((5, 2, 32))), ValueError), (dict(q_weight=torch.zeros(64, dtype=torch.bfloat16)), ValueError),
    (dict(), ValueError)])
def test_append_binding_refuses(q8, kw, err):
    with pytest.raises(err):
        (sas.append_paged_q8 if q8 else sas.append_paged)(**_ap(q8, **kw))


@pytest.mark.parametrize("kw,err", [
    (dict(k_scale=torch.ones((5, 1))), ValueError), (dict(v_cache=torch.zeros((5, 2, 64, 128))), TypeError),
    (dict(idx=torch.zeros((3, 2, 2), dtype=torch.int64)), TypeError), (dict(cnt=torch.zeros((3, 1), dtype=torch.int32)), ValueError),
    (dict(), ValueError)])
def test_decode_q8_binding_refuses(kw, err):
    f8 = torch.float8_e4m3fn
    d = dict(q=torch.zeros((3, 8, 128), dtype=torch.bfloat16), k_cache=torch.zeros((5, 2, 64, 128), dtype=f8),
             v_cache=torch.zeros((5, 2, 64, 128), dtype=f8), k_scale=torch.ones((5, 2)), v_scale=torch.ones((5, 2)),
             page_table=torch.zeros((3, 2), dtype=torch.int32), kv_len=torch.ones(3, dtype=torch.int32),
             idx=torch.zeros((3, 2, 2), dtype=torch.int32), cnt=torch.zeros((3, 2), dtype=torch.int32),
             log_gate=torch.zeros((3, 2, 2)))
    d.update(kw)
    with pytest.raises(err):
        sas.decode_paged_q8(**d)


# ---------------------------------------------------------------------------------------- page arithmetic on the host
@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src = d / "rows.cpp"
    src.write_text('''#include "page_rows.h"
extern "C" int tiles(int has_cu, int lo, int hi, int n, long long T, int max_new, int kv, int max_pages, int max_pos,
                     long long* out) {
    sas::SeqNew s = sas::seq_new(has_cu != 0, lo, hi, n, T, max_new, kv, max_pages, max_pos);
    if (s.bad) return -1;
    int m = 0;
    for (int i = 0; i < sas::max_tiles(max_new); ++i) {
        sas::PageTile t = sas::page_tile(s, i);
        if (t.hi <= t.lo) continue;
        out[4 * m] = t.block; out[4 * m + 1] = t.lo; out[4 * m + 2] = t.hi; out[4 * m + 3] = t.row; ++m;
    }
    return m;
}
extern "C" unsigned base(int lo, int n) { return sas::seq_tile_base(lo, n); }
extern "C" int max_tiles(int n) { return sas::max_tiles(n); }
extern "C" int sexp(unsigned bits) { return sas::scale_exp(bits); }
extern "C" int ok(float s) { return sas::scale_ok(s); }
''')
    so = d / "rows.so"
    csrc = os.path.join(ROOT, "trainable_gated_block_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", csrc, str(src), "-o", str(so)],
                   check=True)
    h = ctypes.CDLL(str(so))
    h.tiles.argtypes = [ctypes.c_int] * 4 + [ctypes.c_longlong] + [ctypes.c_int] * 4 + [ctypes.c_void_p]
    h.ok.argtypes = [ctypes.c_float]
    return h


def _tiles(h, *a):
    out = np.zeros(4 * 4096, dtype=np.int64)
    m = h.tiles(*a, out.ctypes.data)
    return m if m < 0 else [tuple(r) for r in out[:4 * m].reshape(m, 4)]


@pytest.mark.parametrize("start", [0, 1, 63, 64, 65, 100])
@pytest.mark.parametrize("count", [1, 2, 63, 64, 65, 128, 200])
@pytest.mark.parametrize("slack", [0, 70])
def test_tiles_cover_each_new_row_once(rows, start, count, slack):
    got = _tiles(rows, 1, 10, 10 + count, 0, 10 + count, count + slack, start + count, 16, 1024)
    want = [(p // 64, p % 64, 10 + p - start) for p in range(start, start + count)]
    assert [(b, r, row + r - lo) for b, lo, hi, row in got for r in range(lo, hi)] == want
    assert len({b for b, *_ in got}) == len(got)


def test_tile_indices_suffice_for_every_sequence(rows):
    """Between the tile bases of neighbouring sequences lie as many indices as the rows can touch blocks,
    whatever the first position."""
    for lo in list(range(0, 130)) + [10 ** 6 + 63]:
        for count in list(range(0, 200)) + [4095, 4096, 4097]:
            room = rows.base(lo + count, 8) - rows.base(lo, 7)
            assert room >= (count + 62) // 64 + 1
            if count:
                assert max(len(_tiles(rows, 1, lo, lo + count, 7, 1 << 30, count, s + count, 1 << 20, 1 << 30))
                           for s in (0, 1, 62, 63)) <= min(room, rows.max_tiles(count))


@pytest.mark.parametrize("args,bad", [
    ((0, 0, 0, 5, 8, 1, 1, 4, 1000), False), ((0, 0, 0, 5, 8, 1, 0, 4, 1000), False),      # one token; padding
    ((0, 0, 0, 5, 8, 1, -3, 4, 1000), True), ((0, 0, 0, 5, 8, 1, 257, 4, 1000), True),     # negative; pages run out
    ((0, 0, 0, 5, 8, 1, 11, 4, 10), True), ((0, 0, 0, 5, 8, 1, 10, 4, 10), False),         # rotation table runs out
    ((1, 3, 3, 0, 8, 4, 77, 4, 1000), False), ((1, 3, 2, 0, 8, 4, 77, 4, 1000), True),     # no new tokens; reversed
    ((1, -1, 2, 0, 8, 4, 77, 4, 1000), True), ((1, -1, -1, 0, 8, 4, 77, 4, 1000), True),
    ((1, 5, 9, 0, 8, 4, 77, 4, 1000), True), ((1, 0, 5, 0, 8, 4, 77, 4, 1000), True),      # past T; above max_new
    ((1, 0, 4, 0, 8, 4, 3, 4, 1000), True),                                                # more new than all
    ((1, 2147483647, -2147483648, 0, 8, 4, 3, 4, 1000), True), ((1, -2147483648, 2147483647, 0, 8, 4, 3, 4, 1000), True),
    ((0, 0, 0, 5, 8, 1, 2147483647, 2147483647, 2147483647), False)])
def test_sequences_that_break_the_terms(rows, args, bad):
    got = _tiles(rows, *args)
    assert (got == -1) == bad
    if not bad:
        for b, lo, hi, row in got:
            assert 0 <= b < args[7] and 0 <= lo < hi <= 64 and 0 <= row < args[4]


def test_scale_exponent(rows):
    for a in (0.0, 1e-30, 1.0, 1.75, 1.7500001, 447.9, 448.0, 448.1, 3.4e38, 2.0 ** -100, 1e-45):
        bits = int(np.array(a, dtype=np.float32).view(np.uint32))
        assert 2.0 ** rows.sexp(bits) == R.scale_of(float(np.float32(a))), a
    assert not rows.ok(0.0) and not rows.ok(float("nan")) and not rows.ok(float("inf")) and not rows.ok(-1.0)
    assert rows.ok(2.0 ** -100) and rows.ok(2.0 ** 120) and not rows.ok(2.0 ** -101)
