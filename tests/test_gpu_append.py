"""append_paged and append_paged_q8 through the C ABI against the fp64 reference, and a run of append,
scoring and decode as a serving loop makes them.

Tolerances (u = 2^-24): q, k: 2^-8 |y| + 24 u (|a| + |b|) (as for qk_norm_rope); values: exact in bf16.
8-bit codes: half an e4m3 step, 2^-4 |x| or 2^-10 of the scale in the subnormal range, plus the fp32 part.
Pooled keys: 64 terms and two products, 67 u of the mean magnitude.
"""
import math

import numpy as np
import pytest
import torch

from oracle import sas_oracle as O
from oracle import serving_oracle as R
from trainable_gated_block_b200 import build, sas

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    sas.lib()


class Cache:
    """Pages filled with random contents, on the GPU, and the calls on them."""

    def __init__(self, q8, P, Hkv, D, seed):
        g = torch.Generator().manual_seed(seed)
        self.q8, self.P, self.Hkv, self.D = q8, P, Hkv, D
        x = [torch.randn((P, Hkv, 64, D), generator=g) for _ in range(2)]
        if q8:
            self.k, self.v = ((t * 100).clamp(-448, 448).to(F8).cuda() for t in x)
            self.ks, self.vs = (torch.randint(-9, -5, (P, Hkv), generator=g).float().exp2().cuda() for _ in range(2))
        else:
            self.k, self.v = (t.to(torch.bfloat16).cuda() for t in x)
            self.ks = self.vs = None
        self.kpool = torch.full((P, Hkv, D), 3.0, device="cuda")

    def append(self, q, k, v, table, pt, kv_len, w=(None, None), **kw):
        pages = (self.k, self.v, self.ks, self.vs) if self.q8 else (self.k, self.v)
        fn = sas.append_paged_q8 if self.q8 else sas.append_paged
        return fn(q, k, v, table, *pages, pt, kv_len, q_weight=w[0], k_weight=w[1], eps=EPS, kpool=self.kpool, **kw)

    def host(self):
        d = dict(k=self.k.cpu(), v=self.v.cpu(), kpool=self.kpool.cpu())
        if self.q8:
            d.update(ks=self.ks.cpu(), vs=self.vs.cpu())
        return d


def _tokens(T, Hq, Hkv, D, seed, fused=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((T, (Hq + 2 * Hkv) * D), generator=g) * scale).to(torch.bfloat16)
    q, k, v = (t.view(T, -1, D) for t in qkv.split((Hq * D, Hkv * D, Hkv * D), dim=1))
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16) for _ in range(2)]
    dev = qkv.cuda()
    qd, kd, vd = (t.view(T, -1, D) for t in dev.split((Hq * D, Hkv * D, Hkv * D), dim=1))
    if not fused:
        qd, kd, vd = qd.contiguous(), kd.contiguous(), vd.contiguous()
    return (q, k, v, w), (qd, kd, vd, [t.cuda() for t in w])


def _check_store(cache, before, after, items, name, x, pair):
    """Pages after an append of rows x [T, Hkv, D] (fp64); everything else as it was."""
    touched = torch.zeros((cache.P, 64), dtype=torch.bool)
    b, a = before[name], after[name]
    for page, rows in items.items():
        lo = rows[0][0]
        r = [i for i, _, _ in rows]
        t = [i for _, i, _ in rows]
        touched[page, r] = True
        new, mag = np.moveaxis(x[t], 1, 0), np.moveaxis(pair[t], 1, 0)           # [Hkv, rows, D]
        got = R.f64(a[page][:, r])
        if not cache.q8:
            tol = 2.0 ** -8 * np.abs(new) + 24 * U * mag
            assert np.all(np.abs(got - new) <= tol), (name, page)
            continue
        touched[page, :lo] = True
        for h in range(cache.Hkv):
            old = float(before[name + "s"][page, h])
            need = R.scale_of(np.abs(new[h]).max())
            want = old if lo and need <= old else need
            s = float(after[name + "s"][page, h])
            assert s == want, (name, page, h, s, want)
            tol = np.maximum(2.0 ** -4 * np.abs(new[h]), 2.0 ** -10 * s) + 24 * U * mag[h]
            assert np.all(np.abs(s * got[h] - new[h]) <= tol), (name, page, h)
            if lo:
                was, now = R.f64(b[page, h, :lo]) * old, R.f64(a[page, h, :lo]) * s
                assert np.all(np.abs(was - now) <= (0.0 if s == old else 2.0 ** -10 * s)), (name, page, h)
    raw = torch.uint8 if cache.q8 else torch.int16
    same = (a.view(raw) == b.view(raw)).all(-1).all(1)                          # [P, 64]
    assert bool((same | touched).all()), f"{name}: a row outside the call changed"
    if cache.q8:
        idle = [p for p in range(cache.P) if p not in items]
        assert torch.equal(before[name + "s"][idle], after[name + "s"][idle])


def _check_call(cache, tok, dev, table, pt, kv, cu, max_new, with_k=True):
    (q, k, v, w), (qd, kd, vd, wd) = tok, dev
    T = q.shape[0]
    before = cache.host()
    out = cache.append(qd, kd, vd, table, pt.cuda(), kv.cuda(), wd, cu_new=None if cu is None else cu.cuda(),
                       max_new=max_new, with_k=with_k)
    torch.cuda.synchronize()
    sas.get_error_flag()
    after = cache.host()
    qo, ko = out if with_k else (out, None)
    rows = R.new_rows(kv.tolist(), None if cu is None else cu.tolist(), T)
    t = [i for _, i, _ in rows]
    pos = np.zeros(T, dtype=np.int64)
    pos[t] = [p for _, _, p in rows]
    tab = table.cpu()
    rq, pq = R.norm_rope(q, w[0], tab, pos, EPS)
    rk, pk = R.norm_rope(k, w[1], tab, pos, EPS)
    assert np.all(np.abs(R.f64(qo)[t] - rq[t]) <= 2.0 ** -8 * np.abs(rq[t]) + 24 * U * pq[t])
    if with_k:
        assert np.all(np.abs(R.f64(ko)[t] - rk[t]) <= 2.0 ** -8 * np.abs(rk[t]) + 24 * U * pk[t])
    items = R.page_items(kv.tolist(), None if cu is None else cu.tolist(), T, pt.tolist())
    _check_store(cache, before, after, items, "k", rk, pk)
    _check_store(cache, before, after, items, "v", R.f64(v), np.zeros(v.shape))
    full = {p for p, r in items.items() if r[-1][0] == 63}
    for p in range(cache.P):
        if p not in full:
            assert torch.equal(after["kpool"][p], before["kpool"][p])
            continue
        keys = R.f64(after["k"][p]) * (R.f64(after["ks"][p])[:, None, None] if cache.q8 else 1.0)
        tol = 67 * U * np.abs(keys).mean(1)
        assert np.all(np.abs(R.f64(after["kpool"][p]) - keys.mean(1)) <= tol), p
    return qo, ko, after


def _layout(starts, news, seed, spare=2):
    """Page table with the pages of every block of each sequence, in random order."""
    blocks = [(s + n + 63) // 64 for s, n in zip(starts, news)]
    P = sum(blocks) + spare
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).tolist()
    pt = torch.zeros((len(starts), max(max(blocks), 1) + 1), dtype=torch.int32)
    for i, b in enumerate(blocks):
        for j in range(b):
            pt[i, j] = perm.pop()
    return P, pt


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 2, 1), (128, 5, 5), (64, 12, 3)])
def test_single_tokens(q8, D, Hq, Hkv):
    """One token for each sequence at every kind of row: a page's first, inner and last, and padding entries."""
    starts = [0, 1, 62, 63, 64, 127, 128, 200, 0]
    news = [1] * 8 + [0]
    P, pt = _layout(starts, news, seed=D)
    kv = torch.tensor([s + n for s, n in zip(starts, news)], dtype=torch.int32)
    kv[8] = 0                                                   # padding
    tok, dev = _tokens(9, Hq, Hkv, D, seed=Hq)
    cache = Cache(q8, P, Hkv, D, seed=1)
    qo, ko, _ = _check_call(cache, tok, dev, sas.rope_table(300, D), pt, kv, None, 1)
    assert torch.all(qo[8] == 0) and torch.all(ko[8] == 0)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,starts,news", [
    (128, 8, 2, [0], [1]), (128, 8, 2, [0], [64]), (128, 8, 2, [0], [65]), (128, 4, 4, [63], [2]),
    (128, 40, 8, [0, 30, 64, 5, 100], [200, 100, 64, 0, 1]), (64, 2, 1, [0, 3, 63, 1], [300, 61, 1, 130]),
    (64, 6, 2, [10, 0, 70], [0, 0, 5])])
def test_pieces_of_prompts(q8, D, Hq, Hkv, starts, news):
    P, pt = _layout(starts, news, seed=sum(news))
    T = sum(news)
    kv = torch.tensor([s + n for s, n in zip(starts, news)], dtype=torch.int32)
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    tok, dev = _tokens(T, Hq, Hkv, D, seed=T + D)
    _check_call(Cache(q8, P, Hkv, D, seed=2), tok, dev, sas.rope_table(400, D), pt, kv, cu, max(news) + 7)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 6, 3), (128, 10, 5), (128, 6, 6), (128, 7, 7), (64, 9, 9), (64, 5, 1), (64, 3, 3)])
def test_heads_that_do_not_fill_a_unit(q8, D, Hq, Hkv):
    """Pieces that start and end inside pages, with counts of heads that leave a last unit part empty."""
    starts, news = [20, 0, 63], [140, 64, 1]
    P, pt = _layout(starts, news, seed=Hkv)
    kv = torch.tensor([s + n for s, n in zip(starts, news)], dtype=torch.int32)
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    tok, dev = _tokens(sum(news), Hq, Hkv, D, seed=Hq + D)
    _check_call(Cache(q8, P, Hkv, D, seed=26), tok, dev, sas.rope_table(200, D), pt, kv, cu, max(news))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_mean_keys_by_prompt_and_by_token_have_the_same_bits(q8, D):
    """Without rotation. In 8-bit pages of values on the codes' grid the sums are exact too."""
    Hq = Hkv = 3
    g = torch.Generator().manual_seed(27)
    if q8:
        k = torch.randint(-15, 16, (128, Hkv, D), generator=g).float()
        k[::64] = 448.0                 # a page's first row sets its scale to 1
    else:
        k = torch.randn((128, Hkv, D), generator=g)
    k = k.to(torch.bfloat16).cuda()
    q = torch.zeros((128, Hq, D), dtype=torch.bfloat16, device="cuda")
    table = torch.cat((torch.ones((128, D // 2)), torch.zeros((128, D // 2))), dim=1).cuda()
    pt = torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    a, b = Cache(q8, 2, Hkv, D, seed=28), Cache(q8, 2, Hkv, D, seed=28)
    a.append(q, k, k, table, pt, torch.tensor([128], dtype=torch.int32).cuda(),
             cu_new=torch.tensor([0, 128], dtype=torch.int32).cuda(), max_new=128)
    for i in range(128):
        b.append(q[i:i + 1], k[i:i + 1], k[i:i + 1], table, pt, torch.tensor([i + 1], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    sas.get_error_flag()
    assert torch.equal(a.k.float(), b.k.float()) and torch.equal(a.kpool, b.kpool)
    if q8:
        assert torch.all(a.ks == 1.0) and torch.all(b.ks == 1.0)
        assert torch.equal(a.kpool.double(), k.view(2, 64, Hkv, D).double().mean(1)[[1, 0]])    # page 1: the first block


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 6, 3)])
def test_single_tokens_of_some_sequences(q8, D, Hq, Hkv):
    """cu_new with max_new 1: sequences that bring a token and others that bring none."""
    starts, news = [63, 5, 130, 64, 0], [1, 0, 1, 0, 1]
    P, pt = _layout(starts, news, seed=21)
    kv = torch.tensor([s + n for s, n in zip(starts, news)], dtype=torch.int32)
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    tok, dev = _tokens(3, Hq, Hkv, D, seed=22)
    _check_call(Cache(q8, P, Hkv, D, seed=23), tok, dev, sas.rope_table(140, D), pt, kv, cu, 1)


@pytest.mark.parametrize("q8", [False, True])
def test_many_sequences_and_long_pieces(q8):
    """More units and tiles than the resident CTAs take at a time, by token and by piece."""
    D, Hq, Hkv = 128, 20, 4
    g = torch.Generator().manual_seed(24)
    starts = torch.randint(0, 300, (150,), generator=g).tolist()
    P, pt = _layout(starts, [1] * 150, seed=25)
    tok, dev = _tokens(150, Hq, Hkv, D, seed=26)
    kv = torch.tensor([s + 1 for s in starts], dtype=torch.int32)
    _check_call(Cache(q8, P, Hkv, D, seed=27), tok, dev, sas.rope_table(400, D), pt, kv, None, 1)
    starts, news = [70, 0, 129], [2700, 1999, 641]
    P, pt = _layout(starts, news, seed=28)
    tok, dev = _tokens(sum(news), Hq, Hkv, D, seed=29)
    kv = torch.tensor([s + n for s, n in zip(starts, news)], dtype=torch.int32)
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    _check_call(Cache(q8, P, Hkv, D, seed=30), tok, dev, sas.rope_table(2800, D), pt, kv, cu, max(news))


@pytest.mark.parametrize("q8", [False, True])
def test_rows_behind_the_last_sequence_stay(q8):
    """cu_new ends before T, and starts after row 0: the rows outside are neither stored nor written."""
    P, pt = _layout([5], [70], seed=4)
    tok, dev = _tokens(80, 4, 2, 128, seed=5, fused=False)
    cu = torch.tensor([3, 73], dtype=torch.int32)
    kv = torch.tensor([75], dtype=torch.int32)
    cache = Cache(q8, P, 2, 128, seed=6)
    _check_call(cache, tok, dev, sas.rope_table(80, 128), pt, kv, cu, 70)
    import ctypes
    q, k, v, w = dev
    qo = torch.full((80, 4, 128), 9.0, device="cuda", dtype=torch.bfloat16)
    ko = torch.full((80, 2, 128), 9.0, device="cuda", dtype=torch.bfloat16)
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())   # noqa: E731
    table, ptd, cud, kvd = sas.rope_table(80, 128), pt.cuda(), cu.cuda(), kv.cuda()
    head = [p(q), 512, p(k), 256, p(v), 256, p(w[0]), p(w[1]), p(table), 80, p(cud), 1, 70, 80, p(kvd), p(ptd),
            pt.shape[1], P, 4, 2, 128, 64, EPS, p(qo), p(ko), p(cache.k), p(cache.v)]
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if q8:
        assert sas.lib().sas_append_paged_q8(*head, p(cache.ks), p(cache.vs), None, st) == sas.SAS_OK
    else:
        assert sas.lib().sas_append_paged(*head, None, st) == sas.SAS_OK
    torch.cuda.synchronize()
    for t in (qo, ko):
        assert torch.all(t[:3] == 9) and torch.all(t[73:] == 9) and not torch.any((t[3:73] == 9).all(-1))


@pytest.mark.parametrize("q8", [False, True])
def test_rotation_only(q8):
    P, pt = _layout([0], [40], seed=4)
    (q, k, v, _), (qd, kd, vd, _) = _tokens(40, 4, 2, 64, seed=6)
    cu, kv = torch.tensor([0, 40], dtype=torch.int32), torch.tensor([40], dtype=torch.int32)
    _check_call(Cache(q8, P, 2, 64, seed=7), (q, k, v, (None, None)), (qd, kd, vd, (None, None)),
                sas.rope_table(40, 64), pt, kv, cu, 40, with_k=False)


@pytest.mark.parametrize("q8", [False, True])
def test_bad_sequences_and_pages_are_skipped(q8):
    """Lengths that break the terms and page ids outside the cache: flagged, nothing of them stored, the
    others unaffected."""
    D, Hq, Hkv = 128, 4, 2
    cache = Cache(q8, 6, Hkv, D, seed=8)
    tok, dev = _tokens(6, Hq, Hkv, D, seed=9)
    table = sas.rope_table(100, D)
    #  sequence:      ok  bad page   page id -1   past max_pages   past the table   ok
    kv = torch.tensor([5, 70, 3, 200, 101, 65], dtype=torch.int32)
    pt = torch.tensor([[0, 0], [1, 6], [-1, 1], [2, 2], [2, 2], [2, 3]], dtype=torch.int32)
    before = cache.host()
    sas.get_error_flag()
    cache.append(*dev[:3], table, pt.cuda(), kv.cuda(), dev[3])
    with pytest.raises(sas.SasError):
        sas.get_error_flag()
    after = cache.host()
    (q, k, v, w) = tok
    pos = np.array([4, 0, 0, 0, 0, 64])
    rk, pk = R.norm_rope(k, w[1], table.cpu(), pos, EPS)
    items = {0: [(4, 0, 4)], 3: [(0, 5, 64)]}
    _check_store(cache, before, after, items, "k", rk, pk)
    _check_store(cache, before, after, items, "v", R.f64(v), np.zeros(v.shape))
    # a piece longer than max_new, bounds that run backwards, and a good one between them
    cu = torch.tensor([0, 4, 2, 3], dtype=torch.int32)
    kv = torch.tensor([10, 10, 10], dtype=torch.int32)
    pt = torch.tensor([[0], [1], [2]], dtype=torch.int32)
    before = cache.host()
    cache.append(*dev[:3], table, pt.cuda(), kv.cuda(), dev[3], cu_new=cu.cuda(), max_new=3)
    with pytest.raises(sas.SasError):
        sas.get_error_flag()
    after = cache.host()
    rk, pk = R.norm_rope(k, w[1], table.cpu(), np.full(6, 9), EPS)
    _check_store(cache, before, after, {2: [(9, 2, 9)]}, "k", rk, pk)


def test_q8_old_scales_outside_the_range_are_flagged():
    cache = Cache(True, 4, 2, 64, seed=8)
    tok, dev = _tokens(3, 2, 2, 64, seed=9)
    cache.ks[0, 0], cache.ks[1, 1], cache.vs[2, 0] = 0.0, float("nan"), float("inf")
    before = cache.host()
    kv = torch.tensor([5, 5, 5], dtype=torch.int32)
    pt = torch.tensor([[0], [1], [2]], dtype=torch.int32)
    sas.get_error_flag()
    cache.append(*dev[:3], sas.rope_table(10, 64), pt.cuda(), kv.cuda(), dev[3])
    with pytest.raises(sas.SasError):
        sas.get_error_flag()
    after = cache.host()
    k, k0 = after["k"].view(torch.uint8), before["k"].view(torch.uint8)
    v, v0 = after["v"].view(torch.uint8), before["v"].view(torch.uint8)
    assert torch.equal(k[0, 0], k0[0, 0]) and torch.equal(k[1, 1], k0[1, 1]) and torch.equal(v[2, 0], v0[2, 0])
    assert not torch.equal(k[0, 1], k0[0, 1]) and not torch.equal(v[0, 0], v0[0, 0])
    # the same garbage where the page starts anew is no matter
    kv = torch.tensor([1, 1, 1], dtype=torch.int32)
    cache.append(*dev[:3], sas.rope_table(10, 64), pt.cuda(), kv.cuda(), dev[3])
    torch.cuda.synchronize()
    sas.get_error_flag()
    assert torch.isfinite(cache.ks[:3]).all() and torch.isfinite(cache.vs[:3]).all()


def test_q8_scale_growth_row_by_row():
    """64 single-token steps whose values grow by 1.5 each: the scale follows, older rows keep their values
    up to the codes' subnormals, and the page's mean key comes with its last row."""
    D, Hkv = 64, 2
    cache = Cache(True, 3, Hkv, D, seed=10)
    table = sas.rope_table(64, D)
    pt = torch.tensor([[1]], dtype=torch.int32)
    g = torch.Generator().manual_seed(11)
    for i in range(64):
        x = torch.randn((1, 4 * Hkv // 2 + 2 * Hkv, D), generator=g) * 1e-3 * 1.5 ** (i if i < 40 else 40)
        x = x.to(torch.bfloat16)
        q, k, v = x[:, :4], x[:, 4:6], x[:, 6:8]
        xd = x.cuda()
        kv = torch.tensor([i + 1], dtype=torch.int32)
        _check_call(cache, (q, k, v, (None, None)), (xd[:, :4], xd[:, 4:6], xd[:, 6:8], (None, None)), table, pt, kv,
                    None, 1)


def test_q8_special_values():
    """Zero pages, values under the least scale, the largest bf16, NaN and infinities."""
    D = 64
    table = torch.cat((torch.ones((64, D // 2)), torch.zeros((64, D // 2))), 1).cuda()     # no turn
    cache = Cache(True, 6, 1, D, seed=12)
    x = torch.zeros((6, 1, D))
    x[1] = 1e-30
    x[2, 0, 3] = 3.0e38
    x[3, 0, :3] = torch.tensor([float("nan"), 2.0, float("inf")])
    x[4] = float("nan")
    x[5] = torch.linspace(-448, 448, D)
    x = x.to(torch.bfloat16).cuda()
    pt = torch.arange(6, dtype=torch.int32)[:, None].contiguous().cuda()
    kv = torch.ones(6, dtype=torch.int32).cuda()
    cache.append(x, x, x, table, pt, kv)
    torch.cuda.synchronize()
    sas.get_error_flag()
    for codes, scale in ((cache.k, cache.ks), (cache.v, cache.vs)):
        s, row = scale[:, 0].cpu(), codes[:, 0, 0].float().cpu()
        assert s.tolist() == [2.0 ** -64, 2.0 ** -64, 2.0 ** 120,
                              2.0 ** -7, 2.0 ** -64, 1.0]
        assert torch.all(row[0] == 0) and torch.all(row[1] == 0) and torch.all(row[4].isnan())
        assert row[3, :3].isnan().tolist() == [True, False, True] and float(row[3, 1] * s[3]) == 2.0
        assert float((row[2] * s[2] - x[2, 0].float().cpu()).abs().max()) <= 2.0 ** -4 * 3.0e38
        assert torch.all((row[5] - x[5, 0].float().cpu()).abs() <= 2.0 ** -4 * x[5, 0].float().cpu().abs() + 2.0 ** -10)


@pytest.mark.parametrize("q8", [False, True])
def test_one_call_equals_token_by_token(q8):
    """bf16 pages: the same bits. 8-bit pages: the same scales, and codes that may differ where a value fell
    below the normal range before the scale grew (within 2^-9 of the scale: two roundings)."""
    D, Hq, Hkv, n = 128, 4, 2, 150
    table = sas.rope_table(n, D)
    pt = torch.tensor([[2, 0, 1]], dtype=torch.int32).cuda()
    _, (q, k, v, w) = _tokens(n, Hq, Hkv, D, seed=13)
    a, b = Cache(q8, 4, Hkv, D, seed=14), Cache(q8, 4, Hkv, D, seed=14)
    qa = a.append(q, k, v, table, pt, torch.tensor([n], dtype=torch.int32).cuda(), w,
                  cu_new=torch.tensor([0, n], dtype=torch.int32).cuda(), max_new=n)
    qb = [b.append(q[i:i + 1], k[i:i + 1], v[i:i + 1], table, pt, torch.tensor([i + 1], dtype=torch.int32).cuda(), w)
          for i in range(n)]
    torch.cuda.synchronize()
    sas.get_error_flag()
    assert torch.equal(qa, torch.cat(qb))
    if not q8:
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.kpool, b.kpool)
        return
    assert torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert float((x.float() - y.float()).abs().max()) <= 2.0 ** -9


@pytest.mark.parametrize("q8", [False, True])
def test_other_stream_and_replayed_graph(q8):
    """A decode step captured once and replayed with new tokens and lengths in the captured buffers."""
    D, Hq, Hkv, N = 128, 8, 2, 3
    table = sas.rope_table(200, D)
    pt = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32).cuda()
    _, (q, k, v, w) = _tokens(4 * N, Hq, Hkv, D, seed=15)
    a, b = Cache(q8, 6, Hkv, D, seed=16), Cache(q8, 6, Hkv, D, seed=16)
    buf = [torch.zeros((N, H, D), dtype=torch.bfloat16, device="cuda") for H in (Hq, Hkv, Hkv)]
    kv = torch.zeros(N, dtype=torch.int32, device="cuda")           # capture stores nothing: padding entries
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.append(*buf, table, pt, kv, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = a.append(*buf, table, pt, kv, w)
    for step in range(4):
        lens = torch.tensor([62 + step, 0 if step == 1 else 10 + step, 1 + step], dtype=torch.int32).cuda()
        part = [t[N * step:N * step + N] for t in (q, k, v)]
        for x, y in zip(buf, part):
            x.copy_(y)
        kv.copy_(lens)
        graph.replay()
        ref = b.append(*part, table, pt, lens, w)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    sas.get_error_flag()
    raw = torch.uint8
    assert torch.equal(a.k.view(raw), b.k.view(raw)) and torch.equal(a.v.view(raw), b.v.view(raw))
    assert torch.equal(a.kpool, b.kpool)


@pytest.mark.parametrize("q8", [False, True])
def test_serving_loop_against_reference(q8):
    """Prompts of different lengths, then decode steps: append (norm, rotation, pages, pooled keys), scoring,
    selection and decode, each step checked against the fp64 decode over the cache as it stands."""
    D, Hq, Hkv, K, steps = 128, 8, 2, 2, 6
    lens = [190, 61, 130]
    N, T = len(lens), sum(lens)
    P, pt = _layout(lens, [steps] * N, seed=17)
    table = sas.rope_table(256, D)
    cache = Cache(q8, P, Hkv, D, seed=18)
    tok, dev = _tokens(T, Hq, Hkv, D, seed=19)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    qo, ko, _ = _check_call(cache, tok, dev, table, pt, torch.tensor(lens, dtype=torch.int32), cu, max(lens))
    # the prompts' own attention on the rotated tokens
    s = torch.randn((N, Hkv, 3, 3), generator=torch.Generator().manual_seed(20))
    sel = sas.select_varlen(s.cuda(), K, cu.cuda())
    o, _ = sas.attn_fwd_varlen(qo, ko, dev[2].contiguous(), cu.cuda(), max(lens), *sel[:3])
    ri, rc, rg, _ = O.select_varlen(s, K, cu)
    ro, _ = O.attn_fwd_varlen(qo.cpu(), ko.cpu(), tok[2], cu, ri, rc, rg, 1 / math.sqrt(D), max(lens))
    assert float(np.abs(R.f64(o) - ro).max()) <= 1e-2
    ptd = pt.cuda()
    for step in range(steps):
        kv = torch.tensor([n + step + 1 for n in lens], dtype=torch.int32)
        tok, dev = _tokens(N, Hq, Hkv, D, seed=100 + step)
        q, _, after = _check_call(cache, tok, dev, table, pt, kv, None, 1)
        s, idx, cnt, gate, _ = sas.score_select_decode(q, cache.kpool, ptd, kv.cuda(), K, 4)
        if q8:
            o, lse = sas.decode_paged_q8(q, cache.k, cache.v, cache.ks, cache.vs, ptd, kv.cuda(), idx, cnt, gate)
        else:
            o, lse = sas.decode_paged(q, cache.k, cache.v, ptd, kv.cuda(), idx, cnt, gate)
        torch.cuda.synchronize()
        sas.get_error_flag()
        keys = R.f64(after["k"]) * (R.f64(after["ks"])[:, :, None, None] if q8 else 1.0)
        vals = R.f64(after["v"]) * (R.f64(after["vs"])[:, :, None, None] if q8 else 1.0)
        sref = O.standin_scores_decode(q.cpu(), keys, pt, kv, np.zeros((N, Hkv, 4)))
        nh = O.decode_history(kv)
        for n in range(N):
            assert np.abs(R.f64(s)[n, :, :nh[n]] - sref[n, :, :nh[n]]).max(initial=0.0) <= 1e-5
        ro, rl = O.decode(q.cpu(), keys, vals, pt, kv, idx.cpu(), cnt.cpu(), gate.cpu(), 1 / math.sqrt(D))
        assert float(np.abs(R.f64(o) - ro).max()) <= 1e-2 and float(np.abs(R.f64(lse) - rl).max()) <= 1e-2


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of the cache; only rows of the pages in use are looked at."""
    D, Hq, Hkv, P = 128, 16, 8, 70000                            # 4.6 GB for each cache
    table = sas.rope_table(200, D)
    tok, dev = _tokens(130, Hq, Hkv, D, seed=31)
    cu, kv = torch.tensor([0, 130], dtype=torch.int32), torch.tensor([130], dtype=torch.int32)
    where = torch.tensor([[P - 1, 12345, P - 2]], dtype=torch.int32)
    big, small = Cache.__new__(Cache), Cache(True, 3, Hkv, D, seed=32)
    big.q8, big.P, big.Hkv, big.D = True, P, Hkv, D
    big.k, big.v = (torch.empty((P, Hkv, 64, D), dtype=F8, device="cuda") for _ in range(2))
    big.ks, big.vs = (torch.zeros((P, Hkv), device="cuda") for _ in range(2))
    big.kpool = torch.zeros((P, Hkv, D), device="cuda")
    for c, pt in ((big, where), (small, torch.tensor([[0, 1, 2]], dtype=torch.int32))):
        c.append(*dev[:3], table, pt.cuda(), kv.cuda(), dev[3], cu_new=cu.cuda(), max_new=130)
        one = [t[:1].contiguous() for t in dev[:3]]
        c.append(*one, table, pt.cuda(), torch.tensor([131], dtype=torch.int32).cuda(), dev[3])
    torch.cuda.synchronize()
    sas.get_error_flag()
    raw, at = torch.uint8, where[0].long().cuda()
    for a, b in ((big.k, small.k), (big.v, small.v)):
        a, b = a.view(raw)[at], b.view(raw)
        assert torch.equal(a[:2], b[:2]) and torch.equal(a[2, :, :3], b[2, :, :3])
    assert torch.equal(big.ks[at], small.ks) and torch.equal(big.vs[at], small.vs)
    assert torch.equal(big.kpool[at[:2]], small.kpool[:2])
