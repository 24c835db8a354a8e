"""Special values, bad scales and bad sequences in pieces of prompts for 8-bit pages, whose kernel decides on a
page's scales for several heads and rows at a time."""
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as R
from tests.test_gpu_append import EPS, F8, U, Cache, _check_store, _tokens
from trainable_gated_block_b200 import build, sas

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    sas.lib()


def _no_turn(n, D):
    return torch.cat((torch.ones((n, D // 2)), torch.zeros((n, D // 2))), 1).cuda()


def _want(x):
    """Scale and codes of one page and head [rows, D]: infinities as NaN, neither has a part in the scale."""
    x = torch.where(x.isinf(), math.nan, x.double())
    top = x.abs().nan_to_num(0.0).max()
    s = R.scale_of(float(top))
    return s, (x / s).float().to(F8)


@pytest.mark.parametrize("D,H", [(64, 1), (64, 5), (128, 4), (128, 6), (128, 9)])
def test_special_values_in_a_prompt(D, H):
    """Blocks with an infinity in one head, NaN rows, zeros, values under the least scale and the largest ones,
    each followed by a plain block; rows on the codes' grid. With mean keys."""
    blocks, T = 9, 9 * 64
    g = torch.Generator().manual_seed(D + H)
    x = torch.randint(-15, 16, (blocks, 64, H, D), generator=g).float()
    x[:, 0] = 448.0                                 # scale 1, and all values on the grid
    x[1, 7, H // 2, 3], x[1, 9, 0, 5] = math.inf, -math.inf
    x[3, 5:9] = math.nan
    x[3, 11, H - 1, D - 1] = math.inf
    x[4, :, 0] = 0.0
    x[6, :, H - 1] = 1e-30
    x[7, :, :, 1] = 3.0e38
    x[7, 3, 0, 0] = -math.inf
    x = x.to(torch.bfloat16)
    dev = x.view(T, H, D).cuda()
    cache = Cache(True, blocks + 1, H, D, seed=1)
    pt = torch.randperm(blocks, generator=g).to(torch.int32)[None].contiguous()
    before = cache.host()
    cache.append(dev, dev, dev, _no_turn(T, D), pt.cuda(), torch.tensor([T], dtype=torch.int32).cuda(),
                 cu_new=torch.tensor([0, T], dtype=torch.int32).cuda(), max_new=T)
    torch.cuda.synchronize()
    sas.get_error_flag()
    after = cache.host()
    # the rotation by (1, 0): n_a 1 - n_b 0, so a NaN or an infinity of a key makes its partner NaN (infinity times 0)
    lo, hi = x.double().split(D // 2, dim=-1)
    turned = torch.cat((lo - hi * 0.0, hi + lo * 0.0), dim=-1)
    for b in range(blocks):
        p = int(pt[0, b])
        for h in range(H):
            for c, sc, values in (("v", "vs", x), ("k", "ks", turned)):
                s, codes = _want(values[b, :, h])
                got = after[c][p, h].float()
                assert float(after[sc][p, h]) == s, (b, h)
                assert torch.equal(got.isnan(), codes.float().isnan()), (b, h)
                assert torch.equal(got.nan_to_num(0.0), codes.float().nan_to_num(0.0)), (b, h)
            mean = (codes.double() * s).mean(0)
            pool = after["kpool"][p, h].double()
            assert torch.equal(pool.isnan(), mean.isnan()), (b, h)
            keep = ~mean.isnan()
            tol = 67 * U * (codes.double() * s).abs().mean(0)
            assert torch.all((pool - mean)[keep].abs() <= tol[keep]), (b, h)
    for name in after:
        assert torch.equal(after[name][blocks].view(torch.uint8), before[name][blocks].view(torch.uint8))


@pytest.mark.parametrize("D,H", [(64, 3), (128, 5)])
def test_bad_old_scales_of_pages_that_fill(D, H):
    """Old scales without a value on pages that this call goes on with and fills: flagged, that page and head stay
    as they are (also their mean key); the other heads and the blocks behind them are stored."""
    starts, news = [30, 10, 50], [200, 54, 90]
    g = torch.Generator().manual_seed(H)
    cache = Cache(True, 14, H, D, seed=2)
    pt = torch.tensor([[0, 1, 2, 3], [4, 0, 0, 0], [5, 6, 7, 0]], dtype=torch.int32)
    pt[1, 1:], pt[2, 3] = 12, 13                    # not used
    cache.ks[0, 1], cache.ks[4, 0], cache.vs[4, H - 1], cache.vs[5, 1] = 0.0, math.nan, math.inf, 2.0 ** -101
    T = sum(news)
    x = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    kv = torch.tensor([s + n for s, n in zip(starts, news)], dtype=torch.int32)
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    before = cache.host()
    sas.get_error_flag()
    dev = x.cuda()
    q, k = cache.append(dev, dev, dev, _no_turn(300, D), pt.cuda(), kv.cuda(), cu_new=cu.cuda(), max_new=200, with_k=True)
    torch.cuda.synchronize()
    with pytest.raises(sas.SasError):
        sas.get_error_flag()
    after = cache.host()
    assert torch.equal(q.cpu(), x) and torch.equal(k.cpu(), x)
    items = R.page_items(kv.tolist(), cu.tolist(), T, pt.tolist())
    skipped = {"k": [(0, 1), (4, 0)], "v": [(4, H - 1), (5, 1)]}
    for c in "kv":
        for p, h in skipped[c]:
            assert torch.equal(after[c][p, h].view(torch.uint8), before[c][p, h].view(torch.uint8)), (c, p, h)
            assert torch.equal(after[c + "s"][p, h].view(torch.int32), before[c + "s"][p, h].view(torch.int32))
        # the others, with the skipped ones as if the call had not been made for them
        b, a = ({n: t.clone() for n, t in d.items()} for d in (before, after))
        for p, h in skipped[c]:
            for d in (b, a):
                d[c][p, h], d[c + "s"][p, h] = before[c][(p + 1) % 8, 0], 1.0
        for p, rows in items.items():
            heads = [h for h in range(H) if (p, h) not in skipped[c]]
            part = Cache.__new__(Cache)
            part.q8, part.P, part.Hkv, part.D = True, 1, len(heads), D
            sub = [{n: t[p:p + 1][:, heads] for n, t in d.items()} for d in (b, a)]
            ref = R.f64(x)[:, heads]
            _check_store(part, sub[0], sub[1], {0: rows}, c, ref, np.abs(ref))
    full = {p for p, r in items.items() if r[-1][0] == 63}
    for p in range(cache.P):
        for h in range(H):
            if p in full and (p, h) not in skipped["k"]:
                keys = R.f64(after["k"][p, h]) * float(after["ks"][p, h])
                assert np.all(np.abs(R.f64(after["kpool"][p, h]) - keys.mean(0)) <= 67 * U * np.abs(keys).mean(0))
            else:
                assert torch.equal(after["kpool"][p, h], before["kpool"][p, h]), (p, h)


@pytest.mark.parametrize("q8", [False, True])
def test_a_good_sequence_among_bad_ones(q8):
    """Pieces longer than max_new and bounds that run backwards: the one good sequence has its q, k and v; the rows
    of the others stay."""
    D, Hq, Hkv = 128, 4, 2
    cache = Cache(q8, 4, Hkv, D, seed=8)
    (q, k, v, w), dev = _tokens(6, Hq, Hkv, D, seed=9)
    table = sas.rope_table(100, D)
    cu = torch.tensor([0, 4, 2, 3], dtype=torch.int32)
    kv = torch.tensor([10, 10, 10], dtype=torch.int32)
    pt = torch.tensor([[0], [1], [2]], dtype=torch.int32)
    before = cache.host()
    sas.get_error_flag()
    qo, ko = cache.append(*dev[:3], table, pt.cuda(), kv.cuda(), dev[3], cu_new=cu.cuda(), max_new=3, with_k=True)
    torch.cuda.synchronize()
    with pytest.raises(sas.SasError):
        sas.get_error_flag()
    after = cache.host()
    pos = np.full(6, 9)
    rq, pq = R.norm_rope(q, w[0], table.cpu(), pos, EPS)
    rk, pk = R.norm_rope(k, w[1], table.cpu(), pos, EPS)
    _check_store(cache, before, after, {2: [(9, 2, 9)]}, "k", rk, pk)
    _check_store(cache, before, after, {2: [(9, 2, 9)]}, "v", R.f64(v), np.zeros(v.shape))
    for out, ref, pair in ((qo, rq, pq), (ko, rk, pk)):
        assert np.all(np.abs(R.f64(out)[2] - ref[2]) <= 2.0 ** -8 * np.abs(ref[2]) + 24 * U * pair[2])
    assert torch.equal(after["kpool"], before["kpool"])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("head", [0, 63, 64])
def test_mean_key_of_the_largest_values(D, head):
    """A page of values near the largest, filled by a piece, by a token, or by both: its mean is as large."""
    x = torch.full((64, 2, D), 3.0e38).to(torch.bfloat16)
    x[:, 1] *= -0.5
    dev, table = x.cuda(), _no_turn(64, D)
    cache = Cache(True, 2, 2, D, seed=3)
    pt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    kv = [torch.tensor([i], dtype=torch.int32).cuda() for i in range(65)]
    if head:
        cache.append(dev[:head], dev[:head], dev[:head], table, pt, kv[head],
                     cu_new=torch.tensor([0, head], dtype=torch.int32).cuda(), max_new=64)
    for i in range(head, 64):
        cache.append(dev[i:i + 1], dev[i:i + 1], dev[i:i + 1], table, pt, kv[i + 1])
    torch.cuda.synchronize()
    sas.get_error_flag()
    keys = cache.k[0].double().cpu() * cache.ks[0].double().cpu()[:, None, None]
    mean = keys.mean(1)
    assert torch.all((cache.kpool[0].double().cpu() - mean).abs() <= 67 * U * mean.abs())
    assert float(mean.abs().max()) > 2.9e38
