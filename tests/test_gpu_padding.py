"""Padding entries (kv_len 0) through a decode step of a fixed batch: append, scores, selection, decode. They leave
no error behind and change nothing for the other sequences."""
import math

import pytest
import torch

from tests.test_gpu_append import Cache, _layout, _tokens
from trainable_gated_block_b200 import build, sas

pytestmark = pytest.mark.gpu
D, HQ, HKV, K = 128, 8, 2, 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    sas.lib()


def _step(cache, dev, table, pt, kv, w):
    q = cache.append(*dev, table, pt, kv, w)
    s, idx, cnt, gate, lse_s = sas.score_select_decode(q, cache.kpool, pt, kv, K, 4)
    if cache.q8:
        o, lse = sas.decode_paged_q8(q, cache.k, cache.v, cache.ks, cache.vs, pt, kv, idx, cnt, gate)
    else:
        o, lse = sas.decode_paged(q, cache.k, cache.v, pt, kv, idx, cnt, gate)
    return dict(q=q, idx=idx, cnt=cnt, gate=gate, lse_s=lse_s, o=o, lse=lse)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_decode_step_with_padding(q8, graph):
    """One batch with two padding entries, another without them: the same bits for the sequences in both."""
    lens = [190, 0, 61, 130, 0]
    real = [0, 2, 3]
    P, pt = _layout(lens, [1] * 5, seed=17)
    table = sas.rope_table(256, D)
    kv = torch.tensor([n + 1 if n else 0 for n in lens], dtype=torch.int32).cuda()
    _, (q, k, v, w) = _tokens(5, HQ, HKV, D, seed=19, fused=False)
    pt, at = pt.cuda(), torch.tensor(real).cuda()
    a, b = Cache(q8, P, HKV, D, seed=18), Cache(q8, P, HKV, D, seed=18)
    sas.get_error_flag()
    if graph:
        g = torch.cuda.CUDAGraph()
        buf = torch.zeros_like(kv)                  # padding entries alone while it is captured
        _step(a, (q, k, v), table, pt, buf, w)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            got = _step(a, (q, k, v), table, pt, buf, w)
        buf.copy_(kv)
        g.replay()
    else:
        got = _step(a, (q, k, v), table, pt, kv, w)
    torch.cuda.synchronize()
    sas.get_error_flag()                            # nothing is flagged
    want = _step(b, [t[at].contiguous() for t in (q, k, v)], table, pt[at].contiguous(), kv[at].contiguous(), w)
    torch.cuda.synchronize()
    sas.get_error_flag()
    for name in want:
        assert torch.equal(got[name][at], want[name]), name
    raw = torch.uint8 if q8 else torch.int16
    assert torch.equal(a.k.view(raw), b.k.view(raw)) and torch.equal(a.v.view(raw), b.v.view(raw))
    pad = torch.tensor([1, 4]).cuda()
    assert torch.all(got["cnt"][pad] == 0) and torch.all(got["idx"][pad] == -1)
    assert torch.all(got["gate"][pad] == -math.inf) and torch.all(got["lse_s"][pad] == -math.inf)
    assert torch.all(got["o"][pad] == 0) and torch.all(got["lse"][pad] == -math.inf)


@pytest.mark.parametrize("ld_s", [20, 700])
def test_selection_of_padding(ld_s):
    """Both kernels of the selection (rows by warps and by CTAs); a negative length is flagged as before."""
    g = torch.Generator().manual_seed(3)
    s = torch.randn((4, 2, ld_s), generator=g)
    s[2] = float("nan")                             # not read
    kv = torch.tensor([64 * ld_s, 70, 0, 1], dtype=torch.int32)
    sas.get_error_flag()
    idx, cnt, gate, lse_s = sas.select(s.cuda(), 3, kv_len=kv.cuda())
    torch.cuda.synchronize()
    sas.get_error_flag()
    assert cnt.cpu().view(4, 2).tolist() == [[3, 3], [1, 1], [0, 0], [0, 0]]
    assert torch.all(idx.view(4, -1)[2:] == -1) and torch.all(lse_s.view(4, -1)[2:] == -math.inf)
    kv[2] = -1
    sas.select(s.cuda(), 3, kv_len=kv.cuda())
    torch.cuda.synchronize()
    with pytest.raises(sas.SasError):
        sas.get_error_flag()


def test_bf16_decode_of_a_negative_length_is_flagged():
    x = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((2, 4, D), (3, 2, 64, D), (3, 2, 64, D))]
    pt = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    sel = (torch.zeros((2, 2, 1), dtype=torch.int32, device="cuda"), torch.zeros((2, 2), dtype=torch.int32, device="cuda"),
           torch.zeros((2, 2, 1), device="cuda"))
    sas.get_error_flag()
    sas.decode_paged(*x, pt, torch.tensor([5, -1], dtype=torch.int32).cuda(), *sel)
    torch.cuda.synchronize()
    with pytest.raises(sas.SasError):
        sas.get_error_flag()
