"""Kernels that are placed while the kernel in front of them still runs: they read what that one writes by ordinary
loads, and a run of calls gives the same bits with and without waiting in between."""
import glob
import math
import os
import re

import pytest
import torch

from trainable_gated_block_b200 import build, sas

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trainable_gated_block_b200", "csrc")
READ_ONLY = re.compile(r"__ldg|__ldcs?\b|ld\.global\.nc|__restrict__")


def _code(path):
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_no_read_only_loads_where_kernels_start_early():
    """Sources of kernels behind after_previous() (with the headers that only they use), and the body of any other
    kernel that waits for the grid in front by itself."""
    early = {p for p in glob.glob(os.path.join(CSRC, "*.cu")) if '"dependent.cuh"' in _code(p)}
    assert {os.path.basename(p) for p in early} >= {"append.cu", "decode_q8.cu", "norm_rope.cu"}
    for p in sorted(early) + [os.path.join(CSRC, h) for h in ("head_row.cuh", "page_rows.h", "dependent.cuh", "sm100.cuh")]:
        assert not READ_ONLY.search(_code(p)), p
    for p in sorted(set(glob.glob(os.path.join(CSRC, "*.cu"))) - early):
        text = _code(p)
        for kernel in re.split(r"(?=__global__)", text)[1:]:
            if "griddepcontrol.wait" in kernel:
                head = kernel[:kernel.index("griddepcontrol.wait")]
                body = kernel[:kernel.index("\n}\n")]
                assert not READ_ONLY.search(head) and not READ_ONLY.search(body), p


@pytest.mark.gpu
@pytest.mark.parametrize("K,scored", [(3, False), (120, False), (3, True), (100, True)])
def test_calls_back_to_back_have_the_bits_of_calls_one_by_one(K, scored):
    """Steps of norm + rotation, append into 8-bit pages, scores and selection (or a fixed one) and decode, each
    reading what the call in front has written (queries, keys, pages, scales that grow, mean keys, selections),
    with every step's result kept."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    sas.lib()
    N, Hq, Hkv, D, steps = 24, 16, 4, 128, 70
    g = torch.Generator().manual_seed(7)
    table = sas.rope_table(9000, D)
    blocks = K + 8
    start = torch.randint(64 * (K + 1), 64 * (blocks - 2), (N,), generator=g, dtype=torch.int32)
    start[:4] = 64 * (K + 2) - torch.arange(4, dtype=torch.int32)
    pt = torch.randperm(N * blocks, generator=g).to(torch.int32).view(N, blocks).cuda()
    idx = torch.stack([torch.randperm(K + 1, generator=g)[:K].sort().values for _ in range(N * Hkv)])
    sel = (idx.view(N, Hkv, K).to(torch.int32).cuda(), torch.full((N, Hkv), K, dtype=torch.int32, device="cuda"),
           -torch.rand((N, Hkv, K), generator=g).cuda())
    qk = (torch.randn((steps, N, (Hq + 2 * Hkv) * D), generator=g) * 1.1 ** torch.arange(steps)[:, None, None]).to(torch.bfloat16)
    qkv = [t.unflatten(-1, (-1, D)) for t in qk.cuda().split((Hq * D, Hkv * D, Hkv * D), dim=-1)]
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    codes = [(torch.randn((N * blocks, Hkv, 64, D), generator=g) * 60).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.randint(-9, -4, (N * blocks, Hkv), generator=g).float().exp2() for _ in range(2)]
    lens = [(start + i + 1).cuda() for i in range(steps)]

    def run(wait):
        pages = [t.cuda() for t in codes] + [t.cuda() for t in scales]
        kpool = pages[0].float().mean(2) * pages[2][:, :, None]
        out = []
        torch.cuda.synchronize()
        for i in range(steps):
            q, k = sas.qk_norm_rope(qkv[0][i], qkv[1][i], table, *w, positions=lens[i])
            if wait:
                torch.cuda.synchronize()
            q = sas.append_paged_q8(q, k, qkv[2][i], table, *pages, pt, lens[i], *w, kpool=kpool)
            if wait:
                torch.cuda.synchronize()
            kept = sas.score_select_decode(q, kpool, pt, lens[i], K, blocks)[1:4] if scored else sel
            if wait:
                torch.cuda.synchronize()
            out.append((q, kpool.clone(), *sas.decode_paged_q8(q, *pages, pt, lens[i], *kept)))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        sas.get_error_flag()
        return out, pages

    (one, a), (many, b) = run(True), run(False)
    for x, y in zip(one, many):
        assert all(torch.equal(s, t) for s, t in zip(x, y))
        assert all(math.isfinite(float(t.float().abs().max())) for t in y)
    assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b))
    assert not torch.equal(a[2].cpu(), scales[0]) and not torch.equal(a[3].cpu(), scales[1])
