"""decode_paged_q8 through the C ABI against the fp64 reference, whose decode_q8 derives each row's error
bound: fp32 logits and sums, fp16 probabilities, one rounding of the output to bf16."""
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as R
from trainable_gated_block_b200 import build, sas

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    sas.lib()


def _codes(P, Hkv, g, lo=-9, hi=-4):
    x = (torch.randn((P, Hkv, 64, D), generator=g) * 90).clamp(-448, 448).to(F8)
    return x, torch.randint(lo, hi, (P, Hkv), generator=g).float().exp2()


def _make(lens, Hq, Hkv, K, seed, ld=None):
    g = torch.Generator().manual_seed(seed)
    N = len(lens)
    pages = [(n + 63) // 64 for n in lens]
    P = max(1, sum(pages))
    perm = torch.randperm(P, generator=g).to(torch.int32)
    pt = torch.zeros((N, max(max(pages), 1)), dtype=torch.int32)
    at = 0
    for i, p in enumerate(pages):
        pt[i, :p] = perm[at:at + p]
        at += p
    kc, ks = _codes(P, Hkv, g)
    vc, vs = _codes(P, Hkv, g)
    kv = torch.tensor(lens, dtype=torch.int32)
    q = torch.randn((N, Hq, D), generator=g).to(torch.bfloat16)
    s = torch.randn((N, Hkv, max(1, pt.shape[1])), generator=g)
    idx = torch.full((N, Hkv, K), -1, dtype=torch.int32)
    cnt = torch.zeros((N, Hkv), dtype=torch.int32)
    gate = torch.full((N, Hkv, K), -math.inf)
    for n in range(N):
        nh = max(0, (lens[n] - 1) // 64)
        c = min(K, nh)
        for h in range(Hkv):
            if c:
                top = s[n, h, :nh].topk(c).indices.sort().values
                idx[n, h, :c] = top.to(torch.int32)
                gate[n, h, :c] = s[n, h, top] - s[n, h, :nh].logsumexp(0)
            cnt[n, h] = c
    return dict(q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, page_table=pt, kv_len=kv, idx=idx, cnt=cnt,
                log_gate=gate)


def _run(x, flag=False, **kw):
    out = sas.decode_paged_q8(**{k: v.cuda() for k, v in x.items()}, **kw)
    torch.cuda.synchronize()
    if flag:
        with pytest.raises(sas.SasError):
            sas.get_error_flag()
    else:
        sas.get_error_flag()
    return out


def _ref(x, sm=1 / math.sqrt(D)):
    return R.decode_q8(x["q"], x["k_cache"], x["v_cache"], x["k_scale"], x["v_scale"], x["page_table"], x["kv_len"],
                       x["idx"], x["cnt"], x["log_gate"], sm)


def _check(out, ref, rows=slice(None)):
    o, lse = (R.f64(t)[rows] for t in out)
    ro, rl, to, tl = (t[rows] for t in ref)
    assert np.all(np.isfinite(o))
    fin = np.isfinite(rl)
    assert np.array_equal(np.isfinite(lse), fin)
    assert np.all(np.abs(o - ro) <= to), float((np.abs(o - ro) / np.maximum(to, 1e-300)).max())
    assert np.all(np.abs(lse[fin] - rl[fin]) <= tl[fin])


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (3, 1), (8, 2), (10, 2), (6, 1), (14, 2), (8, 1), (32, 8)])
@pytest.mark.parametrize("lens,K", [([1], 2), ([64], 0), ([65, 130, 64, 700], 3), ([0, 129, 0, 1], 1),
                                    ([1000, 7, 513], 20)])
def test_against_reference(Hq, Hkv, lens, K):
    x = _make(lens, Hq, Hkv, K, seed=Hq * 100 + len(lens) + K)
    out = _run(x)
    _check(out, _ref(x))
    for n, length in enumerate(lens):
        if length == 0:                       # padding entries
            assert torch.all(out[0][n] == 0) and torch.all(out[1][n] == -math.inf)


def test_every_length_of_the_current_block():
    x = _make(list(range(1, 65)) + [64 + i for i in range(1, 65, 7)], 4, 1, 1, seed=3)
    _check(_run(x), _ref(x))


def test_many_sequences_share_the_ctas():
    x = _make([100 + 37 * i for i in range(40)], 16, 4, 5, seed=4)
    _check(_run(x), _ref(x))


def test_enough_slots_for_the_many_warp_kernel():
    """N Hkv (K + 1) slots above ten for each of ten warps on every SM; the sequences share pages."""
    N, Hq, Hkv, K = 64, 16, 8, 30
    x = _make([64 * 3 + 1] * N, Hq, Hkv, K, seed=20)
    g = torch.Generator().manual_seed(21)
    P, blocks = x["k_cache"].shape[0], [int(b) for b in torch.randint(0, 45, (N,), generator=g)]
    x["page_table"] = torch.randint(0, P, (N, 45), generator=g, dtype=torch.int32)
    x["kv_len"] = torch.tensor([64 * b + 1 + 7 * (i % 9) for i, b in enumerate(blocks)], dtype=torch.int32)
    for n, b in enumerate(blocks):
        c = min(K, b)
        x["cnt"][n] = c
        x["idx"][n], x["log_gate"][n] = -1, -math.inf
        for h in range(Hkv):
            x["idx"][n, h, :c] = torch.randperm(b, generator=g)[:c].sort().values.to(torch.int32)
            x["log_gate"][n, h, :c] = -torch.rand(c, generator=g) * 4
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert N * Hkv * (K + 1) >= 10 * 10 * sms
    _check(_run(x), _ref(x))


@pytest.mark.parametrize("Hq,Hkv,N,K", [
    # one slot for each warp of a cluster of 32, 24, 16, 12, 8, 6, 4 and 3 warps; an empty selection
    (32, 8, 6, 31), (8, 8, 1, 20), (8, 8, 12, 15), (8, 4, 2, 10), (28, 4, 1, 7), (4, 4, 1, 5), (5, 1, 1, 3), (7, 1, 2, 1),
    (6, 2, 3, 0),
    # more slots than warps; a second wave of clusters
    (8, 8, 6, 32), (32, 8, 7, 31), (8, 1, 48, 5), (8, 1, 49, 5), (16, 8, 16, 20), (8, 8, 20, 18), (8, 8, 30, 13),
    (16, 8, 40, 9), (8, 8, 96, 5), (8, 8, 130, 5),
    # the device's ranges: few items with many slots, odd waves
    (8, 8, 2, 40), (8, 8, 75, 6), (8, 8, 75, 24)])
def test_every_way_to_cut_the_work(Hq, Hkv, N, K):
    x = _make([(2100 + 300 * n) % 2600 for n in range(N)], Hq, Hkv, K, seed=30 + N + K)
    _check(_run(x), _ref(x))


@pytest.mark.parametrize("N,Hq,Hkv,K", [(3, 24, 8, 620), (1, 8, 8, 1900), (3, 16, 8, 300), (2, 2, 1, 700)])
def test_few_items_with_many_slots(N, Hq, Hkv, K):
    """Fewer than 28 items: the device's ranges, up to 25 slots long. The sequences share pages."""
    x = _make([64 * 20] * N, Hq, Hkv, 0, seed=40)
    g = torch.Generator().manual_seed(41)
    P, blocks = x["k_cache"].shape[0], K + 40
    x["page_table"] = torch.randint(0, P, (N, blocks + 1), generator=g, dtype=torch.int32)
    x["kv_len"] = torch.tensor([64 * blocks + 9 + n for n in range(N)], dtype=torch.int32)
    x["cnt"] = torch.full((N, Hkv), K, dtype=torch.int32)
    x["idx"] = torch.stack([torch.randperm(blocks, generator=g)[:K].sort().values for _ in range(N * Hkv)])
    x["idx"] = x["idx"].view(N, Hkv, K).to(torch.int32)
    x["log_gate"] = -torch.rand((N, Hkv, K), generator=g) * 4
    _check(_run(x), _ref(x))


def test_all_history_of_a_long_sequence():
    x = _make([64 * 300 + 5], 8, 2, 300, seed=5)
    _check(_run(x, sm_scale=0.03), _ref(x, 0.03))


def test_scales_far_apart():
    """Pages whose value scales differ by 2^30, query rows of very different sizes, and scales that are no
    power of two."""
    x = _make([64 * 6 + 3, 200], 8, 2, 4, seed=6)
    g = torch.Generator().manual_seed(7)
    x["v_scale"] = x["v_scale"] * torch.randint(-30, 1, x["v_scale"].shape, generator=g).float().exp2()
    x["k_scale"] = x["k_scale"] * (0.5 + torch.rand(x["k_scale"].shape, generator=g))
    x["q"] = (x["q"].float() * torch.randint(-20, 3, (2, 8, 1), generator=g).float().exp2()).to(torch.bfloat16)
    _check(_run(x), _ref(x))


def test_rows_past_the_end_and_unused_pages_do_not_matter():
    """NaN codes behind the last token and in pages that are not kept, NaN scales of those pages."""
    x = _make([64 * 5 + 9], 4, 1, 2, seed=8)
    ref = _run(x)
    nan = torch.tensor(float("nan")).to(F8)
    used = {int(x["page_table"][0, j]) for j in x["idx"][0, 0].tolist()} | {int(x["page_table"][0, 5])}
    for c in ("k_cache", "v_cache"):
        raw = x[c].view(torch.uint8)
        raw[int(x["page_table"][0, 5]), :, 9:] = nan.view(torch.uint8)
        for p in range(6):
            if p not in used:
                raw[p] = nan.view(torch.uint8)
    for s in ("k_scale", "v_scale"):
        for p in range(6):
            if p not in used:
                x[s][p] = float("nan")
    out = _run(x)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


def test_gates_that_close_blocks():
    """A gate of -inf or of the type's lowest value removes its block; a large one takes all."""
    x = _make([64 * 4 + 20], 4, 1, 3, seed=9)
    x["log_gate"][0, 0] = torch.tensor([-math.inf, torch.finfo(torch.float32).min, -1.0])
    y = {k: v.clone() for k, v in x.items()}
    y["idx"][0, 0] = torch.tensor([int(x["idx"][0, 0, 2]), -1, -1])
    y["log_gate"][0, 0] = torch.tensor([-1.0, -math.inf, -math.inf])
    y["cnt"][0, 0] = 1
    _check(_run(x), _ref(y))


def test_a_closed_block_is_left_out_whatever_it_holds():
    x = _make([300, 450, 200], 4, 2, 3, seed=12)
    x["log_gate"][1, :, 1] = -math.inf
    x["log_gate"][2] = -math.inf
    x["log_gate"][2, :, 1] = torch.finfo(torch.float32).min
    want = _run(x)
    y = dict(x, log_gate=x["log_gate"].clone())
    y["log_gate"][2] = -math.inf
    _check(want, _ref(y))
    for n, i in ((1, 1), (2, 0), (2, 1), (2, 2)):
        for h in range(2):
            page = int(x["page_table"][n, x["idx"][n, h, i]])
            for cache in ("k_cache", "v_cache"):
                x[cache].view(torch.uint8)[page, h, 5:40] = 0x7f          # NaN
    got = _run(x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_block_named_twice_counts_twice():
    x = _make([400, 1000], 8, 2, 4, seed=13)
    x["idx"][:, :, 2] = x["idx"][:, :, 1]
    x["log_gate"][:, :, 2] = x["log_gate"][:, :, 1] - 0.5
    _check(_run(x), _ref(x))


def test_nan_in_a_query_or_a_key_reaches_its_rows_only():
    x = _make([64 * 3 + 1, 64 * 3 + 1], 8, 2, 3, seed=10)
    ref = _ref(x)
    x["q"][0, 2, 7] = float("nan")
    raw = x["k_cache"].view(torch.uint8)
    raw[int(x["page_table"][1, 1]), 1, 5, 3] = 0x7f
    o, lse = _run(x)
    bad = torch.zeros((2, 8), dtype=torch.bool)
    bad[0, 2] = True
    bad[1, 4:] = True
    assert torch.equal(o.isnan().all(-1).cpu(), bad) and torch.equal(lse.isnan().cpu(), bad)
    keep = ~bad.numpy()
    assert np.all(np.abs(R.f64(o) - ref[0])[keep] <= ref[2][keep])


def test_bad_pages_scales_and_lengths_are_skipped():
    x = _make([64 * 3 + 2, 64 * 3 + 2, 64 * 3 + 2, 70, 64 * 2 + 1], 4, 2, 3, seed=11)
    sas.get_error_flag()
    y = {k: v.clone() for k, v in x.items()}
    P = x["k_cache"].shape[0]
    y["page_table"][0, 1] = P                       # a page id outside the cache
    y["k_scale"][int(x["page_table"][1, 0])] = 0.0  # scales without a value
    y["v_scale"][int(x["page_table"][1, 2])] = math.inf
    y["idx"][2, 0, 0] = 3                           # not a history block
    y["kv_len"][3] = 64 * 4 + 1                     # longer than the page table
    out = _run(y, flag=True)
    z = {k: v.clone() for k, v in x.items()}

    def keep(n, h, left):
        z["idx"][n, h] = torch.tensor((left + [-1] * 3)[:3])
        z["log_gate"][n, h] = torch.tensor([float(x["log_gate"][n, h, i]) for i in left] + [-math.inf] * (3 - len(left)))
        z["cnt"][n, h] = len(left)

    for h in range(2):
        keep(0, h, [0, 2])
        keep(1, h, [1])
    keep(2, 0, [1, 2])
    z["kv_len"][3] = 0
    _check(out, _ref(z))
    # a sequence that keeps nothing readable: o 0, lse -inf
    y = {k: v.clone() for k, v in x.items()}
    y["page_table"][4] = -1
    out = _run(y, flag=True)
    assert torch.all(out[0][4] == 0) and torch.all(out[1][4] == -math.inf)
    y = {k: v.clone() for k, v in x.items()}
    y["cnt"][0, 0], y["cnt"][1, 1] = 9, -2          # counts out of range are clamped
    out = _run(y, flag=True)
    z = {k: v.clone() for k, v in x.items()}
    z["cnt"][1, 1] = 0
    _check(out, _ref(z))


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of the cache (only the pages in use are written)."""
    x = _make([64 * 4 + 30, 64 * 2], 16, 8, 3, seed=12)
    used = x["k_cache"].shape[0]
    P = 70000                                       # 4.6 GB for each cache
    big = {}
    where = torch.linspace(P - 1, 3, used).long()
    for c in ("k_cache", "v_cache"):
        big[c] = torch.empty((P, 8, 64, D), dtype=F8, device="cuda")
        big[c].view(torch.uint8)[where.cuda()] = x[c].view(torch.uint8).cuda()
    for s in ("k_scale", "v_scale"):
        big[s] = torch.zeros((P, 8), device="cuda")
        big[s][where.cuda()] = x[s].cuda()
    rest = {k: v.cuda() for k, v in x.items() if k not in big}
    rest["page_table"] = where.to(torch.int32)[x["page_table"].long()].cuda()
    out = sas.decode_paged_q8(**big, **rest)
    torch.cuda.synchronize()
    sas.get_error_flag()
    _check(out, _ref(x))


@pytest.mark.parametrize("K,none", [(6, True), (40, False)])
def test_repeats_streams_and_graphs(K, none):
    """The same bits every time: on another stream, and from two captured graphs that share a workspace (which
    few block slots do not use)."""
    x = {k: v.cuda() for k, v in _make([64 * 9 + 3, 300, 0, 64 * 50], 8, 2, K, seed=13).items()}
    ws = torch.empty(sas.decode_q8_workspace_bytes(4, 8, 2, D, K), dtype=torch.uint8, device="cuda")
    assert (ws.numel() == 256) == none
    first = sas.decode_paged_q8(**x, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = sas.decode_paged_q8(**x)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sas.decode_paged_q8(**x, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    sas.get_error_flag()
    for other in (second, *outs):
        assert torch.equal(first[0], other[0]) and torch.equal(first[1], other[1])


def test_no_sequences_and_no_lse():
    x = {k: v.cuda() for k, v in _make([70], 4, 2, 1, seed=14).items()}
    o, lse = sas.decode_paged_q8(**x, with_lse=False)
    assert lse is None and torch.equal(o, sas.decode_paged_q8(**x)[0])
    e = {k: (v if k in ("k_cache", "v_cache", "k_scale", "v_scale") else v[:0]) for k, v in x.items()}
    o, lse = sas.decode_paged_q8(**e)
    assert o.shape == (0, 4, D) and lse.shape == (0, 4)
