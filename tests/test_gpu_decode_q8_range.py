"""decode_paged_q8 where the weights and the value scales of an item's blocks lie far apart, against the fp64
reference and its error bounds (oracle/serving_oracle.py, decode_q8)."""
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as R
from tests.test_gpu_decode_q8 import D, _check, _make, _ref, _run
from trainable_gated_block_b200 import build, sas

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    sas.lib()


def shared(N, Hq, Hkv, K, blocks, seed, pages=40):
    """N sequences of `blocks` history blocks that share a few pages; every head keeps K of them, block 0 among
    them, with gates in -4 .. 0. The current blocks hold 20 to 63 tokens."""
    x = _make([64 * pages], Hq, Hkv, 0, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    x["q"] = torch.randn((N, Hq, D), generator=g).to(torch.bfloat16)
    x["page_table"] = torch.randint(0, pages, (N, blocks + 1), generator=g, dtype=torch.int32)
    x["kv_len"] = torch.tensor([64 * blocks + 20 + 7 * n % 44 for n in range(N)], dtype=torch.int32)
    x["cnt"] = torch.full((N, Hkv), K, dtype=torch.int32)
    rest = [1 + torch.randperm(blocks - 1, generator=g)[:K - 1].sort().values for _ in range(N * Hkv)]
    idx = torch.stack([torch.cat((torch.zeros(1, dtype=torch.long), r)) for r in rest])
    x["idx"] = idx.view(N, Hkv, K).to(torch.int32)
    x["log_gate"] = -torch.rand((N, Hkv, K), generator=g) * 4
    return x


def _check_up_to_infinity(out, ref):
    """_check where codes of 448 times 2^120 reach 5.9e38, beyond the largest bf16 value of 3.39e38: a result
    that is surely beyond it is an infinity of its sign, one that may be on either side is so or within its bound."""
    o, (ro, rl, to, tl) = R.f64(out[0]), ref
    top = float(torch.finfo(torch.bfloat16).max)
    inf = np.isinf(o) & (np.sign(o) == np.sign(ro))
    assert np.all(inf[np.abs(ro) - to > top])
    beyond = inf & (np.abs(ro) + to > top)
    assert np.mean(beyond) < 0.01
    _check((torch.from_numpy(np.where(beyond, ro, o)), out[1]), ref)


# one slot for each warp of a cluster; two and three slots for each of a cluster's warps; the device's ranges
CUTS = [(1, 8, 8, 4), (130, 8, 8, 5), (64, 8, 4, 8), (75, 8, 8, 6)]


@pytest.mark.parametrize("N,Hq,Hkv,K", CUTS)
@pytest.mark.parametrize("hi,lo", [(63, -64), (120, -7), (120, -100), (64, -64), (-70, -100)])
def test_value_scales_at_the_ends_of_their_range(N, Hq, Hkv, K, hi, lo):
    """Pages of value scales 2^hi and 2^lo in one item: all of their tokens count in the softmax sum, and each
    page's values in o."""
    x = shared(N, Hq, Hkv, K, K + 3, seed=50 + K)
    big = torch.rand(x["v_scale"].shape, generator=torch.Generator().manual_seed(hi - lo)) < 0.5
    x["v_scale"] = torch.where(big, 2.0 ** hi, 2.0 ** lo).float()
    _check_up_to_infinity(_run(x), _ref(x))


def test_equal_logits_of_two_pages_far_apart():
    """Two blocks of equal logits whose scales differ by 2^127: lse = log 128 and o the mean of all values."""
    x = shared(1, 8, 8, 1, 1, seed=60, pages=2)
    x["q"].zero_()
    x["log_gate"].zero_()
    x["kv_len"][0] = 128
    x["page_table"][0] = torch.tensor([0, 1])
    x["v_scale"][0], x["v_scale"][1] = 2.0 ** 63, 2.0 ** -64
    o, lse = _run(x)
    mean = x["v_cache"][0].double().sum(1) * 2.0 ** 63 / 128
    assert float((lse.cpu() - math.log(128)).abs().max()) <= 1e-5
    assert torch.all((o[0].cpu().double() - mean).abs() <= 2.0 ** -7 * mean.abs() + 2.0 ** 63 * 1e-3)


def test_a_page_with_one_channel_far_out():
    """One page of a range holds a value 2^14 times the others' in one channel; the other blocks are 2^-13 of
    its weight. Their values in the other channels are not lost beside it."""
    x = shared(64, 8, 8, 200, 230, seed=70)
    pages = x["k_cache"].shape[0]
    x["page_table"] = torch.where(x["page_table"] == 0, 1, x["page_table"])
    x["page_table"][:, 0] = 0                       # block 0 of every sequence, and no other
    assert pages == 40 and not bool((x["page_table"][:, 1:] == 0).any())
    x["log_gate"][:, :, 0], x["log_gate"][:, :, 1:] = 0.0, -9.0
    raw = x["v_cache"].float()
    raw[0, :, :, 1:] = 0
    x["v_cache"] = raw.to(x["v_cache"].dtype)
    x["v_scale"][:] = 2.0 ** -8
    x["v_scale"][0] = 2.0 ** 6
    _check(_run(x), _ref(x))


def test_small_weights_beside_one_large():
    """12,800 tokens of weights e^-18 and below behind a block whose values are zero: o is theirs alone."""
    x = shared(64, 8, 8, 200, 230, seed=80)
    x["page_table"][:, 1:] = x["page_table"][:, 1:].clamp(min=1)
    x["page_table"][:, 0] = x["page_table"][:, -1] = 0          # the first kept and the current block
    x["v_cache"].view(torch.uint8)[0] = 0
    x["log_gate"][:, :, 0], x["log_gate"][:, :, 1:] = 0.0, -18.0
    _check(_run(x), _ref(x))


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 1), (10, 2), (8, 1)])
def test_values_that_cancel(Hq, Hkv):
    """Two tokens of nearly equal weights and opposite values: what the weights lose would show in o."""
    x = _make([2] * 64, Hq, Hkv, 0, seed=90)
    x["q"] = x["q"] * 0.005
    raw = (x["v_cache"].view(torch.uint8) | 0x60) & 0x7e            # codes of 32 to 448
    raw[:, :, 1] = raw[:, :, 0] | 0x80
    x["v_cache"] = raw.view(x["v_cache"].dtype)
    _check(_run(x), _ref(x))


def test_a_closed_block_is_left_out_whatever_its_page_and_scales():
    """Behind a gate of -inf or the lowest fp32 value, pages with scales without a value and page ids outside the
    cache are neither read nor flagged."""
    x = _make([64 * 6 + 10, 64 * 5 + 1, 64 * 4], 4, 2, 4, seed=95)
    for n in range(3):
        x["idx"][n, 1], x["cnt"][n, 1] = x["idx"][n, 0], x["cnt"][n, 0]
    low = torch.finfo(torch.float32).min
    x["log_gate"][0, :, 1], x["log_gate"][0, :, 2], x["log_gate"][1, :, 0] = -math.inf, low, low
    x["log_gate"][2, :, :3] = -math.inf
    want = _run(x)
    _check(want, _ref(dict(x, log_gate=torch.where(x["log_gate"] == low, -math.inf, x["log_gate"]))))
    closed = [(0, 1), (0, 2), (1, 0), (2, 0), (2, 1), (2, 2)]
    bad = [0.0, float("nan"), math.inf, -1.0, None, None]
    for (n, i), b in zip(closed, bad):
        block = int(x["idx"][n, 0, i])
        page = int(x["page_table"][n, block])
        if b is None:
            x["page_table"][n, block] = -5 if i == 1 else x["k_cache"].shape[0]
        else:
            x["k_scale"][page], x["v_scale"][page] = b, b
    got = _run(x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("size", [-133, -127, -120, -60, 0, 60, 100])
def test_queries_of_any_size(size):
    """Query rows down to bf16's subnormals beside key scales that make their logits count, and large ones."""
    x = _make([64 * 5 + 3, 200, 64 * 4], 8, 2, 3, seed=97)
    q = torch.randint(-7, 8, x["q"].shape, generator=torch.Generator().manual_seed(98)).double() * 2.0 ** size
    x["q"] = q.to(torch.bfloat16)
    assert torch.equal(x["q"].double(), q)
    x["k_scale"] = x["k_scale"] * 2.0 ** min(max(-size - 2, -90), 125)
    _check(_run(x, sm_scale=0.5), _ref(x, 0.5))
