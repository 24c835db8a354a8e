"""qk_norm_rope and its gradient through the C ABI against the fp64 reference.

Tolerances (u = 2^-24, half a step of fp32; h = half a step of the output type, 2^-24 or 2^-8 relative):
* outputs: h |y| + 24 u (|a| + |b|), a and b the rotation pair. The sum of squares has 16 terms in a
  lane and 3 exchanges (19 roundings, half of them in the root), the mean and eps add one, rsqrtf is
  within 2 ulp (4 u), the two products and the rotation 2 each: under 18 u.
* dq, dk: h |dx| + 80 u M, M the same expression on magnitudes: 1/rms and the normalised value carry 15 u
  each, the dot product 39 u, its product with the value 16 more.
* weight gradients: (17 + adds) u times the sum of the terms' magnitudes; a sum passes at most `adds`
  additions (4 in a unit, the units of a slot, the slots of a CTA, the CTAs).
"""
import math

import numpy as np
import pytest
import torch

from oracle import sas_oracle as O
from oracle import serving_oracle as R
from tests.parity_util import check_grad, check_out
from trainable_gated_block_b200 import build, inputs, sas

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6
DTYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f32": (torch.float32, U)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    sas.lib()


def _make(dtype, D, shape, Hq, Hkv, seed, fused=True, max_pos=70000, scale=1.0):
    dt = DTYPES[dtype][0]
    g = torch.Generator().manual_seed(seed)
    T = math.prod(shape)
    qkv = (torch.randn((T, (Hq + 2 * Hkv) * D), generator=g) * scale).to(dt)
    q, k, _ = qkv.split((Hq * D, Hkv * D, Hkv * D), dim=1)
    q, k = q.view(*shape, Hq, D), k.view(*shape, Hkv, D)
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt) for _ in range(2)]
    dq, dk = (torch.randn(t.shape, generator=g).to(dt) for t in (q, k))
    pos = torch.randint(0, max_pos, shape, generator=g, dtype=torch.int32)
    return q, k, w, dq, dk, pos


def _strided(t):
    """t on the GPU with its strides (parts of one projection's output)."""
    base = t.as_strided((t.untyped_storage().nbytes() // t.element_size(),), (1,), 0).cuda()
    return base.as_strided(t.shape, t.stride(), t.storage_offset())


def _check(got, ref, tol, what):
    err = np.abs(R.f64(got) - ref)
    assert np.all(np.isfinite(R.f64(got))), what
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {float((err - tol).max()):.3e} over"


def _adds(T, H, D):
    slots = 256 // (D // 16)
    units = T * -(-H // 4)
    return 4 + max(1, math.ceil(units / slots)) + slots + 64


def _compare(dtype, D, shape, Hq, Hkv, table, x, weights=True, positions=True, adds=None):
    q, k, w, dq, dk, pos = x
    h = DTYPES[dtype][1]
    T = math.prod(shape)
    wq, wk = w if weights else (None, None)
    p = pos if positions else None
    qd, kd = _strided(q), _strided(k)
    wd = [None if t is None else t.cuda() for t in (wq, wk)]
    pd = None if p is None else p.cuda()
    y = sas.qk_norm_rope(qd, kd, table, *wd, positions=pd, eps=EPS)
    grads = sas.qk_norm_rope_bwd(dq.cuda(), dk.cuda(), qd, kd, table, *wd, positions=pd, eps=EPS)
    torch.cuda.synchronize()
    sas.get_error_flag()
    at = (p if p is not None else torch.arange(shape[-1]).expand(shape)).reshape(-1).numpy()
    tab = table.cpu()
    for i, (t, up, wt, H) in enumerate(((q, dq, wq, Hq), (k, dk, wk, Hkv))):
        name = "qk"[i]
        rows = t.reshape(T, H, D)
        ref, pair = R.norm_rope(rows, wt, tab, at, EPS)
        assert y[i].is_contiguous() and y[i].shape == t.shape
        _check(y[i].reshape(T, H, D), ref, h * np.abs(ref) + 24 * U * pair, name)
        dx, dw, mag, wmag = R.norm_rope_bwd(up.reshape(T, H, D), rows, wt, tab, at, EPS)
        _check(grads[i].reshape(T, H, D), dx, h * np.abs(dx) + 80 * U * mag, "d" + name)
        if weights:
            _check(grads[2 + i], dw, (17 + (adds or _adds(T, H, D))) * U * wmag, f"d{name}_weight")
        else:
            assert grads[2 + i] is None
    return y, grads


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("shape,Hq,Hkv", [((1,), 2, 1), ((5,), 32, 8), ((67,), 40, 8), ((2, 33), 5, 5), ((3, 1), 3, 1),
                                          ((1, 130), 8, 2), ((1031,), 1, 1), ((2, 300), 9, 3)])
def test_against_reference(dtype, D, shape, Hq, Hkv):
    table = sas.rope_table(70000, D)
    x = _make(dtype, D, shape, Hq, Hkv, seed=math.prod(shape) + D + Hq)
    _compare(dtype, D, shape, Hq, Hkv, table, x)


@pytest.mark.parametrize("dtype,D,shape,fused,weights,positions", [
    ("bf16", 128, (2, 77), True, True, False), ("f32", 64, (50,), False, True, False),
    ("bf16", 64, (90,), True, False, True), ("f32", 128, (1, 40), False, False, False)])
def test_without_positions_or_weights(dtype, D, shape, fused, weights, positions):
    table = sas.rope_table(max(shape) if not positions else 70000, D)
    x = _make(dtype, D, shape, 4, 2, seed=9, fused=fused)
    _compare(dtype, D, shape, 4, 2, table, x, weights=weights, positions=positions)


@pytest.mark.parametrize("dtype,D,T,Hq,Hkv", [("bf16", 64, 9001, 12, 4), ("bf16", 128, 4001, 40, 8),
                                              ("f32", 128, 1601, 40, 8)])
def test_many_tokens_use_every_cta(dtype, D, T, Hq, Hkv):
    """More units than the resident CTAs hold at a time; the last two are beyond eight for each row slot, where
    a CTA does query and key units. Additions of a weight gradient's sum: at most 4 in a unit, 20 units of a
    slot, 64 slots, 32 in each of the last two steps."""
    table = sas.rope_table(70000, D)
    x = _make(dtype, D, (T,), Hq, Hkv, seed=5)
    _compare(dtype, D, (T,), Hq, Hkv, table, x, adds=4 + 20 + 64 + 64)


def test_extreme_rows():
    """Zero rows, tiny and large ones: eps bounds the first, the norm removes the size of the others."""
    table = sas.rope_table(70000, 128)
    q, k, w, dq, dk, pos = _make("f32", 128, (6,), 4, 4, seed=6, fused=False)
    q[0], q[1], q[2] = 0, q[1] * 1e-12, q[2] * 1e12
    k[3] = 0
    _compare("f32", 128, (6,), 4, 4, table, (q, k, w, dq, dk, pos))


def test_nan_stays_in_its_row():
    table = sas.rope_table(64, 128)
    q, k, w, dq, dk, _ = _make("bf16", 128, (7,), 4, 2, seed=7, fused=False)
    clean = sas.qk_norm_rope(q.cuda(), k.cuda(), table, w[0].cuda(), w[1].cuda())
    q[3, 2, 5] = float("nan")
    q[4, 1, 0] = float("inf")
    y, yk = sas.qk_norm_rope(q.cuda(), k.cuda(), table, w[0].cuda(), w[1].cuda())
    bad = torch.zeros((7, 4), dtype=torch.bool)
    bad[3, 2] = bad[4, 1] = True
    got = ~torch.isfinite(y).all(-1).cpu()
    assert torch.equal(got, bad) and torch.equal(yk, clean[1])
    assert torch.equal(y[~bad.cuda()], clean[0][~bad.cuda()])


def test_positions_outside_the_table_are_flagged():
    table = sas.rope_table(10, 64)
    q, k, w, dq, dk, _ = (t for t in _make("f32", 64, (4,), 3, 1, seed=8, fused=False))
    pos = torch.tensor([3, 10, -1, 9], dtype=torch.int32)
    args = [q.cuda(), k.cuda(), table, w[0].cuda(), w[1].cuda()]
    sas.get_error_flag()
    y, yk = sas.qk_norm_rope(*args, positions=pos.cuda())
    with pytest.raises(sas.SasError):
        sas.get_error_flag()
    g = sas.qk_norm_rope_bwd(dq.cuda(), dk.cuda(), *args, positions=pos.cuda())
    with pytest.raises(sas.SasError):
        sas.get_error_flag()
    for t in (y, yk, g[0], g[1]):
        assert torch.all(t[1:3] == 0) and torch.all(t[[0, 3]].abs().amax((1, 2)) > 0)
    keep = [0, 3]
    ref = sas.qk_norm_rope_bwd(dq[keep].cuda(), dk[keep].cuda(), q[keep].cuda(), k[keep].cuda(), *args[2:],
                               positions=pos[keep].cuda())
    for a, b in ((g[2], ref[2]), (g[3], ref[3])):               # flagged rows add nothing
        assert float((a - b).abs().max()) <= 16 * U * float(b.abs().max() + 16)


def test_no_tokens():
    table = sas.rope_table(4, 128)
    e = torch.empty((0, 4, 128), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(128, device="cuda", dtype=torch.bfloat16)
    y = sas.qk_norm_rope(e, e, table, w, w)
    assert y[0].shape == e.shape
    g = sas.qk_norm_rope_bwd(e, e, e, e, table, w, w)
    assert torch.all(g[2] == 0) and torch.all(g[3] == 0)
    assert sas.qk_norm_rope_bwd(e, e, e, e, table)[2] is None


def test_repeats_are_equal_and_other_streams_and_graphs_work():
    table = sas.rope_table(4096, 128)
    q, k, w, dq, dk, _ = (t for t in _make("bf16", 128, (2, 2000), 8, 2, seed=10, fused=False))
    args = [q.cuda(), k.cuda(), table, w[0].cuda(), w[1].cuda()]
    up = [dq.cuda(), dk.cuda()]

    def call():
        return (*sas.qk_norm_rope(*args), *sas.qk_norm_rope_bwd(*up, *args))

    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = call()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_training_chain_against_reference():
    """norm + rotation, select, attention, its backward, the gradient of norm + rotation: the whole chain from
    the projections' outputs to their gradients, against the fp64 chain on the same inputs."""
    B, S, Hq, Hkv, D, K = 1, 320, 4, 2, 128, 2
    NQB = S // 64
    q, k, w, do, _, _ = _make("bf16", D, (B, S), Hq, Hkv, seed=11)
    g = torch.Generator().manual_seed(12)
    v = torch.randn((B, S, Hkv, D), generator=g).to(torch.bfloat16)
    s = torch.randn((B, Hkv, NQB, NQB), generator=g)
    table = sas.rope_table(S, D)
    sc = 1.0 / math.sqrt(D)
    qd, kd, wd = _strided(q), _strided(k), [t.cuda() for t in w]
    qr, kr = sas.qk_norm_rope(qd, kd, table, *wd)
    sel = sas.select(s.cuda(), K)
    o, lse = sas.attn_fwd(qr, kr, v.cuda(), *sel[:3], sc)
    dqr, dkr, dv, ds = sas.attn_bwd(qr, kr, v.cuda(), o, do.cuda(), lse, s.cuda(), sel[3], *sel[:3], sc)
    dq, dk, dwq, dwk = sas.qk_norm_rope_bwd(dqr, dkr, qd, kd, table, *wd)
    torch.cuda.synchronize()
    sas.get_error_flag()
    pos, tab = np.arange(S), table.cpu()
    rq = R.norm_rope(q[0], w[0], tab, pos, EPS)[0][None]
    rk = R.norm_rope(k[0], w[1], tab, pos, EPS)[0][None]
    idx, cnt, lg, _ = O.select(s, K, O.prefill_history(NQB))
    ro, _ = O.attn_fwd(rq, rk, v, idx, cnt, lg, sc)
    rdq, rdk, rdv, rds, _ = O.attn_bwd(rq, rk, v, do, idx, cnt, lg, s, sc)
    check_out(o, ro, "bf16", "chain o")
    gq, gwq, _, _ = R.norm_rope_bwd(rdq[0], q[0], w[0], tab, pos, EPS)
    gk, gwk, _, _ = R.norm_rope_bwd(rdk[0], k[0], w[1], tab, pos, EPS)
    for a, b, what in ((dq[0], gq, "dq"), (dk[0], gk, "dk"), (dwq, gwq, "dq_weight"), (dwk, gwk, "dk_weight"),
                       (dv, rdv, "dv"), (ds, rds, "ds")):
        check_grad(a, b, "bf16", "chain " + what)
