"""CPU pins of the fp64 reference of the operators around the attention calls."""
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as R
from trainable_gated_block_b200 import sas


def test_norm_rope_gradient_against_differences():
    rng = np.random.default_rng(0)
    T, H, D, eps = 3, 2, 8, 1e-3
    x, dy, w = rng.normal(size=(T, H, D)), rng.normal(size=(T, H, D)), rng.normal(size=D)
    table = sas.rope_table(16, D, base=100.0, device="cpu")
    pos = np.array([0, 15, 7])
    dx, dw, _, _ = R.norm_rope_bwd(dy, x, w, table, pos, eps)

    def loss(x, w):
        return float((R.norm_rope(x, w, table, pos, eps)[0] * dy).sum())

    h = 1e-6
    for i in np.ndindex(T, H, D):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) <= 1e-7
    for i in range(D):
        e = np.zeros(D)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) <= 1e-7


def test_rotation_keeps_norms_and_relative_positions():
    rng = np.random.default_rng(1)
    D = 64
    table = sas.rope_table(2000, D, device="cpu")
    a, b = rng.normal(size=(1, 1, D)), rng.normal(size=(1, 1, D))
    dots = []
    for p in (0, 5, 1000):
        ra, rb = R.rotate(a, table, [p + 17]), R.rotate(b, table, [p])
        assert abs(np.linalg.norm(ra) / np.linalg.norm(a) - 1) <= 1e-6
        dots.append(float((ra * rb).sum()))
    assert max(dots) - min(dots) <= 1e-5 * np.linalg.norm(a) * np.linalg.norm(b)
    ref = R.rotate(R.rotate(a, table, [9]), table, [9], sign=-1.0)
    assert np.abs(ref - a).max() <= 1e-6


def test_rope_table_far_positions():
    t = sas.rope_table(1 << 20, 4, base=1e6, device="cpu")
    p = (1 << 20) - 1
    for i, f in enumerate((1.0, 1e6 ** -0.5)):
        assert abs(float(t[p, i]) - math.cos(p * f)) <= 1e-7
        assert abs(float(t[p, 2 + i]) - math.sin(p * f)) <= 1e-7


@pytest.mark.parametrize("amax,exp", [(448.0, 0), (448.0001, 1), (224.0, -1), (1.75, -8), (1.76, -7), (0.0, -64),
                                      (1e-30, -64), (3.3e38, 120)])
def test_scale_of(amax, exp):
    assert R.scale_of(amax) == 2.0 ** exp
    if exp > -64:
        assert amax <= 448 * 2.0 ** exp and amax > 448 * 2.0 ** (exp - 1)


def test_decode_q8_equals_decode_of_the_values():
    g = torch.Generator().manual_seed(2)
    N, Hq, Hkv, D, P, K = 2, 4, 2, 16, 6, 2
    q = torch.randn((N, Hq, D), generator=g)
    kc, vc = (torch.randn((P, Hkv, 64, D), generator=g) for _ in range(2))
    ks, vs = (torch.rand((P, Hkv), generator=g) + 0.5 for _ in range(2))
    pt = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32)
    kv = torch.tensor([150, 64 + 1], dtype=torch.int32)
    idx = torch.tensor([[[0, 1], [1, -1]], [[0, -1], [-1, -1]]], dtype=torch.int32)
    cnt = torch.tensor([[2, 1], [1, 0]], dtype=torch.int32)
    gate = -torch.rand((N, Hkv, K), generator=g)
    o, lse, _, _ = R.decode_q8(q, kc, vc, ks, vs, pt, kv, idx, cnt, gate, 0.25)
    ro, rl = R.O.decode(q.double(), kc.double() * ks[:, :, None, None].double(),
                        vc.double() * vs[:, :, None, None].double(), pt, kv, idx, cnt, gate, 0.25)
    assert np.abs(o - ro).max() <= 1e-12 and np.abs(lse - rl).max() <= 1e-12
