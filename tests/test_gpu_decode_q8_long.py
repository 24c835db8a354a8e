"""decode_paged_q8 with more slots for a warp than it resolves at a time (32) and than its list holds (64), on the
clusters and on the device's ranges, with batches of slots that hold nothing."""
import math

import pytest
import torch

from tests.test_gpu_decode_q8 import _check, _ref, _run
from tests.test_gpu_decode_q8_range import shared
from trainable_gated_block_b200 import build, sas

pytestmark = pytest.mark.gpu
CLUSTER_WARPS = (32, 24, 16, 12, 8, 6, 4, 3)     # of an item


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    sas.lib()


def _slots_of_a_warp(N, Hq, Hkv, K):
    """The fewest slots that the longest stream of a warp can have, by what the workspace says of the way taken."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sas.decode_q8_workspace_bytes(N, Hq, Hkv, 128, K) == 256:
        # clusters: resident together as far as that goes, twelve warps an SM
        warps = next((w for w in CLUSTER_WARPS if N * Hkv * w <= 12 * sms), CLUSTER_WARPS[-1])
        return -(-(K + 1) // warps)
    slots = N * Hkv * (K + 1)
    return -(-slots // ((4 if slots <= 32 * 4 * sms else 10) * sms))        # ranges of four or of ten warps an SM


@pytest.mark.parametrize("N,Hq,Hkv,K,ranges,fewest", [
    (75, 8, 8, 30, True, 32), (2, 16, 8, 1180, True, 32),       # ranges of four warps: one full batch
    (75, 8, 8, 66, True, 27), (75, 32, 8, 70, True, 27),        # of ten warps, over the ends of items
    (75, 40, 8, 170, True, 65), (3, 8, 8, 4100, True, 65),      # the same, within an item
    (64, 8, 8, 330, False, 65), (64, 40, 8, 290, False, 65),    # three warps an item
    (8, 32, 8, 2100, False, 65),                                # 24 warps an item
    (24, 16, 8, 530, False, 65)])                               # eight
def test_many_slots_a_warp(N, Hq, Hkv, K, ranges, fewest):
    x = shared(N, Hq, Hkv, K, K + 40, seed=N + K)
    assert (sas.decode_q8_workspace_bytes(N, Hq, Hkv, 128, K) != 256) == ranges
    assert _slots_of_a_warp(N, Hq, Hkv, K) >= fewest
    rows = _some(N, 6)
    _check_rows(x, rows)


@pytest.mark.parametrize("N,Hq,Hkv,K", [(75, 8, 8, 200), (64, 8, 8, 500)])
def test_batches_of_slots_that_hold_nothing(N, Hq, Hkv, K):
    """Whole batches of slots without an entry: short selections, padding entries, sequences of one token and
    selections whose gates are closed, among others of full length."""
    x = shared(N, Hq, Hkv, K, K + 40, seed=N)
    for n in range(N):
        kind = n % 5
        if kind == 1:
            x["kv_len"][n], x["cnt"][n] = 0, 0
        elif kind == 2:
            x["kv_len"][n], x["cnt"][n] = 1 + n % 64, 0
        elif kind == 3:
            x["cnt"][n] = n % 70
        elif kind == 4:
            x["log_gate"][n, :, 5:K - 3] = -math.inf
    for n in range(N):
        c = int(x["cnt"][n, 0])
        x["idx"][n, :, c:], x["log_gate"][n, :, c:] = -1, -math.inf
    _check_rows(x, sorted(set(_some(N, 6)) | {0, 1, 2, 3, 4}))


def _some(N, k):
    return sorted({round(i * (N - 1) / (k - 1)) for i in range(k)})


def _check_rows(x, rows):
    """All sequences run, these are compared (the reference takes its time)."""
    o, lse = _run(x)
    at = torch.tensor(rows)
    part = {k: (v if k in ("k_cache", "v_cache", "k_scale", "v_scale") else v[at]) for k, v in x.items()}
    _check((o.cpu()[at], lse.cpu()[at]), _ref(part))
