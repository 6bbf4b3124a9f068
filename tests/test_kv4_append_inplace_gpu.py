"""mq_kv4_append with the queries written over themselves, where the other half of
a rotated pair is loaded again from the same memory."""
import numpy as np
import pytest
import torch

from dense_sparse_w4a4_amd import ops
from test_kv4_gpu import _assert_append, _table, _to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ops.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 32), (64, 48), (128, 16), (128, 64), (128, 96), (128, 112)])
def test_queries_in_place_with_some_channels_rotated(D, rot, norm, inter, dtype):
    """Views of one projection's output, bit for bit against the oracle."""
    rng = np.random.default_rng([D, rot])
    T, hq, hk = 41, 6, 2
    qkv = _to(rng.standard_normal((T, (hq + 2 * hk) * D)), dtype).cuda()
    q = qkv[:, :hq * D].view(T, hq, D)
    k = qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
    v = qkv[:, (hq + hk) * D:].view(T, hk, D)
    w = [_to(0.5 + rng.random(D), dtype).cuda() for _ in range(2)] if norm else (None, None)
    cache = ops.kv4_cache(3, 32, hk, D)
    _assert_append(cache, q, k, v, rng.permutation(96)[:T].tolist(), rng.integers(0, 90, T), _table(90, rot), w[0], w[1],
                   inter, q_out=q)
