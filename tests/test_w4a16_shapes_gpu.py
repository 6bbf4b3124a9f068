"""mq_w4a16_linear over the range of its activations and of its launch shapes,
against the fp64 product.

Bound, beside test_w4a16_gpu.py's per output: the root mean square error.  A sum
with an error e is rounded to within |round(y) - y| + 2 |e| of y, so the error's rms
is at most that of rounding the exact product plus 2 rms(e).  e: fp32 sums of a
group's products (for bf16 of terms up to 18 times the codes' own, random signs:
2^-24 * 18 * sqrt(8) additions, some 2^-18 of the sum), of groups and of waves (up
to 2^-24 * sqrt(200)): below 2^-14 of the outputs' rms."""
import numpy as np
import pytest
import torch

import oracle
from dense_sparse_w4a4_amd import ops
from test_w4a16_gpu import DTYPES, _check, _layer, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ops.lib()
    yield
    torch.cuda.synchronize()


def _rms(x):
    top = max(float(np.abs(x).max()), 1e-300)
    return top * float(np.sqrt(np.mean((x / top) ** 2)))


def _check_rms(y, ref, dtype):
    rounded = torch.from_numpy(ref).to(dtype).double().numpy()
    got, best = _rms(y.double().cpu().numpy() - ref), _rms(rounded - ref)
    assert got <= best + 2.0 ** -13 * _rms(ref), (got / _rms(ref), best / _rms(ref))


@pytest.mark.parametrize("M", [1, 9, 40])
@pytest.mark.parametrize("size", [1e-38, 1e-36, 1e33, 1e35, 3e36])
def test_bf16_activations_near_the_smallest_and_largest(M, size):
    """Finite activations to some 3e38, whose outputs are inside bf16's range, and
    subnormal ones."""
    layer, packed = _layer(512, 512, 64, 0.1)
    x = (_x(M, 512, torch.float32, 8) * size).clamp(-3e38, 3e38).to(torch.bfloat16)
    y = ops.w4a16_linear(x.cuda(), layer)
    _check(y, x, packed, torch.bfloat16)
    _check_rms(y, oracle.w4a16_reference(x.double().numpy(), packed), torch.bfloat16)


def test_host_layers_and_workspaces_are_refused():
    layer, _ = _layer(512, 512, 64, 0.1)
    host = ops.PackedLayer(layer.N, layer.K, layer.block, layer.qw.cpu(), layer.sw.cpu(), layer.row_ptr, layer.col_idx,
                           layer.qr, layer.sr)
    x = _x(4, 512, torch.float16).cuda()
    with pytest.raises(ValueError, match="device tensors"):
        ops.w4a16_linear(x, host)
    # (a layer of zeros whose inputs are split over workgroups, so that one is needed)
    N, K, M = 4096, 8192, 16
    need = ops.w4a16_linear_workspace(M, N, K)
    assert need > 0
    zeros = ops.PackedLayer(N, K, 64, torch.zeros((N // 16, K // 128, 64, 16), dtype=torch.uint8, device="cuda"),
                            torch.zeros((N, K // 128), dtype=torch.float16, device="cuda"),
                            *(layer.row_ptr[:0], layer.col_idx[:0], layer.qr[:0], layer.sr[:0]))
    x = _x(M, K, torch.float16).cuda()
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for bad in (torch.empty(need, dtype=torch.uint8), one.expand(need), torch.zeros(2 * need, dtype=torch.uint8,
                                                                                     device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            ops.w4a16_linear(x, zeros, workspace=bad)
    assert not ops.w4a16_linear(x, zeros, workspace=one).any()  # too small: one of its own
