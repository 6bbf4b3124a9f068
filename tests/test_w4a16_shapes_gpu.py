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


_made = {}


def _random_layer(N, K, b):
    """A layer of random codes (a tenth of its blocks as residual), its fp64 weights
    and, per input, its rows' scales, on the device."""
    if (N, K, b) not in _made:
        _made.clear()
        torch.cuda.empty_cache()
        g = torch.Generator(device="cuda").manual_seed(N + K + b)
        signed = lambda p: (torch.stack([p & 15, p >> 4], -1).flatten(-2).long() + 8) % 16 - 8  # noqa: E731

        def codes(*shape):
            return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
        qw = codes(N // 16, K // 128, 64, 16)
        sw = (0.004 + 0.004 * torch.rand((N, K // 128), device="cuda", generator=g)).half()
        grid = torch.rand((N // b, K // b), device="cuda", generator=g) < 0.1
        rows, cols = grid.nonzero(as_tuple=True)
        row_ptr = torch.zeros(N // b + 1, dtype=torch.int32, device="cuda")
        row_ptr[1:] = grid.sum(1).cumsum(0)
        qr = codes(len(rows), b, b // 2)
        sr = (0.001 * torch.rand((len(rows), b), device="cuda", generator=g)).half()
        # lane (r, c) of a slab holds channel r's inputs 32 c .. 32 c + 31 of a group
        q = qw.view(N // 16, K // 128, 4, 16, 16).permute(0, 3, 1, 2, 4).reshape(N, K // 2)
        scale = sw.double().repeat_interleave(128, 1)
        w = signed(q).double() * scale
        at = lambda t: t.view(N // b, b, K // b, b)  # noqa: E731
        at(w)[rows, :, cols] += signed(qr).double() * sr.double()[..., None]
        at(scale)[rows, :, cols] += sr.double()[..., None]
        layer = ops.PackedLayer(N, K, b, qw, sw, row_ptr, cols.int(), qr, sr)
        _made[N, K, b] = layer, w, scale
    return _made[N, K, b]


def _check_random(y, x, made, dtype):
    layer, w, scale = made
    x64 = x.double().cuda()
    ref = x64 @ w.t()
    mag = x64.abs() @ w.abs().t() if dtype == torch.float16 else 2 * 144 * (x64.abs() @ scale.t())
    out = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    tol = out * ref.abs() + (128 + layer.K // 128 + 16) * 2.0 ** -23 * mag + 2.0 ** -24
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst err/tol {float((err / tol).max()):.3f}"
    _check_rms(y, ref.cpu().numpy(), dtype)


# (M, N, K, block, whether the inputs are split over workgroups): every launch shape
# that layers of N 4096 .. 51200 and K 4096 .. 25600 get for 1 .. 4096 tokens, at
# smaller sizes.  Token tiles, slabs, waves of a workgroup:
SHAPES = [
    (2, 2048, 4096, 64, False),      # 1, 1, 8, activations read by the operand
    (3, 8192, 4096, 128, False),     # 1, 2, 8
    (1, 8192, 4096, 32, False),
    (4, 16384, 1024, 32, False),     # 1, 2, 4
    (2, 16384, 512, 64, False),      # 1, 4, 4
    (7, 2048, 4096, 64, False),      # 1, 1, 8, activations through LDS from here on
    (20, 6144, 4096, 64, False),     # 1, 2, 8
    (9, 8192, 4096, 32, False),
    (33, 6144, 1024, 32, False),     # 1, 2, 4
    (9, 16384, 512, 64, False),      # 1, 4, 4
    (9, 8192, 2048, 64, False),      # 1, 4, 8
    (16, 4096, 8192, 128, True),
    (5, 4096, 12288, 64, True),
    (20, 16384, 2048, 32, False),    # 2, 2, 4
    (20, 8192, 4096, 32, False),     # 2, 2, 8
    (20, 8192, 2048, 64, False),     # 2, 4, 8
    (17, 4096, 8192, 64, True),
    (32, 4096, 12288, 128, True),
    (200, 8192, 2048, 32, False),    # 4, 2, 4
    (40, 8192, 4096, 32, False),     # 4, 2, 8
    (50, 8192, 2048, 128, False),    # 4, 4, 8
    (1025, 4096, 2048, 64, False),
    (100, 2048, 8192, 64, True),
    (33, 4096, 12288, 64, True),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K,b,split", SHAPES)
def test_every_launch_shape(M, N, K, b, split, dtype):
    made = _random_layer(N, K, b)
    assert (ops.w4a16_linear_workspace(M, N, K) > 0) == split
    x = _x(M, K, dtype, 9)
    _check_random(ops.w4a16_linear(x.cuda(), made[0]), x, made, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("M", [16, 20, 50])
def test_split_inputs_given_workspace_strided_output_and_graph(M, dtype):
    """Whatever the workspace holds, rows apart, repeats and graph replays: the
    same bits."""
    N, K = 4096, 8192
    made = _random_layer(N, K, 64)
    need = ops.w4a16_linear_workspace(M, N, K)
    assert need > 0
    x = _x(M, K, dtype, 10)
    xs = x.cuda()
    want = ops.w4a16_linear(xs, made[0])
    _check_random(want, x, made, dtype)
    wide = torch.full((M, N + 256), 7.0, dtype=dtype, device="cuda")
    out = wide[:, 128:128 + N]
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    same = lambda: torch.equal(out.contiguous().view(torch.int16), want.view(torch.int16))  # noqa: E731
    ops.w4a16_linear(xs, made[0], out=out, workspace=ws)
    assert same() and bool((wide[:, :128] == 7).all()) and bool((wide[:, 128 + N:] == 7).all())
    assert bool((ws[need:] == 255).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.w4a16_linear(xs, made[0], out=out, workspace=ws)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same()
        assert torch.equal(ops.w4a16_linear(xs, made[0]).view(torch.int16), want.view(torch.int16))
