"""Attention over the 4-bit cache where masks, scales and zero points go to
their limits: what a row does not see has no effect on it, whatever its bits.

Bounds, beside test_kv4_gpu.py's: a value is s (u - 8) + s (z + 8), two fp32
sums that may cancel.  Each addition (one per 32 tokens, and as many again where
waves and parts are joined) may be off by 2^-24 of a partial sum, at most 8 + Z
times S = sum p s / sum p for zero points with |z + 8| <= Z, so 2^-23 (8 + Z) S
for both.  A weight below fp16's normal numbers is off by 2^-25 where the largest
is at least 2^3, 2^-28 of it: under 2^-19 of A for these contexts."""
import numpy as np
import pytest
import torch

import oracle
from dense_sparse_w4a4_amd import ops
from test_kv4_gpu import _batch, _device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ops.lib()
    yield
    torch.cuda.synchronize()


def _held(cache, table, n):
    """Word indexes (page, offset) of a sequence's first n tokens."""
    t = np.arange(n)
    page = cache["kq"].shape[2]
    return table[t // page], t % page


def _expect(cache, table, lens, news, q, causal, window, scale):
    """fp64 (o, lse, bound of o, bound of lse) over the whole batch."""
    parts, at = [], 0
    q64 = q.double().numpy()
    D = q.shape[2]
    for i, (n, m) in enumerate(zip(lens, news)):
        k, v = oracle.kv4_read(cache, table[i], n)
        p, off = _held(cache, table[i], n)
        ks, vs = cache["ksz"][p, :, off].astype(np.float64), cache["vsz"][p, :, off].astype(np.float64)
        qq = q64[at:at + m]
        ref = lambda x: oracle.attention_reference(qq, k, x, causal, window, scale)  # noqa: E731
        o, lse = ref(v)
        A, _ = ref(np.abs(v))
        S, _ = ref(np.repeat(vs[..., :1], D, -1))
        Z = np.abs(vs[..., 1] + 8).max(initial=0)
        d = 2.0 ** -18 * abs(scale) * 15 * ks[..., 0].max(initial=0) * np.abs(qq).sum(-1)
        sums = 2.0 ** -23 * (8 + Z) * S * 2 * (n / 32 + 1)
        parts.append((o, lse, (2.0 ** -11 + 2 * d[..., None] + 2.0 ** -16 + 2.0 ** -19) * A + sums, d))
        at += m
    o, lse, tol, d = (np.concatenate(x) for x in zip(*parts))
    out = 2.0 ** -11 if q.dtype == torch.float16 else 2.0 ** -8
    with np.errstate(invalid="ignore"):
        return o, lse, out * np.abs(o) + tol + 2.0 ** -24, d + 2.0 ** -20 * np.abs(lse) + 2.0 ** -16


def _run(cache, table, lens, news, q, causal=True, window=0, scale=None, max_q=None):
    lse = torch.full(q.shape[:2], 5.0, dtype=torch.float32, device="cuda")
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32).cuda()
    out = ops.kv4_attention(q.cuda(), _device(cache), torch.from_numpy(table).cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), starts, max_q=max_q, causal=causal,
                            window=window, scale=scale, lse=lse)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _close(got, want, rows=slice(None)):
    (o, lse), (ro, rl, tol, ltol) = got, want
    err = np.abs(o[rows] - ro[rows])
    assert np.all(err <= tol[rows]), f"o: worst err/tol {np.nanmax(err / tol[rows]):.3f}, nan {np.isnan(err).sum()}"
    empty = np.isinf(rl[rows])
    assert np.array_equal(lse[rows][empty], rl[rows][empty])
    assert np.all(np.abs(lse[rows][~empty] - rl[rows][~empty]) <= ltol[rows][~empty])


def _copy(cache):
    return {n: x.copy() for n, x in cache.items()}


BATCH = ([300, 65, 129, 40], [37, 20, 5, 40])
ODD = [np.nan, np.inf, -np.inf, 65504, -65504]


@pytest.mark.parametrize("hq,hk,D,dtype", [(8, 2, 128, torch.float16), (8, 1, 64, torch.bfloat16)])
def test_zero_points_of_tokens_that_no_row_sees(hq, hk, D, dtype):
    """Tokens below every row's window hold any zero point, in the steps that
    are read for the tokens beside them."""
    lens, news = BATCH
    cache, table, q = _batch(lens, news, hq, hk, D, 32, dtype, seed=20)
    want = _expect(cache, table, lens, news, q, True, 21, D ** -0.5)
    rng = np.random.default_rng(20)
    bad = _copy(cache)
    for i, (n, m) in enumerate(zip(lens, news)):
        p, off = _held(cache, table[i], max(0, n - m - 20))
        for name in ("ksz", "vsz"):
            bad[name][p, :, off, 1] = rng.choice(ODD, (len(p), hk))
    for max_q in (1, 40):
        print(f"hq={hq} D={D} max_q={max_q}", flush=True)
        _close(_run(bad, table, lens, news, q, window=21, max_q=max_q), want)


@pytest.mark.parametrize("name", ["ksz", "vsz"])
@pytest.mark.parametrize("odd", [np.nan, np.inf, -np.inf])
def test_zero_points_reach_only_the_rows_that_see_them(name, odd):
    """Row i of a sequence of 90 with 30 queries sits at 60 + i and sees the last
    25 tokens: token 70's zero point is in rows 10 .. 29, token 47's in rows 0 .. 11."""
    lens, news = [90], [30]
    cache, table, q = _batch(lens, news, 4, 2, 128, 32, torch.float16, seed=21)
    want = _expect(cache, table, lens, news, q, True, 25, 128 ** -0.5)
    for t, sees in ((70, np.arange(10, 30)), (47, np.arange(0, 12))):
        bad = _copy(cache)
        p, off = _held(cache, table[0], 90)
        bad[name][p[t], :, off[t], 1] = odd
        others = np.setdiff1d(np.arange(30), sees)
        for max_q in (1, 30):
            got = _run(bad, table, lens, news, q, window=25, max_q=max_q)
            assert not np.isfinite(got[0][sees]).any()
            _close(got, want, others)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_q", [1, 100])
def test_zero_points_are_exact_whole_numbers(D, max_q):
    """One visible token: its weight is 1, and the output is the held value s (u
    + z) rounded once (the sum p may be off by fp32's rounding), for zero points up to the largest of fp16."""
    zeros = [2040, 2041, 2043, 2045, 2047, 2048, 2050, 4092, 16368, 16400, 65504]
    zeros = np.array([-z for z in zeros] + [0, -7, -8] + zeros, np.float64)
    n = len(zeros)
    cache, table, q = _batch([1] * n, [1] * n, 4, 2, D, 32, torch.float16, seed=22)
    cache["vsz"][table[:, 0], :, 0] = np.stack([np.full(n, 0.5), zeros], -1)[:, None, :]
    exact = np.stack([oracle.kv4_read(cache, table[i], 1)[1][0] for i in range(n)]).repeat(2, 1)  # [n, 4, D]
    got, _ = _run(cache, table, [1] * n, [1] * n, q, max_q=max_q)
    half = 0.5 * np.spacing(np.abs(exact).astype(np.float16)).astype(np.float64)
    err = np.abs(got - exact)
    assert np.all(err <= half * (1 + 2.0 ** -8)), (err / half).max(axis=(1, 2))


@pytest.mark.parametrize("hq,hk,D,dtype", [(8, 2, 128, torch.float16), (8, 1, 64, torch.bfloat16)])
@pytest.mark.parametrize("size", [0.01, 0.001, 2.0 ** -20])
def test_value_scales_of_unseen_tokens(hq, hk, D, dtype, size):
    """The largest value scales, infinities and NaN, on tokens that no row sees
    (below the window) and on tokens that only later rows see."""
    lens, news = BATCH
    cache, table, q = _batch(lens, news, hq, hk, D, 32, dtype, seed=23)
    for i, n in enumerate(lens):
        p, off = _held(cache, table[i], n)
        cache["vsz"][p, :, off, 0] = (cache["vsz"][p, :, off, 0].astype(np.float32) * (size * 8)).astype(np.float16)
    want = _expect(cache, table, lens, news, q, True, 21, D ** -0.5)
    for odd in (65504, np.inf, np.nan):
        bad = _copy(cache)
        rows, at = [], 0
        for i, (n, m) in enumerate(zip(lens, news)):
            p, off = _held(cache, table[i], n)
            hidden = np.arange(max(0, n - m - 20))
            late = n - m + m // 2  # seen by the rows from m // 2 on
            bad["vsz"][p[hidden], :, off[hidden], 0] = odd
            bad["vsz"][p[late], :, off[late], 0] = odd
            rows += range(at, at + m // 2)
            at += m
        for max_q in (1, 40):
            print(f"hq={hq} D={D} size={size} odd={odd} max_q={max_q}", flush=True)
            _close(_run(bad, table, lens, news, q, window=21, max_q=max_q), want, np.array(rows))


@pytest.mark.parametrize("max_q", [1, 100])
@pytest.mark.parametrize("place", [0, 40, 299])
def test_a_large_value_scale_without_weight(place, max_q):
    """A visible token of the largest value scale, whose score is so low that it
    does not count, leaves the other tokens' weights as precise as without it."""
    lens, news = [300, 300], [1, 20]
    cache, table, q = _batch(lens, news, 8, 2, 128, 32, torch.float16, seed=24)
    q = q.abs()
    for i, n in enumerate(lens):
        p, off = _held(cache, table[i], n)
        cache["ksz"][p, :, off, 1] = -7
        cache["vsz"][p, :, off, 0] = (cache["vsz"][p, :, off, 0].astype(np.float32) * 0.01).astype(np.float16)
        cache["kq"][p[place], :, off[place]] = 0
        cache["ksz"][p[place], :, off[place]] = 0.4, -20  # score about -90
        cache["vsz"][p[place], :, off[place], 0] = 65504
    want = _expect(cache, table, lens, news, q, True, 0, 128 ** -0.5)
    _close(_run(cache, table, lens, news, q, max_q=max_q), want)


@pytest.mark.parametrize("max_q", [1, 100])
@pytest.mark.parametrize("rising", [True, False])
def test_value_scales_against_scores(rising, max_q):
    """Scores that rise along the context while value scales fall from the
    largest to small ones (or the other way round): the weights that count are
    small (or come first)."""
    n = 400
    lens, news = [n, n], [1, 20]
    cache, table, q = _batch(lens, news, 8, 2, 128, 32, torch.float16, seed=25)
    q = q.abs()
    t = np.arange(n) if rising else np.arange(n)[::-1]
    for i in range(2):
        p, off = _held(cache, table[i], n)
        cache["ksz"][p, :, off, 0] = 0.2
        cache["ksz"][p, :, off, 1] = np.round(-22 + t / 20)[:, None]
        cache["vsz"][p, :, off, 0] = (60000 * 2.0 ** (-t / 13.0))[:, None]
    want = _expect(cache, table, lens, news, q, True, 0, 128 ** -0.5)
    _close(_run(cache, table, lens, news, q, max_q=max_q), want)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 30])
def test_windows_as_large_as_an_int(window):
    """A window past every context hides nothing, also where a sequence has more
    queries than tokens."""
    lens, news = [3, 70, 0, 200, 1], [7, 3, 2, 40, 65]
    for D in (64, 128):
        cache, table, q = _batch(lens, news, 8, 4, D, 32, torch.float16, seed=26)
        want = _expect(cache, table, lens, news, q, True, 0, D ** -0.5)
        for max_q in (1, 65):
            print(f"window={window} D={D} max_q={max_q}", flush=True)
            _close(_run(cache, table, lens, news, q, window=window, max_q=max_q), want)


@pytest.mark.parametrize("max_q", [1, 100])
def test_host_and_overlapping_workspaces_are_refused(max_q):
    cache = ops.kv4_cache(4, 32, 2, 64)
    q = torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda")
    args = (q, cache, torch.zeros((3, 2), dtype=torch.int32, device="cuda"),
            torch.ones(3, dtype=torch.int32, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda"), max_q)
    need = ops.kv4_attention_workspace(3, 3, 4, 2, 64, max_q)
    assert need > 0
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for bad in (torch.empty(need, dtype=torch.uint8), one.expand(need)):
        with pytest.raises(ValueError, match="workspace"):
            ops.kv4_attention(*args, workspace=bad)
    assert not ops.kv4_attention(*args, workspace=one).any()


@pytest.mark.parametrize("scale", [-3.0, 3.0])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 50])
def test_sharp_softmax_under_windows(D, scale, window):
    """Outputs and log-sums where nearly all weight is on one token."""
    lens, news = [300, 70, 3, 0], [9, 40, 1, 1]
    cache, table, q = _batch(lens, news, 8, 2, D, 32, torch.float16, seed=27)
    want = _expect(cache, table, lens, news, q, True, window, scale)
    for max_q in (1, 40):
        _close(_run(cache, table, lens, news, q, window=window, scale=scale, max_q=max_q), want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_q", [1, 100])
def test_precision_of_scores(D, dtype, max_q):
    """One visible token: the log-sum is its score.  Root mean square error over
    that of the scores: the key codes' products lose two bits, 1.1e-7 (the error was
    1.8e-6 where they lost six); the chain of sums of codes, about twice the score
    before the zero point's share is added, 1.1e-7; the queries' sum, scale and units
    0.7e-7: 1.7e-7 in all, held to 2^-21."""
    n = 512
    cache, table, q = _batch([1] * n, [1] * n, 8, 2, D, 32, dtype, seed=28)
    _, lse, _, _ = _expect(cache, table, [1] * n, [1] * n, q, True, 0, D ** -0.5)
    _, got = _run(cache, table, [1] * n, [1] * n, q, max_q=max_q)
    assert np.sqrt(np.mean((got - lse) ** 2)) <= 2.0 ** -21 * np.sqrt(np.mean(lse ** 2))
