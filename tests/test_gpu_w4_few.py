"""GPU: the W4A16 product for few tokens against its 64-bit form, within the
error its roundings can add up to (tests/rules_ref.py)."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import rules_ref
from tests.few_ref import same_bits

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


def _weights(rng, N, K, g, z_range=(0, 16)):
    """Any codes, scales of both signs, zero points of a range (numpy)."""
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = (rng.uniform(0.5, 2.0, (N, K // g)) * rng.choice([-0.01, 0.01], (N, K // g))).astype(np.float16)
    z = rng.integers(*z_range, (N, K // g)).astype(np.float16)
    return q, s, z


def _dev(w, g, tiled=False):
    p = (*[torch.from_numpy(a).cuda() for a in w], g)
    return dg.pack_tiled(p) if tiled else p


def _x(rng, T, K, dtype):
    x = rng.standard_normal((T, K)) * np.exp(rng.standard_normal(K))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def _check(y, x, w, g):
    want, bound = rules_ref.linear(x, *w, g, y.dtype)
    err = np.abs(y.cpu().double().numpy() - want)
    assert (err <= bound).all(), (err / bound).max()


SHAPES = [(1, 64, 1), (1, 128, 16), (2, 192, 5), (3, 704, 2111), (1, 2816, 300), (5, 2816, 1030), (7, 64, 4097),
          (8, 128, 20000), (15, 1088, 33), (16, 4096, 256), (17, 256, 100), (31, 2816, 47), (33, 960, 1000),
          (47, 128, 16400), (48, 8192, 40), (49, 1152, 255), (64, 2816, 513), (64, 64, 15), (64, 16384, 16),
          (4, 28672, 20), (1, 100096, 3), (20, 40960, 18), (12, 5632, 2000),
          (3, 35264, 50), (16, 8256, 33), (9, 12352, 9000), (64, 4160, 5000), (30, 3008, 9000), (16, 6400, 40000)]


@pytest.mark.parametrize("xt", [F16, BF16], ids=str)
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_shapes(T, K, N, xt):
    rng = np.random.default_rng([T, K, N])
    x = _x(rng, T, K, xt)
    for g in (64, 128):
        if K % g:
            continue
        w = _weights(rng, N, K, g)
        yt = [F32, F16, BF16][(T + N + g // 64) % 3]
        y = dg.w4a16_linear_few(x.cuda(), _dev(w, g), dtype=yt)
        assert y.shape == (T, N) and y.dtype == yt
        _check(y, x, w, g)
        if N % 16 == 0:
            assert same_bits(dg.w4a16_linear_few(x.cuda(), _dev(w, g, True), dtype=yt), y)


@pytest.mark.parametrize("T", range(1, 65, 3))
def test_every_number_of_tokens(T):
    # each token's results depend on its own row only
    rng = np.random.default_rng(T)
    K, N = 832, 272
    x = _x(rng, 64, K, BF16).cuda()
    w = _weights(rng, N, K, 64)
    wd = _dev(w, 64, T % 2 == 0)
    y = dg.w4a16_linear_few(x[:T], wd, dtype=F32)
    _check(y, x[:T].cpu(), w, 64)
    for t in {0, T // 2, T - 1}:
        _check(dg.w4a16_linear_few(x[t:t + 1], wd, dtype=F32), x[t:t + 1].cpu(), w, 64)
        other = x[:T].clone()
        other[torch.arange(T, device="cuda") != t] *= -3
        assert same_bits(dg.w4a16_linear_few(other, wd, dtype=F32)[t], y[t])


@pytest.mark.parametrize("xt", [F16, BF16], ids=str)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("K,g", [(256, 128), (256, 64), (2816, 128), (1600, 64)])
def test_one_hot(K, g, tiled, xt):
    # each output is one weight (q - z) s, exactly: every code, channel, place
    # of K and token has its own
    rng = np.random.default_rng(K + g)
    N = 48
    q, s, z = _weights(rng, N, K, g, (-2048, 2049))
    at = rng.permutation(K)
    w = (rules_ref.codes(q) - np.repeat(z.astype(np.float64), g, 1)) * np.repeat(s.astype(np.float64), g, 1)
    for k0 in range(0, K, 64):
        ks = at[k0:k0 + 64]
        x = torch.zeros((len(ks), K), dtype=xt, device="cuda")
        x[torch.arange(len(ks)), torch.from_numpy(ks).cuda()] = 1
        y = dg.w4a16_linear_few(x, _dev((q, s, z), g, tiled), dtype=F32)
        assert np.array_equal(y.cpu().double().numpy(), w[:, ks].T)


@pytest.mark.parametrize("xt", [F16, BF16], ids=str)
def test_zero_points(xt):
    # zero points far outside the codes, and not whole
    rng = np.random.default_rng(9)
    for z_range in ((-2048, 2049), (0, 1), (1000, 1025), (-40, -10)):
        T, K, N, g = 6, 512, 80, 128
        q, s, z = _weights(rng, N, K, g, z_range)
        z = (z.astype(np.float32) + rng.random(z.shape)).astype(np.float16)
        x = _x(rng, T, K, xt)
        _check(dg.w4a16_linear_few(x.cuda(), _dev((q, s, z), g), dtype=F32), x, (q, s, z), g)


@pytest.mark.parametrize("xt", [F16, BF16], ids=str)
@pytest.mark.parametrize("skip", [1, 5, 8])
@pytest.mark.parametrize("T", [1, 4, 21, 64])
def test_strided(T, skip, xt):
    # rows apart from an odd element on, into a slice; the rest untouched
    rng = np.random.default_rng([T, skip])
    K, N, g = 704, 1003, 64
    wide = _x(rng, T, K + skip, xt).cuda()
    w = _weights(rng, N, K, g)
    for yt in (F32, F16, BF16):
        buf = torch.full((T + 2, N + 9), 7.0, dtype=yt, device="cuda")
        y = buf[1:T + 1, skip:skip + N]
        assert dg.w4a16_linear_few(wide[:, skip:], _dev(w, g), out=y) is y
        _check(y, wide[:, skip:].cpu(), w, g)
        rest = buf.clone()
        rest[1:T + 1, skip:skip + N] = 7.0
        assert (rest == 7.0).all()


@pytest.mark.parametrize("xt", [F16, BF16], ids=str)
def test_values_at_the_edges(xt):
    # zeros, subnormals, the largest values; a token with a NaN or an infinity
    # has NaN or infinite results and leaves the others alone
    rng = np.random.default_rng(4)
    T, K, N, g = 20, 384, 64, 128
    w = _weights(rng, N, K, g)
    x = _x(rng, T, K, xt)
    fi = torch.finfo(xt)
    x[0] = 0
    x[1] = torch.from_numpy(rng.integers(-9, 10, K)).to(torch.float32).mul(fi.smallest_normal / 16).to(xt)
    x[2] = 65000 if xt is F16 else 2.0 ** 99
    y = dg.w4a16_linear_few(x.cuda(), _dev(w, g), dtype=F32)
    _check(y, x, w, g)
    assert (y[0] == 0).all()
    bad = x.clone()
    bad[3, 200], bad[9, 0], bad[16, 383] = float("nan"), float("inf"), float("-inf")
    yb = dg.w4a16_linear_few(bad.cuda(), _dev(w, g), dtype=F32)
    hit = torch.zeros(T, dtype=torch.bool, device="cuda")
    hit[[3, 9, 16]] = True
    assert not torch.isfinite(yb[hit]).any()
    assert same_bits(yb[~hit], y[~hit])


def test_reruns_and_graph():
    rng = np.random.default_rng(6)
    for T, K, N in ((1, 2816, 4096), (9, 2816, 2111), (40, 1408, 3000)):
        x = _x(rng, T, K, F16).cuda()
        w = _dev(_weights(rng, N, K, 128), 128)
        first = dg.w4a16_linear_few(x, w, dtype=F32)
        for _ in range(5):
            assert same_bits(dg.w4a16_linear_few(x, w, dtype=F32), first)
        out = torch.empty_like(first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dg.w4a16_linear_few(x, w, out=out)
        for i in range(4):
            x.copy_(_x(rng, T, K, F16))
            graph.replay()
            assert same_bits(out, dg.w4a16_linear_few(x, w, dtype=F32))


def test_agrees_with_the_layer_for_many_tokens():
    rng = np.random.default_rng(2)
    x = _x(rng, 33, 2816, F16).cuda()
    w = _dev(_weights(rng, 512, 2816, 128), 128, True)
    a, b = dg.w4a16_linear(x, w), dg.w4a16_linear_few(x, w)
    assert (a.float() - b.float()).abs().max() <= 2e-3 * b.float().abs().max()


def test_refusals():
    rng = np.random.default_rng(1)
    w = _dev(_weights(rng, 32, 128, 64), 64)
    x = torch.zeros((2, 128), dtype=F16, device="cuda")
    with pytest.raises(TypeError):
        dg.w4a16_linear_few(x.float(), w)
    with pytest.raises(TypeError):
        dg.w4a16_linear_few(x, w, dtype=torch.float64)
    with pytest.raises(ValueError, match="shapes"):
        dg.w4a16_linear_few(x[:, :64], w)
    with pytest.raises(ValueError, match="contiguous"):
        dg.w4a16_linear_few(x.t()[:2], w)
    with pytest.raises(ValueError, match="out"):
        dg.w4a16_linear_few(x, w, out=torch.zeros((2, 31), device="cuda"))
    with pytest.raises(dg.Dgw4Error, match="UNSUPPORTED"):
        dg.w4a16_linear_few(torch.zeros((65, 128), dtype=F16, device="cuda"), w)
    assert dg.w4a16_linear_few(x[:0], w).shape == (0, 32)


def test_offsets_past_32_bits():
    # weights and scales past 2 GiB, rows of x and y far apart: the last channels
    # of the last tokens
    g = torch.Generator(device="cuda").manual_seed(3)
    N, K, T = 1100003, 4096, 3
    q = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8, generator=g)
    s = (torch.rand((N, K // 64), device="cuda", generator=g) * 0.01).half()
    z = torch.randint(0, 16, (N, K // 64), device="cuda", generator=g).half()
    assert q.numel() > 2 ** 31
    wide = torch.zeros((T, 800_000_000), device="cuda", dtype=torch.float16)
    x = wide[:, -K:]
    x.copy_(torch.randn((T, K), device="cuda", generator=g))
    out = torch.zeros((T, 800_000_000), device="cuda", dtype=torch.float16)
    y = out[:, -N:]
    dg.w4a16_linear_few(x, (q, s, z, 64), out=y)
    for part in (slice(0, 40), slice(524270, 524310), slice(N - 40, N)):
        _check(y[:, part], x.cpu(), [v[part].cpu().numpy() for v in (q, s, z)], 64)
    assert (out[:, :-N] == 0).all()
