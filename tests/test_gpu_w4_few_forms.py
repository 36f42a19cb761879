"""GPU: the W4A16 product for few tokens in every form that a call can take: each
kernel, each split of K over its waves, with one turn of channels a workgroup and
with several, x in one chunk and in several (an even and an odd number of them).
tests/test_w4_few_plan.py asks the library's own choice that the sizes here do
reach each. Against the 64-bit form, computed on the GPU by plain operations."""
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import rules_ref
from tests.few_ref import U32, same_bits

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


# Both group sizes, both layouts.
SHAPES = [
    # x whole, eight waves
    (4, 128, 16), (3, 640, 65712), (1, 1152, 16400), (8, 1280, 65632), (3, 2176, 8208), (11, 2560, 32912),
    (6, 4224, 16), (6, 4736, 17200), (5, 1408, 140000),
    # x whole, sixteen waves
    (15, 2432, 33536), (15, 2432, 100560), (15, 2432, 17824), (13, 2816, 71296), (15, 2432, 9280), (16, 4096, 11264),
    (15, 2560, 33328), (15, 4224, 4128), (11, 4736, 16752), (5, 8320, 16), (6, 9600, 8368),
    # chunks of 2048 columns, up to 16 tokens
    (15, 5376, 49856), (14, 5376, 102176), (16, 5632, 65008), (14, 5248, 8240), (15, 4992, 20704), (26, 4608, 16),
    (15, 5248, 4192), (9, 12288, 9008),
    # chunks of 512 columns, blocks of up to 32 tokens
    (29, 1152, 32816), (19, 1152, 65584), (20, 1408, 20000), (25, 1280, 65552), (32, 2816, 70000), (61, 1152, 1040),
    (30, 2560, 34064), (64, 2816, 8192), (17, 896, 33008),
    # and up to 64
    (62, 1152, 32896), (36, 1152, 65664), (33, 896, 70000), (37, 1152, 16416), (44, 1280, 65616),
    (40, 2816, 70000), (49, 1152, 8208), (50, 1408, 9008), (64, 2816, 16384), (47, 2560, 33040), (64, 1024, 262144),
]
# Groups of 64, their number odd, row-major, odd channels.
RAGGED = [
    (6, 192, 17), (13, 576, 65627), (2, 1088, 16497), (7, 1216, 65657), (3, 2240, 8201), (14, 2496, 32871),
    (7, 4160, 17), (6, 4672, 16787),
    (15, 2752, 33173), (15, 2624, 102739), (15, 2624, 16705), (14, 2624, 68449), (14, 2624, 8215), (15, 2880, 33675),
    (10, 4160, 4139), (15, 4672, 16657), (4, 8384, 17), (6, 9280, 8231),
    (15, 4928, 50803), (15, 4800, 105155), (15, 5184, 8331), (15, 4800, 21313), (56, 4544, 17), (15, 5056, 4429),
    (20, 1088, 32921), (29, 1088, 66027), (22, 1088, 16405), (24, 1216, 65647), (59, 1088, 1033), (20, 2496, 33033),
    (39, 1088, 32863), (53, 1088, 65689), (50, 1088, 16391), (51, 1216, 65553), (59, 1088, 8197), (42, 2496, 32923),
]


def _weights(gen, N, K, g):
    """Any codes, scales of both signs, whole zero points."""
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (torch.rand((N, K // g), device="cuda", generator=gen) * 0.015 + 0.005).half()
    sign = torch.randint(0, 2, s.shape, device="cuda", generator=gen).half() * 2 - 1
    z = torch.randint(0, 16, s.shape, device="cuda", generator=gen).half()
    return q, s * sign, z


def _reference(x, q, s, z, g, dtype):
    """rules_ref.linear, with its bound, on the GPU: x and the weights where they
    are, channels a block at a time."""
    T, K = x.shape
    N = q.shape[0]
    xd = x.double()
    y = torch.empty((T, N), dtype=torch.float64, device="cuda")
    size = torch.empty_like(y)
    step = max(1, (1 << 26) // K)
    for n0 in range(0, N, step):
        n = slice(n0, min(N, n0 + step))
        c = torch.stack((q[n] & 15, q[n] >> 4), dim=-1).view(-1, K // g, g).double()
        sc, zp = s[n].double()[..., None], z[n].double()[..., None]
        y[:, n] = xd @ ((c - zp) * sc).view(-1, K).t()
        size[:, n] = xd.abs() @ (sc.abs() * (31 + (16 + zp).abs())).expand(-1, -1, g).reshape(-1, K).t()
    bound = 1.01 * U32 * (g + K / g + 22) * size
    return y, bound + rules_ref.HALF_STEP[dtype] * (y.abs() + bound) + rules_ref.TINY[dtype]


def _x(gen, T, K, dtype):
    x = torch.randn((T, K), device="cuda", generator=gen)
    return (x * torch.exp(torch.randn(K, device="cuda", generator=gen))).to(dtype)


def _run(T, K, N, groups, xt):
    gen = torch.Generator(device="cuda").manual_seed(T * 1000003 + K * 1009 + N)
    x = _x(gen, T, K, xt)
    for i, g in enumerate(groups):
        w = _weights(gen, N, K, g)
        yt = [F32, F16, BF16][(T + K // 64 + i) % 3]
        y = dg.w4a16_linear_few(x, (*w, g), dtype=yt)
        want, bound = _reference(x, *w, g, yt)
        err = (y.double() - want).abs()
        assert bool((err <= bound).all()), float((err / bound).max())
        if N % 16 == 0:
            tiled = dg.pack_tiled((*w, g))
            assert same_bits(dg.w4a16_linear_few(x, tiled, dtype=yt), y)
        # again, into rows apart: the same bits, nothing beside them
        out = torch.full((T, N + 3), 7.0, dtype=yt, device="cuda")
        dg.w4a16_linear_few(x, (*w, g), out=out[:, 1:N + 1])
        assert same_bits(out[:, 1:N + 1], y)
        assert bool((out[:, 0] == 7.0).all() and (out[:, N + 1:] == 7.0).all())


@pytest.mark.parametrize("xt", [F16, BF16], ids=str)
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_forms(T, K, N, xt):
    _run(T, K, N, (64, 128), xt)


@pytest.mark.parametrize("xt", [F16, BF16], ids=str)
@pytest.mark.parametrize("T,K,N", RAGGED)
def test_ragged_forms(T, K, N, xt):
    _run(T, K, N, (64,), xt)


@pytest.mark.parametrize("T,K,N", [(15, 2624, 68449), (15, 4800, 21313), (24, 1216, 65647), (42, 2496, 32923)])
def test_tokens_stay_apart(T, K, N):
    # several turns: a NaN or an infinity in a token leaves the others' bits alone
    gen = torch.Generator(device="cuda").manual_seed(N)
    x, w = _x(gen, T, K, BF16), (*_weights(gen, N, K, 64), 64)
    y = dg.w4a16_linear_few(x, w, dtype=F32)
    bad = x.clone()
    bad[3, K - 1], bad[T - 1, 0] = float("nan"), float("inf")
    yb = dg.w4a16_linear_few(bad, w, dtype=F32)
    hit = torch.zeros(T, dtype=torch.bool, device="cuda")
    hit[[3, T - 1]] = True
    assert not torch.isfinite(yb[hit]).any()
    assert same_bits(yb[~hit], y[~hit])


def test_reference_is_the_host_form():
    gen = torch.Generator(device="cuda").manual_seed(1)
    for g in (64, 128):
        x, w = _x(gen, 5, 384, F16), _weights(gen, 33, 384, g)
        y, bound = _reference(x, *w, g, F16)
        y0, bound0 = rules_ref.linear(x.cpu(), *[v.cpu().numpy() for v in w], g, F16)
        assert abs(y.cpu().numpy() - y0).max() <= 1e-12 * abs(y0).max()
        assert abs(bound.cpu().numpy() - bound0).max() <= 1e-12 * bound0.max()
