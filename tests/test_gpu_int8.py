"""GPU: 8-bit row quantisation and the 8-bit products against their
definitions, bit for bit (the sums are exact integers and every rounding is
stated, so there is one right answer; tests/few_ref.py)."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import few_ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


def _acts(rng, rows, K, dtype):
    x = torch.from_numpy(rng.standard_normal((rows, K), dtype=np.float32))
    x *= torch.from_numpy(np.exp(rng.standard_normal(K)).astype(np.float32))
    return x.to(dtype)


def _codes(rng, rows, K, low=-127):
    q = rng.integers(low, 128, (rows, K), dtype=np.int8)
    s = np.exp(rng.standard_normal(rows) - 5).astype(np.float32)
    return q, s


def _dev(*a):
    return [torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in a]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 16), (3, 17), (5, 2816), (300, 100), (2, 16384),
                                    (7, 4097), (2, 70001), (1000, 33)])
def test_quantize_rows(rows, K, dtype):
    rng = np.random.default_rng([rows, K])
    x = _acts(rng, rows, K, dtype)
    q, s = dg.quantize_rows_i8(x.cuda())
    rq, rs = few_ref.quantize_rows(x)
    assert q.shape == rq.shape
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy().view(np.int32), rs.view(np.int32))


# both sides of each length at which another number of threads takes a row, and
# every length of a last vector
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,K", [(70, K) for K in (1, 2, 7, 8, 9, 10, 11, 12, 13, 14, 15, 127, 128, 129, 383, 384,
                                                      385, 767, 768, 769, 1023, 1024, 1025, 1535, 1536, 1537, 2999,
                                                      4095, 4096, 4097, 8191, 8192, 8193, 16383, 16385)] +
                         [(8191, 1601), (8200, 1601), (8195, 2998)])
def test_quantize_lengths(rows, K, dtype):
    rng = np.random.default_rng([rows, K, 1])
    x = _acts(rng, rows, K, dtype)
    x[-1] = 0
    x[-1, K - 1] = -0.25                  # the row's maximum in its last column
    if rows >= 70:
        x[3, K // 2] = float("nan")
        x[5, K - 1] = float("inf")
    q, s = dg.quantize_rows_i8(x.cuda())
    rq, rs = few_ref.quantize_rows(x)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_edges(dtype):
    # zeros, one sign, ties of the rounding, the type's extremes and subnormals,
    # NaN and infinities: each row on its own
    K = 300
    fi = torch.finfo(dtype)
    x = torch.zeros((12, K), dtype=dtype)
    x[1, 7] = -3
    x[2] = torch.arange(K).to(dtype) - 100
    x[3, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5]).to(dtype)
    x[3, 4:130] = (torch.arange(126) + 0.5).to(dtype)
    x[4, 3] = fi.max
    x[4, 4] = -fi.max
    x[5, 3] = fi.tiny
    x[6, 250] = fi.smallest_normal * fi.eps          # the smallest subnormal
    x[6, 251] = -3 * fi.smallest_normal * fi.eps
    x[7, 299] = float("nan")
    x[8, 0] = float("inf")
    x[9, 1] = float("-inf")
    x[10, 2], x[10, 3] = float("nan"), float("inf")
    x[11] = -0.0
    x[7:11, 9] = 2
    q, s = dg.quantize_rows_i8(x.cuda())
    rq, rs = few_ref.quantize_rows(x)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert few_ref.same_bits(s, torch.from_numpy(rs))
    assert torch.isnan(s[7:11]).all() and (s[[0, 11]] == 1).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("skip", [1, 3, 8, 13])
def test_quantize_strided(dtype, skip):
    # rows apart, from an odd element on; outputs into slices, the rest untouched
    rng = np.random.default_rng(skip)
    wide = _acts(rng, 21, 150 + skip, dtype).cuda()
    x = wide[:, skip:]
    q = torch.full((23, 192), 55, dtype=torch.int8, device="cuda")
    s = torch.full((23,), 9.0, device="cuda")
    dg.quantize_rows_i8(x, out=(q[:21, 16:176], s[:21]))
    rq, rs = few_ref.quantize_rows(x.cpu())
    assert np.array_equal(q[:21, 16:176].cpu().numpy(), rq)
    assert np.array_equal(s[:21].cpu().numpy(), rs)
    assert (q[21:] == 55).all() and (q[:, :16] == 55).all() and (q[:, 176:] == 55).all()
    assert (s[21:] == 9).all()


PRODUCTS = [(1, 16, 1), (1, 2816, 300), (2, 64, 17), (3, 4096, 64), (5, 48, 1000), (8, 704, 129),
            (16, 1024, 255), (17, 2816, 77), (31, 80, 33), (33, 16384, 40), (64, 256, 256),
            (65, 272, 515), (100, 1008, 90), (128, 704, 513), (200, 128, 1030), (257, 320, 257),
            (300, 2816, 700), (513, 144, 260), (1030, 64, 31), (1, 131056, 5), (40, 131056, 18)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,K,N", PRODUCTS)
def test_product(T, K, N, dtype):
    rng = np.random.default_rng([T, K, N])
    (xq, xs), (wq, ws) = _codes(rng, T, K), _codes(rng, N, K)
    xd, sd, wd, vd = _dev(xq, xs, wq, ws)
    y = dg.w8a8_linear(xd, sd, (wd, vd), dtype=dtype)
    assert few_ref.same_bits(y, few_ref.product(xq, xs, wq, ws, dtype))


# each tile of the product, K in whole turns of its parts and not (the last
# parts' stages past K), channels and tokens that end inside a tile
@pytest.mark.parametrize("T,K,N", [(770, 16, 11565), (646, 144, 13129), (200, 144, 40001), (657, 16, 9631),
                                   (587, 144, 9625), (835, 16, 4549), (322, 144, 10061), (194, 704, 8146),
                                   (200, 832, 7998), (250, 2800, 4001), (36, 16, 8293), (33, 144, 9906),
                                   (35, 48, 4868), (35, 176, 5205), (59, 112, 35), (77, 4112, 81),
                                   (40, 8208, 35), (65, 6000, 100)])
def test_product_tiles(T, K, N):
    rng = np.random.default_rng([T, K, N])
    (xq, xs), (wq, ws) = _codes(rng, T, K), _codes(rng, N, K)
    xd, sd, wd, vd = _dev(xq, xs, wq, ws)
    for dtype in TYPES:
        y = dg.w8a8_linear(xd, sd, (wd, vd), dtype=dtype)
        assert few_ref.same_bits(y, few_ref.product(xq, xs, wq, ws, dtype))


# the tiles with K in two and four parts that few sizes reach
@pytest.mark.parametrize("T,K,N", [(250, 2816, 4001), (180, 4000, 4099), (256, 2560, 4095), (40, 8192, 35),
                                   (33, 10240, 90), (95, 9104, 70)])
def test_product_tiles_in_parts(T, K, N):
    test_product_tiles(T, K, N)


@pytest.mark.parametrize("T", [1, 9, 70, 300])
def test_product_extremes(T):
    # the largest sums (all codes -128 at the longest K), zeros, and scales
    # whose products overflow, vanish or are NaN
    K, N = 131056, 34
    xq = np.full((T, K), -128, dtype=np.int8)
    wq = np.full((N, K), -128, dtype=np.int8)
    wq[1] = 127
    wq[2] = 0
    xs = np.geomspace(1e-30, 1e30, T).astype(np.float32)
    xs[0] = np.nan
    ws = np.geomspace(1e-10, 1e10, N).astype(np.float32)
    xd, sd, wd, vd = _dev(xq, xs, wq, ws)
    for dtype in TYPES:
        y = dg.w8a8_linear(xd, sd, (wd, vd), dtype=dtype)
        assert few_ref.same_bits(y, few_ref.product(xq, xs, wq, ws, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,K,N,pad", [(3, 64, 50, 5), (40, 96, 130, 3), (150, 192, 300, 1),
                                       (260, 128, 256, 8)])
def test_product_strided(T, K, N, pad, dtype):
    # operands and output inside wider tensors; what lies between stays
    rng = np.random.default_rng([T, N])
    xq, xs = _codes(rng, T, K + 48)
    wq, ws = _codes(rng, N, K + 32)
    xd, sd, wd, vd = _dev(xq, xs, wq, ws)
    big = torch.full((T + 2, N + 2 * pad), 3.0, dtype=dtype, device="cuda")
    y = big[1:T + 1, pad:pad + N]
    dg.w8a8_linear(xd[:, 32:32 + K], sd, (wd[:, 16:16 + K], vd), out=y)
    assert few_ref.same_bits(y, few_ref.product(xq[:, 32:32 + K], xs, wq[:, 16:16 + K], ws, dtype))
    assert (big[0] == 3).all() and (big[-1] == 3).all()
    assert (big[:, :pad] == 3).all() and (big[:, pad + N:] == 3).all()


@pytest.mark.parametrize("xtype", TYPES, ids=str)
@pytest.mark.parametrize("T,K,N", [(1, 1, 1), (1, 2816, 512), (1, 16384, 100), (2, 100, 65), (4, 2816, 1000),
                                   (8, 17, 300), (13, 2000, 48), (16, 333, 257), (17, 500, 70),
                                   (130, 2816, 300), (3, 70001, 20)])
def test_product_from_activations(T, K, N, xtype):
    rng = np.random.default_rng([T, K, N, 1])
    x = _acts(rng, T, K, xtype)
    Kp = (K + 15) // 16 * 16
    wq, ws = _codes(rng, N, Kp)                   # the columns past K hold anything
    wd, vd = _dev(wq, ws)
    rq, rs = few_ref.quantize_rows(x)
    n = dg.w8a8_workspace_bytes(T, K)
    ws_buf = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    for dtype in TYPES:
        y = dg.w8a8_linear_tokens(x.cuda(), (wd, vd), dtype=dtype, workspace=ws_buf)
        assert few_ref.same_bits(y, few_ref.product(rq, rs, wq, ws, dtype)), dtype
        q, s = dg.quantize_rows_i8(x.cuda())
        assert few_ref.same_bits(y, dg.w8a8_linear(q, s, (wd, vd), dtype=dtype))


@pytest.mark.parametrize("T", [2, 9, 40])
def test_activations_strided_and_nonfinite(T):
    rng = np.random.default_rng(T)
    wide = _acts(rng, T, 403, torch.bfloat16)
    wide[T // 2, 200] = float("nan")
    wide[0, 300] = float("inf")
    x = wide[:, 3:]
    wq, ws = _codes(rng, 70, 400)
    wd, vd = _dev(wq, ws)
    big = torch.full((T + 1, 75), 3.0, device="cuda")
    y = dg.w8a8_linear_tokens(wide.cuda()[:, 3:], (wd, vd), out=big[:T, 2:72])
    rq, rs = few_ref.quantize_rows(x)
    assert few_ref.same_bits(y, few_ref.product(rq, rs, wq, ws, torch.float32))
    assert torch.isnan(y[0]).all() and torch.isnan(y[T // 2]).all()
    assert (big[T] == 3).all() and (big[:, :2] == 3).all() and (big[:, 72:] == 3).all()


# 512 workgroups take 16 channels at a time: a few that take a second turn,
# several whole rounds, several batches of K a turn, and both sides of the size
# (16384 blocks of channels) from which a turn is two neighbouring blocks, with
# an odd last one
@pytest.mark.parametrize("T,K,N", [(1, 600, 8193), (5, 300, 8200), (6, 1000, 8208), (6, 2900, 24603),
                                   (1, 9000, 16401), (5, 3600, 24590), (2, 6500, 9000), (6, 64, 57361),
                                   (1, 600, 262128), (6, 600, 262129), (5, 600, 262145), (5, 3600, 262149),
                                   (6, 80, 524305)])
def test_few_tokens_in_turns(T, K, N):
    g = torch.Generator(device="cuda").manual_seed(N + T)
    x = torch.randn((T, K), device="cuda", generator=g).to(torch.bfloat16)
    wq = torch.randint(-127, 128, (N, (K + 15) // 16 * 16), dtype=torch.int8, device="cuda", generator=g)
    ws = torch.rand(N, device="cuda", generator=g) + 0.5
    q, s = dg.quantize_rows_i8(x)
    rq, rs = few_ref.quantize_rows(x.cpu())
    for dtype in TYPES:
        y = dg.w8a8_linear_tokens(x, (wq, ws), dtype=dtype)
        assert few_ref.same_bits(y, dg.w8a8_linear(q, s, (wq, ws), dtype=dtype)), dtype
        for n0 in (0, 8192 - 40, N // 2, N - 80):
            n1 = min(N, n0 + 80)
            ref = few_ref.product(rq, rs, wq[n0:n1].cpu().numpy(), ws[n0:n1].cpu().numpy(), dtype)
            assert few_ref.same_bits(y[:, n0:n1], ref), (dtype, n0)
    # into rows that lie apart, replayed: what lies between stays
    big = torch.full((T + 1, N + 7), 3.0, device="cuda")
    ws_buf = torch.empty(dg.w8a8_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
    out = big[:T, 3:3 + N]
    want = dg.w8a8_linear(q, s, (wq, ws), dtype=torch.float32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.w8a8_linear_tokens(x, (wq, ws), out=out, workspace=ws_buf)
    for _ in range(3):
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert few_ref.same_bits(out, want)
    assert (big[T] == 3).all() and (big[:, :3] == 3).all() and (big[:, 3 + N:] == 3).all()


def test_empty_batch():
    w = (torch.zeros((8, 32), dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda"))
    assert dg.w8a8_linear(w[0][:0], w[1][:0], w).shape == (0, 8)
    assert dg.w8a8_linear_tokens(torch.empty((0, 32), device="cuda"), w).shape == (0, 8)
    q, s = dg.quantize_rows_i8(torch.empty((0, 20), device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0,)


def test_offsets_past_32_bits():
    # outputs, weights and activations whose byte offsets pass 2^32: the last
    # rows and columns of each
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GiB")
    g = torch.Generator(device="cuda").manual_seed(1)
    # weights of 4.3 GB
    N, K = 33000, 131056
    wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    ws = torch.rand(N, device="cuda", generator=g)
    for T in (2, 40):
        xq = torch.randint(-127, 128, (T, K), dtype=torch.int8, device="cuda", generator=g)
        xs = torch.rand(T, device="cuda", generator=g)
        y = dg.w8a8_linear(xq, xs, (wq, ws), dtype=torch.float32)
        for n0 in (0, N - 40):
            ref = few_ref.product(xq.cpu().numpy(), xs.cpu().numpy(), wq[n0:n0 + 40].cpu().numpy(),
                                  ws[n0:n0 + 40].cpu().numpy(), torch.float32)
            assert few_ref.same_bits(y[:, n0:n0 + 40], ref), (T, n0)
    # activations of 4.3 GB, quantised and multiplied as they are
    wq2, ws2 = wq[:20].contiguous(), ws[:20].contiguous()
    xs = torch.rand(N, device="cuda", generator=g)
    y = dg.w8a8_linear(wq, xs, (wq2, ws2), dtype=torch.float32)
    ref = few_ref.product(wq[-50:].cpu().numpy(), xs[-50:].cpu().numpy(), wq2.cpu().numpy(),
                          ws2.cpu().numpy(), torch.float32)
    assert few_ref.same_bits(y[-50:], ref)
    del wq, y
    # an output of 4.4 GB
    T, N, K = 4200, 262144, 16
    xq = torch.randint(-127, 128, (T, K), dtype=torch.int8, device="cuda", generator=g)
    wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    xs, ws = torch.rand(T, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    y = dg.w8a8_linear(xq, xs, (wq, ws), dtype=torch.float32)
    ref = few_ref.product(xq[-60:].cpu().numpy(), xs[-60:].cpu().numpy(), wq[-300:].cpu().numpy(),
                          ws[-300:].cpu().numpy(), torch.float32)
    assert few_ref.same_bits(y[-60:, -300:], ref)
    # rows of activations past 2^32 bytes
    x = torch.randn((70000, 16384), dtype=torch.float32, device="cuda", generator=g)
    q, s = dg.quantize_rows_i8(x)
    rq, rs = few_ref.quantize_rows(x[-3:].cpu())
    assert np.array_equal(q[-3:].cpu().numpy(), rq) and np.array_equal(s[-3:].cpu().numpy(), rs)


def test_more_threads_than_a_launch_takes():
    # rows in two launches; channels past what the smallest tiles' grid can hold
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GiB")
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = (1 << 27) + 5
    x = torch.randint(-3, 4, (rows, 1), dtype=torch.int8, device="cuda", generator=g).half()
    q, s = dg.quantize_rows_i8(x)
    # the code of a row's only value is 127 with its sign, or 0
    assert torch.equal(q[:, 0], (torch.sign(x[:, 0]) * 127).to(torch.int8)) and not q[:, 1:].any()
    _, rs = few_ref.quantize_rows(torch.arange(4).half()[:, None])
    assert torch.equal(s, torch.from_numpy(rs).cuda()[x[:, 0].abs().long()])
    del x, q, s
    N, K = (1 << 29) + 17, 16
    wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    ws = torch.rand(N, device="cuda", generator=g)
    xq = torch.randint(-127, 128, (1, K), dtype=torch.int8, device="cuda", generator=g)
    xs = torch.rand(1, device="cuda", generator=g)
    y = dg.w8a8_linear(xq, xs, (wq, ws), dtype=torch.float16)
    for n0 in (0, N // 2, N - 400):
        ref = few_ref.product(xq.cpu().numpy(), xs.cpu().numpy(), wq[n0:n0 + 400].cpu().numpy(),
                              ws[n0:n0 + 400].cpu().numpy(), torch.float16)
        assert few_ref.same_bits(y[:, n0:n0 + 400], ref), n0


def test_longest_row():
    # the most columns a row may have: the last step of every thread passes 2^31.
    # Codes against the definition in fp32, over the whole row and with the row's
    # maximum in its last column; the memory around them stays
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GiB")
    K, pad = 2**31 - 17, 1 << 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((1, K), dtype=torch.float16, device="cuda").normal_(generator=g)
    x[0, K - 1] = -200
    big = torch.full((K + 1 + 2 * pad,), 55, dtype=torch.int8, device="cuda")
    q, s = big[pad:pad + K + 1].view(1, K + 1), torch.empty(1, device="cuda")
    dg.quantize_rows_i8(x, out=(q, s))
    torch.cuda.synchronize()
    scale = np.float32(200) / np.float32(127)
    assert s.item() == scale
    assert (big[:pad] == 55).all() and (big[pad + K + 1:] == 55).all() and q[0, K] == 0
    step = 1 << 26
    for k in range(0, K, step):
        # the quotient in 64 bits rounded to 32 is the one of fp32
        want = torch.round((x[0, k:k + step].double() / s.double()).float()).clamp_(-127, 127).to(torch.int8)
        assert torch.equal(q[0, k:min(k + step, K)], want), k
    for part in (slice(0, 20000), slice(K - 20000, K)):     # and by the host's division
        want = np.rint(x[0, part].float().cpu().numpy() / scale)
        assert np.array_equal(q[0, part].cpu().numpy(), want.astype(np.int8))


def test_more_rows_than_32_bits():
    # refused, whatever the memory holds (as 2^32 + 3 rows modulo 2^32 it would
    # be three)
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GiB")
    x = torch.zeros((2**32 + 3, 1), dtype=torch.float16, device="cuda")
    w = (torch.zeros((4, 16), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda"))
    out = (torch.zeros((3, 16), dtype=torch.int8, device="cuda"), torch.zeros(3, device="cuda"))
    for call in (lambda: dg.quantize_rows_i8(x, out=out), lambda: dg.w8a8_linear_tokens(x, w)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
