"""GPU: the routed-expert layer for few tokens (dgw4_moe_few, _routed) against
its plain 64-bit form, element by element within the bound that counts the
kernel's roundings (tests/few_ref.py), and the identities that hold bit for
bit: reruns, the two weight layouts, routed against router + layer, graph
replays, padding."""
import numpy as np
import pytest
import torch

import w4a16_grouped_moe_amd as dg
from tests import few_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    dg.lib()


class Case:
    def __init__(self, T, E, topk, d, m, gg=128, dgr=64, seed=0, same_sign=False):
        rng = np.random.default_rng([seed, T, E, topk, d, m])
        self.T, self.E, self.topk, self.d, self.m = T, E, topk, d, m
        gw = rng.standard_normal((E, 2 * m, d), dtype=np.float32) * np.float32(0.02)
        dw = rng.standard_normal((E, d, m), dtype=np.float32) * np.float32(0.02)
        if same_sign:                     # groups of one sign: zero points off the grid
            gw, dw = np.abs(gw), -np.abs(dw)
        self.gu = (*dg.quantize_rtn(torch.from_numpy(gw).cuda(), gg), gg)
        self.dn = (*dg.quantize_rtn(torch.from_numpy(dw).cuda(), dgr), dgr)
        self.x = torch.from_numpy(rng.standard_normal((T, d), dtype=np.float32)).half().cuda()
        self.logits = torch.from_numpy(rng.standard_normal((T, E), dtype=np.float32) * 2).cuda()
        self.ids, self.w = dg.router(self.logits, topk)

    def tiled(self):
        return dg.pack_tiled(self.gu), dg.pack_tiled(self.dn)

    def check(self, out, what="", x=None, ids=None, w=None):
        host = lambda p: (*(t.cpu().numpy() for t in p[:3]), p[3])
        ref, bound = few_ref.moe((self.x if x is None else x).cpu().numpy(),
                                 (self.ids if ids is None else ids).cpu().numpy(),
                                 (self.w if w is None else w).cpu().numpy(),
                                 host(self.gu), host(self.dn), self.E)
        err = np.abs(out.cpu().numpy().astype(np.float64) - ref)
        print(f"[few] {what} worst error / bound {np.nanmax(err / bound):.3f}", flush=True)
        assert (err <= bound).all(), what


SHAPES = [
    dict(T=1, E=8, topk=2, d=512, m=192),
    dict(T=1, E=1, topk=1, d=128, m=64),
    dict(T=1, E=24, topk=8, d=2816, m=704),            # the layer's widths, one token
    dict(T=3, E=20, topk=8, d=2816, m=704),
    dict(T=7, E=5, topk=3, d=256, m=64, gg=64),
    dict(T=16, E=16, topk=4, d=384, m=320),
    dict(T=64, E=9, topk=8, d=512, m=192),             # 512 assignments, several tiles an expert
    dict(T=512, E=3, topk=1, d=256, m=128, dgr=128),   # one choice each, many tiles
    dict(T=33, E=1000, topk=15, d=128, m=64),          # many experts
    dict(T=2, E=70, topk=64, d=128, m=64),             # the widest choice
    dict(T=5, E=6, topk=2, d=4096, m=1408, gg=64, dgr=128),
    dict(T=9, E=4, topk=2, d=640, m=64, gg=128, dgr=64, same_sign=True),
    # past 64 assignments: every number of steps and scale pieces of down
    dict(T=20, E=4, topk=4, d=256, m=704),
    dict(T=17, E=5, topk=4, d=128, m=1024),
    dict(T=33, E=3, topk=2, d=128, m=1408),
    dict(T=70, E=2, topk=1, d=256, m=2048),
    dict(T=23, E=6, topk=3, d=128, m=768, dgr=128),
    dict(T=40, E=6, topk=2, d=384, m=1408, gg=64, dgr=128),
    # up to 64: halves of m in one step and in several
    dict(T=4, E=3, topk=2, d=128, m=1408),
    dict(T=3, E=4, topk=4, d=256, m=2048),
    dict(T=2, E=3, topk=1, d=128, m=64, dgr=64),
    dict(T=1, E=3, topk=3, d=8192, m=128),             # the most groups of d
    # routing inside the first launch: more than 128 experts, the widest choice
    dict(T=7, E=200, topk=5, d=128, m=64),
    dict(T=1, E=256, topk=64, d=128, m=64),
    dict(T=64, E=129, topk=1, d=128, m=64),
    # up to 64 assignments whose H does not fit down's LDS, or whose down is apart
    dict(T=6, E=9, topk=8, d=2304, m=1408),
    dict(T=64, E=4, topk=1, d=2304, m=1024),
    dict(T=8, E=10, topk=8, d=128, m=2048),
    dict(T=8, E=9, topk=8, d=512, m=704),
    dict(T=2, E=9, topk=8, d=1536, m=1408, dgr=128),
    dict(T=4, E=9, topk=8, d=2304, m=1408),            # 90 KB of H
    dict(T=8, E=9, topk=8, d=2432, m=704),
    dict(T=17, E=4, topk=4, d=128, m=4096, dgr=128),   # the longest m
    dict(T=2, E=5, topk=4, d=256, m=4096, dgr=128),
    dict(T=2, E=5, topk=4, d=2304, m=4096, dgr=128),
    # every number of groups that a wave holds, where K's last share is short
    dict(T=2, E=4, topk=2, d=1152, m=128, gg=128, dgr=128),
    dict(T=3, E=4, topk=2, d=1920, m=320, gg=128, dgr=64),
    dict(T=3, E=4, topk=2, d=576, m=384, gg=64, dgr=128),
    dict(T=2, E=4, topk=3, d=1472, m=512, gg=64, dgr=128),
    dict(T=1, E=4, topk=2, d=2112, m=640, gg=64, dgr=128),
    dict(T=25, E=4, topk=3, d=960, m=320, gg=64, dgr=64),
    dict(T=25, E=4, topk=3, d=1280, m=512, gg=128, dgr=128),
    dict(T=22, E=3, topk=3, d=256, m=128, gg=64, dgr=64),
    dict(T=34, E=3, topk=2, d=1088, m=576, gg=64, dgr=64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_matches_plain_form(shape):
    c = Case(**shape)
    out = dg.moe_few(c.x, c.ids, c.w, c.gu, c.dn)
    c.check(out, str(shape))
    # the tiled layout, a rerun into a used workspace, and the form from logits
    gu, dn = c.tiled()
    n = dg.moe_few_workspace_bytes(c.T, c.topk, c.E, c.d, c.m, gu[3], dn[3])
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    for pair in ((gu, dn), (c.gu, dn), (gu, c.dn), (gu, dn)):
        again = dg.moe_few(c.x, c.ids, c.w, *pair, workspace=ws)
        assert few_ref.same_bits(out, again)
    routed = dg.moe_few_routed(c.x, c.logits, c.topk, gu, dn, workspace=ws)
    assert few_ref.same_bits(out, routed)


@pytest.mark.parametrize("E", [5, 64, 65, 128, 130, 256])
def test_routing_edges(E):
    # ties to the lower id, +0 and -0 equal, negative values, subnormals and the
    # extremes of fp32: the form from logits chooses and weighs as the router
    T, topk = 8, min(E, 8)
    c = Case(T=T, E=E, topk=topk, d=128, m=64, seed=11)
    rng = np.random.default_rng(E)
    lg = np.round(rng.standard_normal((T, E)) * 2).astype(np.float32)      # many ties
    lg[1] = 0.5
    lg[2] = np.where(np.arange(E) % 2 == 0, np.float32(0.0), np.float32(-0.0))
    lg[3] = -np.abs(lg[3]) - 1
    lg[4] = rng.choice(np.array([1e-40, -1e-40, 3.4e38, -3.4e38, 0], dtype=np.float32), E)
    lg[5, :] = -3.4e38
    lg[6] = rng.standard_normal(E) * 1e-3
    logits = torch.from_numpy(lg).cuda()
    ids, w = dg.router(logits, topk)
    assert few_ref.same_bits(dg.moe_few_routed(c.x, logits, topk, c.gu, c.dn),
                             dg.moe_few(c.x, ids, w, c.gu, c.dn))


def test_agrees_with_the_layer():
    # the tile path of the same layer, within both paths' roundings (1e-2 of
    # the largest output, the layer's stated tolerance)
    c = Case(T=12, E=16, topk=8, d=2816, m=704, seed=3)
    a = dg.moe_few(c.x, c.ids, c.w, c.gu, c.dn).double()
    b = dg.moe_forward(c.x, c.ids, c.w, c.gu, c.dn).double()
    assert (a - b).abs().max() <= 2e-2 * b.abs().max()


def test_dead_ids_and_padding():
    # ids outside [0, E) count for nothing, a token without live ids gets
    # zeros, whatever its row of x or its weights hold
    c = Case(T=10, E=6, topk=3, d=256, m=128, seed=4)
    ids, w, x = c.ids.clone(), c.w.clone(), c.x.clone()
    ids[3] = -1
    ids[4, 1] = 6
    ids[5, 0] = -2**31
    ids[6, 2] = 2**31 - 1
    ids[9] = 99
    w[3] = float("nan")
    w[9] = float("inf")
    w[4, 1] = float("nan")
    x[3], x[9] = float("nan"), float("inf")
    clean = x.clone()
    clean[3], clean[9] = 0, 0
    out = dg.moe_few(x, ids, w, c.gu, c.dn)
    assert not out[3].any() and not out[9].any()
    c.check(out, "dead ids", x=clean, ids=ids, w=torch.nan_to_num(w, 0, 0, 0))
    none = dg.moe_few(x, torch.full_like(ids, -1), w, c.gu, c.dn)
    assert not none.any()


def test_equal_ids_each_count():
    c = Case(T=5, E=4, topk=4, d=256, m=64, seed=5)
    ids = torch.tensor([[2, 2, 2, 2], [0, 1, 0, 1], [3, 3, 0, 0], [1, 2, 3, 0], [2, 2, 2, 1]],
                       dtype=torch.int32, device="cuda")
    c.check(dg.moe_few(c.x, ids, c.w, c.gu, c.dn), "equal ids", ids=ids)


def test_one_expert_takes_everything():
    c = Case(T=64, E=5, topk=1, d=256, m=64, seed=6)
    ids = torch.full_like(c.ids, 4)
    c.check(dg.moe_few(c.x, ids, c.w, c.gu, c.dn), "one expert", ids=ids)


def test_nan_stays_in_its_row():
    c = Case(T=17, E=3, topk=2, d=256, m=64, seed=7)
    base = dg.moe_few(c.x, c.ids, c.w, c.gu, c.dn)
    x = c.x.clone()
    x[8, 5] = float("nan")
    out = dg.moe_few(x, c.ids, c.w, c.gu, c.dn)
    keep = [t for t in range(17) if t != 8]
    assert few_ref.same_bits(out[keep], base[keep])
    assert torch.isnan(out[8]).all()


def test_writes_only_its_rows():
    c = Case(T=6, E=8, topk=2, d=256, m=64, seed=8)
    big = torch.full((9, 256), 7.0, dtype=torch.float16, device="cuda")
    n = dg.moe_few_workspace_bytes(6, 2, 8, 256, 64)
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    dg.moe_few(c.x, c.ids, c.w, c.gu, c.dn, workspace=ws[:n], out=big[:6])
    assert (big[6:] == 7.0).all() and (ws[n:] == 0xA5).all()
    c.check(big[:6], "guarded")


def test_empty_batch():
    c = Case(T=1, E=4, topk=2, d=128, m=64)
    out = dg.moe_few(c.x[:0], c.ids[:0], c.w[:0], c.gu, c.dn)
    assert out.shape == (0, 128)
    assert dg.moe_few_routed(c.x[:0], c.logits[:0], 2, c.gu, c.dn).shape == (0, 128)


def test_captured_and_replayed():
    c = Case(T=4, E=12, topk=3, d=512, m=192, seed=9)
    gu, dn = c.tiled()
    n = dg.moe_few_workspace_bytes(4, 3, 12, 512, 192, gu[3], dn[3])
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    x, lg = c.x.clone(), c.logits.clone()
    out = torch.empty((4, 512), dtype=torch.float16, device="cuda")
    dg.moe_few_routed(x, lg, 3, gu, dn, workspace=ws[0], out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.moe_few_routed(x, lg, 3, gu, dn, workspace=ws[0], out=out)
    for i in range(4):
        x.copy_(torch.roll(c.x, i, 0) * (1 + 0.1 * i))
        lg.copy_(torch.roll(c.logits, i, 1))
        graph.replay()
        eager = dg.moe_few_routed(x, lg, 3, gu, dn, workspace=ws[1])
        torch.cuda.synchronize()
        assert few_ref.same_bits(out, eager), i


def test_two_streams():
    c = Case(T=8, E=16, topk=4, d=512, m=192, seed=10)
    base = dg.moe_few(c.x, c.ids, c.w, c.gu, c.dn)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(base) for _ in range(2)]
    n = dg.moe_few_workspace_bytes(8, 4, 16, 512, 192)
    wss = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, o, ws in zip(streams, outs, wss):
            with torch.cuda.stream(st):
                dg.moe_few(c.x, c.ids, c.w, c.gu, c.dn, workspace=ws, out=o)
    torch.cuda.synchronize()
    assert few_ref.same_bits(outs[0], base) and few_ref.same_bits(outs[1], base)
