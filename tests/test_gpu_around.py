"""Norm, adapters and router balance as a program runs them: together with the
8-bit product and the gated block, on streams, in graphs, with shared scratch memory."""

import pytest
import torch

import lru_expert_cache_amd as ft
from tests import around_case as ac
from tests import dense_case as dc

pytestmark = pytest.mark.gpu


def _scratch(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda").fill_(0xFF)


class Serving:
    """A block's entry in a serving step: the norm leaves the sum, 16-bit rows and codes; the codes go through the
    shared 8-bit projection, the rows through the requests' adapters, which add to its 32-bit results."""

    def __init__(self, T, H, N, R=16, n=5, seed=0):
        self.T, self.H, self.N = T, H, N
        self.norm = ac.Norm(T, H, seed=seed)
        self.ad = ac.Adapters(T, H, N, R, n, "bf16", "fp32", seed=seed)
        g = ac.gen(50 + seed)
        w = torch.randn(N, H, generator=g, device="cuda") * H**-0.5
        self.w, self.ws = torch.empty(N, H, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
        ft.ft_moe_int_quantize(ft.FT_DT_F32, N, H, w, self.w, self.ws)
        self.m = ft.make_int_matmul(T, H, N, ft.FT_DT_F32)
        e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        self.sum, self.y, self.codes, self.scale = e(T, H), e(T, H), e(T, H, t=torch.int8), e(T, t=torch.float32)
        self.p, self.out = e(T, N, t=torch.float32), e(T, N)
        self.w1, self.w2 = _scratch(ft.ft_moe_int_matmul_work(self.m)), self.ad.work()
        torch.cuda.synchronize()

    def run(self, stream=None):
        n, a = self.norm, self.ad
        ft.ft_moe_rms_norm_forward(n.d, n.x, n.residual, n.weight, self.sum, self.y, self.codes, self.scale, stream)
        ft.ft_moe_int_matmul(self.m, self.codes, self.scale, self.w, self.ws, self.p, self.w1, stream)
        ft.ft_moe_adapters_apply(a.d, self.y, a.ids, a.a, a.b, a.scale, self.p, self.out, self.w2, stream)

    def outputs(self):
        return (self.sum, self.y, self.codes, self.scale, self.p, self.out)


@pytest.mark.parametrize("T,H,N", [(1, 256, 128), (33, 1024, 520), (300, 777, 333)])
def test_serving_step(T, H, N):
    """Each step's results against the 64-bit values for what the step before left."""
    s = Serving(T, H, N)
    s.run()
    torch.cuda.synchronize()
    ref = s.norm.forward_reference()
    for k, v in (("sum", s.sum), ("y", s.y)):
        ac.check(v, ref[k], k)
    assert torch.equal(s.codes, ref["codes"]) and torch.equal(s.scale, ref["scale"])
    ac.check(s.p, dc.int_product_reference(s.codes, s.scale, s.w, s.ws, torch.float32), "projection")
    s.ad.x, s.ad.base = s.y, s.p
    ac.check(s.out, s.ad.reference(), "out")


class Training:
    """A training step's block: norm, router logits and their balance, the gated block on the norm's rows; then the
    gradients of all of it back to the stream."""

    def __init__(self, T, H, I, E, k, seed=0):
        self.T, self.H, self.E, self.k = T, H, E, k
        self.norm, self.ffn = ac.Norm(T, H, "bf16", "fp32", seed=seed), dc.Ffn(T, H, I, seed=seed)
        self.bal = ac.Balance(T, E, k, masked=0.1, seed=seed)
        self.router = torch.randn(E, H, generator=ac.gen(60 + seed), device="cuda") * H**-0.5
        e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        f = torch.float32
        self.sum, self.y, self.out, self.gu = e(T, H, t=f), e(T, H), e(T, H), e(T, 2 * I)
        self.sel, self.w, self.counts, self.loss = e(T, k, t=torch.int32), e(T, k, t=f), e(E + 1, t=torch.int32), e(1, t=f)
        self.dz, self.dx_ffn, self.dy = e(T, E, t=f), e(T, H), e(T, H)
        self.dw = [e(I, H), e(I, H), e(H, I)]
        self.dx, self.dres, self.dweight = e(T, H), e(T, H, t=f), e(H)
        n, b, g = self.norm, self.bal, self.ffn
        self.work = [_scratch(v) for v in (ft.ft_moe_balance_work(b.d), ft.ft_moe_gated_ffn_work(g.desc),
                                           ft.ft_moe_gated_ffn_work(g.desc, True), ft.ft_moe_rms_norm_work(n.d))]
        torch.cuda.synchronize()

    def run(self, stream=None):
        n, b, g = self.norm, self.bal, self.ffn
        ft.ft_moe_rms_norm_forward(n.d, n.x, n.residual, n.weight, self.sum, self.y, stream=stream)
        torch.mm(self.y.float(), self.router.t(), out=b.z)
        ft.ft_moe_balance_forward(b.d, b.z, b.valid, self.sel, self.w, self.counts, self.loss, self.work[0], stream)
        ft.ft_moe_gated_ffn_forward(g.desc, self.y, g.wg, g.wu, g.wd, self.out, self.gu, self.work[1], stream)
        ft.ft_moe_gated_ffn_backward(g.desc, self.y, g.wg, g.wu, g.wd, self.gu, g.dy, self.dx_ffn, *self.dw, self.work[2], stream)
        ft.ft_moe_balance_backward(b.d, b.z, b.valid, self.sel, self.w, self.counts, b.dw, b.dloss, self.dz, stream)
        torch.add(self.dx_ffn, torch.mm(self.dz, self.router), out=self.dy)
        ft.ft_moe_rms_norm_backward(n.d, self.sum, n.weight, self.dy, n.dsum, self.dx, self.dres, self.dweight, self.work[3], stream)

    def outputs(self):
        return (self.sum, self.y, self.out, self.sel, self.w, self.counts, self.loss, self.dz, self.dx_ffn, *self.dw, self.dx,
                self.dres, self.dweight)


@pytest.mark.parametrize("T,H,I,E,k", [(5, 64, 48, 8, 2), (200, 512, 256, 60, 6)])
def test_training_step(T, H, I, E, k):
    """Each step's results against the 64-bit values for what the step before left."""
    s = Training(T, H, I, E, k)
    s.run()
    torch.cuda.synchronize()
    n, b, g = s.norm, s.bal, s.ffn
    ref = n.forward_reference()
    ac.check(s.sum, ref["sum"], "sum")
    ac.check(s.y, ref["y"], "y")
    r = b.reference()
    assert torch.equal(s.sel, r["sel"]) and torch.equal(s.counts, r["counts"])
    ac.check(s.w, r["w"], "w")
    ac.check(s.loss, r["loss"], "loss")
    ac.check(s.dz, b.backward_reference(), "dlogits")
    g.x = s.y
    (ry, rgu) = g.forward_reference()
    dc.check(s.out, ry, "out")
    dc.check(s.gu, rgu, "gu")
    for v, q, name in zip((s.dx_ffn, *s.dw), g.backward_reference(s.gu), ("dx", "dwg", "dwu", "dwd")):
        dc.check(v, q, name)
    n.s, n.dy = s.sum, s.dy
    for name, q in n.backward_reference().items():
        ac.check({"dx": s.dx, "dresidual": s.dres, "dweight": s.dweight}[name], q, name)


def _replayed(make, change):
    s = make()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.run(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run(torch.cuda.current_stream())
    g = ac.gen(8)
    for _ in range(4):
        change(s, g)
        s.run(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        want = [v.clone() for v in s.outputs()]
        for v in s.outputs():
            v.fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), want))


@pytest.mark.parametrize("T", [1, 40, 700])
def test_serving_graph_replays(T):
    """Other tokens and other adapters for each replay."""

    def change(s, g):
        s.norm.x.copy_(torch.randn(s.T, s.H, generator=g, device="cuda"))
        s.ad.ids.copy_(torch.randint(-1, s.ad.count, (s.T,), generator=g, device="cuda"))

    _replayed(lambda: Serving(T, 512, 264), change)


@pytest.mark.parametrize("T", [30, 2500])
def test_training_graph_replays(T):
    def change(s, g):
        s.norm.x.copy_(torch.randn(s.T, s.H, generator=g, device="cuda"))
        s.bal.valid.copy_(torch.rand(s.T, generator=g, device="cuda") < 0.8)

    _replayed(lambda: Training(T, 256, 128, 40, 4), change)


def test_graphs_that_share_scratch_memory_in_turn():
    """Two captured calls with the same scratch memory, replayed one after the other."""
    a, b = Serving(100, 512, 264, seed=1), Serving(90, 512, 264, seed=2)
    work = _scratch(max(a.w2.numel(), b.w2.numel()))
    a.w2 = b.w2 = work
    want, graphs = [], []
    for s in (a, b):
        s.run(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        want.append([v.clone() for v in s.outputs()])
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.run(torch.cuda.current_stream())
        graphs.append(graph)
    for _ in range(3):
        for s in (a, b):
            for v in s.outputs():
                v.fill_(77)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            assert all(torch.equal(x, y) for x, y in zip(s.outputs(), w))


def test_two_streams_at_once():
    """Calls on two streams, each with scratch memory of its own, do not disturb each other."""
    steps = [Serving(500, 1024, 520, seed=i) for i in range(2)] + [Training(700, 512, 256, 64, 8, seed=i) for i in range(2)]
    want = []
    for s in steps:
        s.run(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        want.append([v.clone() for v in s.outputs()])
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s in steps:
            for v in s.outputs():
                v.fill_(77)
        torch.cuda.synchronize()
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run(stream)
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(x, y) for x, y in zip(s.outputs(), w))


def test_host_memory_is_refused():
    n, a, b = ac.Norm(4, 32), ac.Adapters(4, 32, 16, 8, 2), ac.Balance(4, 8, 2)
    host = torch.empty(64, 64)
    for call in (lambda: ft.ft_moe_rms_norm_forward(n.d, n.x, n.residual, host, None, n.dy),
                 lambda: ft.ft_moe_rms_norm_forward(n.d, n.x, n.residual, n.weight, None, host),
                 lambda: ft.ft_moe_rms_norm_backward(n.d, n.s, n.weight, n.dy, None, host, work=n.work()),
                 lambda: ft.ft_moe_adapters_apply(a.d, a.x, a.ids.cpu(), a.a, a.b, a.scale, a.base, a.apply(), a.work()),
                 lambda: ft.ft_moe_adapters_apply(a.d, a.x, a.ids, a.a, a.b, a.scale, a.base, host, a.work()),
                 lambda: ft.ft_moe_balance_backward(b.d, b.z, None, None, None, host, None, None, torch.empty_like(b.z))):
        with pytest.raises(ft.FtError) as e:
            call()
        assert e.value.code == ft.FT_E_INVALID and "memory of device" in str(e.value)


def test_columns_of_one_buffer():
    """Input and output rows that lie beside each other are no overlap."""
    buf = torch.randn(30, 300, device="cuda").to(torch.bfloat16)
    n = ac.Norm(30, 100)
    n.d.ld_x = n.d.ld_y = n.d.ld_residual = 300
    x, res, y = buf[:, :100], buf[:, 100:200], buf[:, 200:]
    n.x, n.residual = x.clone(), res.clone()
    ref = n.forward_reference()
    ft.ft_moe_rms_norm_forward(n.d, x, res, n.weight, None, y)
    ac.check(y, ref["y"], "y")
    assert torch.equal(x, n.x) and torch.equal(res, n.residual)
