"""The 8-bit layer's operators one behind the other, as a serving program runs
them: norm, router, experts with the residual, norm, gated product, 8-bit rows,
product with the residual. Every step against the plain form on what the step
before gave, and the whole run captured into a graph."""
import numpy as np
import pytest

import serve_layer_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


def num(t):
    return t.float().cpu().numpy()


class Layer:
    def __init__(self, sv, n_in, n_mid, experts, wide):
        g = torch.Generator().manual_seed(3)
        mat = lambda *s: torch.randn(s, generator=g) / np.sqrt(s[-1])
        quant = lambda w: sv.qr_quantize_rows_i8(w.reshape(-1, w.shape[-1]).cuda())
        self.sv, self.n_in, self.n_mid, self.wide = sv, n_in, n_mid, wide
        parts = []
        for r, k in ((n_mid, n_in), (n_mid, n_in), (n_in, n_mid)):
            c, s = quant(mat(experts, r, k))
            parts += [c.view(experts, r, -1), s.view(experts, r)]
        self.experts = sv.MoeExperts(*parts, n_in=n_in, n_mid=n_mid)
        self.plain_experts = {n: p.cpu().numpy() for n, p in zip(("gate", "gated", "up", "upd", "down", "downd"), parts)}
        for n, k in (("gate", n_in), ("up", n_in), ("down", n_mid)):
            self.plain_experts[n] = self.plain_experts[n][..., :k]
        self.router = mat(experts, n_in).to(BF16).cuda() * 3
        self.norms = [(1 + 0.1 * torch.randn(n_in, generator=g)).to(BF16).cuda() for _ in range(2)]
        self.gate, self.up, self.down = quant(mat(wide, n_in)), quant(mat(wide, n_in)), quant(mat(n_in, wide))

    def run(self, x, residual):
        """All steps' outputs by name."""
        sv, o = self.sv, {}
        o["c1"], o["s1"], o["t1"], o["y1"] = sv.qr_norm_rows_i8(x, self.norms[0], residual=residual, y=True)
        o["ids"], o["wt"] = sv.qr_moe_route(o["y1"], self.router, 2)
        o["m"] = sv.qr_moe_i8(o["c1"], o["s1"], self.experts, o["ids"], o["wt"], residual=o["t1"])
        o["c2"], o["s2"], _, _ = sv.qr_norm_rows_i8(o["m"], self.norms[1])
        o["g"] = sv.qr_matmul_i8_ex(*self.gate, o["c2"], o["s2"], self.n_in, act="silu", up=self.up[0], upd=self.up[1])
        o["c3"], o["s3"] = sv.qr_quantize_rows_i8(o["g"])
        o["out"] = sv.qr_matmul_i8_ex(*self.down, o["c3"], o["s3"], self.wide, residual=o["m"])
        return o

    def check(self, o, x, residual):
        n, w = self.n_in, self.wide
        eq = lambda a, b: np.count_nonzero(a != b) <= 1 + a.size // 100000 and np.max(np.abs(a - b), initial=0) <= 1
        t, y = plain.norm(num(x), num(residual), num(self.norms[0]), 1e-6, BF16)
        assert np.array_equal(num(o["t1"]), t)
        c, s, _ = plain.code_rule(y)
        assert eq(o["c1"].cpu().numpy()[:, :n].astype(int), c.astype(int)) and np.allclose(num(o["s1"]), s, rtol=2.0 ** -23)
        ids, wt = plain.route(o["y1"].double().cpu().numpy(), self.router.double().cpu().numpy(), 2, "softmax", None, True, 1.0)
        assert np.array_equal(o["ids"].cpu().numpy(), ids) and np.allclose(num(o["wt"]), wt, rtol=2.0 ** -23)
        want, bound = plain.experts(self.plain_experts, o["c1"].cpu().numpy()[:, :n], num(o["s1"]), o["ids"].cpu().numpy(),
                                    num(o["wt"]), "silu", num(o["t1"]), BF16)
        assert np.all(np.abs(num(o["m"]) - want) <= bound)
        _, y = plain.norm(num(o["m"]), None, num(self.norms[1]), 1e-6, BF16)
        c, s, _ = plain.code_rule(y)
        assert eq(o["c2"].cpu().numpy()[:, :n].astype(int), c.astype(int)) and np.allclose(num(o["s2"]), s, rtol=2.0 ** -23)
        host = lambda p, k: (p[0].cpu().numpy()[:, :k], num(p[1]))
        x2 = host((o["c2"], o["s2"]), n)
        want, bound = plain.product(*host(self.gate, n), *x2, None, "silu", host(self.up, n) + (None,), None, BF16)
        assert np.all(np.abs(num(o["g"]) - want) <= bound)
        want, bound = plain.product(*host(self.down, w), *host((o["c3"], o["s3"]), w), None, "none", None, num(o["m"]), BF16)
        assert np.all(np.abs(num(o["out"]) - want) <= bound)


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_a_layer(sv, tokens):
    print(f"layer {tokens}", flush=True)
    layer = Layer(sv, 256, 192, 12, 700)
    g = torch.Generator().manual_seed(tokens)
    new = lambda: (torch.randn((tokens, 256), generator=g).to(BF16).cuda(), (3 * torch.randn((tokens, 256), generator=g)).to(BF16).cuda())
    x, r = new()
    layer.check(layer.run(x, r), x, r)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = layer.run(x, r)
    for _ in range(3):
        nx, nr = new()
        x.copy_(nx), r.copy_(nr)
        graph.replay()
        torch.cuda.synchronize()
        layer.check(out, x, r)
        eager = layer.run(x, r)
        assert all(torch.equal(out[k], eager[k]) for k in out)
