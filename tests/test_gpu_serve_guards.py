"""The 8-bit layer's operators on operands that lie between guards: every byte
before the first row and behind the last one (and the scratch memory's) holds a
pattern, which changes no result when it changes and is there after the call. In
turn the patterns are NaN (code -1, an id that is no expert), zeros (an id that
is one) and the largest codes and values."""
import numpy as np
import pytest

from test_gpu_serve_i8_ex import case as product_case
from test_gpu_serve_i8_ex import check as check_product
from test_gpu_serve_moe import Case, check_route, route_case
from test_gpu_serve_norm import check as check_norm
from test_gpu_serve_norm import rows as norm_rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
FILLS = (0xff, 0x00, 0x7f)
GUARD = 4096


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


def say(*a):
    print(*a, flush=True)


class Guarded:
    """Tensors in the middle of buffers of one pattern."""

    def __init__(self, fill):
        self.fill, self.parts = fill, []

    def _part(self, nbytes):
        buf = torch.full((nbytes + 2 * GUARD,), self.fill, dtype=torch.uint8, device="cuda")
        self.parts.append((buf, nbytes))
        return buf[GUARD:GUARD + nbytes]

    def __call__(self, t):
        if t is None:
            return None
        t = torch.from_numpy(np.ascontiguousarray(t)) if isinstance(t, np.ndarray) else t
        part = self._part(t.numel() * t.element_size()).view(t.dtype).view(t.shape)
        part.copy_(t)
        return part

    def new(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        return self._part(n).view(dtype).view(shape)

    def check(self):
        for buf, n in self.parts:
            assert (buf[:GUARD] == self.fill).all() and (buf[GUARD + n:] == self.fill).all()


def same(outs):
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n_rows,n", [(1, 1), (7, 129), (3, 513), (5, 2049), (514, 2053), (2, 4101), (513, 4103), (3, 8203),
                                      (2, 16391)])
def test_norm(sv, n_rows, n, dtype):
    say(f"guards: norm {n_rows}x{n} {dtype}")
    x, r, w = norm_rows(n_rows, n, 1, dtype), norm_rows(n_rows, n, 2, dtype), norm_rows(1, n, 3, dtype)[0].contiguous()
    outs = []
    for fill in FILLS:
        g = Guarded(fill)
        out = dict(total=g.new((n_rows, n), dtype), y=g.new((n_rows, n), dtype),
                   codes=g.new((n_rows, sv.qr_i8_row_bytes(n)), torch.int8), scales=g.new((n_rows,), F32))
        got = sv.qr_norm_rows_i8(g(x), g(w), 1e-5, residual=g(r), **out)
        check_norm(got, x, r, w, 1e-5, True)
        g.check()
        outs.append(got)
    same(outs)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("t,r,k", [(1, 3, 130), (5, 30, 1200), (17, 33, 64), (33, 40, 129), (48, 4097, 128), (20, 3001, 1000),
                                   (65, 200, 129), (100, 2050, 384), (300, 4100, 520), (700, 11001, 70), (2500, 5000, 90)])
def test_product(sv, t, r, k, up, dtype):
    say(f"guards: product {t}x{r}x{k} up={up} {dtype}")
    c = product_case(t, r, k, dtype, up, True, True)
    outs = []
    for fill in FILLS:
        g = Guarded(fill)
        u = c["up"] or (None, None, None)
        y = sv.qr_matmul_i8_ex(g(c["w"][0]), g(c["w"][1]), g(c["x"][0]), g(c["x"][1]), k, bias=g(c["bias"]), act="silu",
                               up=g(u[0]), upd=g(u[1]), up_bias=g(u[2]), residual=g(c["residual"]), out=g.new((t, r), dtype))
        if fill == FILLS[0]:
            check_product(y, c, k, "silu", dtype)
        g.check()
        outs.append((y,))
    same(outs)


# one launch of few experts; 16x16 and 32x32 tiles in 64 bits; rough logits, with
# as many experts as each size of the choice takes
@pytest.mark.parametrize("t,e,k,top_k,xt,wt", [(5, 7, 65, 3, BF16, BF16), (3, 5, 129, 2, F32, BF16), (1, 300, 129, 8, BF16, BF16),
                                               (17, 70, 1001, 5, F32, F32), (40, 1001, 333, 7, BF16, F32),
                                               (5003, 41, 33, 2, BF16, BF16), (5003, 41, 97, 2, F32, F32),
                                               (2049, 257, 2049, 8, BF16, BF16), (6001, 90, 2003, 1, BF16, BF16),
                                               (1301, 1001, 1003, 4, BF16, BF16)])
def test_route(sv, t, e, k, top_k, xt, wt):
    x, w, b = route_case(t, e, k, 7, xt, wt)
    outs = []
    for fill in FILLS:
        say(f"guards: route {t}x{e}x{k} {xt} {wt} {fill:#x}")
        g = Guarded(fill)
        got = sv.qr_moe_route(g(x), g(w), top_k, score="sigmoid", bias=g(b), ids=g.new((t, top_k), torch.int32),
                              weights=g.new((t, top_k), F32),
                              workspace=g.new((sv.qr_moe_route_workspace_bytes(e, t, k),), torch.uint8))
        if fill == FILLS[0]:
            check_route(got, x, w, top_k, "sigmoid", b, True, 1.0)
        g.check()
        outs.append(got)
    same(outs)


@pytest.mark.parametrize("t,e,k,n_in,n_mid", [(1, 1, 1, 1, 1), (3, 3, 2, 129, 65), (33, 2, 1, 141, 300), (70, 3, 1, 333, 100),
                                              (33, 2, 2, 140, 4201), (20, 1, 1, 100, 4103), (257, 5, 2, 73, 67), (65, 64, 6, 150, 64)])
def test_experts(sv, t, e, k, n_in, n_mid):
    say(f"guards: experts {t} tokens, {k} of {e}, {n_in}x{n_mid}")
    c = Case(t, e, k, n_in, n_mid, seed=t)
    if t > 1:
        c.ids[t // 2] = -1                      # a padded token
    outs = []
    for fill in FILLS:
        g = Guarded(fill)
        f, s = c.full, c.layer
        ex = sv.MoeExperts(g(f["gate"]), g(s["gated"]), g(f["up"]), g(s["upd"]), g(f["down"]), g(s["downd"]), n_in, n_mid)
        y = sv.qr_moe_i8(g(c.x), g(c.xd), ex, g(c.ids), g(c.weights), residual=g(c.residual), dtype=F32,
                         out=g.new((t, n_in), F32), workspace=g.new((sv.qr_moe_i8_workspace_bytes(ex, t, k),), torch.uint8))
        if fill == FILLS[0]:
            c.check(y, F32)
        g.check()
        outs.append((y,))
    same(outs)
