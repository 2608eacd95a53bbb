"""Calls of the 8-bit layer's operators at the ends of what they allow and where
their kernels change: long sums and many pairs of an expert, rows and tables of
the longest kind, views, several streams at once, a second device."""
import numpy as np
import pytest

import serve_layer_plain as plain
from test_gpu_serve_i8_ex import call, case
from test_gpu_serve_i8_ex import check as check_product
from test_gpu_serve_moe import Case, check_route, dev, route_case
from test_gpu_serve_norm import check as check_norm
from test_gpu_serve_norm import rows as norm_rows

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


def say(*a):
    print(*a, flush=True)


# few pairs and more than 64, both with more than 12 an expert and sums of 4096
# and longer; pairs that fill one workgroup's 512 slots and one more token
@pytest.mark.parametrize("t,e,k,n_in,n_mid", [(20, 1, 1, 100, 4100), (33, 2, 2, 140, 4200), (64, 1, 1, 70, 4096),
                                              (65, 2, 1, 90, 4160), (512, 6, 1, 64, 130), (513, 6, 1, 64, 130),
                                              (256, 5, 2, 72, 64), (257, 5, 2, 72, 64), (21, 3, 3, 64, 64),
                                              (22, 3, 3, 64, 64), (48, 4, 2, 17, 4097)])
def test_experts_where_the_kernels_change(sv, t, e, k, n_in, n_mid):
    say(f"experts {t} tokens, {k} of {e}, {n_in}x{n_mid}")
    c = Case(t, e, k, n_in, n_mid, seed=t)
    c.check(c.run(sv, torch.float32), torch.float32)


@pytest.mark.parametrize("n_in,n_mid", [(131072, 3), (5, 131072), (131071, 64), (40, 70000)])
def test_longest_rows_of_experts(sv, n_in, n_mid):
    say(f"experts {n_in}x{n_mid}")
    c = Case(2, 2, 2, n_in, n_mid, seed=1)
    c.check(c.run(sv, torch.float32), torch.float32)


@pytest.mark.parametrize("t,n_in", [(1, 131072), (40, 131071), (3, 100003)])
def test_longest_rows_of_the_router(sv, t, n_in):
    say(f"route {t}x{n_in}")
    x, w, b = route_case(t, 9, n_in, 5, BF16, torch.float32)
    check_route(sv.qr_moe_route(x.cuda(), w.cuda(), 4, bias=dev(b)), x, w, 4, "softmax", b, True, 1.0)


def test_many_tokens_of_the_router(sv):
    say("route 70000")
    x, w, _ = route_case(70000, 5, 33, 6, BF16, BF16)
    check_route(sv.qr_moe_route(x.cuda(), w.cuda(), 2, score="sigmoid", renorm=False), x, w, 2, "sigmoid", None, False, 1.0)


def test_logits_near_each_other_in_64_bits(sv):
    """Rows of the router that differ in the last place of one value: fp32 sums
    would not tell them apart."""
    say("near ties")
    rng = np.random.default_rng(3)
    for n_in in (640, 7168):
        row = rng.standard_normal(n_in).astype(np.float32)
        w = np.repeat(row[None], 12, axis=0)
        for e in range(12):
            w[e, 7 * e + 3] = np.nextafter(w[e, 7 * e + 3], np.float32(9.0 if e % 3 else -9.0))
        x = torch.from_numpy(rng.standard_normal((50, n_in)).astype(np.float32))
        w = torch.from_numpy(w)
        check_route(sv.qr_moe_route(x.cuda(), w.cuda(), 5), x, w, 5, "softmax", None, True, 1.0)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_longest_sums_of_a_gated_product(sv, act):
    say(f"gated {act}")
    for t, r, k in ((3, 5, 131072), (70, 40, 131071), (40, 17, 20000)):
        c = case(t, r, k, torch.float32, True, True, True)
        check_product(call(sv, c, k, act, torch.float32), c, k, act, torch.float32)


def test_scales_at_the_ends_of_their_range(sv):
    """Token scales above 2^96 and tiny ones, through gate and residual."""
    say("scales")
    t, r, k = 20, 40, 300
    c = case(t, r, k, torch.float32, False, True, True)
    c["x"][1][::2] = np.float32(2.0) ** 110
    c["x"][1][1::2] = np.float32(2.0) ** -100
    c["w"][1][:] *= np.float32(2.0) ** -115
    check_product(call(sv, c, k, "none", torch.float32), c, k, "none", torch.float32)
    check_product(call(sv, c, k, "relu", torch.float32), c, k, "relu", torch.float32)


def test_views_as_operands(sv):
    """Single tokens and columns of larger tensors, whose strides mean nothing or
    more than a row."""
    say("views")
    buf = norm_rows(8, 400, 1, BF16).cuda()
    one = buf[3:4, 8:264]                                  # one row: any stride
    got = sv.qr_norm_rows_i8(one, None, 1e-6, residual=buf[5:6, 8:264], total=buf[7:8, 100:356])
    check_norm(got, norm_rows(8, 400, 1, BF16)[3:4, 8:264], norm_rows(8, 400, 1, BF16)[5:6, 8:264], None, 1e-6, False)
    c = Case(6, 5, 2, 200, 100, seed=2)
    big = torch.zeros((12, 2), dtype=torch.int32, device="cuda")
    big[4:10] = dev(c.ids)
    y = sv.qr_moe_i8(dev(c.x), dev(c.xd), c.experts(sv), big[4:10], dev(c.weights), dtype=torch.float32)
    c.check(y, torch.float32, residual=False)
    with pytest.raises(ValueError):
        sv.qr_moe_i8(dev(c.x), dev(c.xd), c.experts(sv), big[::2], dev(c.weights))


def test_calls_on_several_streams_at_once(sv):
    """Each with its own scratch memory; the results do not depend on what runs
    beside them."""
    say("streams")
    cases = [Case(t, 9, 2, 260, 330, seed=t) for t in (1, 7, 40, 90)]
    args = [(dev(c.x), dev(c.xd), c.experts(sv), dev(c.ids), dev(c.weights)) for c in cases]
    routes = [route_case(t, 64, 900, t, BF16, BF16) for t in (1, 30, 200, 700)]
    gpu = [(x.cuda(), w.cuda()) for x, w, _ in routes]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = []
    for _ in range(5):
        for i, s in enumerate(streams):
            outs.append((i, sv.qr_moe_i8(*args[i], dtype=torch.float32, stream=s), sv.qr_moe_route(*gpu[i], 6, stream=s)))
    torch.cuda.synchronize()
    first = {}
    for i, y, (ids, wt) in outs:
        if i not in first:
            cases[i].check(y, torch.float32, residual=False)
            check_route((ids, wt), *routes[i][:2], 6, "softmax", None, True, 1.0)
            first[i] = (y, ids, wt)
        assert all(torch.equal(a, b) for a, b in zip(first[i], (y, ids, wt)))


def test_on_a_device_that_is_not_current(sv):
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    c = Case(5, 4, 2, 130, 100, seed=3)
    with torch.cuda.device(1):
        args = (dev(c.x), dev(c.xd), c.experts(sv), dev(c.ids), dev(c.weights))
    c.check(sv.qr_moe_i8(*args, dtype=torch.float32), torch.float32, residual=False)


def test_rows_that_are_not_there_are_not_read(sv):
    """Operands that end where their last row ends, each the last bytes of its
    allocation: what lies behind is other memory, filled with NaN patterns."""
    say("ends of buffers")
    def last(t):
        """t as the last bytes of a larger buffer of 0xff."""
        n = t.numel() * t.element_size()
        buf = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
        at = (4096 // 16) * 16
        part = buf[at:at + n].view(t.dtype).view(t.shape)
        part.copy_(t)
        return part
    c = Case(3, 3, 2, 129, 65, seed=9)
    full = c.full
    ex = sv.MoeExperts(last(dev(full["gate"])), last(dev(c.layer["gated"])), last(dev(full["up"])), last(dev(c.layer["upd"])),
                       last(dev(full["down"])), last(dev(c.layer["downd"])), 129, 65)
    y = sv.qr_moe_i8(last(dev(c.x)), last(dev(c.xd)), ex, last(dev(c.ids)), last(dev(c.weights)), dtype=torch.float32)
    c.check(y, torch.float32, residual=False)
    x, w, _ = route_case(5, 7, 65, 1, BF16, BF16)
    check_route(sv.qr_moe_route(last(x.cuda()), last(w.cuda()), 3), x, w, 3, "softmax", None, True, 1.0)


def test_the_norm_of_rows_around_each_kernels_end(sv):
    say("norm ends")
    for n_rows, k in ((512, 4096), (513, 4096), (513, 2049), (600, 8192), (513, 4104), (520, 8200), (3, 16385), (2, 32768),
                      (514, 512), (513, 513)):
        for dtype in (torch.float32, BF16):
            x, r = norm_rows(n_rows, k, k, dtype), norm_rows(n_rows, k, k + 1, dtype)
            got = sv.qr_norm_rows_i8(x.cuda(), None, 1e-5, residual=r.cuda(), y=True)
            check_norm(got, x, r, None, 1e-5, True)
