"""The serving calls at the ends of what their headers allow: most heads and
groups, codes of -128, caches and tables without blocks, calls that overlap in
time, and the same rows through views that lie differently."""
import numpy as np
import pytest

import serve_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_serve_kv8 import check_attention, check_cache, dev, fresh, make_kv, say, sv  # noqa: E402,F401


@pytest.mark.parametrize("n_out,n_tok", [(70, 1), (70, 20), (140, 150), (6200, 30)])
def test_product_of_smallest_codes(sv, n_out, n_tok):
    """-128 * -128 * 131071 is the largest sum that 31 bits hold."""
    say(f"codes of -128 {n_out}x{n_tok}")
    n_in = 131071
    w, x = [torch.full((n, 131072), -128, dtype=torch.int8, device="cuda") for n in (n_out, n_tok)]
    w[:, n_in:] = 0
    x[:, n_in:] = 0
    x[0] *= -1                   # (wraps: -128 again)
    one = lambda n: torch.ones(n, device="cuda")
    y = sv.qr_matmul_i8(w, one(n_out), x, one(n_tok), n_in, dtype=torch.float32)
    assert bool((y == float(np.float32(128 * 128 * n_in))).all())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("new", [[1, 1], [3, 0]])
def test_most_query_heads_of_a_head(sv, new, bf16):
    say(f"group 1024 new={new} bf16={bf16}")
    check_attention(sv, [100, 33], new, 1024, 1, 64, 32, bf16, seed=1)


@pytest.mark.parametrize("new", [[1, 1], [40, 20]])
def test_most_heads(sv, new):
    say(f"1024 heads new={new}")
    heads, dim, block, n_blocks = 1024, 64, 32, 4
    table = np.array([[2, 0], [3, -1]], dtype=np.int32)
    lens = np.array([40, 20])
    cu = plain.offsets(lens)
    kv = make_kv(cu[-1], heads, dim, 3, True)
    cache, ref = fresh(sv, n_blocks, heads, dim, block), plain.PlainCache(n_blocks, heads, dim, block)
    sv.qr_kv8_append(cache, kv[0].cuda(), kv[1].cuda(), dev(cu), dev(lens), dev(table))
    ref.append([x.float().numpy() for x in kv], cu, lens, table)
    check_cache(cache, ref, slice(None))
    got = sv.qr_kv8_read(cache, dev(cu), dev(lens), dev(table), cu[-1])
    for j in range(2):
        want = np.concatenate([ref.values(table[s], lens[s])[j] for s in range(2)])
        assert torch.equal(got[j].cpu(), torch.from_numpy(want.astype(np.float32)))
    check_attention(sv, [40, 20], new, 1, heads, dim, block, True, seed=2, table=np.where(table < 0, 1, table))


def test_no_blocks(sv):
    """A cache without blocks, a table without columns: nothing is a token."""
    say("no blocks")
    cu, lens = dev([0, 3, 4]), dev([70, 1])
    kv = [x.cuda() for x in make_kv(4, 2, 64, 1, False)]
    q = torch.ones((4, 4, 64), device="cuda")
    for n_blocks, width in ((0, 3), (5, 0), (0, 0)):
        cache = sv.kv8_cache(n_blocks, 2, 64, 32, "cuda")
        before = [t.clone() for t in cache]
        table = torch.zeros((2, width), dtype=torch.int32, device="cuda")
        sv.qr_kv8_append(cache, kv[0], kv[1], cu, lens, table)
        for a, b in zip(before, cache):
            assert torch.equal(a.view(torch.int8), b.view(torch.int8))
        k, v = sv.qr_kv8_read(cache, cu, lens, table, 4)
        out = sv.qr_attention_kv8(q, cache, cu, lens, table)
        for t in (k, v, out):
            assert bool((t == 0).all())


def test_views_that_lie_differently(sv):
    """Keys and values apart in types of stride, from fp32 and bf16, and
    outputs side by side with their queries in one buffer."""
    say("views")
    heads, dim, block, n = 2, 64, 32, 75
    g = torch.Generator().manual_seed(4)
    table, cu, lens = dev([[2, 0, 1]]), dev([0, n]), dev([n])
    for dtype in (torch.float32, torch.bfloat16):
        wide = torch.randn((n, heads + 3, dim), generator=g).to(dtype).cuda()
        k = wide[:, 1:1 + heads]
        v = torch.randn((2 * n, heads, dim), generator=g).to(dtype).cuda()[::2]
        a, b = [fresh(sv, 3, heads, dim, block) for _ in range(2)]
        sv.qr_kv8_append(a, k, v, cu, lens, table)
        sv.qr_kv8_append(b, k.contiguous(), v.contiguous(), cu, lens, table)
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        both = torch.full((n, 2, heads + 1, dim), 9.0, dtype=dtype, device="cuda")
        sv.qr_kv8_read(a, cu, lens, table, n, k=both[:, 0, 1:], v=both[:, 1, :heads])
        want = sv.qr_kv8_read(a, cu, lens, table, n, dtype=dtype)
        assert torch.equal(both[:, 0, 1:], want[0]) and torch.equal(both[:, 1, :heads], want[1])
        assert bool((both[:, 0, 0] == 9).all()) and bool((both[:, 1, heads] == 9).all())
        # queries and outputs, in either order, as parts of one buffer
        for new in (n, 3):
            buf = torch.randn((new, 2, 4, dim), generator=g).to(dtype).cuda()
            one = dev([0, new])
            for qi in (0, 1):
                q = buf[:, qi].clone()
                expect = sv.qr_attention_kv8(q, a, one, lens, table)
                sv.qr_attention_kv8(buf[:, qi], a, one, lens, table, out=buf[:, 1 - qi])
                assert torch.equal(buf[:, 1 - qi], expect) and torch.equal(buf[:, qi], q)
            with pytest.raises(Exception, match="overlap"):
                sv.qr_attention_kv8(buf[:, 0], a, one, lens, table, out=buf[:, 0])
            with pytest.raises(Exception, match="overlap"):
                sv.qr_attention_kv8(buf.view(new, 8, dim)[:, 1:5], a, one, lens, table, out=buf.view(new, 8, dim)[:, 4:8])


def test_calls_that_overlap_in_time(sv):
    """Two streams with work of their own, and one cache that both read."""
    say("two streams")
    heads, dim, block, n = 4, 128, 64, 6000
    cache = fresh(sv, 100, heads, dim, block)
    table, lens = dev([np.arange(100)]), dev([n])
    k, v = [x.cuda() for x in make_kv(n, heads, dim, 3, True)]
    sv.qr_kv8_append(cache, k, v, dev([0, n]), lens, table)
    qs = [torch.randn((m, 16, dim), generator=torch.Generator().manual_seed(m)).to(torch.bfloat16).cuda()
          for m in (1, 200)]
    cus = [dev([0, 1]), dev([0, 200])]
    want = [sv.qr_attention_kv8(q, cache, cu, lens, table) for q, cu in zip(qs, cus)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(sv.qr_attention_kv8(qs[i], cache, cus[i], lens, table, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o, want[i])
