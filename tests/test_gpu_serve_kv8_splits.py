"""Attention of few rows whose tokens are split over workgroups, against 64-bit
arithmetic: every width, few splits and many, sequences that use all of them,
some and one in the same call. And what other tests look at only in part: every
block of a cache that a captured graph writes, and whose memory a call takes."""
import numpy as np
import pytest

import serve_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_serve_kv8 import check_attention, dev, fresh, make_kv, say, sv  # noqa: E402,F401


def splits_taken(sv, lens, new, group, heads, dim, block, width):
    """Splits for which the call sizes its workspace (units of 16 rows)."""
    n_tok, n_seq = sum(new), len(lens)
    cache = sv.kv8_cache(1, heads, dim, block, "cuda")
    ws = sv.qr_attention_kv8_workspace_bytes(cache, group * heads, n_tok, n_seq, width)
    one = (n_tok * group // 16 + n_seq) * heads * 16 * (dim + 2) * 4
    assert ws % one == 0
    return ws // one


# lens, new, table width in blocks of 64, splits
FEW = [([1500, 300, 40], [1, 1, 1], 24, 6), ([1090, 17], [1, 0], 18, 5), ([2040, 2040], [3, 2], 32, 8),
       ([1100], [1], 20, 5)]
MANY = [([10000, 2500, 100], [1, 1, 1], 160, 40), ([4700, 0], [2, 0], 75, 19)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,heads", [(1, 3), (4, 2), (10, 1)])
def test_splits(sv, group, heads, dim, bf16):
    for lens, new, width, splits in FEW + MANY:
        say(f"splits={splits} dim={dim} group={group} bf16={bf16} lens={lens}")
        assert splits_taken(sv, lens, new, group, heads, dim, 64, width) == splits
        check_attention(sv, lens, new, group, heads, dim, 64, bf16, seed=dim + splits, width=width)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_splits_of_a_window(sv, dim, bf16):
    """Windows that end in the middle of the splits, and rows without tokens."""
    for window in (3, 700, 2000):
        say(f"split window={window} dim={dim} bf16={bf16}")
        check_attention(sv, [5000, 900, 0], [2, 1, 1], 4, 1, dim, 128, bf16, seed=window, width=50, window=window)


@pytest.mark.parametrize("block", [32, 128])
def test_most_splits(sv, block):
    say(f"128 splits block={block}")
    width = 40000 // block
    assert splits_taken(sv, [39000], [1], 4, 1, 256, block, width) == 128
    check_attention(sv, [39000], [1], 4, 1, 256, block, True, seed=block, width=width)


def test_every_block_that_a_graph_writes(sv):
    """Appends and attention captured once and replayed with other lengths,
    beside the same calls made eagerly: whole caches, bit for bit."""
    say("graph, all blocks")
    heads, dim, block, n_seq, width = 2, 64, 32, 5, 40
    n_blocks = n_seq * width + 10
    table = dev(np.random.default_rng(3).permutation(n_blocks)[:n_seq * width].reshape(n_seq, width))
    start = np.array([0, 5, 31, 64, 1000])
    kv = [x.cuda() for x in make_kv(int(start.sum()), heads, dim, 4, True)]
    caches = [fresh(sv, n_blocks, heads, dim, block) for _ in range(2)]
    for c in caches:
        sv.qr_kv8_append(c, kv[0], kv[1], dev(plain.offsets(start)), dev(start), table)
    cu, lens = dev(np.arange(n_seq + 1)), dev(start + 1)
    k, v = [x.cuda() for x in make_kv(n_seq, heads, dim, 5, True)]
    q = torch.zeros((n_seq, 4 * heads, dim), dtype=torch.bfloat16, device="cuda")

    def step(c):
        sv.qr_kv8_append(c, k, v, cu, lens, table)
        return sv.qr_attention_kv8(q, c, cu, lens, table)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[1])
    for i in range(40):          # past the end of a block in every sequence
        for dst, src in zip((k, v), make_kv(n_seq, heads, dim, 100 + i, True)):
            dst.copy_(src)
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)))
        lens.copy_(dev(start + 1 + i))
        want = step(caches[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        for a, b in zip(caches[0], caches[1]):
            assert torch.equal(a.view(torch.int8), b.view(torch.int8)), i


def stream_of(t):
    """The stream that the memory of t belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def test_memory_comes_from_the_stream_of_the_call(sv, monkeypatch):
    """Outputs and workspaces that a call allocates, for a torch stream, for a
    handle and for the current stream."""
    say("owners")
    heads, dim, block, n = 2, 64, 32, 1500
    table, cu, lens, one = dev([np.arange(50)]), dev([0, n]), dev([n]), dev([0, 3])
    k, v = [x.cuda() for x in make_kv(n, heads, dim, 3, True)]
    q = k.repeat(1, 2, 1)[:3].contiguous()
    cache = fresh(sv, 50, heads, dim, block)
    made = []
    new = sv._new
    monkeypatch.setattr(sv, "_new", lambda *a: made.append(new(*a)) or made[-1])

    def calls(stream):
        made.clear()
        sv.qr_kv8_append(cache, k, v, cu, lens, table, stream=stream)
        o = sv.qr_attention_kv8(q, cache, one, lens, table, stream=stream)
        sv.qr_kv8_read(cache, cu, lens, table, n, stream=stream)
        x, xd = sv.qr_quantize_rows_i8(o.view(3, -1), stream=stream)
        sv.qr_matmul_i8(x, xd, x, xd, 4 * dim, stream=stream)
        torch.cuda.synchronize()
        assert len(made) == 7 and made[0].dtype == torch.bfloat16 and made[1].dtype == torch.uint8
        return {stream_of(t) for t in made}

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    here = torch.cuda.current_stream().cuda_stream
    assert here != side.cuda_stream
    assert calls(None) == {here}
    assert calls(side) == {side.cuda_stream}
    assert calls(side.cuda_stream) == {side.cuda_stream}
    with torch.cuda.stream(side):
        assert calls(None) == {side.cuda_stream}
