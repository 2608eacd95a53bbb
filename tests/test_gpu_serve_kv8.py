"""The paged 8-bit cache and attention over it on the GPU, through the C-ABI,
against the plain CPU forms: codes, scales and values bit for bit, attention
within the bound that serve_plain.attention derives."""
import numpy as np
import pytest

import serve_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


def say(*a):
    print(*a, flush=True)


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def make_kv(n, heads, dim, seed, bf16):
    g = torch.Generator().manual_seed(seed)
    kv = [torch.randn((n, heads, dim), generator=g) * torch.exp(torch.randn((n, 1, 1), generator=g)) for _ in range(2)]
    return [x.to(torch.bfloat16) for x in kv] if bf16 else kv


def check_cache(cache, ref, blocks):
    """Scales and codes of the given blocks, bit for bit."""
    want = ref.device_tensors()
    for got, exp in zip(cache, want):
        a, b = got.cpu()[blocks], exp[blocks]
        if a.dtype == torch.float32:
            a, b = a.view(torch.int32), b.view(torch.int32)
        assert torch.equal(a, b)


def fresh(sv, n_blocks, heads, dim, block):
    c = sv.kv8_cache(n_blocks, heads, dim, block, "cuda")
    for t in c:
        t.zero_()
    return c


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("dim,block,heads", [(64, 32, 3), (128, 64, 2), (256, 128, 1), (128, 32, 8), (64, 128, 1)])
def test_append_in_steps_and_read(sv, dim, block, heads, bf16):
    """Chunks that start and end anywhere in a block, one token at a time
    among them; scales that grow and codes that follow."""
    say(f"append dim={dim} block={block} heads={heads} bf16={bf16}")
    rng = np.random.default_rng(dim + block)
    lens = np.array([0, 0, 0, 0])
    final = [3 * block + 5, 1, 2 * block, 150]
    n_blocks = sum(-(-n // block) for n in final) + 2
    table = plain.table_for(final, block, n_blocks, rng)
    cache, ref = fresh(sv, n_blocks, heads, dim, block), plain.PlainCache(n_blocks, heads, dim, block)
    steps = [[7, 1, 2 * block, 40], [1, 0, 0, 1], [block, 0, 0, 1], [1, 0, 0, 7]]
    steps.append([f - sum(st[i] for st in steps) for i, f in enumerate(final)])
    for i, new in enumerate(steps):
        lens = lens + np.array(new)
        cu = plain.offsets(new)
        kv = make_kv(cu[-1], heads, dim, 100 * i + dim, bf16)
        ref.append([x.float().numpy() for x in kv], cu, lens, table)
        sv.qr_kv8_append(cache, kv[0].cuda(), kv[1].cuda(), dev(cu), dev(lens), dev(table))
        check_cache(cache, ref, slice(None))
        before = [t.clone() for t in cache]
        sv.qr_kv8_append(cache, kv[0].cuda(), kv[1].cuda(), dev(cu), dev(lens), dev(table))
        for a, b in zip(before, cache):    # writing the same rows again changes nothing
            live = table[table >= 0]
            assert torch.equal(a[live].view(torch.int8), b[live].view(torch.int8))
    cu = plain.offsets(lens)
    for dtype in (torch.float32, torch.bfloat16):
        got = sv.qr_kv8_read(cache, dev(cu), dev(lens), dev(table), cu[-1], dtype=dtype)
        for j in range(2):
            want = np.concatenate([ref.values(table[s], lens[s])[j] for s in range(4)])
            want = torch.from_numpy(want.astype(np.float32)).to(dtype)   # the 64-bit product is exact
            assert torch.equal(got[j].cpu(), want)


def test_append_edges(sv):
    """Absent blocks, positions below zero, rows of no sequence, zeros,
    values whose scale underflows, infinities and NaN."""
    say("append edges")
    heads, dim, block, n_blocks = 2, 64, 32, 12
    table = np.array([[3, -1, 5], [12, 7, 0], [1, 2, 100], [9, 10, 11]], dtype=np.int32)
    lens = np.array([90, 70, 5, 130])      # the last one passes its table
    new = [90, 70, 9, 130]                 # the third one's rows start below 0
    cu = plain.offsets(new)
    kv = make_kv(cu[-1] + 6, heads, dim, 5, False)
    kv[0][cu[0] + 3, 0] = 0
    kv[0][cu[1] + 40, 1, 7] = float("inf")
    kv[1][cu[1] + 50, 0, 9] = float("nan")
    kv[0][cu[3]:cu[3] + 32] = 0
    kv[1][cu[3] + 32:cu[3] + 64] = 1e-44
    ref = plain.PlainCache(n_blocks, heads, dim, block)
    cache = fresh(sv, n_blocks, heads, dim, block)
    for step in range(2):                  # the second: one more token each
        if step:
            lens, new = lens + 1, [1, 1, 1, 1]
            cu = plain.offsets(new)
            kv = make_kv(cu[-1] + 6, heads, dim, 6, False)
        ref.append([x.numpy() for x in kv], cu, lens, table)
        sv.qr_kv8_append(cache, kv[0].cuda(), kv[1].cuda(), dev(cu), dev(lens), dev(table))
        got = [cache.kd.cpu().numpy(), cache.vd.cpu().numpy()]
        for j in range(2):
            assert np.array_equal(np.nan_to_num(got[j], nan=-1), np.nan_to_num(ref.scales[j], nan=-1))
        k, v = cache.k.cpu(), cache.v.cpu()
        assert torch.equal(k, ref.device_tensors()[0]) and torch.equal(v, ref.device_tensors()[1])
    assert np.isnan(got[0][7, 1]) and np.isnan(got[1][7, 0]) and np.isnan(got[0]).sum() == 1
    # reading: zeros where there is no token, rows of no sequence untouched
    lens, new = np.array([91, 71, 6, 131]), [91, 71, 10, 131]
    cu = plain.offsets(new)
    out = [torch.full((cu[-1] + 6, heads, dim), 7.0, device="cuda") for _ in range(2)]
    sv.qr_kv8_read(cache, dev(cu), dev(lens), dev(table), cu[-1] + 6, k=out[0], v=out[1])
    for j in range(2):
        o = out[j].cpu().numpy()
        assert (o[cu[-1]:] == 7).all()
        for s in range(4):
            val, _ = [ref.values(table[s], lens[s])[i] for i in (j, 2)]
            skip = max(0, new[s] - lens[s])
            assert (o[cu[s]:cu[s] + skip] == 0).all()
            np.testing.assert_array_equal(o[cu[s] + skip:cu[s + 1]], val[lens[s] - new[s] + skip:].astype(np.float32))


def test_strided_keys_and_values(sv):
    """k, v and q as parts of one fused projection."""
    say("strided k, v")
    heads, dim, block, n = 2, 64, 32, 70
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn((n, 8 * dim), generator=g).to(torch.bfloat16).cuda()
    q, k, v = [t.view(n, -1, dim) for t in torch.split(qkv, [4 * dim, 2 * dim, 2 * dim], dim=1)]
    table, cu, lens = dev([[2, 0, 1]]), dev([0, n]), dev([n])
    a, b = [fresh(sv, 3, heads, dim, block) for _ in range(2)]
    sv.qr_kv8_append(a, k, v, cu, lens, table)
    sv.qr_kv8_append(b, k.contiguous(), v.contiguous(), cu, lens, table)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    out = torch.full((n, 6, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    sv.qr_attention_kv8(q, a, cu, lens, table, out=out[:, 1:5])
    assert torch.equal(out[:, 1:5], sv.qr_attention_kv8(q.contiguous(), a, cu, lens, table))
    assert bool((out[:, 0] == 3).all()) and bool((out[:, 5] == 3).all())


def check_attention(sv, lens, new, group, heads, dim, block, bf16, window=0, seed=0, table=None, width=None,
                    scale=None, pad=0, spread=1.0, hot=0.0):
    rng = np.random.default_rng(seed)
    if table is None:
        n_blocks = sum(-(-max(0, n) // block) for n in lens) + 1
        table = plain.table_for(lens, block, n_blocks, rng, width)
    else:
        n_blocks = int(table.max()) + 1
    ref = plain.PlainCache(n_blocks, heads, dim, block)
    for j in range(2):
        ref.codes[j][:] = rng.integers(-127, 128, ref.codes[j].shape)
        ref.scales[j][:] = np.exp(spread * rng.standard_normal(ref.scales[j].shape)) * 0.01
    cache = sv.Kv8Cache(*[t.cuda() for t in ref.device_tensors()])
    cu = plain.offsets(new)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((cu[-1] + pad, group * heads, dim), generator=g) * (1.0 + hot)
    q = q.to(torch.bfloat16) if bf16 else q
    sc = dim ** -0.5 if scale is None else scale
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    sv.qr_attention_kv8(q.cuda(), cache, dev(cu), dev(lens), dev(table), scale=scale, window=window, out=out)
    want, bound = plain.attention(q.double().numpy(), ref, cu, lens, table, sc, window, bf16)
    got = out.double().cpu().numpy()
    assert (got[cu[-1]:] == 7).all()
    got, want, bound = got[:cu[-1]], want[:cu[-1]], bound[:cu[-1]]
    if bf16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    else:
        bound = bound + 2.0 ** -24 * np.abs(want)
    assert np.all(np.isfinite(got))
    bad = np.abs(got - want) > bound
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside the bound, worst "
                           f"{np.max(np.abs(got - want) / np.maximum(bound, 1e-300)):.2f}x, first at {np.argwhere(bad)[0]}")
    return out


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("dim,block", [(64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("group,heads", [(1, 3), (4, 2), (8, 1), (20, 1)])
def test_decode(sv, dim, block, group, heads, bf16):
    say(f"decode dim={dim} block={block} group={group} bf16={bf16}")
    lens = [1, 31, 32, 33, 64, 65, 200, 700]
    check_attention(sv, lens, [1] * 8, group, heads, dim, block, bf16, seed=dim + group)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("dim,block", [(64, 64), (128, 128), (256, 32)])
@pytest.mark.parametrize("group,heads", [(1, 2), (3, 1), (4, 1)])
def test_prompts_and_chunks(sv, dim, block, group, heads, bf16):
    say(f"chunks dim={dim} block={block} group={group} bf16={bf16}")
    check_attention(sv, [150, 40, 129, 300], [150, 17, 1, 70], group, heads, dim, block, bf16, seed=dim + group)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("window", [1, 5, 32, 33, 100, 10 ** 12])
@pytest.mark.parametrize("lens,new", [([300, 90, 1], [1, 1, 1]), ([200, 70, 400], [200, 3, 130])])
def test_windows(sv, lens, new, window, bf16):
    say(f"window={window} lens={lens} bf16={bf16}")
    check_attention(sv, lens, new, 2, 2, 64, 32, bf16, window=window, seed=window % 97)


@pytest.mark.parametrize("bf16", [True, False])
def test_one_long_sequence_splits(sv, bf16):
    say(f"long bf16={bf16}")
    check_attention(sv, [9001], [1], 4, 1, 128, 64, bf16, seed=3)
    check_attention(sv, [5000, 3], [2, 1], 2, 2, 64, 32, bf16, seed=4, width=400)
    check_attention(sv, [4000], [70], 1, 1, 64, 32, bf16, seed=5)
    check_attention(sv, [900, 2500], [60, 70], 2, 1, 128, 128, bf16, seed=6, window=1500)


@pytest.mark.parametrize("bf16", [True, False])
def test_many_groups_for_one_workgroup(sv, bf16):
    """So many sequences and heads that no tokens are split: blocks and
    scales are looked up several times within a workgroup."""
    say(f"unsplit bf16={bf16}")
    check_attention(sv, [8400] + [1] * 31, [1] * 32, 1, 64, 64, 32, bf16, seed=21)
    check_attention(sv, [2300] + [60] * 7, [130] + [60] * 7, 1, 64, 64, 64, bf16, seed=22)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("new", [[60, 9, 33, 100], [1, 1, 1, 1], [40, 90, 200, 100]])
def test_absent_tokens_and_empty_rows(sv, new, bf16):
    """Evicted and out-of-range blocks, rows before position 0, a sequence
    past its table, an empty one, rows of no sequence."""
    say(f"absent new={new} bf16={bf16}")
    table = np.array([[3, -1, 5, 8], [-1, 7, 0, 4], [1, 2, 100, -7], [-1, -1, -1, -1]], dtype=np.int32)
    lens = [100, 64, 200, 90]
    t2 = np.concatenate([table, np.full((2, 4), -1, np.int32)])
    check_attention(sv, lens + [0, 0], new + [0, 5], 3, 2, 64, 32, bf16, seed=1,
                    table=np.where(t2 == 100, 9, t2) if bf16 else np.where(t2 == 100, -2, t2), pad=11)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("hot,spread", [(30.0, 0.5), (0.0, 6.0), (8.0, 3.0)])
def test_peaked_weights_and_uneven_scales(sv, hot, spread, bf16):
    say(f"hot={hot} spread={spread} bf16={bf16}")
    check_attention(sv, [500, 260], [1, 1], 4, 1, 128, 32, bf16, seed=7, hot=hot, spread=spread)
    check_attention(sv, [300, 260], [300, 40], 2, 1, 64, 32, bf16, seed=8, hot=hot, spread=spread)


def test_negative_scale_factor_and_zero(sv):
    say("scale factors")
    for scale in (-0.2, 0.0, 1e-20):
        check_attention(sv, [130, 70], [1, 70], 2, 1, 64, 32, True, seed=2, scale=scale)
        check_attention(sv, [130, 70], [1, 2], 2, 1, 64, 32, True, seed=2, scale=scale)


def test_rows_before_the_first_sequence(sv):
    """A part of a batch: cu starts behind rows of others."""
    say("part of a batch")
    rng = np.random.default_rng(13)
    lens, table = [70, 40], plain.table_for([70, 40], 32, 8, rng)
    cache = sv.kv8_cache(8, 2, 64, 32, "cuda")
    k, v = [x.cuda() for x in make_kv(110, 2, 64, 3, True)]
    sv.qr_kv8_append(cache, k, v, dev([0, 70, 110]), dev(lens), dev(table))
    q = torch.randn((100, 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for new in ([1, 3], [30, 20]):
        cu = plain.offsets(new)
        want = sv.qr_attention_kv8(q[:cu[-1]], cache, dev(cu), dev(lens), dev(table))
        shifted = torch.cat([q[:50], q[:cu[-1]]])
        out = torch.full_like(shifted, 7.0)
        sv.qr_attention_kv8(shifted, cache, dev([50 + c for c in cu]), dev(lens), dev(table), out=out)
        assert bool((out[:50] == 7).all())
        # (the two calls may take different kernels: each output within half a
        # step of bf16 and 2^-10 of the values' size of the exact one)
        got, ref = out[50:].double(), want.double()
        big = float(v.abs().max())
        assert bool(((got - ref).abs() <= 2 * (2.0 ** -8 * ref.abs() + 2.0 ** -10 * big)).all())
        read = sv.qr_kv8_read(cache, dev([50 + c for c in cu]), dev(lens), dev(table), 50 + cu[-1], k=torch.full(
            (50 + cu[-1], 2, 64), 7.0, device="cuda"))
        assert bool((read[0][:50] == 7).all())
        assert torch.equal(read[0][50:], sv.qr_kv8_read(cache, dev(cu), dev(lens), dev(table), cu[-1])[0])

@pytest.mark.parametrize("new", [[1, 1], [128, 200]])
def test_nan_blocks_reach_only_the_rows_that_see_them(sv, new):
    say(f"NaN blocks new={new}")
    heads, dim, block = 2, 64, 32
    lens = [256, 200]
    rng = np.random.default_rng(9)
    table = plain.table_for(lens, block, 20, rng)
    ref = plain.PlainCache(20, heads, dim, block)
    for j in range(2):
        ref.codes[j][:] = rng.integers(-127, 128, ref.codes[j].shape)
        ref.scales[j][:] = 0.01
    bad_k, bad_v = 5, 3                    # blocks of sequence 0 and 1
    ref.scales[0][table[0, bad_k], 0] = np.nan
    ref.scales[1][table[1, bad_v], 1] = np.nan
    ref.codes[1][table[1, bad_v], 1] = 0
    cache = sv.Kv8Cache(*[t.cuda() for t in ref.device_tensors()])
    cu = plain.offsets(new)
    for dtype in (torch.float32, torch.bfloat16):
        q = torch.randn((cu[-1], 4, dim), generator=torch.Generator().manual_seed(1)).to(dtype)
        q[0, 3] = float("nan")
        for window in (0, 40):
            out = sv.qr_attention_kv8(q.cuda(), cache, dev(cu), dev(lens), dev(table), window=window)
            nan = torch.isnan(out).cpu()
            want = torch.zeros_like(nan)
            for s, (blk, hs) in enumerate([(bad_k, (0, 1)), (bad_v, (2, 3))]):
                for i in range(new[s]):
                    p = lens[s] - new[s] + i
                    lo = max(0, p - window + 1) if window else 0
                    if lo < (blk + 1) * block and p >= blk * block:
                        want[cu[s] + i, list(hs)] = True
            want[0, 3] = True
            assert torch.equal(nan, want)


def test_shared_prefix_blocks(sv):
    """Two sequences read the same blocks."""
    say("shared prefix")
    table = np.array([[4, 1, 2, 0], [4, 1, 3, -1]], dtype=np.int32)
    check_attention(sv, [120, 90], [1, 1], 4, 2, 128, 32, True, seed=12, table=table)
    check_attention(sv, [120, 90], [60, 26], 4, 2, 128, 32, False, seed=12, table=table)


def test_offsets_past_32_bits(sv):
    """Blocks behind the first 4 GiB of codes."""
    say("offsets past 32 bits")
    heads, dim, block = 8, 128, 64
    n_blocks = (1 << 32) // (heads * dim * block) + 40
    cache = sv.kv8_cache(n_blocks, heads, dim, block, "cuda")
    n = 300
    lo = np.arange(5, dtype=np.int32)[None]
    hi = (n_blocks - 1 - np.arange(5, dtype=np.int32))[None]
    k, v = [x.cuda() for x in make_kv(n, heads, dim, 1, True)]
    cu, lens = dev([0, n]), dev([n])
    outs, reads = [], []
    for t in (lo, hi):
        table = dev(t)
        sv.qr_kv8_append(cache, k, v, cu, lens, table)
        reads.append(sv.qr_kv8_read(cache, cu, lens, table, n))
        for new in (1, 300):
            outs.append(sv.qr_attention_kv8(k[:new].repeat(1, 2, 1), cache, dev([0, new]), lens, table))
    assert torch.equal(reads[0][0], reads[1][0]) and torch.equal(reads[0][1], reads[1][1])
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])


@pytest.mark.parametrize("most", [1, 3, 90])
def test_many_sequences(sv, most):
    """More sequences than a wave looks at at once, empty ones among them, at
    the ends too; written, read and attended to."""
    say(f"many sequences most={most}")
    rng = np.random.default_rng(most)
    n_seq, heads, dim, block = 200, 1, 64, 32
    new = rng.integers(0, most + 1, n_seq)
    new[[0, 63, 64, 127, 128, 199]] = [0, most, 0, most, most, 0]
    if most == 90:
        new = np.where(rng.random(n_seq) < 0.3, 0, np.maximum(new, 75))
    lens = new + rng.integers(0, 40, n_seq) * (new > 0)
    n_blocks = int(sum(-(-int(n) // block) for n in lens))
    table = plain.table_for(lens, block, n_blocks, rng)
    cache, ref = fresh(sv, n_blocks, heads, dim, block), plain.PlainCache(n_blocks, heads, dim, block)
    cu = plain.offsets(lens)
    kv = make_kv(cu[-1], heads, dim, most, True)
    sv.qr_kv8_append(cache, kv[0].cuda(), kv[1].cuda(), dev(cu), dev(lens), dev(table))
    ref.append([x.float().numpy() for x in kv], cu, lens, table)
    check_cache(cache, ref, slice(None))
    got = sv.qr_kv8_read(cache, dev(cu), dev(lens), dev(table), cu[-1])
    for j in range(2):
        want = np.concatenate([ref.values(table[s], lens[s])[j] for s in range(n_seq)])
        assert torch.equal(got[j].cpu(), torch.from_numpy(want.astype(np.float32)))
    check_attention(sv, [int(n) for n in lens], [int(n) for n in new], 1, heads, dim, block, True, seed=most,
                    table=table)


def test_calls_on_a_stream_of_their_own(sv):
    """Outputs and scratch that the calls allocate belong to the stream they
    are given, as a torch stream or as a handle."""
    say("own stream")
    heads, dim, block, n = 2, 64, 32, 1500
    table, cu, lens = dev([np.arange(50)]), dev([0, n]), dev([n])
    k, v = [x.cuda() for x in make_kv(n, heads, dim, 3, True)]
    q = k.repeat(1, 2, 1)[:3].contiguous()
    one = dev([0, 3])
    w, wd = sv.qr_quantize_rows_i8(torch.randn((200, 4 * dim), device="cuda"))

    def chain(stream):
        cache = fresh(sv, 50, heads, dim, block)
        torch.cuda.synchronize()
        sv.qr_kv8_append(cache, k, v, cu, lens, table, stream=stream)
        o = sv.qr_attention_kv8(q, cache, one, lens, table, stream=stream)
        back = sv.qr_kv8_read(cache, cu, lens, table, n, stream=stream)
        x, xd = sv.qr_quantize_rows_i8(o.view(3, -1), stream=stream)
        y = sv.qr_matmul_i8(w, wd, x, xd, 4 * dim, stream=stream)
        torch.cuda.synchronize()
        return o, *back, x, xd, y

    want = chain(None)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for a, b in zip(chain(stream), want):
            assert torch.equal(a, b)


def test_graph_of_a_decode_step(sv):
    """Quantized projections, append and attention captured once and replayed
    with other lengths, against the same calls made eagerly."""
    say("graph")
    heads, group, dim, block, n_seq = 2, 4, 64, 32, 5
    hidden, n_q = 512, 8
    g = torch.Generator().manual_seed(2)
    wqkv, wqkv_d = sv.qr_quantize_rows_i8((torch.randn(((n_q + 2 * heads) * dim, hidden), generator=g) * 0.05).cuda())
    wo, wo_d = sv.qr_quantize_rows_i8((torch.randn((hidden, n_q * dim), generator=g) * 0.05).cuda())
    width, n_blocks = 40, 210
    table = dev(np.random.default_rng(3).permutation(n_blocks)[:n_seq * width].reshape(n_seq, width))
    start = np.array([0, 5, 31, 64, 1000])
    cu0 = plain.offsets(start)
    kv = [x.cuda() for x in make_kv(cu0[-1], heads, dim, 4, True)]
    caches = [fresh(sv, n_blocks, heads, dim, block) for _ in range(2)]
    for c in caches:
        sv.qr_kv8_append(c, kv[0], kv[1], dev(cu0), dev(start), table)
    cu = dev(np.arange(n_seq + 1))
    x = torch.zeros((n_seq, hidden), dtype=torch.bfloat16, device="cuda")
    lens = dev(start + 1)

    def step(c):
        xq, xd = sv.qr_quantize_rows_i8(x)
        qkv = sv.qr_matmul_i8(wqkv, wqkv_d, xq, xd, hidden)
        q, k, v = [t.view(n_seq, -1, dim) for t in torch.split(qkv, [n_q * dim, heads * dim, heads * dim], dim=1)]
        sv.qr_kv8_append(c, k, v, cu, lens, table)
        o = sv.qr_attention_kv8(q, c, cu, lens, table)
        oq, od = sv.qr_quantize_rows_i8(o.view(n_seq, -1))
        return sv.qr_matmul_i8(wo, wo_d, oq, od, hidden)

    inputs = [torch.randn((n_seq, hidden), generator=g).to(torch.bfloat16).cuda() for _ in range(5)]
    x.copy_(inputs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(caches[1])
    for i, inp in enumerate(inputs):
        x.copy_(inp)
        lens.copy_(dev(start + 1 + i))
        want = step(caches[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        for a, b in zip(caches[0], caches[1]):
            live = table.reshape(-1)[:1]
            assert torch.equal(a[live.long()].view(torch.int8), b[live.long()].view(torch.int8))


def test_projections_cache_and_attention_together(sv):
    """A prompt and then single tokens through an attention layer, against
    64-bit arithmetic on the values that the codes stand for."""
    say("layer")
    heads, group, dim, block = 2, 2, 64, 32
    hidden, n_q = 256, 4
    rng = np.random.default_rng(6)
    wqkv = (rng.standard_normal(((n_q + 2 * heads) * dim, hidden)) * 0.08).astype(np.float32)
    w, wd = plain.quantize_rows(wqkv)
    gw, gwd = sv.qr_quantize_rows_i8(torch.from_numpy(wqkv).cuda())
    assert np.array_equal(gw.cpu().numpy(), w)
    n_blocks = 16
    table = np.array([[3, 9, 1, 14], [7, 0, 5, 2]], dtype=np.int32)
    cache, ref = fresh(sv, n_blocks, heads, dim, block), plain.PlainCache(n_blocks, heads, dim, block)
    lens = np.array([0, 0])
    for new in ([45, 100], [1, 1], [1, 1], [3, 0]):
        lens = lens + np.array(new)
        cu = plain.offsets(new)
        x = rng.standard_normal((cu[-1], hidden)).astype(np.float32)
        xq, xd = sv.qr_quantize_rows_i8(torch.from_numpy(x).cuda())
        qkv = sv.qr_matmul_i8(gw, gwd, xq, xd, hidden, dtype=torch.float32)
        px, pd = plain.quantize_rows(x)
        want, mag = plain.product(w, wd, px, pd)
        assert np.all(np.abs(qkv.double().cpu().numpy() - want) <= 4 * 2.0 ** -24 * mag)
        q, k, v = [t.view(cu[-1], -1, dim) for t in torch.split(qkv, [n_q * dim, heads * dim, heads * dim], dim=1)]
        sv.qr_kv8_append(cache, k, v, dev(cu), dev(lens), dev(table))
        ref.append([k.cpu().numpy(), v.cpu().numpy()], cu, lens, table)
        out = sv.qr_attention_kv8(q, cache, dev(cu), dev(lens), dev(table))
        want, bound = plain.attention(q.double().cpu().numpy(), ref, cu, lens, table, dim ** -0.5, 0, False)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound + 2.0 ** -24 * np.abs(want))
