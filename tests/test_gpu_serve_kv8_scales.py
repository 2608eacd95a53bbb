"""Attention over blocks whose value scales lie far apart, against 64-bit
arithmetic: how well a row knows the values of a quiet block must not depend on
a loud one that it barely attends to, whatever kernel the call takes."""
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


def attention(q, ref, n_new, length, table_row, scale, window, fp16_weights, floor=2.0 ** -31):
    """(out, bound) of the last n_new tokens of one sequence in 64 bits, q
    float64 [n_new, n_q, dim].

    The bound is serve_plain.attention's, with u = 2^-24, except that the floor
    of the weights counts each token with its own values: a weight enters in
    fp16 (fp32 rows: as two parts), off by 2^-11 (2^-22) of itself or, where it
    or its second part is subnormal, by half a step, 2^-25. The largest weight
    is at least 2^10 there, times 2^-1 for the mantissa and 2^-3 for the
    exponent of a value scale that goes into it: 2^-31 of the largest weight."""
    u = 2.0 ** -24
    k, v, present = ref.values(table_row, length)
    dim, group = q.shape[2], q.shape[1] // k.shape[1]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n_new):
        p = length - n_new + i
        idx = np.arange(max(0, p - window + 1) if window else 0, p + 1)
        idx = idx[present[idx]]
        for h in range(q.shape[1]):
            kk, vv = k[idx, h // group], v[idx, h // group]
            sc = scale * (kk @ q[i, h])
            mag = np.max(abs(scale) * (np.abs(kk) @ np.abs(q[i, h])))
            w = np.exp(sc - np.max(sc))
            tot = np.sum(w)
            out[i, h] = (w @ vv) / tot
            spread = min(np.max(sc) - np.min(sc), 200.0)
            e = (2 * dim + 12) * u * mag + u * (spread * 1.5 + 11) + (3 * (len(idx) // 32 + 2) + 608) * u
            e += 2.0 ** -11 if fp16_weights else 2.0 ** -22
            bound[i, h] = (e * ((w @ np.abs(vv)) / tot + np.abs(out[i, h]))
                           + floor / tot * np.sum(np.abs(vv), axis=0))
    step = 2.0 ** -8 if fp16_weights else 2.0 ** -24     # the output type's
    return out, bound + step * (np.abs(out) + bound)


def check(sv, dim, bf16, loud, far, away, n_new, window=0, n_blocks=5, block=32, length=None):
    """The block in slot `loud` has value scales 2^far times the others', and
    keys that lower its scores by `away`; every other channel of its values is
    zero."""
    rng = np.random.default_rng(7 * dim + far + loud)
    heads, group = 2, 2
    length = n_blocks * block - 9 if length is None else length
    ref = plain.PlainCache(n_blocks, heads, dim, block)
    table = rng.permutation(n_blocks).astype(np.int32)[None]
    for j in range(2):
        ref.codes[j][:] = rng.integers(-127, 128, ref.codes[j].shape)
        ref.scales[j][:] = 0.01 * np.exp(0.3 * rng.standard_normal(ref.scales[j].shape))
    at = table[0, loud]
    ref.codes[0][at] = -127
    ref.scales[0][at] = away / (127 * dim ** 0.5)        # queries are 1 on average
    ref.codes[1][at, ..., 1::2] = 0
    ref.scales[1][np.arange(n_blocks) != at] *= np.float32(2.0 ** -far)
    q = 1.0 + 0.1 * torch.randn((n_new, heads * group, dim), generator=torch.Generator().manual_seed(far))
    q = q.to(torch.bfloat16) if bf16 else q
    cache = sv.Kv8Cache(*[t.cuda() for t in ref.device_tensors()])
    out = sv.qr_attention_kv8(q.cuda(), cache, dev([0, n_new]), dev([length]), dev(table), window=window)
    want, bound = attention(q.double().numpy(), ref, n_new, length, table[0], dim ** -0.5, window, bf16)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    off = np.abs(got - want)
    bad = off > bound                                    # (a row of one token may be 0 with a bound of 0)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside the bound, worst {np.max(off[bad] / bound[bad]):.3g}x"


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("loud", [0, 2, 4])
@pytest.mark.parametrize("far", [2, 3, 4, 9, 16, 28, 36, 70])
def test_a_loud_block_barely_attended(sv, far, loud, dim, bf16):
    for n_new in (50, 1):     # 100 rows a head, then two: both kernels
        say(f"loud block far={far} slot={loud} dim={dim} bf16={bf16} new={n_new}")
        check(sv, dim, bf16, loud, far, 42.0, n_new)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("far", [4, 20, 40])
def test_a_loud_block_attended(sv, far, bf16):
    """Half of the channels hold nothing of the loud block."""
    for n_new in (50, 1):
        say(f"loud attended far={far} bf16={bf16} new={n_new}")
        check(sv, 128, bf16, 1, far, 0.5, n_new)


@pytest.mark.parametrize("bf16", [True, False])
def test_rows_that_do_and_do_not_see_the_loud_block(sv, bf16):
    """A window that ends within the rows of a wave, and the rows of a prompt
    that begin before the loud block."""
    say(f"window bf16={bf16}")
    check(sv, 64, bf16, 1, 30, 42.0, 90, window=60)
    check(sv, 128, bf16, 2, 30, 42.0, 151)
    check(sv, 256, bf16, 2, 30, 42.0, 90, window=60)


@pytest.mark.parametrize("bf16", [True, False])
def test_a_loud_block_in_a_split_sequence(sv, bf16):
    say(f"split bf16={bf16}")
    for loud in (0, 40, 79):
        check(sv, 64, bf16, loud, 30, 42.0, 20, n_blocks=80)


@pytest.mark.parametrize("loud", [0, 2, 4])
@pytest.mark.parametrize("far", [3, 4, 12, 16, 20, 24])
def test_weights_of_quiet_tokens_one_by_one(sv, far, loud):
    """Every channel holds the value of one quiet token, and every quiet token
    has the score 0: an output is that token's weight, with nothing added to
    it. fp32 rows keep 2^-22 of it, their two fp16 parts. Beside that count, in
    u = 2^-24: 14 for an exponent of up to 20 (a difference of scores, 10, 9
    and 1), 6 for exp2, the mantissa's logarithm and its reciprocal, 60 for the
    sum of the weights (six groups of 32, two chains of eight in each, halves,
    rescales), 3 for the quotient, its scale and the output: 83 u."""
    say(f"weights far={far} slot={loud}")
    dim, block, heads, group, length, n_new = 128, 32, 2, 2, 160, 50
    rng = np.random.default_rng(far + loud)
    ref = plain.PlainCache(5, heads, dim, block)
    for j in range(2):
        ref.scales[j][:] = 0.01 * np.exp(0.3 * rng.standard_normal(ref.scales[j].shape))
    ref.codes[0][loud] = -127
    ref.scales[0][loud] = 42 / (127 * dim ** 0.5)
    ref.scales[1][np.arange(5) != loud] *= np.float32(2.0 ** -far)
    quiet = [p for p in range(length) if p // block != loud]
    for c, p in enumerate(quiet):
        ref.codes[1][p // block, :, p % block, c] = 100
    cache = sv.Kv8Cache(*[t.cuda() for t in ref.device_tensors()])
    q = torch.ones((n_new, heads * group, dim))
    table = np.arange(5, dtype=np.int32)[None]
    got = sv.qr_attention_kv8(q.cuda(), cache, dev([0, n_new]), dev([length]), dev(table)).double().cpu().numpy()
    value = np.array([ref.scales[1][p // block].astype(np.float64) * 100 for p in quiet])     # [channel, kv head]
    for i in range(n_new):
        pos = length - n_new + i
        seen = np.array([p <= pos for p in quiet])
        others = max(0, min(block, pos + 1 - loud * block)) * np.exp(-42.0)
        want = np.where(seen[:, None], value / (seen.sum() + others), 0.0).T.repeat(group, axis=0)
        off = np.abs(got[i] - want) / np.where(want > 0, want, 1.0)
        assert off.max() <= 2.0 ** -22 + 83 * 2.0 ** -24, f"row {i}: {off.max():.3g}"


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n_new", [120, 50, 1])
@pytest.mark.parametrize("zero", [[0], [2], [0, 1, 2], [4], [0, 1, 2, 3, 4]])
def test_blocks_of_scale_zero(sv, zero, n_new, bf16):
    """Their codes stand for zeros, whatever they are."""
    say(f"zero blocks={zero} bf16={bf16} new={n_new}")
    for dim in (64, 128, 256):
        rng = np.random.default_rng(dim)
        ref = plain.PlainCache(5, 1, dim, 32)
        for j in range(2):
            ref.codes[j][:] = rng.integers(-127, 128, ref.codes[j].shape)
            ref.scales[j][:] = 0.01 * np.exp(rng.standard_normal(ref.scales[j].shape))
        ref.scales[1][zero] = 0
        table = np.arange(5, dtype=np.int32)[None]
        q = torch.randn((n_new, 2, dim), generator=torch.Generator().manual_seed(n_new))
        q = q.to(torch.bfloat16) if bf16 else q
        cache = sv.Kv8Cache(*[t.cuda() for t in ref.device_tensors()])
        out = sv.qr_attention_kv8(q.cuda(), cache, dev([0, n_new]), dev([155]), dev(table))
        want, bound = attention(q.double().numpy(), ref, n_new, 155, table[0], dim ** -0.5, 0, bf16)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)


@pytest.mark.parametrize("loud", [0, 2, 4])
@pytest.mark.parametrize("far", [80, 95, 120])
def test_scales_out_of_reach_of_each_other(sv, far, loud):
    """Beyond factors of 2^70 weights lose a bit for each bit of distance, and
    nothing overflows."""
    for n_new, away in ((50, 42.0), (50, 0.5), (1, 42.0)):
        say(f"out of reach far={far} slot={loud} new={n_new}")
        dim, heads = 128, 1
        rng = np.random.default_rng(far)
        ref = plain.PlainCache(5, heads, dim, 32)
        for j in range(2):
            ref.codes[j][:] = rng.integers(-127, 128, ref.codes[j].shape)
            ref.scales[j][:] = 0.01
        ref.codes[0][loud] = -127
        ref.scales[0][loud] = away / (127 * dim ** 0.5)
        ref.scales[1][:] = np.float32(2.0 ** -far)
        ref.scales[1][loud] = 1.0
        table = np.arange(5, dtype=np.int32)[None]
        q = torch.ones((n_new, 2, dim))
        cache = sv.Kv8Cache(*[t.cuda() for t in ref.device_tensors()])
        out = sv.qr_attention_kv8(q.cuda(), cache, dev([0, n_new]), dev([155]), dev(table)).double().cpu().numpy()
        floor = min(1.0, 2.0 ** (-31 + far - 70))
        want, bound = attention(q.double().numpy(), ref, n_new, 155, table[0], dim ** -0.5, 0, False, floor)
        assert np.all(np.isfinite(out)) and np.all(np.abs(out - want) <= bound)
