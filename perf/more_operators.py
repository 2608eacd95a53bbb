"""Cases, plain forms and framework calls of the 8-bit layer around attention.

Four operators, as a serving program runs them one behind the other:

  norm     the residual's addition, a root-mean-square norm, and the row of 8-bit
           codes with one scale that the next product reads.
  product  an 8-bit product whose epilogue takes the bias, the activation, the
           gate's second product and the residual.
  route    the router of a mixture of experts: scores of every expert, the
           largest few of each token and their weights.
  experts  the experts of a few tokens: gated 8-bit products, their weighted sum
           and the residual.

`own` selects the framework's kernels; otherwise `run` computes the same
operators with elementary torch operations: in 32 bits, and in 64 where a value
is compared with others or rounded to a code next.
"""
import math

import torch

own = False

_DEV = "cuda"
_EPS = 1e-6
_BLOCK = 64          # channels of a hidden row that share one scale


# --------------------------------------------------------------------------
# cases

def _norm(name, rows, n, dtype="bf16", residual=True, y=False):
    return {"name": name, "op": "norm", "rows": rows, "n": n, "dtype": dtype, "residual": residual, "y": y}


def _product(name, tokens, n_out, n_in, dtype="bf16", act="none", up=False, bias=False, residual=False):
    return {"name": name, "op": "product", "tokens": tokens, "n_out": n_out, "n_in": n_in, "dtype": dtype,
            "act": act, "up": up, "bias": bias, "residual": residual}


def _route(name, tokens, experts, n_in, top_k, dtype="bf16", score="softmax", bias=False, renorm=True):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "n_in": n_in, "top_k": top_k,
            "dtype": dtype, "score": score, "bias": bias, "renorm": renorm}


def _experts(name, tokens, experts, top_k, n_in, n_mid, dtype="bf16", residual=True):
    return {"name": name, "op": "experts", "tokens": tokens, "experts": experts, "top_k": top_k, "n_in": n_in,
            "n_mid": n_mid, "dtype": dtype, "residual": residual}


def listed():
    return [
        # one sequence's decode step: latency
        _norm("norm_1x4096", 1, 4096),
        # a ragged prompt in front of a router, which reads the normed row itself
        _norm("norm_333x7168_f32", 333, 7168, dtype="f32", y=True),
        # a prefill batch
        _norm("norm_8192x4096", 8192, 4096),
        # gate and up projection of one token: the weights' bytes
        _product("gated_1", 1, 11008, 4096, act="silu", up=True),
        # the down projection of a short ragged prompt, with what follows it
        _product("down_333_f32", 333, 4096, 11008, dtype="f32", bias=True, residual=True),
        # gate and up projection of a prefill batch: the matrix cores
        _product("gated_8192", 8192, 11008, 4096, act="silu", up=True),
        # the router of one token: latency
        _route("route_1", 1, 256, 7168, 8),
        # the router of a prompt's chunk: scores by sigmoid, experts chosen with a bias
        _route("route_2048", 2048, 256, 7168, 8, score="sigmoid", bias=True),
        # eight of 256 experts for one token
        _experts("experts_1", 1, 256, 8, 7168, 2048),
        # a decode batch that meets most of the 256 experts
        _experts("experts_64", 64, 256, 8, 7168, 2048),
        # few large experts, all of them busy, 32-bit outputs
        _experts("experts_23_f32", 23, 8, 2, 4096, 11008, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _whole(rng, n, step):
    """A usual width (whole steps) more often than an odd one."""
    return -(-n // step) * step if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(("norm", "product", "route", "experts"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "norm":
        rows, n = _log(rng, 1, 8192), _whole(rng, _log(rng, 64, 16384), 128)
        while rows * n > 8192 * 4096:
            rows = max(1, rows // 2)
        c = _norm("", rows, n, dtype, rng.random() < 0.7, rng.random() < 0.4)
    elif op == "product":
        tokens = _log(rng, 1, 6000)
        n_out, n_in = _whole(rng, _log(rng, 200, 12000), 128), _whole(rng, _log(rng, 200, 12000), 128)
        up = rng.random() < 0.5
        while 2.0 * tokens * n_out * n_in * (2 if up else 1) > 8e11:
            tokens = max(1, tokens // 2)
        c = _product("", tokens, n_out, n_in, dtype, rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")), up,
                     rng.random() < 0.4, rng.random() < 0.5)
    elif op == "route":
        tokens, experts = _log(rng, 1, 2048), _whole(rng, _log(rng, 4, 384), 8)
        n_in, top_k = _whole(rng, _log(rng, 128, 8192), 64), min(experts, rng.choice((1, 2, 4, 6, 8)))
        while 2.0 * tokens * experts * n_in > 2.0 * 2048 * 256 * 7168:
            tokens = max(1, tokens // 2)
        c = _route("", tokens, experts, n_in, top_k, dtype, rng.choice(("softmax", "softmax", "sigmoid")),
                   rng.random() < 0.3, rng.random() < 0.7)
    else:
        tokens, experts = _log(rng, 1, 128), _whole(rng, _log(rng, 2, 128), 8)
        top_k = min(experts, rng.choice((1, 2, 4, 8)))
        n_in, n_mid = _whole(rng, _log(rng, 200, 7168), 128), _whole(rng, _log(rng, 100, 4096), 64)
        while 3.0 * experts * n_in * n_mid > 2e9:
            n_in, n_mid = max(200, n_in * 3 // 4), max(100, n_mid * 3 // 4)
        c = _experts("", tokens, experts, top_k, n_in, n_mid, dtype, rng.random() < 0.6)
    del c["name"]
    return c


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


# --------------------------------------------------------------------------
# inputs (from the seed alone)

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(2_000_003 + seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=_DEV)


def _hidden(g, rows, n):
    """Rows of a hidden state: a few loud channels, as models have them."""
    x = _randn(g, rows, n)
    loud = torch.rand(n, generator=g, device=_DEV) < 0.004
    return torch.where(loud, x * 12.0, x)


def _codes(x):
    """Rows in 8 bits with one scale each, as a user's program has them in
    hand: codes int8 [n, width up to 128s], scales."""
    x = x.float()
    amax = x.abs().amax(dim=1)
    inv = (127.0 / amax.double()).float()
    codes = torch.zeros((x.shape[0], -(-x.shape[1] // 128) * 128), dtype=torch.int8, device=x.device)
    codes[:, :x.shape[1]] = torch.round(x * inv[:, None])
    return codes, (amax.double() / 127.0).float()


def _weight_rows(g, rows, n):
    """Weights of about 0.02, a different size per channel, in 8 bits."""
    w = _randn(g, rows, n).mul_(0.02)
    w *= torch.exp(0.3 * _randn(g, rows, 1))
    return _codes(w)


def _expert_rows(g, experts, rows, n):
    codes = torch.empty((experts, rows, -(-n // 128) * 128), dtype=torch.int8, device=_DEV)
    scales = torch.empty((experts, rows), device=_DEV)
    step = max(1, (1 << 28) // (rows * n))
    for a in range(0, experts, step):
        b = min(experts, a + step)
        c, s = _weight_rows(g, (b - a) * rows, n)
        codes[a:b], scales[a:b] = c.view(b - a, rows, -1), s.view(b - a, rows)
    return codes, scales


def _choices(g, case):
    """Experts of every token, distinct ones, some more popular than others,
    and their weights."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    liked = torch.rand((t, e), generator=g, device=_DEV) + 0.3 * torch.rand(e, generator=g, device=_DEV)
    ids = liked.argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    w = torch.rand((t, k), generator=g, device=_DEV) + 0.1
    return ids, w / w.sum(dim=1, keepdim=True)


def _inputs(case, seed):
    g, dt = _gen(seed), _dtype(case)
    if case["op"] == "norm":
        st = {"x": _hidden(g, case["rows"], case["n"]).to(dt), "g": (1.0 + 0.1 * _randn(g, case["n"])).to(dt)}
        st["residual"] = (4.0 * _hidden(g, case["rows"], case["n"])).to(dt) if case["residual"] else None
    elif case["op"] == "product":
        t, r, k = case["tokens"], case["n_out"], case["n_in"]
        st = {"x": _codes(_hidden(g, t, k).to(dt)), "w": _weight_rows(g, r, k)}
        st["up"] = _weight_rows(g, r, k) if case["up"] else None
        st["bias"] = _randn(g, r) if case["bias"] else None
        st["up_bias"] = _randn(g, r) if case["bias"] and case["up"] else None
        st["residual"] = _randn(g, t, r).to(dt) if case["residual"] else None
    elif case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["n_in"]
        st = {"x": _hidden(g, t, k).to(dt), "w": (_randn(g, e, k) * 1.5 / math.sqrt(k)).to(dt)}
        st["bias"] = 0.1 * _randn(g, e) if case["bias"] else None
    else:
        t, e, h, f = case["tokens"], case["experts"], case["n_in"], case["n_mid"]
        st = {"x": _codes(_hidden(g, t, h).to(dt))}
        for name, rows, n in (("gate", f, h), ("up", f, h), ("down", h, f)):
            st[name] = _expert_rows(g, e, rows, n)
        st["ids"], st["weights"] = _choices(g, case)
        st["residual"] = _randn(g, t, h).to(dt) if case["residual"] else None
    return st


# --------------------------------------------------------------------------
# state and passes

def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own and case["op"] == "experts":
        from post_weight_quantization_row_amd import serve
        # the handle of the weights, checked once when a model is loaded
        st["layer"] = serve.MoeExperts(*st["gate"], *st["up"], *st["down"], n_in=case["n_in"], n_mid=case["n_mid"])
    return st


def run(st):
    return (_run_own if own else _run_plain)(st["case"], st)


def _values(case, codes, scales):
    """What the codes stand for, in the type of the rows."""
    out = torch.empty((codes.shape[0], case["n"]), dtype=_dtype(case), device=codes.device)
    return torch.mul(codes[:, :case["n"]], scales[:, None], out=out)


def _run_own(case, st):
    from post_weight_quantization_row_amd import serve
    if case["op"] == "norm":
        codes, scales, total, y = serve.qr_norm_rows_i8(st["x"], st["g"], _EPS, residual=st["residual"], y=case["y"])
        return [_values(case, codes, scales)] + [t for t in (total, y) if t is not None]
    if case["op"] == "product":
        w, up = st["w"], st["up"] or (None, None)
        return serve.qr_matmul_i8_ex(*w, *st["x"], case["n_in"], bias=st["bias"], act=case["act"], up=up[0], upd=up[1],
                                     up_bias=st["up_bias"], residual=st["residual"], dtype=_dtype(case))
    if case["op"] == "route":
        return serve.qr_moe_route(st["x"], st["w"], case["top_k"], score=case["score"], bias=st["bias"],
                                  renorm=case["renorm"])
    return serve.qr_moe_i8(*st["x"], st["layer"], st["ids"], st["weights"], residual=st["residual"],
                           dtype=_dtype(case))


def _act(name, x):
    if name == "relu":
        return torch.clamp_min(x, 0.0)
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _plain_norm(case, st):
    dt, x = _dtype(case), st["x"]
    total = None
    if st["residual"] is not None:
        x = total = (x.float() + st["residual"].float()).to(dt)
    # codes are next to a border now and then: the row's factor in 64 bits
    x64 = x.double()
    r = 1.0 / torch.sqrt((x64 * x64).sum(dim=1, keepdim=True) / case["n"] + _EPS)
    y = (x64 * r).float() * st["g"].float()
    codes, scales = _codes(y)
    out = [_values(case, codes, scales)]
    if total is not None:
        out.append(total)
    if case["y"]:
        out.append(y.to(dt))
    return out


def _plain_product(case, st):
    def product(w, bias):
        p = torch.matmul(st["x"][0].float(), w[0].float().t()) * st["x"][1][:, None] * w[1][None, :]
        return p if bias is None else p + bias

    y = _act(case["act"], product(st["w"], st["bias"]))
    if case["up"]:
        y = y * product(st["up"], st["up_bias"])
    if case["residual"]:
        y = y + st["residual"].float()
    return y.to(_dtype(case))


def _plain_route(case, st):
    # the choice is next to a border now and then: 64 bits
    logits = torch.matmul(st["x"].double(), st["w"].double().t())
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = score / score.sum(dim=1, keepdim=True)
    by = score if st["bias"] is None else score + st["bias"].double()
    # a stable order: ties go to the lowest index
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :case["top_k"]]
    w = torch.gather(score, 1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), w.float()


def _plain_experts(case, st):
    k, h, f = case["top_k"], case["n_in"], case["n_mid"]
    x, xd = st["x"]
    wide = st["down"][0].shape[2]
    outs = []
    step = max(1, 16 // k)   # tokens whose experts' weights are gathered at once
    for a in range(0, case["tokens"], step):
        ids = st["ids"][a:a + step].reshape(-1).long()
        rows = x[a:a + step].double().repeat_interleave(k, dim=0)
        d = xd[a:a + step].repeat_interleave(k)[:, None]

        def product(w):
            # whole sums over 2^24, which 32 bits would round, in 64
            s = torch.bmm(w[0][ids].double(), rows[:, :, None])[:, :, 0]
            return s.float() * d * w[1][ids]

        gate, up = product(st["gate"]).double(), product(st["up"]).double()
        mid = torch.zeros((len(ids), wide), device=x.device)
        mid[:, :f] = (gate / (1.0 + torch.exp(-gate)) * up).float()
        mid = mid.view(len(ids), -1, _BLOCK)
        amax = mid.abs().amax(dim=2, keepdim=True)
        inv = (127.0 / amax.double()).float()
        inv = torch.where(torch.isfinite(inv), inv, torch.zeros_like(inv))
        mid = (torch.round(mid * inv) * (amax.double() / 127.0).float()).view(len(ids), wide)
        o = torch.bmm(st["down"][0][ids].float(), mid[:, :, None])[:, :, 0] * st["down"][1][ids]
        outs.append((o.view(-1, k, h) * st["weights"][a:a + step, :, None]).sum(dim=1))
    y = torch.cat(outs)
    if case["residual"]:
        y = y + st["residual"].float()
    return y.to(_dtype(case))


def _run_plain(case, st):
    return {"norm": _plain_norm, "product": _plain_product, "route": _plain_route,
            "experts": _plain_experts}[case["op"]](case, st)


# --------------------------------------------------------------------------
# the work of one pass

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        r, n = case["rows"], case["n"]
        moved = e + 1 + (2 * e if case["residual"] else 0) + (e if case["y"] else 0)
        # the values of the codes go out in the type of the rows
        return {"bytes": r * n * (moved + e) + n * e + 4 * r, "flops": 8 * r * n}
    if case["op"] == "product":
        t, r, k, m = case["tokens"], case["n_out"], case["n_in"], 2 if case["up"] else 1
        return {"bytes": t * k + 4 * t + m * (r * k + 4 * r + (4 * r if case["bias"] else 0)) +
                t * r * e * (2 if case["residual"] else 1), "flops": 2 * m * t * r * k}
    if case["op"] == "route":
        t, r, k = case["tokens"], case["experts"], case["n_in"]
        return {"bytes": (t + r) * k * e + 8 * t * case["top_k"], "flops": 2 * t * r * k}
    t, h, f, k, n = case["tokens"], case["n_in"], case["n_mid"], case["top_k"], case["experts"]
    met = n * (1.0 - (1.0 - k / n) ** t)   # distinct experts, on average
    return {"bytes": met * (3 * h * f + 4 * (2 * f + h)) + t * h * (1 + e * (2 if case["residual"] else 1)) + 8 * t * k,
            "flops": 6 * t * k * h * f}


# --------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms

def _r32(x):
    """A 64-bit value rounded to the 32 bits in which the definition holds it."""
    return x.to(torch.float32).to(torch.float64)


def _exact_codes(v):
    """Values that rows (the last dimension) in 8 bits with one scale stand for."""
    top = v.abs().max(dim=-1, keepdim=True).values
    mult = _r32(torch.full_like(top, 127.0).div(top))
    code = _r32(v * mult).round()
    return torch.where(top > 0, code * _r32(top / 127.0), torch.zeros_like(v))


def _exact_act(name, x):
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return x * 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
    if name == "gelu_tanh":
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x.relu() if name == "relu" else x


def _exact_norm(case, st):
    x, out = st["x"].double(), []
    if case["residual"]:
        s = (x + st["residual"].double()).to(torch.float32).to(_dtype(case))
        out, x = [s.double()], s.double()
    rms = x.square().mean(dim=1, keepdim=True).add(_EPS).sqrt()
    y = _r32(_r32(x / rms) * st["g"].double())
    return [_exact_codes(y)] + out + ([y] if case["y"] else [])


def _exact_product(case, st):
    def one(w, bias):
        s = torch.mm(st["x"][0].double(), w[0].double().t().contiguous())
        s = s * (st["x"][1].double().unsqueeze(1) * w[1].double())
        return s if bias is None else s + bias.double()

    y = _exact_act(case["act"], one(st["w"], st["bias"]))
    y = y * one(st["up"], st["up_bias"]) if case["up"] else y
    return y + st["residual"].double() if case["residual"] else y


def _exact_route(case, st):
    x, w = st["x"].double(), st["w"].double()
    logit = torch.stack([torch.mv(x, row) for row in w], dim=1)
    score = torch.sigmoid(logit) if case["score"] == "sigmoid" else torch.softmax(logit, dim=1)
    left = score if st["bias"] is None else score + st["bias"].double()
    left, ids = left.clone(), []
    for _ in range(case["top_k"]):
        best = left == left.max(dim=1, keepdim=True).values
        at = best.to(torch.int8).argmax(dim=1)        # the first of equal ones
        ids.append(at)
        left[torch.arange(len(at), device=at.device), at] = -math.inf
    ids = torch.stack(ids, dim=1)
    wt = torch.gather(score, 1, ids)
    return ids.to(torch.int32), wt / wt.sum(dim=1, keepdim=True) if case["renorm"] else wt


def _exact_experts(case, st):
    f = case["n_mid"]
    x, xd = st["x"][0].double(), st["x"][1].double()
    y = torch.zeros((case["tokens"], case["n_in"]), dtype=torch.float64, device=x.device)
    for e in range(case["experts"]):
        t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        if not len(t):
            continue
        g, u = (_r32(_r32(torch.mm(x[t], st[n][0][e].double().t().contiguous()) * xd[t, None]) * st[n][1][e].double())
                for n in ("gate", "up"))
        mid = _r32(g * torch.sigmoid(g) * u)
        mid = torch.nn.functional.pad(mid, (0, -f % _BLOCK)).view(len(t), -1, _BLOCK)
        mid = _exact_codes(mid).view(len(t), -1)[:, :f]
        o = torch.mm(mid, st["down"][0][e, :, :f].double().t().contiguous()) * st["down"][1][e].double()
        y[t] += o * st["weights"][t, j].double()[:, None]
    return y + st["residual"].double() if case["residual"] else y


def exact(case, seed):
    st = _inputs(case, seed)
    return {"norm": _exact_norm, "product": _exact_product, "route": _exact_route,
            "experts": _exact_experts}[case["op"]](case, st)
