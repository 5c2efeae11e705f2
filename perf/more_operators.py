"""The MXFP8 operators around attention, as cases to measure: quantization of
activations and weights, the RMS norm with the residual's addition and an
8-bit output, the matrix product with bias, activation and residual, the
choice of experts from router logits, and the mixture-of-experts layer of a
few tokens, in a plain form (torch operations in 32 bits) and through the
package.

MXFP8: e4m3 codes [rows, K] with a scale 2^E per 32 values of a row, kept as
the byte E + 127 [rows, K / 32]; E is the smallest from -100 up with
amax <= 448 * 2^E.

Cases are plain dicts; a case fixes every size and which experts tokens go to
(drawn from its own "route" number), a seed fixes every other value."""
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
GROUP = 32


# ---------------------------------------------------------------- cases

def listed():
    return [
        # attention outputs of a decode batch, before the output projection
        dict(name="quantize 48", op="quantize", T=48, K=4096, dtype="bf16"),
        # a weight matrix at load
        dict(name="quantize weights", op="quantize", T=11264, K=4096, dtype="bf16"),
        # the norm before a projection, one token: latency
        dict(name="norm 1", op="norm", T=1, K=4096, residual=True, normed=False),
        # a prefill batch, whose normed values the router reads in bf16 too
        dict(name="norm 7000", op="norm", T=7000, K=5120, residual=True, normed=True),
        # output projection of one token onto the residual stream
        dict(name="linear 1", op="linear", T=1, N=4096, K=4096, act="none", bias=False, residual=True, quantized=False),
        # gate and up projections of a decode batch, 8-bit for the down projection
        dict(name="linear 48 swiglu", op="linear", T=48, N=12288, K=4096, act="swiglu", bias=False, residual=False,
             quantized=True),
        # a prefill batch with bias and activation, an odd number of tokens
        dict(name="linear 2501 gelu", op="linear", T=2501, N=13824, K=5120, act="gelu_tanh", bias=True, residual=False,
             quantized=False),
        # gate and up projections of a prefill batch
        dict(name="linear 6000 swiglu", op="linear", T=6000, N=8192, K=4096, act="swiglu", bias=False, residual=False,
             quantized=True),
        # a decode batch's routing with sigmoid scores, a selection bias and groups of experts
        dict(name="route 48 grouped", op="route", T=48, E=256, topk=8, scoring="sigmoid", bias=True, groups=8,
             topk_groups=4),
        # a prefill batch's routing by softmax
        dict(name="route 9000", op="route", T=9000, E=64, topk=6, scoring="softmax", bias=False, groups=1, topk_groups=1),
        # one token through its experts
        dict(name="moe 1", op="moe", T=1, E=64, topk=8, K=4096, F=1024, residual=True, route=1),
        # a decode batch that reaches nearly every expert
        dict(name="moe 48", op="moe", T=48, E=64, topk=8, K=4096, F=1024, residual=False, route=2),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "linear", "linear", "linear", "route", "moe", "moe"])
    if op == "quantize":
        return dict(op=op, T=_log(rng, 1, 9000), K=GROUP * _log(rng, 2, 160), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 7000), K=GROUP * _log(rng, 2, 224), residual=rng.random() < 0.7,
                    normed=rng.random() < 0.3)
    if op == "linear":
        act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh", "swiglu", "swiglu"])
        quantized = rng.random() < 0.4
        N = GROUP * _log(rng, 2, 256) if quantized or rng.random() < 0.7 else _log(rng, 50, 8000)
        return dict(op=op, T=rng.choice([_log(rng, 1, 128), _log(rng, 1, 6000)]), N=N, K=GROUP * _log(rng, 2, 128), act=act,
                    bias=rng.random() < 0.3, residual=not quantized and rng.random() < 0.4, quantized=quantized)
    if op == "route":
        scoring = rng.choice(["softmax", "sigmoid"])
        E = rng.choice([8, 16, 40, 64, 128, 160, 256, 384])
        groups = rng.choice([1, 4, 8 if E > 8 else 2]) if scoring == "sigmoid" else 1
        return dict(op=op, T=_log(rng, 1, 9000), E=E, topk=rng.randint(1, 8 if groups == 1 else 2), scoring=scoring,
                    bias=scoring == "sigmoid", groups=groups, topk_groups=rng.randint(1, groups))
    E = rng.choice([8, 16, 40, 64])
    return dict(op=op, T=rng.choice([1, _log(rng, 1, 48), _log(rng, 1, 128)]), E=E, topk=rng.randint(1, 8),
                K=GROUP * _log(rng, 8, 128), F=GROUP * _log(rng, 4, 32), residual=rng.random() < 0.5,
                route=rng.randrange(1000, 1 << 30))


def _experts(case):
    """The experts of each token, from the case alone: some are more popular than others."""
    rng = random.Random(case["route"])
    popular = [rng.random() + 0.15 for _ in range(case["E"])]
    got = []
    for _ in range(case["T"]):
        keys = sorted(range(case["E"]), key=lambda e: rng.random() ** (1.0 / popular[e]), reverse=True)
        got.append(keys[:case["topk"]])
    return got


def _held(rows, K):
    """Bytes of a quantized matrix."""
    return rows * K + rows * K // GROUP


def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        E, k = case["E"], case["topk"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    K = case["K"]
    if op == "quantize":
        return {"bytes": T * K * (2 if case["dtype"] == "bf16" else 4) + _held(T, K), "flops": 2 * T * K}
    if op == "norm":
        return {"bytes": 2 * T * K * (1 + 2 * case["residual"] + case["normed"]) + 2 * K + _held(T, K), "flops": 5 * T * K}
    if op == "linear":
        N = case["N"]
        rows = 2 * N if case["act"] == "swiglu" else N
        out = _held(T, N) if case["quantized"] else 2 * T * N
        return {"bytes": _held(T, K) + _held(rows, K) + out + 2 * rows * case["bias"] + 2 * T * N * case["residual"],
                "flops": 2 * T * rows * K}
    F, experts = case["F"], _experts(case)
    active = len({e for x in experts for e in x})
    pairs = sum(len(x) for x in experts)
    return {"bytes": active * 3 * _held(F, K) + _held(T, K) + 8 * pairs + 2 * T * K * (1 + case["residual"]),
            "flops": 6 * pairs * F * K}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def activations(rows, K):
        # rows of unlike sizes, and some columns that are large in every row
        size = torch.exp2(normal(rows, 1)) * torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 12.0, 1.0)
        return (torch.randn((rows, K), generator=g, device="cuda", dtype=torch.bfloat16) * size.to(torch.bfloat16))

    def weights(rows, K):
        # quantized part by part, as a checkpoint's matrices are
        parts = [torch.randn((min(16384, rows - i), K), generator=g, device="cuda", dtype=torch.bfloat16)
                 for i in range(0, rows, 16384)]
        codes, scales = zip(*(_quantize(x.float() * K ** -0.5) for x in parts))
        return torch.cat(codes), _padded(torch.cat(scales))

    op, T = case["op"], case["T"]
    s = dict(case)
    if op == "route":
        s["logits"] = 2.0 * normal(T, case["E"])
        s["correction"] = 0.1 * normal(case["E"]) if case["bias"] else None
        return s
    K = case["K"]
    if op == "quantize":
        s["x"] = activations(T, K).to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        return s
    if op == "norm":
        s["x"] = activations(T, K)
        s["weight"] = (1.0 + 0.2 * normal(K)).to(torch.bfloat16)
        s["stream"] = activations(T, K) * 4 if case["residual"] else None
        return s
    codes, scales = _quantize(activations(T, K).float())
    s.update(x=codes, x_scale=_padded(scales))
    s["stream"] = normal(T, case["N"] if op == "linear" else K).to(torch.bfloat16) if case["residual"] else None
    if op == "linear":
        rows = 2 * case["N"] if case["act"] == "swiglu" else case["N"]
        s["w"], s["w_scale"] = weights(rows, K)
        s["offset"] = (0.3 * normal(rows)).to(torch.bfloat16) if case["bias"] else None
        return s
    E, F = case["E"], case["F"]
    w13, w13_scale = weights(E * 2 * F, K)
    w2, w2_scale = weights(E * K, F)
    s.update(w13=w13.view(E, 2 * F, K), w13_scale=w13_scale.unflatten(0, (E, 2 * F)), w2=w2.view(E, K, F),
             w2_scale=w2_scale.unflatten(0, (E, K)))
    s["ids"] = torch.tensor(_experts(case), dtype=torch.int32, device="cuda")
    w = torch.rand((T, case["topk"]), generator=g, device="cuda") + 0.05
    s["weights"] = w / w.sum(1, keepdim=True)
    return s


def _padded(scales):
    """Scale bytes in rows a multiple of 4 bytes apart."""
    rows, n = scales.shape
    held = torch.zeros((rows, -(-n // 4) * 4), dtype=torch.uint8, device=scales.device)
    held[:, :n] = scales
    return held[:, :n]


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"quantize": _plain_quantize, "norm": _norm, "linear": _linear, "route": _route, "moe": _moe}[s["op"]](s)


def _own(s):
    import sparse_mla_attention_fp8_gb300 as smla
    if s["op"] == "quantize":
        codes, scales = smla.mxfp8_quantize(s["x"])
        return [codes.view(E4M3), scales.view(E8M0)]
    if s["op"] == "norm":
        n = smla.rms_norm_mxfp8(s["x"], s["weight"], 1e-6, residual=s["stream"], normed=s["normed"])
        return [n.codes.view(E4M3), n.scales.view(E8M0), n.normed, n.residual]
    if s["op"] == "linear":
        out = smla.linear_mxfp8(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["offset"], activation=s["act"],
                                residual=s["stream"], quantized=s["quantized"])
        return [out[0].view(E4M3), out[1].view(E8M0)] if s["quantized"] else out
    if s["op"] == "route":
        return smla.moe_route(s["logits"], s["topk"], scoring=s["scoring"], bias=s["correction"], num_groups=s["groups"],
                              topk_groups=s["topk_groups"])
    return smla.moe_mxfp8(s["x"], s["x_scale"], s["ids"], s["weights"], s["w13"], s["w13_scale"], s["w2"], s["w2_scale"],
                          residual=s["stream"])


def _two_to(e):
    """2^e, exactly, for whole e of normal float32 powers: by its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponents(y):
    """E of each group of 32 values."""
    amax = y.abs().unflatten(-1, (-1, GROUP)).amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)  # 448 is 0.875 * 2^9
    return torch.where(amax > 0, e, -100).clamp(min=-100)


def _quantize(y):
    """Codes and scale bytes of y, in 32 bits."""
    e = _exponents(y)
    codes = (y.unflatten(-1, (-1, GROUP)) * _two_to(-e)[..., None]).to(E4M3)
    return codes.flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    return (codes.view(E4M3).float().unflatten(-1, (-1, GROUP)) * _two_to(scales.int() - 127)[..., None]).flatten(-2)


def _quantized(y):
    codes, scales = _quantize(y)
    return [codes.view(E4M3), scales.view(E8M0)]


def _plain_quantize(s):
    return _quantized(s["x"].float())


def _norm(s):
    h = s["x"] if s["stream"] is None else (s["x"].float() + s["stream"].float()).to(torch.bfloat16)
    y = h.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    return _quantized(y) + [y.to(torch.bfloat16) if s["normed"] else None, h if s["stream"] is not None else None]


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _linear(s):
    y = torch.matmul(_values(s["x"], s["x_scale"]), _values(s["w"], s["w_scale"]).T)
    if s["offset"] is not None:
        y = y + s["offset"].float()
    if s["act"] == "swiglu":
        gate, up = y.chunk(2, -1)
        y = _silu(gate) * up
    elif s["act"] == "relu":
        y = y.clamp(min=0)
    elif s["act"] == "silu":
        y = _silu(y)
    elif s["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    elif s["act"] == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh((2.0 / torch.pi) ** 0.5 * (y + 0.044715 * y * y * y)))
    if s["stream"] is not None:
        y = y + s["stream"].float()
    return _quantized(y) if s["quantized"] else y.to(torch.bfloat16)


def _route(s):
    x = s["logits"].double()  # (64 bits: near ties)
    T, E = x.shape
    score = torch.softmax(x, -1) if s["scoring"] == "softmax" else 1.0 / (1.0 + torch.exp(-x))
    rank = x if s["correction"] is None else score + s["correction"].double()
    if s["groups"] > 1:
        best = rank.unflatten(1, (s["groups"], -1)).topk(2, -1).values.sum(-1)
        order = best.sort(dim=-1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
        rank = torch.where(kept.repeat_interleave(E // s["groups"], 1), rank, float("-inf"))
    ids = rank.sort(dim=-1, descending=True, stable=True).indices[:, :s["topk"]]
    w = score.gather(1, ids)
    return [ids.int(), (w / w.sum(-1, keepdim=True)).float()]


def _moe(s):
    T, E, F, ids = s["T"], s["E"], s["F"], s["ids"].long()
    x = _values(s["x"], s["x_scale"])
    few = ids.numel() < E  # then each chosen expert by itself, else all experts over all tokens
    experts = ids.flatten() if few else torch.arange(E, device=x.device)
    taken = torch.repeat_interleave(torch.eye(T, device=x.device), ids.shape[1], 1) if few else None
    share = taken * s["weights"].flatten() if few else torch.zeros((T, E), device=x.device).scatter_add_(1, ids, s["weights"])
    y = torch.matmul(x, _values(s["w13"][experts], s["w13_scale"][experts]).transpose(1, 2))  # [experts, T, 2 F]
    y = share.T[..., None] * (_silu(y[..., :F]) * y[..., F:])
    y = torch.where((share.T > 0)[..., None], y, 0.0)
    out = torch.matmul(_values(*_quantize(y)), _values(s["w2"][experts], s["w2_scale"][experts]).transpose(1, 2)).sum(0)
    return (out if s["stream"] is None else out + s["stream"].float()).to(torch.bfloat16)


# ---------------------------------------------------------------- in 64 bits

def _double(codes, scales):
    return codes.view(E4M3).double() * torch.exp2(scales.double() - 127).repeat_interleave(GROUP, -1)


def _power(y):
    """The scale of each group of y, by comparison with every power there is."""
    powers = torch.tensor([2.0 ** e for e in range(-100, 122)], dtype=torch.float64, device=y.device)
    amax = y.abs().reshape(y.shape[0], -1, GROUP).amax(-1)
    return powers[torch.searchsorted(448 * powers, amax)]


def _parts(y):
    """What the codes stand for before their rounding, and nothing for the scales, which are no rounded values."""
    return [y / _power(y).repeat_interleave(GROUP, -1), None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _parts(s["x"].double())
    if op == "norm":
        h = s["x"].double()
        if s["stream"] is not None:
            h = (h + s["stream"].double()).to(torch.bfloat16).double()
        y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["K"] + 1e-6) * s["weight"].double()
        return _parts(y) + [y if case["normed"] else None, h if case["residual"] else None]
    if op == "route":
        x = s["logits"].double().cpu().numpy()
        b = None if s["correction"] is None else s["correction"].double().cpu().numpy()
        return [None, _weights(case, x, b)]
    if op == "linear":
        N = case["N"]
        y = _double(s["x"], s["x_scale"]) @ _double(s["w"], s["w_scale"]).T
        if case["bias"]:
            y += s["offset"].double()
        if case["act"] == "swiglu":
            y = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:]
        elif case["act"] == "relu":
            y = torch.maximum(y, torch.zeros_like(y))
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif case["act"] == "gelu_tanh":
            y = y * torch.sigmoid((8.0 / torch.pi) ** 0.5 * (y + 0.044715 * y ** 3))
        if case["residual"]:
            y = y + s["stream"].double()
        return _parts(y) if case["quantized"] else y
    F, x = case["F"], _double(s["x"], s["x_scale"])
    out = torch.zeros_like(x) if s["stream"] is None else s["stream"].double()
    for e in range(case["E"]):
        t, k = torch.where(s["ids"] == e)
        if t.numel() == 0:
            continue
        y = x[t] @ _double(s["w13"][e], s["w13_scale"][e]).T
        y = s["weights"][t, k].double()[:, None] * (y[:, :F] * torch.sigmoid(y[:, :F]) * y[:, F:])
        p = _power(y).repeat_interleave(GROUP, -1)
        out = out.index_add(0, t, (_nearest(y / p) * p) @ _double(s["w2"][e], s["w2_scale"][e]).T)
    return out


def _nearest(x):
    """x rounded to the nearest e4m3 value, ties to the even one, saturating."""
    size, _ = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = x.abs().clamp(min=2.0 ** -6) / size / 16
    return (torch.round(x / step) * step).clamp(-448, 448)


def _weights(case, x, b):
    import numpy as np
    T, E = x.shape
    if case["scoring"] == "softmax":
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = 1 / (1 + np.exp(-x))
    rank = x if b is None else p + b
    if case["groups"] > 1:
        n = E // case["groups"]
        best = np.sort(rank.reshape(T, case["groups"], n), 2)[:, :, -2:].sum(2)
        kept = np.argsort(-best, 1, kind="stable")[:, :case["topk_groups"]]
        lost = np.ones((T, case["groups"]), bool)
        np.put_along_axis(lost, kept, False, 1)
        rank = np.where(np.repeat(lost, n, 1), -np.inf, rank)
    w = np.take_along_axis(p, np.argsort(-rank, 1, kind="stable")[:, :case["topk"]], 1)
    return w / w.sum(1, keepdims=True)
