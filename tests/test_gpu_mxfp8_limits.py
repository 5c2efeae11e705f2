"""GPU: the MXFP8 operators where float32 runs out, in place, and directly before the library's other calls."""
import numpy as np
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_attention_fp8_gb300 as m
    m.build()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, want, bound):
    bad = ~((got.double() - want).abs() <= bound)
    worst = ((got.double() - want).abs() / bound.clamp(min=1e-300)).amax().item()
    assert not bad.any().item(), f"{int(bad.sum())} of {bad.numel()} outside, worst {worst:.3g} of the bound"


# ---------------------------------------------------------------- activations

@pytest.mark.parametrize("T,N", [(5, 192), (37, 256), (1500, 1056)])
@pytest.mark.parametrize("quantized", [False, True])
def test_gelu_of_negative_values(smla, T, N, quantized):
    """Between -9 and -4 gelu is small beside its argument; what is rounded is to be its own value, not the argument's.
    Every sum is exact: one value of x, 0 or 1, times one of w, -4 to -9, plus a bias of few bits."""
    K = 64
    g = gen(T)
    xv = torch.zeros((T, K), dtype=F64, device="cuda")
    xv[:, 3] = torch.randint(0, 2, (T,), generator=g, device="cuda").double()
    xv[0, 3] = 1
    wv = torch.zeros((N, K), dtype=F64, device="cuda")
    wv[:, 3] = -(torch.randint(8, 18, (N,), generator=g, device="cuda") / 2).double()
    wv[32:64, 3] = -6 - torch.arange(32, device="cuda") % 3  # a group beyond -5.6 alone
    bias = (torch.randint(-15, 16, (N,), generator=g, device="cuda") / 32).float()
    x, w = ref.quantize(xv), ref.quantize(wv)
    z = ref.values(*x) @ ref.values(*w).T + bias.double()
    y = ref.activation("gelu", z)
    # the exponent, z^2 / 2, is off by two or three roundings of 2^-24 and erfc's argument in another form by as much, which
    # z^2 2^-23 covers; exponential, quotient, sum and products by 6 steps of 2^-23
    off = y.abs() * (z * z + 6) * 2.0 ** -23
    got = smla.linear_mxfp8(*x, *w, bias=bias, activation="gelu", quantized=quantized)
    if quantized:
        within(ref.values(*got), y, ref.quantized_bound(y, off))
    else:
        within(got, y, off + 2.0 ** -8 * (y.abs() + off))


def test_gelu_of_infinite_and_large_values(smla):
    z = torch.tensor([float("inf"), 1e30, 100.0, 0.0, -0.0, -20.0, -1e30, float("nan")], device="cuda")
    x, w = (ref.quantize(torch.zeros((rows, 32), dtype=F64, device="cuda")) for rows in (2, 8))
    got = smla.linear_mxfp8(*x, *w, bias=z, activation="gelu")
    want = torch.tensor([float("inf"), 1e30, 100.0, 0.0, 0.0, 0.0, 0.0], device="cuda").to(torch.bfloat16)
    assert torch.equal(got[:, :7], want.expand(2, 7)) and torch.isnan(got[:, 7]).all()


# ---------------------------------------------------------------- routing

def check_route(smla, x, topk, scoring="softmax", bias=None, groups=1, topk_groups=1, masked=None):
    """ids equal; normalized weights off by the exponentials' arguments (2^-24 of their distance from the largest taken
    logit), 32 steps of 2^-24 for exponentials, quotients and sums of up to 32, and three times float32's
    smallest number (two by the exponential, one by the quotient)."""
    ids, w = smla.moe_route(x, topk, scoring=scoring, bias=bias, num_groups=groups, topk_groups=topk_groups)
    known = (x if masked is None else torch.where(masked, float("-inf"), x)).double().cpu().numpy()
    want, ww = ref.route(known, topk, scoring, None if bias is None else bias.double().cpu().numpy(), True, 1.0, groups,
                         topk_groups)
    assert np.array_equal(ids.cpu().numpy(), want)
    taken = np.where(want >= 0, np.take_along_axis(known, want.clip(0), 1), -np.inf)
    top = taken.max(1, keepdims=True)
    far = np.where(want >= 0, top - np.where(want >= 0, taken, top), 0)
    bound = ww * (np.minimum(far, 150) + 32) * 2.0 ** -24 + 3 * 2.0 ** -149
    bad = np.abs(w.double().cpu().numpy() - ww) > bound
    assert not bad.any(), (w.cpu().numpy()[bad.any(1)][:2], ww[bad.any(1)][:2])


@pytest.mark.parametrize("E,groups", [(16, 1), (64, 1), (64, 8), (256, 8)])
@pytest.mark.parametrize("at", [-75.0, -86.0, -90.0, -100.0, -300.0])
def test_route_of_small_sigmoid_scores(smla, at, E, groups):
    """Logits whose float32 scores are 0 or nearly so: their shares are ordinary numbers."""
    x = at + 3 * torch.randn((40, E), generator=gen(E), device="cuda")
    x[20:] *= 1 + 0.1 * torch.rand((20, 1), generator=gen(1), device="cuda")
    for bias in (None, torch.zeros(E, device="cuda")):
        check_route(smla, x, 6, "sigmoid", bias, groups, max(1, groups // 2))


def test_route_of_scores_far_apart(smla):
    """A large score beside ones that float32 holds with few bits or not at all."""
    x = torch.tensor([[-20.0, -84.0, -95.0, -104.0, -200.0], [-60.0, -90.0, -100.0, -110.0, -130.0],
                      [3.0, -90.0, -101.0, -200.0, -60.0], [-100.0, -100.0, -100.0, -100.0, -100.0]], device="cuda")
    for topk in (1, 2, 5):
        check_route(smla, x, topk, "sigmoid")
        check_route(smla, x, topk, "softmax")


def test_route_of_small_softmax_scores(smla):
    """A bias that takes experts whose scores are 0 in float32."""
    g = gen(7)
    x = 2 * torch.randn((30, 32), generator=g, device="cuda")
    x[:, :8] += 150
    bias = torch.where(torch.arange(32, device="cuda") < 8, 0.0, 2.0) + torch.arange(32, device="cuda") / 64
    check_route(smla, x, 4, "softmax", bias)
    check_route(smla, x, 12, "softmax", bias)
    check_route(smla, x, 4, "softmax", bias, groups=4, topk_groups=2)


def test_route_groups_of_large_biases(smla):
    """Groups whose two scores and biases nearly cancel: their sums are off by far more than their size says."""
    g = gen(3)
    x = torch.randn((200, 1), generator=g, device="cuda") + 1e-5 * torch.randn((200, 16), generator=g, device="cuda")
    bias = torch.tensor([1000.0, -1000.0], device="cuda").repeat(8)
    check_route(smla, x.contiguous(), 2, "sigmoid", bias, groups=8, topk_groups=3)
    check_route(smla, x.contiguous(), 2, "softmax", bias, groups=8, topk_groups=3)
    # and only some of them
    few = torch.where(torch.arange(16, device="cuda") < 12, 0.0, bias)
    check_route(smla, x.contiguous(), 2, "sigmoid", few, groups=8, topk_groups=5)


@pytest.mark.parametrize("groups", [1, 4])
def test_route_near_ties_beside_a_nan(smla, groups):
    """NaN masks its expert also where near ties are ranked in 64 bits."""
    g = gen(4)
    x = torch.randn((50, 1), generator=g, device="cuda") + 1e-7 * torch.randint(-3, 4, (50, 32), generator=g, device="cuda")
    masked = torch.rand((50, 32), generator=g, device="cuda") < 0.1
    x = torch.where(masked, float("nan"), x)
    for scoring in ("softmax", "sigmoid"):
        check_route(smla, x, 6, scoring, torch.full((32,), 0.25, device="cuda"), groups, 2 if groups > 1 else 1, masked)


# ---------------------------------------------------------------- waits that run out

def matrix(g, *shape, apart=16):
    """Codes and scale bytes that are drawn as such (no NaN)."""
    codes = torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)
    codes |= torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7
    n = shape[-1] // 32
    scales = torch.randint(112, 118, shape[:-1] + (-(-n // apart) * apart,), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales[..., :n]


def gives_up_and_recovers(smla, call):
    """Calls that unwind, one alone and several in a row, each time with a right one behind them."""
    want = call()
    assert smla.read_device_status() == 0
    for calls in (1, 1, 4):
        smla.mxfp8_give_up(True)
        try:
            for _ in range(calls):
                call()
        finally:
            smla.mxfp8_give_up(False)
        assert smla.read_device_status() == 1
        got = call()
        assert smla.read_device_status() == 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("apart", [4, 16])
@pytest.mark.parametrize("T,N,K,act", [(5, 128, 4096, "none"), (70, 96, 544, "swiglu"), (100, 4096, 2080, "none"),
                                       (1500, 1040, 1056, "none"), (1400, 600, 2080, "swiglu"), (5000, 8192, 512, "gelu")])
def test_linear_unwinds(smla, T, N, K, act, apart):
    """Every form of the product, where copies and products are under way when the waits run out."""
    g = gen(T)
    x, w = matrix(g, T, K, apart=apart), matrix(g, 2 * N if act == "swiglu" else N, K, apart=apart)
    gives_up_and_recovers(smla, lambda: smla.linear_mxfp8(*x, *w, activation=act))


@pytest.mark.parametrize("T", [1, 20, 50, 300])
def test_experts_unwind(smla, T):
    E, topk, K, F = 6, 2, 1056, 544
    g = gen(T)
    x, w13, w2 = matrix(g, T, K), matrix(g, E, 2 * F, K), matrix(g, E, K, F)
    ids = torch.randint(0, E, (T, topk), generator=g, device="cuda").int()
    p = torch.rand((T, topk), generator=g, device="cuda")
    gives_up_and_recovers(smla, lambda: smla.moe_mxfp8(*x, ids, p, *w13, *w2))


@pytest.mark.parametrize("T", [1, 50, 130])
def test_experts_report_in_their_workspace(smla, T):
    """Once in the workspace that the call had, once for the device; another workspace's word stays as it is."""
    E, topk, K, F = 6, 2, 512, 256
    g = gen(T)
    x, w13, w2 = matrix(g, T, K), matrix(g, E, 2 * F, K), matrix(g, E, K, F)
    ids = torch.randint(0, E, (T, topk), generator=g, device="cuda").int()
    p = torch.rand((T, topk), generator=g, device="cuda")
    ws, other = (torch.zeros(smla.moe_mxfp8_workspace_bytes(T, E, topk, F), dtype=torch.uint8, device="cuda") for _ in range(2))
    for held in (0, 119):  # zeroed, and what an uninitialised workspace held
        ws[:4] = held
        smla.mxfp8_give_up(True)
        try:
            smla.moe_mxfp8(*x, ids, p, *w13, *w2, workspace=ws)
        finally:
            smla.mxfp8_give_up(False)
        smla.moe_mxfp8(*x, ids, p, *w13, *w2, workspace=other)
        assert smla.read_device_status(other) == 0
        assert smla.read_device_status(ws) == 1 and smla.read_device_status(ws) == 0
        assert smla.read_device_status() == 1 and smla.read_device_status() == 0
        smla.moe_mxfp8(*x, ids, p, *w13, *w2, workspace=ws)
        assert smla.read_device_status(ws) == 0


# ---------------------------------------------------------------- in place

@pytest.mark.parametrize("T,K", [(1, 512), (6000, 512), (3001, 4096), (2000, 16416), (700, 65536)])
@pytest.mark.parametrize("over", ["x", "residual"])
def test_norm_over_its_inputs(smla, T, K, over):
    """Many rows for each CTA, the sum written over what is read: the same bits as apart."""
    g = gen(K)
    x, r = (torch.randn((T, K), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand(K, generator=g, device="cuda")
    want = smla.rms_norm_mxfp8(x, w, residual=r, normed=True)
    assert torch.equal(want.residual, (x.float() + r.float()).to(torch.bfloat16))
    held = dict(x=x, residual=r)[over].clone()
    a, b = (held, r) if over == "x" else (x, held)
    for _ in range(3):
        held.copy_(dict(x=x, residual=r)[over])
        got = smla.rms_norm_mxfp8(a, w, residual=b, normed=True, residual_out=held)
        assert got.residual.data_ptr() == held.data_ptr()
        assert all(torch.equal(u, v) for u, v in zip(got, want))


@pytest.mark.parametrize("T,N,K,act", [(3, 512, 4096, "none"), (100, 515, 512, "none"), (1500, 2048, 512, "gelu_tanh"),
                                       (1500, 1041, 512, "none"), (1400, 1200, 512, "swiglu")])
def test_linear_over_its_residual(smla, T, N, K, act):
    g = gen(N)
    x, w = matrix(g, T, K), matrix(g, 2 * N if act == "swiglu" else N, K)
    r = torch.randn((T, N), generator=g, device="cuda", dtype=torch.bfloat16)
    want = smla.linear_mxfp8(*x, *w, activation=act, residual=r)
    for _ in range(3):
        held = r.clone()
        assert smla.linear_mxfp8(*x, *w, activation=act, residual=held, out=held).data_ptr() == held.data_ptr()
        assert torch.equal(held, want)


# ---------------------------------------------------------------- behind calls that let theirs start early

def behind_early_signals(smla, payloads, shape, dtype, call, rounds=8):
    """`call(input)` launched directly behind a store that lets its dependents start while a decode before it still runs, and
    then writes the input: two contents in turn, each with the result it has when it lies there."""
    def bf16(*s):
        return torch.randn(s, generator=gen(sum(s)), device="cuda").to(torch.bfloat16)

    T, K, NB = 128, 2048, 64
    q, read = bf16(T, 16, 576), torch.zeros((NB, 64, 656), dtype=torch.uint8, device="cuda")
    indices = torch.randint(0, NB * 64, (T, K), generator=gen(1), device="cuda", dtype=torch.int32)
    table = torch.arange(NB, device="cuda", dtype=torch.int32)[None]
    request = torch.zeros(T, dtype=torch.int32, device="cuda")
    cache = torch.zeros((1, 64, 656), dtype=torch.uint8, device="cuda")
    at = cache[0, 17, 528:656].view(dtype).reshape(shape)  # the position part of a row, which a store copies as it is
    slots, rows, want = torch.full((1,), 17, device="cuda"), [], []
    for p in payloads:
        row = bf16(1, 576)
        row[0, 512:] = p.contiguous().reshape(-1).view(torch.uint8).view(torch.bfloat16)
        rows.append(row)
        got = call(p.contiguous())
        want.append([t.clone() for t in (got if isinstance(got, (tuple, list)) else [got]) if t is not None])
    smla.sparse_mla_decode_fp8(q, read, indices, table, request, 0.1)
    torch.cuda.synchronize()
    for i in range(2 * rounds):
        smla.sparse_mla_decode_fp8(q, read, indices, table, request, 0.1)
        smla.mla_cache_store_fp8(rows[i % 2], slots, cache)
        got = call(at)
        got = [t for t in (got if isinstance(got, (tuple, list)) else [got]) if t is not None]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i % 2], strict=True)), i


def floats(n, dtype, seed):
    return [torch.randn(n, generator=gen(seed + i), device="cuda").to(dtype) for i in range(2)]


def test_quantize_and_norm_wait_for_their_inputs(smla):
    bf = torch.bfloat16
    other, w = floats(64, bf, 1)[0][None], floats(64, bf, 3)[0]
    behind_early_signals(smla, floats(64, bf, 5), (1, 64), bf, lambda x: smla.mxfp8_quantize(x.reshape(1, 64)))
    behind_early_signals(smla, floats(32, torch.float32, 5), (1, 32), torch.float32,
                         lambda x: smla.mxfp8_quantize(x.reshape(1, 32)))
    behind_early_signals(smla, floats(64, bf, 5), (1, 64), bf,
                         lambda x: smla.rms_norm_mxfp8(x.reshape(1, 64), w, residual=other, normed=True))
    behind_early_signals(smla, floats(64, bf, 5), (1, 64), bf,
                         lambda r: smla.rms_norm_mxfp8(other, w, residual=r.reshape(1, 64)))
    behind_early_signals(smla, floats(64, bf, 5), (64,), bf, lambda v: smla.rms_norm_mxfp8(other, v, normed=True))
    behind_early_signals(smla, floats(32, torch.float32, 5), (32,), torch.float32,
                         lambda v: smla.rms_norm_mxfp8(other[:, :32].contiguous(), v, normed=True))


@pytest.mark.parametrize("T,K", [(1, 128), (2500, 128)])
def test_linear_waits_for_its_inputs(smla, T, K):
    """Both kernels: the one of few tokens and the pairs."""
    g = gen(T)
    x, w = matrix(g, T, K), matrix(g, 64, K)
    for bias in (torch.bfloat16, torch.float32):
        N = 64 if bias == torch.bfloat16 else 32
        part = (w[0][:N], w[1][:N])
        behind_early_signals(smla, floats(N, bias, 1), (N,), bias, lambda b: smla.linear_mxfp8(*x, *part, bias=b))
    codes = [matrix(g, 1, 128)[0] for _ in range(2)]
    behind_early_signals(smla, codes, (1, 128), torch.uint8, lambda c: smla.linear_mxfp8(c.reshape(1, 128), x[1][:1], *w))
    scales = [torch.randint(112, 118, (32, 4), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    some = matrix(g, 32, 128)[0]
    behind_early_signals(smla, scales, (32, 4), torch.uint8, lambda s: smla.linear_mxfp8(some, s, *w))
    behind_early_signals(smla, scales, (32, 4), torch.uint8, lambda s: smla.linear_mxfp8(*x, some, s))
    behind_early_signals(smla, floats(64, torch.bfloat16, 3), (1, 64), torch.bfloat16,
                         lambda r: smla.linear_mxfp8(x[0][:1], x[1][:1], *w, residual=r.reshape(1, 64)))


def test_route_and_experts_wait_for_their_inputs(smla):
    g = gen(2)
    f32, E = torch.float32, 32
    logits = torch.randn((3, E), generator=g, device="cuda")
    behind_early_signals(smla, floats(E, f32, 1), (1, E), f32, lambda v: smla.moe_route(v.reshape(1, E), 6))
    behind_early_signals(smla, floats(E, f32, 1), (E,), f32, lambda b: smla.moe_route(logits, 6, scoring="sigmoid", bias=b))
    x, w13, w2 = matrix(g, 4, 128), matrix(g, E, 128, 128), matrix(g, E, 128, 64)
    ids = [torch.randint(0, E, (4, 8), generator=g, device="cuda").int() for _ in range(2)]
    share = [torch.rand((4, 8), generator=g, device="cuda") for _ in range(2)]
    behind_early_signals(smla, ids, (4, 8), torch.int32, lambda i: smla.moe_mxfp8(*x, i.reshape(4, 8), share[0], *w13, *w2))
    behind_early_signals(smla, share, (4, 8), f32, lambda p: smla.moe_mxfp8(*x, ids[0], p.reshape(4, 8), *w13, *w2))


# ---------------------------------------------------------------- with the latent cache's attention

@pytest.mark.parametrize("T,hidden", [(3, 512), (40, 1024), (1500, 256)])
def test_products_around_the_latent_attention(smla, T, hidden):
    """kv_new and q by products, directly followed by the store and the decode that read them early, whose results are
    quantized for the output projection; step after step into the same buffers.  The same bits as with the device idle
    between the calls, and every product within its bound."""
    g = gen(T)
    H, K, NB = 16, 64, 40
    w_kv, w_q, w_o = matrix(g, 576, hidden), matrix(g, H * 576, hidden), matrix(g, hidden, H * 512)
    steps = [torch.randn((T, hidden), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    table = torch.arange(NB, device="cuda", dtype=torch.int32)[None]
    request = torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = torch.randperm(NB * 64, generator=g, device="cuda")[:T]
    indices = slots[torch.randint(0, T, (T, K), generator=g, device="cuda")].int()

    def run(between):
        cache = torch.zeros((NB, 64, 656), dtype=torch.uint8, device="cuda")
        kv, q = (torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in ((T, 576), (T, H * 576)))
        got = []
        torch.cuda.synchronize()
        for s in steps:
            x = smla.mxfp8_quantize(s)
            between()
            smla.linear_mxfp8(*x, *w_kv, out=kv)
            between()
            smla.mla_cache_store_fp8(kv, slots, cache)
            between()
            smla.linear_mxfp8(*x, *w_q, out=q)
            between()
            out, lse = smla.sparse_mla_decode_fp8(q.view(T, H, 576), cache, indices, table, request, 0.002)
            between()
            a = smla.mxfp8_quantize(out.view(T, H * 512))
            between()
            smla.linear_mxfp8(*a, *w_o, residual=s)
            got += [cache.clone(), out, lse, *a]
        torch.cuda.synchronize()
        assert smla.read_device_status() == 0
        # the last step's products
        for y, xv, w in ((kv, x, w_kv), (q, x, w_q)):
            z, off = ref.linear(ref.values(*xv), ref.values(*w), None, "none", None)
            within(y, z, off + 2.0 ** -8 * (z.abs() + off))
        assert torch.equal(ref.values(*a), ref.rounded(out.view(T, H * 512).double()))
        return got

    want = run(torch.cuda.synchronize)
    assert all(torch.isfinite(t.float()).all() for t in want[1::5])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want, strict=True))


# ---------------------------------------------------------------- refusals

def test_flags_without_a_truth_value(smla):
    """The error of asking for it is the call's."""
    g, both = gen(0), torch.tensor([True, False])
    x, w = matrix(g, 2, 64), matrix(g, 32, 64)
    calls = [lambda: smla.linear_mxfp8(*x, *w, quantized=both), lambda: smla.moe_route(torch.zeros((2, 8), device="cuda"), 2, renormalize=both),
             lambda: smla.rms_norm_mxfp8(torch.zeros((2, 64), device="cuda", dtype=torch.bfloat16), quantized=both)]
    for call in calls:
        with pytest.raises(RuntimeError, match="ambiguous") as e:
            call()
        assert e.type is RuntimeError
