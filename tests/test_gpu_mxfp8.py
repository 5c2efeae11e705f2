"""GPU: the MXFP8 operators against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_attention_fp8_gb300 as m
    m.build()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def activations(g, T, K, dtype=torch.bfloat16):
    return (normal(g, T, K) * torch.exp2(2 * normal(g, T, 1)) *
            torch.where(torch.rand(K, generator=g, device="cuda") < 0.03, 20.0, 1.0)).to(dtype)


def within(got, want, bound):
    bad = (got.double() - want).abs() > bound
    worst = ((got.double() - want).abs() / bound.clamp(min=1e-300)).amax().item() if got.numel() else 0
    assert not bad.any().item() and not torch.isnan(got.double()).any().item(), \
        f"{int(bad.sum())} of {bad.numel()} outside, worst {worst:.3g} of the bound"


def matrix(g, rows, K, scale=1.0, apart=16):
    """A quantized matrix and its values."""
    codes, scales = ref.quantize(activations(g, rows, K).double() * scale, apart)
    return codes, scales, ref.values(codes, scales)


# ---------------------------------------------------------------- quantization

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(1, 32), (3, 96), (1, 4096), (257, 160), (64, 1024), (1000, 2080)])
def test_quantize(smla, T, K, dtype):
    x = activations(gen(T + K), T, K, dtype)
    codes, scales = smla.mxfp8_quantize(x)
    want = ref.bytes_of(x.double())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    assert T == 1 or scales.stride(0) % 4 == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_extremes(smla, dtype):
    """Groups of zeros, of infinities alone, with NaN, tiny, huge, at and just beyond a scale's limit."""
    x = torch.zeros((4, 320), device="cuda")
    x[0, 32:64] = float("inf")
    x[0, 64] = float("nan")
    x[0, 65], x[0, 66], x[0, 67] = 3.0, float("-inf"), -0.0
    x[0, 96:128] = 1e-38
    x[0, 128:160] = 3e38
    x[0, 160] = 448.0
    x[0, 192] = 450.0
    x[0, 224] = 2.0 ** -100 * 448
    x[0, 225] = 2.0 ** -104
    x[1, :32] = torch.linspace(-448, 448, 32, device="cuda")
    x[2, :64] = torch.arange(64, device="cuda") * 0.0625 + 16
    x[3, 5] = 1e-45
    x = x.to(dtype)
    codes, scales = smla.mxfp8_quantize(x)
    want = ref.bytes_of(x.double())
    assert torch.equal(scales, want[1])
    same = (codes == want[0]) | (torch.isnan(x) & (codes & 127 == 127))
    assert same.all().item()


def test_quantize_slices_and_outputs(smla):
    """Rows that are slices of longer ones, given outputs, the bytes behind and between left as they were."""
    g = gen(5)
    wide = activations(g, 70, 512)
    x = wide[3:68, 128:128 + 96]
    codes = torch.full((65, 96), 77, dtype=torch.uint8, device="cuda")
    held = torch.full((66, 8), 99, dtype=torch.uint8, device="cuda")
    scales = held[:65, :3]
    got = smla.mxfp8_quantize(x, codes=codes, scales=scales)
    assert got[0].data_ptr() == codes.data_ptr() and got[1].data_ptr() == scales.data_ptr()
    want = ref.bytes_of(x.double())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    assert (held[:, 3:] == 99).all() and (held[65] == 99).all()


def test_quantize_nothing(smla):
    codes, scales = smla.mxfp8_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0, 2)


# ---------------------------------------------------------------- norm

def check_norm(got, x, residual, weight, eps):
    h = x.double()
    if residual is not None:
        h = (x.float() + residual.float()).to(torch.bfloat16).double()
        assert torch.equal(got.residual.double(), h)
    K = x.shape[1]
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    # the sum of K squares within K 2^-24 at most (half of it in the root), the root, the division and three products
    off = y.abs() * (min(K, 512) / 2 + 8) * 2.0 ** -24
    if got.codes is not None:
        within(ref.values(got.codes, got.scales), y, ref.quantized_bound(y, off))
        # and the scale is the smallest, up to the same
        e = got.scales.double() - 127
        amax = y.abs().unflatten(-1, (-1, 32)).amax(-1)
        assert (amax <= 448 * torch.exp2(e) * (1 + 1e-4)).all()
        assert ((amax > 224 * torch.exp2(e) * (1 - 1e-4)) | (e == -100)).all()
    if got.normed is not None:
        within(got.normed, y, off + 2.0 ** -8 * (y.abs() + off) + 2.0 ** -134)


@pytest.mark.parametrize("T,K", [(1, 32), (1, 4096), (5, 96), (9, 256), (33, 576), (3, 1024), (7, 1536), (2, 2080),
                                 (17, 4128), (6, 8192), (4, 12288), (2, 16416), (1, 65536)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(smla, T, K, with_residual):
    g = gen(T * K)
    x = activations(g, T, K)
    r = activations(g, T, K) if with_residual else None
    w = (1 + 0.3 * normal(g, K)).to(torch.bfloat16)
    got = smla.rms_norm_mxfp8(x, w, 1e-6, residual=r, normed=True)
    check_norm(got, x, r, w, 1e-6)
    assert (got.residual is None) == (not with_residual)


@pytest.mark.parametrize("weight", [None, torch.float32])
def test_norm_weights_and_parts(smla, weight):
    g = gen(2)
    x = activations(g, 40, 640)
    w = None if weight is None else 1 + normal(g, 640)
    check_norm(smla.rms_norm_mxfp8(x, w, 1e-3), x, None, w, 1e-3)
    only = smla.rms_norm_mxfp8(x, w, 1e-3, normed=True, quantized=False)
    assert only.codes is None and only.scales is None
    check_norm(only, x, None, w, 1e-3)


def test_norm_in_place_and_slices(smla):
    """The residual stream updated in place; x a slice of a fused projection's rows."""
    g = gen(3)
    wide = activations(g, 50, 1024)
    x, stream = wide[:, 256:768], activations(g, 50, 512)
    before = stream.clone()
    got = smla.rms_norm_mxfp8(x, residual=stream, residual_out=stream)
    assert got.residual.data_ptr() == stream.data_ptr()
    check_norm(got, x, before, None, 1e-6)


def test_norm_of_zero_rows_and_specials(smla):
    """A row of zeros is zeros under every eps > 0; NaN and infinity make their row NaN and no other."""
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    got = smla.rms_norm_mxfp8(x, eps=1e-5, normed=True)
    assert (got.normed[0] == 0).all() and (got.codes[0] & 127 == 0).all()
    assert torch.isnan(got.normed[1]).all()
    assert torch.isnan(got.normed[2, 4]) and (got.normed[2, :4] == 0).all()
    assert (got.codes[1] & 127 == 127).all()
    assert torch.isfinite(got.normed[3].float()).all()


# ---------------------------------------------------------------- linear product

def check_linear(smla, T, N, K, act="none", bias=None, residual=False, quantized=False, seed=0, apart=16):
    g = gen(seed + T + N + K)
    x, xs, xv = matrix(g, T, K, apart=apart)
    rows = 2 * N if act == "swiglu" else N
    w, ws, wv = matrix(g, rows, K, scale=0.3 * K ** -0.5, apart=apart)
    b = None if bias is None else normal(g, rows, dtype=bias)
    r = normal(g, T, N, dtype=torch.bfloat16) if residual else None
    y, off = ref.linear(xv, wv, b, act, r)
    got = smla.linear_mxfp8(x, xs, w, ws, bias=b, activation=act, residual=r, quantized=quantized)
    if quantized:
        assert got[0].shape == (T, N) and got[1].shape == (T, N // 32)
        within(ref.values(*got), y, ref.quantized_bound(y, off))
    else:
        assert got.shape == (T, N) and got.dtype == torch.bfloat16
        within(got, y, off + 2.0 ** -8 * (y.abs() + off) + 2.0 ** -134)
    assert smla.read_device_status() == 0


def test_linear_smallest(smla):
    check_linear(smla, 1, 128, 128)


@pytest.mark.parametrize("apart", [4, 16])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 480, 544, 1024, 1056, 4096])
def test_linear_lengths(smla, K, apart):
    """Rows of scales that end inside a word, a step and a set of steps, on 16-byte boundaries and not."""
    check_linear(smla, 5, 128, K, apart=apart)
    check_linear(smla, 70, 96, K, act="swiglu", apart=apart)


@pytest.mark.parametrize("apart", [4, 16])
@pytest.mark.parametrize("K", [32, 96, 160, 480, 544, 1056, 2080])
def test_linear_lengths_many_tokens(smla, K, apart):
    check_linear(smla, 1500, 1040, K, apart=apart)
    check_linear(smla, 1400, 600, K, act="swiglu", apart=apart)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 96, 97, 128, 129, 300])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_tokens(smla, T, act):
    check_linear(smla, T, 160, 512, act=act)


@pytest.mark.parametrize("N", [1, 2, 31, 33, 127, 129, 250, 1000])
def test_linear_features(smla, N):
    """Odd numbers of features, alone and with bias and residual."""
    check_linear(smla, 19, N, 256)
    check_linear(smla, 130, N, 256, bias=torch.float32, residual=True)
    check_linear(smla, 3, N, 256, act="swiglu", bias=torch.bfloat16, residual=True)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("bias", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", ["bf16", "residual", "mxfp8"])
def test_linear_epilogues(smla, act, bias, out):
    check_linear(smla, 37, 192, 384, act=act, bias=bias, residual=out == "residual", quantized=out == "mxfp8")


@pytest.mark.parametrize("T,N,K", [(1, 32, 32), (40, 96, 2048), (100, 4096, 1024), (1, 2048, 4096), (200, 544, 320)])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_linear_quantized(smla, T, N, K, act):
    check_linear(smla, T, N, K, act=act, quantized=True)


@pytest.mark.parametrize("T,N,K", [(257, 32, 32), (300, 256, 128), (383, 130, 4096), (512, 257, 96), (640, 1000, 256),
                                   (257, 1, 544), (1111, 2080, 1056), (2000, 4096, 512), (5000, 96, 128), (1024, 5120, 64),
                                   (65, 8200, 512), (6001, 33, 256), (100, 6500, 1024)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_many_tokens(smla, T, N, K, act):
    check_linear(smla, T, N, K, act=act)
    if N % 32 == 0:
        check_linear(smla, T, N, K, act=act, quantized=True)
    else:
        check_linear(smla, T, N, K, act=act, bias=torch.bfloat16, residual=True)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("out", ["bf16", "residual", "mxfp8"])
def test_linear_epilogues_many_tokens(smla, act, out):
    check_linear(smla, 1300, 1120, 384, act=act, bias=torch.float32, residual=out == "residual", quantized=out == "mxfp8")


@pytest.mark.parametrize("T,N", [(1277, 4090), (2039, 2816), (1280, 3840), (1019, 2560), (900, 5000), (3400, 2048)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_last_tiles(smla, T, N, act):
    """Tiles beside those that fill the SMs, whole and in parts of fewer tokens, the last ones ragged."""
    check_linear(smla, T, N, 96, act=act, bias=torch.bfloat16, residual=True)
    if N % 32 == 0:
        check_linear(smla, T, N, 64, act=act, quantized=True)


def test_linear_many_tiles(smla):
    check_linear(smla, 1100, 1300, 640, act="gelu", bias=torch.float32)
    check_linear(smla, 1000, 1056, 640, act="swiglu", quantized=True)


def test_linear_slices_and_in_place(smla):
    """x a slice of longer rows, the result written over the residual."""
    g = gen(9)
    wide, wides, wv = matrix(g, 20, 512)
    x, xs, xv = wide[:, 128:384], wides[:, 4:12], wv[:, 128:384]
    w, ws, v = matrix(g, 96, 256, scale=0.05)
    r = normal(g, 20, 96, dtype=torch.bfloat16)
    y, off = ref.linear(xv, v, None, "none", r)
    got = smla.linear_mxfp8(x, xs, w, ws, residual=r, out=r)
    assert got.data_ptr() == r.data_ptr()
    within(got, y, off + 2.0 ** -8 * (y.abs() + off))


def test_linear_views_of_the_codes(smla):
    g = gen(10)
    x, xs, _ = matrix(g, 4, 256)
    w, ws, _ = matrix(g, 64, 256)
    a = smla.linear_mxfp8(x, xs, w, ws)
    b = smla.linear_mxfp8(x.view(torch.float8_e4m3fn), xs.contiguous().view(torch.float8_e8m0fnu), w.view(torch.float8_e4m3fn),
                          ws.contiguous().view(torch.float8_e8m0fnu))
    assert torch.equal(a, b)


def test_linear_nan_stays_in_its_row(smla):
    g = gen(11)
    x, xs, _ = matrix(g, 40, 256)
    w, ws, _ = matrix(g, 64, 256)
    clean = smla.linear_mxfp8(x, xs, w, ws)
    x[7, 100] = 127
    got = smla.linear_mxfp8(x, xs, w, ws)
    assert torch.isnan(got[7]).all()
    keep = torch.arange(40, device="cuda") != 7
    assert torch.equal(got[keep], clean[keep])


# ---------------------------------------------------------------- routing

def check_route(smla, x, topk, scoring="softmax", bias=None, renormalize=True, scale=1.0, groups=1, topk_groups=1):
    ids, w = smla.moe_route(x, topk, scoring=scoring, bias=bias, renormalize=renormalize, scale=scale, num_groups=groups,
                            topk_groups=topk_groups)
    want, ww = ref.route(x.double().cpu().numpy(), topk, scoring, None if bias is None else bias.double().cpu().numpy(),
                         renormalize, scale, groups, topk_groups)
    assert np.array_equal(ids.cpu().numpy(), want)
    # exponentials, sums of up to 512 terms and quotients
    np.testing.assert_allclose(w.double().cpu().numpy(), ww, rtol=64 * 2.0 ** -24, atol=1e-37)


@pytest.mark.parametrize("E,topk", [(1, 1), (8, 2), (32, 32), (40, 3), (64, 6), (100, 8), (128, 1), (256, 8), (384, 8), (512, 32)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(smla, E, topk, scoring, dtype):
    x = (2 * normal(gen(E), 37, E)).to(dtype)  # (bf16 logits have ties)
    check_route(smla, x, topk, scoring)
    check_route(smla, x, topk, scoring, renormalize=False, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,topk", [(256, 8, 4, 8), (64, 32, 3, 2), (12, 2, 1, 6), (160, 4, 4, 6), (512, 16, 2, 8)])
def test_route_groups(smla, scoring, E, groups, kept, topk):
    g = gen(E + groups)
    x = 2 * normal(g, 50, E)
    check_route(smla, x, topk, scoring, bias=0.1 * normal(g, E), groups=groups, topk_groups=kept)
    check_route(smla, x, topk, scoring, groups=groups, topk_groups=kept, renormalize=False)


def test_route_near_ties(smla):
    """Scores plus bias that float32 does not tell apart, and exact ties, which go to the lowest index."""
    g = gen(1)
    x = torch.randint(-2, 3, (200, 64), generator=g, device="cuda").float()
    check_route(smla, x, 8)
    check_route(smla, x, 8, "sigmoid", bias=torch.zeros(64, device="cuda"))
    check_route(smla, x, 8, "sigmoid", bias=torch.zeros(64, device="cuda"), groups=8, topk_groups=3)
    base = normal(g, 200, 1).expand(200, 64)
    near = base + 1e-7 * torch.randint(-3, 4, (200, 64), generator=g, device="cuda")
    check_route(smla, near.contiguous(), 8, "sigmoid", bias=torch.full((64,), 0.25, device="cuda"))
    check_route(smla, near.contiguous(), 8, "softmax", bias=1e-7 * normal(g, 64), groups=4, topk_groups=2)


def test_route_near_ties_of_many(smla):
    """More near ties than a warp has lanes; the last taken and the first left among them."""
    g = gen(2)
    near = normal(g, 100, 1).expand(100, 96) + 1e-7 * torch.randint(-3, 4, (100, 96), generator=g, device="cuda")
    bias = torch.full((96,), 0.25, device="cuda")
    for topk in (1, 8, 31, 32):
        check_route(smla, near.contiguous(), topk, "sigmoid", bias=bias)
    few = 3 * normal(g, 200, 40)
    few[:, 33] = few.sort(dim=1, descending=True).values[:, 31] * (1 + 2.0 ** -23)  # the 32nd's neighbour
    check_route(smla, few, 32, "sigmoid", bias=torch.zeros(40, device="cuda"))
    check_route(smla, few, 32, "softmax", bias=torch.zeros(40, device="cuda"))


def test_route_masked_experts(smla):
    """Masked experts are not taken; where too few are left, id -1 and weight 0."""
    g = gen(4)
    x = normal(g, 6, 48)
    x[0] = float("-inf")
    x[1, 3:] = float("-inf")
    x[2, ::2] = float("-inf")
    x[3, 7] = float("nan")
    x[4, 5] = -0.0
    x[4, 4] = 0.0
    for scoring in ("softmax", "sigmoid"):
        y = x.clone()
        ids, w = smla.moe_route(y, 5, scoring=scoring)
        assert (ids[0] == -1).all() and (w[0] == 0).all()
        assert (ids[1, 3:] == -1).all() and (w[1, 3:] == 0).all() and abs(w[1, :3].sum().item() - 1) < 1e-6
        assert (ids[2] % 2 == 1).all() and not (ids[3] == 7).any()
        y[3, 7] = float("-inf")
        check_route(smla, y, 5, scoring)
        check_route(smla, y, 5, scoring, bias=0.1 * normal(g, 48), groups=4, topk_groups=2)


def test_route_many_tokens(smla):
    check_route(smla, 2 * normal(gen(6), 3001, 64), 6)


# ---------------------------------------------------------------- mixture of experts

def experts(g, E, K, F, apart=16):
    w13 = [matrix(g, 2 * F, K, 0.3 * K ** -0.5) for _ in range(E)]
    w2 = [matrix(g, K, F, 0.3 * F ** -0.5) for _ in range(E)]

    def stacked(ws):
        codes = torch.stack([w[0] for w in ws])
        n = ws[0][1].shape[1]
        held = torch.full((E, codes.shape[1], -(-n // apart) * apart), 255, dtype=torch.uint8, device="cuda")
        for e in range(E):
            held[e, :, :n] = ws[e][1]
        return codes, held[:, :, :n]

    return stacked(w13), stacked(w2), [w[2] for w in w13], [w[2] for w in w2]


def check_moe(smla, T, E, topk, K, F, residual=False, ids=None, seed=0, apart=16, **kw):
    g = gen(seed + T + E + K + F)
    x, xs, xv = matrix(g, T, K, apart=apart)
    (w13, s13), (w2, s2), v13, v2 = experts(g, E, K, F, apart)
    if ids is None:
        ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:topk] for _ in range(T)]).int()
    w = torch.rand(ids.shape, generator=g, device="cuda")
    r = normal(g, T, K, dtype=torch.bfloat16) if residual else None
    y, off = ref.moe(xv, ids, w, v13, v2, r)
    got = smla.moe_mxfp8(x, xs, ids, w, w13, s13, w2, s2, residual=r, **kw)
    within(got, y, off + 2.0 ** -8 * (y.abs() + off) + 2.0 ** -134)
    assert smla.read_device_status() == 0
    return got


def test_moe_smallest(smla):
    check_moe(smla, 1, 1, 1, 128, 128)


@pytest.mark.parametrize("T", [1, 2, 16, 17, 33, 64, 65, 97, 128, 129, 200])
def test_moe_tokens(smla, T):
    check_moe(smla, T, 8, 2, 256, 128, residual=T % 2 == 1)


@pytest.mark.parametrize("apart", [4, 16])
@pytest.mark.parametrize("K,F", [(32, 32), (96, 160), (1024, 32), (160, 544), (480, 1024), (2048, 512), (2080, 480)])
def test_moe_sizes(smla, K, F, apart):
    check_moe(smla, 5, 6, 3, K, F, apart=apart)
    check_moe(smla, 50, 6, 3, K, F, residual=True, apart=apart)
    check_moe(smla, 100, 6, 3, K, F, apart=apart)


@pytest.mark.parametrize("E,topk", [(1, 1), (3, 3), (40, 1), (64, 8), (130, 32)])
def test_moe_experts(smla, E, topk):
    check_moe(smla, 3, E, topk, 128, 64)
    check_moe(smla, 40, E, topk, 128, 64)


def test_moe_ids(smla):
    """Tokens without experts, ids outside, the same expert twice, one expert for all, none at all."""
    E = 5
    ids = torch.tensor([[0, 1], [-1, 3], [7, 2], [4, 4], [-1, -1], [0, 2 ** 30], [-2 ** 31, 1]], dtype=torch.int32, device="cuda")
    check_moe(smla, 7, E, 2, 256, 96, ids=ids, residual=True)
    got = check_moe(smla, 7, E, 2, 256, 96, ids=ids)
    assert (got[4] == 0).all()
    check_moe(smla, 30, E, 2, 256, 96, ids=torch.full((30, 2), 3, dtype=torch.int32, device="cuda"))
    got = check_moe(smla, 30, E, 2, 256, 96, ids=torch.full((30, 2), -1, dtype=torch.int32, device="cuda"))
    assert (got == 0).all()


def test_moe_workspace_and_in_place(smla):
    n = smla.moe_mxfp8_workspace_bytes(20, 8, 2, 96)
    ws = torch.full((n,), 127, dtype=torch.uint8, device="cuda")  # (NaN codes)
    ws[:4] = 0
    check_moe(smla, 20, 8, 2, 256, 96, workspace=ws)
    assert smla.read_device_status(ws) == 0
    with pytest.raises(smla.SmlaError, match="workspace has"):
        check_moe(smla, 20, 8, 2, 256, 96, workspace=ws[:n - 256])


def test_moe_unused_experts_are_not_read(smla):
    """NaN in the weights of an expert that no token goes to."""
    g = gen(3)
    x, xs, _ = matrix(g, 9, 128)
    (w13, s13), (w2, s2), _, _ = experts(g, 4, 128, 64)
    ids = torch.randint(0, 3, (9, 2), generator=g, device="cuda").int()
    w = torch.rand((9, 2), generator=g, device="cuda")
    clean = smla.moe_mxfp8(x, xs, ids, w, w13, s13, w2, s2)
    w13[3], w2[3], s13[3], s2[3] = 127, 127, 255, 255
    assert torch.equal(smla.moe_mxfp8(x, xs, ids, w, w13, s13, w2, s2), clean)


# ---------------------------------------------------------------- offsets beyond 32 bits

def coded(g, *shape):
    """Codes and scale bytes that are drawn as such (no NaN)."""
    codes = torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)
    codes |= torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7
    n = shape[-1] // 32
    scales = torch.randint(116, 122, shape[:-1] + (-(-n // 16) * 16,), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales[..., :n]


def test_quantize_beyond_32_bits(smla):
    T, K = 1_100_001, 2048  # 2.25e9 values
    x = torch.randn((T, K), generator=gen(1), device="cuda", dtype=torch.bfloat16)
    codes, scales = smla.mxfp8_quantize(x)
    for rows in (slice(0, 3), slice(1_048_570, 1_048_580), slice(T - 3, T)):
        want = ref.bytes_of(x[rows].double())
        assert torch.equal(codes[rows], want[0]) and torch.equal(scales[rows], want[1])
    got = smla.rms_norm_mxfp8(x, residual=x, residual_out=x)
    rows = slice(T - 3, T)
    check_norm(smla.MxNorm(got.codes[rows], got.scales[rows], None, None), x[rows], None, None, 1e-6)


@pytest.mark.parametrize("N", [8, 256])
def test_linear_beyond_32_bits(smla, N):
    T, K = 1_100_001, 2048
    g = gen(2)
    x, xs = coded(g, T, K)
    w, ws = coded(g, N, K)
    got = smla.linear_mxfp8(x, xs, w, ws)
    for rows in (slice(0, 3), slice(1_048_570, 1_048_580), slice(T - 3, T)):
        y, off = ref.linear(ref.values(x[rows], xs[rows]), ref.values(w, ws), None, "none", None)
        within(got[rows], y, off + 2.0 ** -8 * (y.abs() + off))


def test_moe_beyond_32_bits(smla):
    E, K, F = 512, 2048, 1056
    g = gen(3)
    w13, s13 = coded(g, E, 2 * F, K)  # 2.2e9 codes
    w2, s2 = coded(g, E, K, F)
    x, xs = coded(g, 3, K)
    ids = torch.tensor([[0, 511], [510, 256], [511, 509]], dtype=torch.int32, device="cuda")
    w = torch.rand((3, 2), generator=g, device="cuda")
    s13, s2 = s13 - 4, s2 - 4  # (activations of ordinary sizes)
    s13, s2 = ([torch.nn.functional.pad(v, (0, -v.shape[2] % 16))[..., :v.shape[2]] for v in (s13, s2)])
    got = smla.moe_mxfp8(x, xs, ids, w, w13, s13, w2, s2)
    used = sorted(set(ids.flatten().tolist()))
    place = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    place[used] = torch.arange(len(used), dtype=torch.int32, device="cuda")
    y, off = ref.moe(ref.values(x, xs), place[ids.long()], w, [ref.values(w13[e], s13[e]) for e in used],
                     [ref.values(w2[e], s2[e]) for e in used], None)
    within(got, y, off + 2.0 ** -8 * (y.abs() + off))


# ---------------------------------------------------------------- together, and how they are called

def layer(smla, t, stream):
    """A decoder layer's way around its attention, with the residual stream updated in place."""
    codes, scales = smla.mxfp8_quantize(t["attended"])
    smla.linear_mxfp8(codes, scales, *t["o"], residual=stream, out=stream)
    n = smla.rms_norm_mxfp8(stream, t["w"], normed=True)
    h = smla.linear_mxfp8(n.codes, n.scales, *t["gate_up"], activation="swiglu", quantized=True)
    smla.linear_mxfp8(*h, *t["down"], residual=stream, out=stream)
    n = smla.rms_norm_mxfp8(stream, t["w"], normed=True)
    logits = (n.normed.float() @ t["router"]).contiguous()
    ids, w = smla.moe_route(logits, 2, scoring="sigmoid", bias=t["bias"], num_groups=2, topk_groups=1)
    return smla.moe_mxfp8(n.codes, n.scales, ids, w, *t["w13"], *t["w2"], residual=stream)


def layer_inputs(T, K, F, E, seed):
    g = gen(seed)
    w13, w2, v13, v2 = experts(g, E, K, F)
    o, gate_up, down = matrix(g, K, 512, 0.02), matrix(g, 2 * F, K, 0.02), matrix(g, K, F, 0.02)
    return dict(attended=normal(g, T, 512, dtype=torch.bfloat16), o=o[:2], gate_up=gate_up[:2], down=down[:2],
                w=(1 + 0.1 * normal(g, K)).to(torch.bfloat16), router=normal(g, K, E) * K ** -0.5, bias=0.1 * normal(g, E),
                w13=w13, w2=w2, stream=normal(g, T, K, dtype=torch.bfloat16),
                values=dict(o=o[2], gate_up=gate_up[2], down=down[2], w13=v13, w2=v2))


@pytest.mark.parametrize("T", [1, 70])
def test_layer(smla, T):
    """The run of them together, every step against the definition on what the step before it left."""
    K, F, E = 256, 128, 8
    t = layer_inputs(T, K, F, E, T)
    v, stream = t["values"], t["stream"].clone()

    def bf16(got, want, off):
        within(got, want, off + 2.0 ** -8 * (want.abs() + off))

    codes, scales = smla.mxfp8_quantize(t["attended"])
    want = ref.linear(ref.values(codes, scales), v["o"], None, "none", stream)
    smla.linear_mxfp8(codes, scales, *t["o"], residual=stream, out=stream)
    bf16(stream, *want)
    n = smla.rms_norm_mxfp8(stream, t["w"], normed=True)
    check_norm(n, stream, None, t["w"], 1e-6)
    h = smla.linear_mxfp8(n.codes, n.scales, *t["gate_up"], activation="swiglu", quantized=True)
    y, off = ref.linear(ref.values(n.codes, n.scales), v["gate_up"], None, "swiglu", None)
    within(ref.values(*h), y, ref.quantized_bound(y, off))
    want = ref.linear(ref.values(*h), v["down"], None, "none", stream)
    smla.linear_mxfp8(*h, *t["down"], residual=stream, out=stream)
    bf16(stream, *want)
    n = smla.rms_norm_mxfp8(stream, t["w"], normed=True)
    logits = (n.normed.float() @ t["router"]).contiguous()
    ids, w = smla.moe_route(logits, 2, scoring="sigmoid", bias=t["bias"], num_groups=2, topk_groups=1)
    out = smla.moe_mxfp8(n.codes, n.scales, ids, w, *t["w13"], *t["w2"], residual=stream)
    bf16(out, *ref.moe(ref.values(n.codes, n.scales), ids, w, v["w13"], v["w2"], stream))
    # and the same run in one go leaves the same bits
    again = t["stream"].clone()
    assert torch.equal(layer(smla, t, again), out) and torch.equal(again, stream)


def test_layer_captured(smla):
    """Captured into a graph and replayed on other inputs, on another stream."""
    t, other = layer_inputs(3, 256, 128, 8, 1), layer_inputs(3, 256, 128, 8, 2)
    stream = torch.cuda.Stream()
    buf = t["stream"].clone()
    layer(smla, t, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        out = layer(smla, t, buf)
    for u in (t, other):
        want_stream = u["stream"].clone()
        merged = dict(t, attended=u["attended"])
        want = layer(smla, merged, want_stream)
        buf.copy_(u["stream"])
        t["attended"].copy_(u["attended"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(buf, want_stream)


def test_refused_tensors(smla):
    """What the binding refuses before the call: shapes, types, strides, devices."""
    g = gen(0)
    x, xs, _ = matrix(g, 4, 64)
    w, ws, _ = matrix(g, 96, 64)
    b = x.new_zeros((4, 64), dtype=torch.bfloat16)
    bad = [
        lambda: smla.mxfp8_quantize(b.half()), lambda: smla.mxfp8_quantize(b[0]), lambda: smla.mxfp8_quantize(b[:, ::2]),
        lambda: smla.mxfp8_quantize(b[:, :40]), lambda: smla.mxfp8_quantize(b[:, 4:36]), lambda: smla.mxfp8_quantize(b[:1].expand(4, 64)),
        lambda: smla.mxfp8_quantize(b, codes=x[:3]), lambda: smla.mxfp8_quantize(b, scales=xs[:, :1]),
        lambda: smla.mxfp8_quantize(b, scales=xs.contiguous()),
        lambda: smla.rms_norm_mxfp8(b.float()), lambda: smla.rms_norm_mxfp8(b, weight=b[0, :32]),
        lambda: smla.rms_norm_mxfp8(b, residual=b[:3]), lambda: smla.rms_norm_mxfp8(b, normed=b[:3]),
        lambda: smla.rms_norm_mxfp8(b, quantized=False),
        lambda: smla.linear_mxfp8(b, xs, w, ws), lambda: smla.linear_mxfp8(x, xs, w[:, :32], ws),
        lambda: smla.linear_mxfp8(x, xs[:3], w, ws), lambda: smla.linear_mxfp8(x, xs, w, ws[:, :1]),
        lambda: smla.linear_mxfp8(x, xs, w[::2], ws[::2]), lambda: smla.linear_mxfp8(x, xs.float(), w, ws),
        lambda: smla.linear_mxfp8(x, xs, w, ws, bias=b[0]), lambda: smla.linear_mxfp8(x, xs, w[:95], ws[:95], activation="swiglu"),
        lambda: smla.linear_mxfp8(x, xs, w, ws, residual=b), lambda: smla.linear_mxfp8(x, xs, w, ws, out=b),
        lambda: smla.linear_mxfp8(x, xs, w[:95], ws[:95], quantized=True),
        lambda: smla.linear_mxfp8(x, xs, w, ws, residual=b.new_zeros((4, 96)), quantized=True),
        lambda: smla.linear_mxfp8(x, xs, w, ws, out_scale=xs), lambda: smla.rms_norm_mxfp8(b, normed=True, quantized=False, codes=x),
        lambda: smla.moe_route(b.half(), 2), lambda: smla.moe_route(b, 0), lambda: smla.moe_route(b, 65),
        lambda: smla.moe_route(b.t(), 2), lambda: smla.moe_route(b, 2, bias=b[0]), lambda: smla.moe_route(b, 2, num_groups=3),
        lambda: smla.moe_route(b, 2, ids=torch.zeros((4, 3), dtype=torch.int32, device="cuda")),
    ]
    (w13, s13), (w2, s2), _, _ = experts(g, 3, 64, 32)
    ids, p = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.ones((4, 2), device="cuda")
    ok = (x, xs, ids, p, w13, s13, w2, s2)
    for i, v in [(0, b), (1, xs[:2]), (2, ids.long()), (2, ids[:3]), (3, p[:, :1]), (3, p.double()), (4, w13[:, :, :32]),
                 (4, w13[0]), (4, w13.transpose(0, 1)), (5, s13[:2]), (5, s13.transpose(0, 1)), (6, w13), (7, s13), (6, w2[:2])]:
        bad.append(lambda i=i, v=v: smla.moe_mxfp8(*ok[:i], v, *ok[i + 1:]))
    bad += [lambda: smla.moe_mxfp8(*ok, residual=b[:2]), lambda: smla.moe_mxfp8(*ok, out=x),
            lambda: smla.moe_mxfp8(*ok, workspace=torch.empty(0, dtype=torch.uint8, device="cuda")),
            lambda: smla.moe_mxfp8(*[v.cpu() for v in ok])]
    for k, call in enumerate(bad):
        with pytest.raises(smla.SmlaError):
            call()
            pytest.fail(f"call {k} was not refused")
    smla.moe_mxfp8(*ok)
    torch.cuda.synchronize()


@pytest.mark.parametrize("experts", [False, True])
def test_a_wait_that_runs_out_is_reported_once(smla, experts):
    assert smla.read_device_status() == 0
    smla.mxfp8_wait_check(experts)
    assert smla.read_device_status() == 1
    assert smla.read_device_status() == 0


def test_streams(smla):
    """Two calls at once on two streams, and a stream that is named."""
    g = gen(8)
    x, xs, _ = matrix(g, 30, 512)
    (w13, s13), (w2, s2), _, _ = experts(g, 8, 512, 256)
    ids = torch.randint(0, 8, (30, 2), generator=g, device="cuda").int()
    w = torch.rand((30, 2), generator=g, device="cuda")
    want = smla.moe_mxfp8(x, xs, ids, w, w13, s13, w2, s2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [smla.moe_mxfp8(x, xs, ids, w, w13, s13, w2, s2, stream=s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(a, want) for a in got)
    q = smla.mxfp8_quantize(want, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(q[0], smla.mxfp8_quantize(want)[0])


def test_results_do_not_change_between_runs(smla):
    g = gen(12)
    x, xs, _ = matrix(g, 3, 4096)
    w, ws, _ = matrix(g, 512, 4096)
    first = smla.linear_mxfp8(x, xs, w, ws)
    for _ in range(10):
        assert torch.equal(smla.linear_mxfp8(x, xs, w, ws), first)
