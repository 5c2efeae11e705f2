"""CPU: the MXFP8 operators' reference on small cases worked by hand, and the
refusals of their entry points (before any device work)."""
import ctypes

import numpy as np
import pytest

import sparse_mla_attention_fp8_gb300 as smla

torch = pytest.importorskip("torch")
import mx_reference as ref  # noqa: E402

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD2 = ctypes.c_void_p(0x10002)
ODD8 = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    smla.build()
    return smla.lib()


# ---------------------------------------------------------------- the reference

def test_quantization_by_hand():
    x = torch.zeros((1, 96), dtype=torch.float64)
    x[0, 0], x[0, 1] = 448.0, -0.3  # scale 2^0: -0.3 lies between -0.28125 and -0.3125
    x[0, 32] = 449.0                # scale 2^1: 224.5 rounds to 224
    codes, scales = ref.bytes_of(x)
    assert scales.tolist() == [[127, 128, 27]]
    assert codes[0, 0] == 126 and codes[0, 32] == 118
    v = ref.values(codes, scales)
    assert v[0, 0] == 448 and v[0, 1] == -0.3125 and v[0, 32] == 448 and (v[0, 64:] == 0).all()


def test_quantization_against_torch():
    x = torch.randn((50, 256), generator=torch.Generator().manual_seed(0)) * 30
    codes, scales = ref.bytes_of(x.double())
    y = (x.unflatten(1, (-1, 32)) * torch.exp2(127 - scales.float())[..., None]).flatten(1)
    assert torch.equal(y.to(torch.float8_e4m3fn).view(torch.uint8), codes)
    assert (y.abs() <= 448).all() and torch.equal(ref.values(codes, scales), ref.rounded(x.double()))


def test_linear_by_hand():
    x = torch.tensor([[1.0, 2.0] + [0.0] * 30], dtype=torch.float64)
    w = torch.zeros((2, 32), dtype=torch.float64)
    w[0, 0], w[1, 1] = 3.0, -0.5
    y, _ = ref.linear(x, w, torch.tensor([0.5, 0.0]), "relu", torch.tensor([[1.0, 1.0]], dtype=torch.bfloat16))
    assert y.tolist() == [[4.5, 1.0]]
    y, _ = ref.linear(x, w, None, "swiglu", None)
    assert abs(y.item() - 3 / (1 + np.exp(-3)) * -1) < 1e-12


def test_route_by_hand():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, 0.0, 2.0]])
    ids, w = ref.route(x, 3, "softmax", None, True, 2.0, 1, 1)
    assert ids.tolist() == [[1, 2, 5]] and abs(w.sum() - 2) < 1e-12 and w[0, 0] == w[0, 1]
    # groups (0, 1, 2) and (3, 4, 5): the first has the larger sum
    ids, _ = ref.route(x, 2, "sigmoid", np.array([0, 0, 0, 0, 0.1, 0.2]), True, 1.0, 2, 1)
    assert ids.tolist() == [[1, 2]]
    ids, w = ref.route(np.full((1, 4), -np.inf), 2, "softmax", None, True, 1.0, 1, 1)
    assert ids.tolist() == [[-1, -1]] and w.tolist() == [[0, 0]]


def test_moe_of_one_expert_is_its_mlp():
    g = torch.Generator().manual_seed(1)
    x = ref.rounded(torch.randn((3, 64), generator=g, dtype=torch.float64))
    w13 = ref.rounded(torch.randn((64, 64), generator=g, dtype=torch.float64))
    w2 = ref.rounded(torch.randn((64, 32), generator=g, dtype=torch.float64))
    ids = torch.tensor([[0, 1], [1, -1], [0, 0]], dtype=torch.int32)
    weights = torch.tensor([[1.0, 1.0], [1.0, 1.0], [0.25, 0.5]])
    out, _ = ref.moe(x, ids, weights, [w13, torch.zeros_like(w13)], [w2, w2], None)
    z = x @ w13.T
    h = z[:, :32] * torch.sigmoid(z[:, :32]) * z[:, 32:]
    assert torch.allclose(out[0], ref.rounded(h[0]) @ w2.T) and (out[1] == 0).all()
    assert torch.allclose(out[2], ref.rounded(0.75 * h[2]) @ w2.T)


# ---------------------------------------------------------------- refusals

def _quantize(L, **kw):
    a = dict(x=FAKE, type=0, stride=64, codes=FAKE, scales=FAKE, ss=4, T=4, K=64)
    a.update(kw)
    return L.mxfp8_quantize(a["x"], a["type"], a["stride"], a["codes"], a["scales"], a["ss"], a["T"], a["K"], None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(K=0), dict(K=-32), dict(K=48), dict(type=2), dict(x=None), dict(x=ODD8),
                                dict(stride=63), dict(stride=60), dict(codes=None), dict(codes=ODD8), dict(scales=None),
                                dict(scales=ODD2), dict(ss=2), dict(ss=0), dict(ss=6), dict(K=160, stride=160, ss=4)])
def test_quantize_refuses(L, kw):
    assert _quantize(L, **kw) == -1 and L.smla_last_error()


def test_nothing_to_do(L):
    assert _quantize(L, T=0, x=None, codes=None, scales=None) == 0
    assert _norm(L, T=0, x=None) == 0
    assert _linear(L, T=0, x=None) == 0
    assert _route(L, T=0, logits=None) == 0
    assert _moe(L, T=0, x=None) == 0


def _norm(L, **kw):
    a = dict(x=FAKE, xs=64, r=None, rs=0, w=FAKE, wt=0, eps=1e-6, codes=FAKE, scales=FAKE, ss=4, normed=None, h=None, T=4, K=64)
    a.update(kw)
    return L.rms_norm_mxfp8(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["wt"], a["eps"], a["codes"], a["scales"], a["ss"],
                            a["normed"], a["h"], a["T"], a["K"], None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(K=40), dict(wt=7), dict(eps=-1e-6), dict(eps=float("nan")), dict(x=None),
                                dict(x=ODD8), dict(xs=72, x=ODD8), dict(xs=60), dict(r=ODD8, rs=64), dict(r=FAKE, rs=32),
                                dict(w=ODD8), dict(codes=None), dict(scales=None), dict(codes=ODD8), dict(ss=2),
                                dict(normed=ODD8), dict(h=ODD8), dict(codes=None, scales=None)])
def test_norm_refuses(L, kw):
    assert _norm(L, **kw) == -1 and L.smla_last_error()


def test_norm_refuses_long_rows(L):
    assert _norm(L, K=65536 + 32, xs=65536 + 32, ss=4096) == -2


def _linear(L, **kw):
    a = dict(x=FAKE, xs=64, sx=FAKE, sxs=4, w=FAKE, sw=FAKE, sws=4, b=None, bt=0, act=0, r=None, rs=0, out=FAKE, codes=None,
             scales=None, ss=0, T=4, N=64, K=64)
    a.update(kw)
    return L.linear_mxfp8(a["x"], a["xs"], a["sx"], a["sxs"], a["w"], a["sw"], a["sws"], a["b"], a["bt"], a["act"], a["r"],
                          a["rs"], a["out"], a["codes"], a["scales"], a["ss"], a["T"], a["N"], a["K"], None)


CODED = dict(out=None, codes=FAKE, scales=FAKE, ss=4)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(N=0), dict(K=16), dict(bt=3), dict(act=-1), dict(act=6), dict(x=None), dict(x=ODD8),
                                dict(xs=72), dict(xs=32), dict(sx=None), dict(sx=ODD2), dict(sxs=2), dict(w=None), dict(w=ODD8),
                                dict(sw=None), dict(sws=0), dict(out=None), dict(out=ctypes.c_void_p(0x10001)),
                                dict(r=FAKE, rs=32), dict(r=ctypes.c_void_p(0x10001), rs=64), dict(b=ctypes.c_void_p(0x10001)),
                                dict(b=ODD2, bt=1), dict(codes=FAKE), dict(scales=FAKE), dict(CODED, N=48), dict(CODED, codes=ODD2),
                                dict(CODED, scales=None), dict(CODED, ss=0)])
def test_linear_refuses(L, kw):
    assert _linear(L, **kw) == -1 and L.smla_last_error()


def test_linear_refuses_a_residual_with_codes(L):
    assert _linear(L, **CODED, r=FAKE, rs=64) == -2


def _route(L, **kw):
    a = dict(logits=FAKE, lt=1, b=None, sc=0, ren=1, scale=1.0, g=1, tg=1, ids=FAKE, w=FAKE, T=4, E=64, topk=8)
    a.update(kw)
    return L.moe_route(a["logits"], a["lt"], a["b"], a["sc"], a["ren"], a["scale"], a["g"], a["tg"], a["ids"], a["w"], a["T"],
                       a["E"], a["topk"], None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(topk=0), dict(g=0), dict(tg=0), dict(tg=2), dict(lt=5), dict(sc=2),
                                dict(g=3, tg=1), dict(g=64, tg=64), dict(E=128, g=64, tg=64), dict(g=16, tg=1), dict(E=4),
                                dict(logits=None), dict(ids=None), dict(w=None)])
def test_route_refuses(L, kw):
    assert _route(L, **kw) == -1 and L.smla_last_error()


@pytest.mark.parametrize("kw", [dict(E=513), dict(E=64, topk=33)])
def test_route_refuses_large(L, kw):
    assert _route(L, **kw) == -2


def _moe(L, **kw):
    a = dict(x=FAKE, xs=64, sx=FAKE, sxs=4, ids=FAKE, g=FAKE, w13=FAKE, s13=FAKE, ss13=4, w2=FAKE, s2=FAKE, ss2=4, r=None, rs=0,
             out=FAKE, T=4, E=8, topk=2, K=64, F=96, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return L.moe_mxfp8(a["x"], a["xs"], a["sx"], a["sxs"], a["ids"], a["g"], a["w13"], a["s13"], a["ss13"], a["w2"], a["s2"],
                       a["ss2"], a["r"], a["rs"], a["out"], a["T"], a["E"], a["topk"], a["K"], a["F"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(topk=0), dict(F=0), dict(F=48), dict(K=48), dict(ids=None), dict(g=None),
                                dict(x=None), dict(x=ODD8), dict(xs=40), dict(sx=ODD2), dict(sxs=3), dict(w13=None),
                                dict(w13=ODD8), dict(s13=None), dict(ss13=0), dict(w2=None), dict(s2=ODD2), dict(ss2=2),
                                dict(out=None), dict(out=ctypes.c_void_p(0x10001)), dict(r=FAKE, rs=16), dict(ws=ODD8)])
def test_moe_refuses(L, kw):
    assert _moe(L, **kw) == -1 and L.smla_last_error()


@pytest.mark.parametrize("kw", [dict(E=513), dict(topk=33), dict(E=512, K=4194304, xs=4194304, sxs=131072)])
def test_moe_refuses_large(L, kw):
    assert _moe(L, **kw) == -2


def test_moe_workspace(L):
    n = smla.moe_mxfp8_workspace_bytes(4, 8, 2, 96)
    assert n > 0 and _moe(L, wsb=n - 1) == -4 and b"needed" in L.smla_last_error()
    for bad in [(-1, 8, 2, 96), (4, 0, 2, 96), (4, 513, 2, 96), (4, 8, 0, 96), (4, 8, 33, 96), (4, 8, 2, 40)]:
        assert smla.moe_mxfp8_workspace_bytes(*bad) == 0
    # rows: the tile's tokens for every expert that they can go to
    assert smla.moe_mxfp8_workspace_bytes(1, 64, 8, 1024) >= 8 * 16 * 1024
    assert smla.moe_mxfp8_workspace_bytes(200, 4, 2, 96) >= 4 * 4 * 64 * 96


def test_names_are_checked():
    with pytest.raises(smla.SmlaError, match="activation"):
        smla.linear_mxfp8(None, None, None, None, activation="tanh")
    with pytest.raises(smla.SmlaError, match="scoring"):
        smla.moe_route(None, 2, scoring="top")


def test_cpu_tensors_are_refused():
    smla.build()
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    b = torch.zeros((2, 64), dtype=torch.uint8)
    s = torch.zeros((2, 4), dtype=torch.uint8)[:, :2]
    for call in (lambda: smla.mxfp8_quantize(x), lambda: smla.rms_norm_mxfp8(x), lambda: smla.linear_mxfp8(b, s, b, s),
                 lambda: smla.moe_route(x, 2), lambda: smla.moe_mxfp8(b, s, b, b, b, s, b, s)):
        with pytest.raises(smla.SmlaError, match="CUDA"):
            call()
