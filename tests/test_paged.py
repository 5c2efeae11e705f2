"""CPU: the paged K/V cache operators' reference on small cases worked by
hand, and the refusals of their entry points (before any device work)."""
import ctypes

import numpy as np
import pytest

import paged_reference as ref
import sparse_mla_attention_fp8_gb300 as smla

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    smla.build()
    return smla.lib()


def test_e4m3_grid():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    theirs = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(theirs), np.isnan(ref.E4M3))
    ok = ~np.isnan(theirs)
    assert np.array_equal(theirs[ok], ref.E4M3[ok])
    assert np.array_equal(ref.e4m3_encode(ref.E4M3[ok]), codes[ok])
    x = np.random.default_rng(0).standard_normal(4000) * 100
    x = np.clip(x, -448, 448).astype(np.float32)
    assert np.array_equal(ref.e4m3_encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_extend_by_hand():
    # request 0: 63 tokens in block 5, 3 new: one new block; request 1: empty, 64 new: one; request 2: nothing
    table = np.array([[5, -1], [-1, -1], [7, 8]], np.int32)
    t, start, lens, req, pos, slot, left, missing = ref.extend(
        [63, 0, 128], [3, 64, 0], table, np.array([1, 2, 3]), 3, 70, 9)
    assert t.tolist() == [[5, 3], [2, -1], [7, 8]]
    assert start.tolist() == [0, 3, 67, 67] and lens.tolist() == [66, 64, 128]
    assert slot[:4].tolist() == [5 * 64 + 63, 3 * 64, 3 * 64 + 1, 2 * 64] and slot[66:].tolist() == [2 * 64 + 63, -1, -1, -1]
    assert req[66:].tolist() == [1, -1, -1, -1] and pos[:4].tolist() == [63, 64, 65, 0] and (left, missing) == (1, 0)


def test_store_by_hand():
    cache, scale = np.zeros((2, 1, 64, 64), np.uint8), np.zeros((2, 1), np.float32)
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, 0], x[1, 0, 1] = 448.0, 449.0
    c, s = ref.store(x[:1], [0, 1], [1], np.array([[1]]), cache, scale)
    assert s[1, 0] == 1.0 and c[1, 0, 0, 0] == 126
    c, s = ref.store(x[1:], [0, 1], [2], np.array([[1]]), c, s)  # needs twice the scale: the first row's code follows
    assert s[1, 0] == 2.0 and ref.E4M3[c[1, 0, 0, 0]] == 224.0 and ref.E4M3[c[1, 0, 1, 1]] == 224.0


def test_attention_of_one_key_is_its_value():
    b = ref.Batch(1, 2, 3, 64, [0, 5], [1, 1], window=1)
    out, lse, _, _ = b.expected()
    for t, (r, p) in enumerate([(0, 0), (1, 5)]):
        for h in range(6):
            blk = b.table[r, 0]
            v = ref.E4M3[b.caches[1][blk, h // 3, p]] * b.scales[1][blk, h // 3]
            assert np.allclose(out[t, h], v, rtol=1e-12)


# ---------------------------------------------------------------- refusals

def _extend(L, **kw):
    a = dict(c=FAKE, q=FAKE, bt=FAKE, fb=FAKE, fc=FAKE, qs=FAKE, sl=FAKE, req=FAKE, pos=FAKE, slot=FAKE, fo=FAKE,
             miss=FAKE, R=2, MB=4, NB=8, F=8, T=3, stream=None)
    a.update(kw)
    return L.paged_blocks_extend(*a.values())


def _release(L, **kw):
    a = dict(rel=FAKE, sl=FAKE, bt=FAKE, fb=FAKE, fc=FAKE, cl=FAKE, fo=FAKE, R=2, MB=4, NB=8, F=8, stream=None)
    a.update(kw)
    return L.paged_blocks_release(*a.values())


def _store(L, **kw):
    a = dict(k=FAKE, ks=256, v=FAKE, vs=256, qs=FAKE, sl=FAKE, bt=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, T=3,
             HK=2, D=128, R=2, MB=4, NB=8, stream=None)
    a.update(kw)
    return L.kv_cache_store_fp8(*a.values())


def _attend(L, **kw):
    a = dict(q=FAKE, qs=512, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, bt=FAKE, sl=FAKE, qst=FAKE, scale=0.1, mq=1, win=0,
             cap=0.0, al=None, pre=None, doc=None, out=FAKE, lse=FAKE, T=3, H=4, HK=2, D=128, R=2, MB=4, NB=8, ws=FAKE,
             wsb=1 << 30, stream=None)
    a.update(kw)
    return L.paged_attention_fp8(*a.values())


@pytest.mark.parametrize("call", [_extend, _release, _store, _attend])
@pytest.mark.parametrize("kw,rc", [(dict(R=-1), -1), (dict(MB=0), -1), (dict(NB=0), -1), (dict(R=8193), -2),
                                   (dict(NB=1 << 26), -2), (dict(MB=1 << 26), -2)])
def test_refuses_bad_batches(L, call, kw, rc):
    assert call(L, **kw) == rc


@pytest.mark.parametrize("kw", [dict(T=-1), dict(F=-1), dict(c=None), dict(bt=None), dict(fb=None), dict(fc=None),
                                dict(qs=None), dict(slot=None), dict(miss=None)])
def test_extend_refuses(L, kw):
    assert _extend(L, **kw) == -1


@pytest.mark.parametrize("kw", [dict(F=-1), dict(rel=None), dict(fb=None), dict(fc=None), dict(cl=None), dict(fo=None)])
def test_release_refuses(L, kw):
    assert _release(L, **kw) == -1


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), -1), (dict(HK=0), -1), (dict(D=96), -2), (dict(k=None), -1), (dict(v=ODD), -1), (dict(ks=255), -1),
    (dict(vs=260), -1), (dict(qs=None), -1), (dict(kc=ODD), -1), (dict(vsc=None), -1), (dict(NB=1 << 24, HK=4), -2),
    (dict(T=0, k=None), 0), (dict(R=0, k=None), 0)])
def test_store_refuses(L, kw, rc):
    assert _store(L, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(H=5), -1), (dict(H=258, qs=258 * 128), -2), (dict(D=192), -2), (dict(MB=(1 << 24) + 1), -2),
    (dict(win=-1), -1), (dict(mq=-1), -1), (dict(cap=-1.0), -1), (dict(cap=float("nan")), -1),
    (dict(cap=float("inf")), -1), (dict(q=None), -1), (dict(q=ODD), -1), (dict(qs=504), -1), (dict(qs=516), -1),
    (dict(out=ODD), -1), (dict(lse=None), -1), (dict(ksc=None), -1), (dict(ws=ctypes.c_void_p(0x10010)), -1),
    (dict(wsb=16), -4), (dict(T=0, q=None), 0), (dict(R=0, q=None), 0)])
def test_attention_refuses(L, kw, rc):
    assert _attend(L, **kw) == rc
    if rc:
        assert L.smla_last_error()


def test_python_binding_has_no_cpu_path():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    c, s = torch.zeros((2, 1, 64, 64), dtype=torch.uint8), torch.zeros((2, 1))
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(smla.SmlaError, match="CUDA"):
        smla.paged_blocks_extend(i, i, torch.zeros((2, 3), dtype=torch.int32), i, i[:1], 2, 2)
    with pytest.raises(smla.SmlaError, match="CUDA"):
        smla.kv_cache_store_fp8(x, x, i, i[:1], i[None, :1], c, c, s, s)
    with pytest.raises(smla.SmlaError, match="CUDA"):
        smla.paged_attention_fp8(x, c, c, s, s, i[None, :1], i[:1], i, 0.1)
