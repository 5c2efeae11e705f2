"""GPU: the paged 8-bit K/V cache operators at the ends of what their entry
points take, against the float64 reference (tests/paged_reference.py)."""
import numpy as np
import pytest

import paged_reference as ref
from helpers import dev, torch_mod
from test_gpu_paged import attend, bf16, check, i32, run_store, smla, store_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- caps

def capped(b):
    """The expected results of a batch with a cap, within what holds without it: the cap's own part
    in the reference's tolerance (2^-20 of the cap) is no limit where the cap is far above the logits."""
    want, want_lse, _, _ = b.expected()
    _, _, tol, ltol = ref.attention(b.q, *b.caches, *b.scales, b.table, b.lens, b.query_start, b.sm_scale, b.window,
                                    0.0, b.slopes, b.prefix, b.doc)
    return want, want_lse, tol, ltol


@pytest.mark.parametrize("cap", [300.0, 1e4, 1e6, 1e9, 1e30])
@pytest.mark.parametrize("G,D,new", [(4, 128, [1, 1]), (3, 64, [2, 5]), (6, 64, [30, 70]), (4, 128, [40, 20])])
def test_wide_caps(smla, G, D, new, cap):  # noqa: F811
    """Caps far above the logits leave them as they are, with few rows and with many."""
    b = ref.Batch(70, 2, G, D, [500, 90], new, softcap=cap)
    check(b, attend(smla, b), capped(b))


@pytest.mark.parametrize("cap", [1e4, 1e6])
@pytest.mark.parametrize("G,D,new", [(4, 128, [1, 1]), (3, 64, [2, 5]), (6, 64, [30, 70])])
def test_wide_caps_beside_rows_that_reach_them(smla, G, D, new, cap):  # noqa: F811
    """One head's logits go up to the cap; the other heads', a hundred thousandth of it, keep their own precision."""
    b = ref.Batch(71, 2, G, D, [500, 90], new, softcap=cap)
    b.q[:, 0] *= np.float32(cap / 4)
    b.q = ref.bf16_round(b.q)
    check(b, attend(smla, b), capped(b))


# ---------------------------------------------------------------- small weights

def small_weights(smla, HK, G, new, top, rest, n, R=4):  # noqa: F811
    """Four requests of n keys that weigh 2^rest each behind a newest block of 64 that weigh 2^top each: (the
    old keys' share of the sum from the kernel, the right one)."""
    torch = torch_mod()
    D, MB = 64, n // 64 + 1
    NB = R * MB
    k = torch.full((NB, HK, 64, D), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    v = k.clone()
    table = torch.randperm(NB, device="cuda").to(torch.int32).view(R, MB)
    v[table[:, -1].long()] = 0
    ks = torch.full((NB, HK), rest / D * np.log(2), device="cuda")
    ks[table[:, -1].long()] = top / D * np.log(2)
    vs = torch.ones((NB, HK), device="cuda")
    lens = i32([n + 64] * R)
    out, _ = smla.paged_attention_fp8(
        torch.ones((R * new, HK * G, D), dtype=torch.bfloat16, device="cuda"), k, v, ks, vs, table, lens,
        i32(np.arange(R + 1) * new), 1.0, max_query_len=new, prefix_lens=lens)
    a, b = 64.0, n * 2.0 ** (rest - top)
    return out.double(), b / (a + b)


@pytest.mark.parametrize("top,rest", [(0, -13.6), (0, -15.4), (0, -17), (0, -18.3), (16, 0), (100, 84.5), (-5, -21.6),
                                      (-12, -23.4), (-40, -52.3)])
@pytest.mark.parametrize("HK,G,new", [(80, 1, 1), (40, 12, 1), (16, 16, 20)])
def test_small_weights_are_not_dropped(smla, HK, G, new, top, rest):  # noqa: F811
    """A tolerance that a result without the small weights misses.  Few rows: equal weights within 2^-24 of the
    largest on average.  Tiles of 256 rows: within 2^-25 of a sum that is kept at 2^4 or more once 512 keys are
    in it, and at 2 here before; the rounding to f16 or two e4m3 terms 2^-7 of the value, to bf16 2^-8, the
    logits' 2^-20 |x|."""
    n = 8000
    out, want = small_weights(smla, HK, G, new, top, rest, n)
    dx = 2.0 ** -20 * max(abs(top), abs(rest))
    steps = n * 2.0 ** -24 / 64 if G * new <= 48 else 512 * 2.0 ** -25 / 2 + n * 2.0 ** -25 / 16
    tol = (2.0 ** -7 + 2.0 ** -8 + 2 * dx) * want + steps
    assert tol < want / 2
    assert (out - want).abs().max().item() <= tol


@pytest.mark.parametrize("HK,G,new", [(80, 64, 1), (80, 1, 60)])
@pytest.mark.parametrize("top,rest", [(-8, -25.1), (-8.9, -25.3), (-7, -24.6)])
def test_many_small_weights_behind_a_weak_start(smla, HK, G, new, top, rest):  # noqa: F811
    """The newest block, alone in its tile of keys, weighs 2^top x 64 (between 2^-3 and 1/2); each of the 25 000
    keys before it less than what f16 holds beside the reference 0.  Within 2^-25 of 2^4 each, the first 512
    within 2^-25 of 64 x 2^top."""
    n = 25088  # the tiles have 128 keys: the newest block shares its tile with none
    out, want = small_weights(smla, HK, G, new, top, rest, n)
    dx = 2.0 ** -20 * max(abs(top), abs(rest))
    tol = (2.0 ** -7 + 2.0 ** -8 + 2 * dx) * want + 512 * 2.0 ** -25 / (64 * 2.0 ** top) + n * 2.0 ** -25 / 16
    assert tol < want / 2
    assert (out - want).abs().max().item() <= tol


# ---------------------------------------------------------------- store

@pytest.mark.parametrize("HK,D,ctx,new", [(2, 128, [9, 40], [1, 1]), (3, 64, [5, 60], [40, 30]), (2, 128, [33, 1], [31, 70])])
def test_store_under_scales_that_are_no_powers_of_two(smla, HK, D, ctx, new):  # noqa: F811
    """A block that another program has begun may have any scale: the codes of the new rows are the quotients'
    nearest, ties to even, and those of the old rows too where the scale grows."""
    lens, start, table, _, x, cache, scale = store_inputs(HK, D, ctx, new, 80)
    rng = np.random.default_rng(81)
    for i in range(2):
        # scales around which products with the rounded reciprocal go wrong, and any others
        scale[i][:] = rng.choice(np.array([3.0, 0.75, 7.0, 0.3, 1.1, 5.0 / 3.0], np.float32), scale[i].shape)
        scale[i][::3] *= rng.uniform(0.5, 2.0, scale[i][::3].shape).astype(np.float32)
        # values half-way between two codes under the scale of their block, as near as bf16 comes to them
        half = (ref.E4M3[8:120] + ref.E4M3[9:121]) / 2
        tie = rng.choice(half, x[i].shape) * rng.choice([-1.0, 1.0], x[i].shape)
        for r in range(len(ctx)):
            b = table[r, ctx[r] // 64]
            t = slice(start[r], start[r + 1])
            x[i][t] = ref.bf16_round(tie[t] * scale[i][b][None, :, None])
        x[i][start[0], 0, 0] = ref.bf16_round(np.array([5000.0]))[0]  # makes one block's scale grow
        x[i][start[1], 0, 1:4] = [np.nan, np.inf, -np.inf]
    run_store(smla, lens, start, table, x, cache, scale)


@pytest.mark.parametrize("old", [14447047.0 * 2 ** -24, 1.9, 0.3])
def test_store_rescales_old_codes_to_the_nearest(smla, old):  # noqa: F811
    """Every finite code under an odd scale that grows to a power of two: 9 x 14447047 lies just below
    half-way between two codes, where its float32 product lies on it."""
    lens, start = np.array([63], np.int32), np.array([0, 1], np.int32)
    codes = np.resize(np.array([c for c in range(256) if c & 127 != 127], np.uint8), (1, 1, 64, 64))
    cache, scale = [codes.copy(), codes.copy()], [np.full((1, 1), old, np.float32) for _ in range(2)]
    x = [np.full((1, 1, 64), 448.0 * 2 ** e, np.float32) for e in (1, 3)]
    run_store(smla, lens, start, np.zeros((1, 1), np.int32), x, cache, scale)


@pytest.mark.parametrize("old", [np.inf, -3.0, -2.0, 1e-40, 3e38])
@pytest.mark.parametrize("n", [1, 40])
def test_store_into_blocks_of_odd_scales(smla, old, n):  # noqa: F811
    """An infinite scale stays and takes codes of 0, a negative or tiny one is replaced; no NaN code is written."""
    rng = np.random.default_rng(82)
    cache = [ref.e4m3_encode(rng.standard_normal((2, 2, 64, 128)) * 100) for _ in range(2)]
    scale = [np.full((2, 2), old, np.float32) for _ in range(2)]
    x = [ref.bf16_round(rng.standard_normal((n, 2, 128))) for _ in range(2)]
    run_store(smla, np.array([20 + n], np.int32), np.array([0, n], np.int32), np.array([[1, 0]], np.int32), x, cache, scale)


# ---------------------------------------------------------------- workspaces

def test_an_empty_workspace_is_refused(smla):  # noqa: F811
    """And not taken for none."""
    torch = torch_mod()
    b = ref.Batch(50, 2, 2, 64, [3], [2])
    with pytest.raises(smla.SmlaError, match="workspace"):
        smla.paged_attention_fp8(bf16(b.q), *(dev(c) for c in b.caches), *(dev(s) for s in b.scales), i32(b.table),
                                 i32(b.lens), i32(b.query_start), 0.1,
                                 workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- failed calls

@pytest.mark.parametrize("many_rows", [False, True])
def test_a_wait_that_runs_out_is_reported_whatever_the_workspace(smla, many_rows):  # noqa: F811
    """A device thread waits in vain, and reports it as the attention's kernels do, into a workspace that nothing
    has cleared (as the ones that calls allocate for themselves): the device's status says so once."""
    torch = torch_mod()
    workspace = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    smla.read_device_status()
    assert smla.read_device_status() == 0
    smla.paged_wait_check(workspace, many_rows=many_rows)
    assert smla.read_device_status(workspace) == 1
    assert smla.read_device_status(workspace) == 0
    del workspace
    assert smla.read_device_status() == 1
    assert smla.read_device_status() == 0


# ---------------------------------------------------------------- launch order

def test_calls_behind_a_store_that_skips_all(smla):  # noqa: F811
    """A decode, a store whose tokens are all skipped, and the paged attention in the workspace that the decode
    uses: the store ends behind the decode, so the attention begins behind it, too."""
    import ctypes

    import smla_inputs as inp
    from helpers import bf16_dev, oracle_cache
    torch = torch_mod()
    case = inp.memory_bound_decode(seed=5, R=9, ctx_lo=300, ctx_hi=2500, K=200, H=16)
    cache = dev(oracle_cache(case))
    args = (bf16_dev(case.q), cache, dev(case.indices), dev(case.block_table), dev(case.req_id_per_token), case.sm_scale)
    b = ref.Batch(90, 2, 4, 128, [2000, 30, 700], [1, 1, 1])
    q, rest = bf16(b.q), [dev(x) for x in b.caches + b.scales + [b.table, b.lens, b.query_start]]
    rows, skip = torch.zeros((9, 576), dtype=torch.bfloat16, device="cuda"), torch.full((9,), -1, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    want = smla.sparse_mla_decode_fp8(*args)

    def p(t):
        return ctypes.c_void_p(t.data_ptr())

    def attend_in_the_librarys_workspace():
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        rc = smla.lib().paged_attention_fp8(p(q), 8 * 128, *(p(x) for x in rest), b.sm_scale, 1, 0, 0.0, None, None, None,
                                            p(out), p(lse), 3, 8, 2, 128, 3, b.table.shape[1], b.NB, None, 0, stream)
        assert rc == 0, smla.lib().smla_last_error()
        return out, lse

    attend_in_the_librarys_workspace()  # (the workspace grows)
    torch.cuda.synchronize()
    expected = b.expected()
    got = []
    for _ in range(20):
        decoded = smla.sparse_mla_decode_fp8(*args)
        smla.mla_cache_store_fp8(rows, skip, cache)
        got.append((decoded, attend_in_the_librarys_workspace()))
    torch.cuda.synchronize()
    for decoded, (out, lse) in got:
        assert torch.equal(decoded[0], want[0]) and torch.equal(decoded[1], want[1])
        check(b, (out.float().cpu().numpy(), lse.cpu().numpy()), expected)


def test_latent_store_directly_behind_the_tables(smla):  # noqa: F811
    """Step after step into the same tables and slot map, each read by the store launched behind it."""
    import oracle
    torch = torch_mod()
    rng = np.random.default_rng(91)
    R, MB, NB, T, steps = 5, 9, 45, 400, 12
    table = torch.full((R, MB), -1, dtype=torch.int32, device="cuda")
    stack, ctx, count = i32(rng.permutation(NB)), i32([0] * R), i32([NB])

    def e(n, t=torch.int32):
        return torch.full((n,), -7, dtype=t, device="cuda")

    out = smla.PagedBatch(e(R + 1), ctx, e(T), e(T), e(T, torch.int64), count, e(1))
    cache = torch.zeros((NB, 64, 656), dtype=torch.uint8, device="cuda")
    news = [rng.integers(0, 60, R) for _ in range(steps)]
    rows = [bf16(rng.standard_normal((T, 576))) for _ in range(steps)]
    d_news = [i32(n) for n in news]
    torch.cuda.synchronize()
    for new, x in zip(d_news, rows):
        smla.paged_blocks_extend(ctx, new, table, stack, count, T, NB, out=out)
        smla.mla_cache_store_fp8(x, out.slot_mapping, cache)
    torch.cuda.synchronize()
    want, w_ctx, w_count = np.zeros((NB, 64, 656), np.uint8), np.zeros(R, np.int32), NB
    w_table = np.full((R, MB), -1, np.int32)
    for new, x in zip(news, rows):
        w_table, _, w_ctx, _, _, slot, w_count, _ = ref.extend(w_ctx, new, w_table, stack.cpu().numpy(), w_count, T, NB)
        oracle.quantize_store(x.cpu().view(torch.int16).numpy().view(np.uint16), slot.astype(np.int64), want)
    assert np.array_equal(table.cpu().numpy(), w_table) and int(count) == w_count
    assert np.array_equal(cache.cpu().numpy(), want)
