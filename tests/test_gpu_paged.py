"""GPU: block tables, the paged 8-bit K/V store and the attention over it,
against the float64 reference (tests/paged_reference.py)."""
import numpy as np
import pytest

import paged_reference as ref
from helpers import dev, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_attention_fp8_gb300 as m
    m.build()
    return m


def bf16(x):
    torch = torch_mod()
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16)


def i32(x):
    return dev(np.asarray(x, np.int32))


# ---------------------------------------------------------------- block tables

EXTEND = [
    # context, new tokens, blocks per row, blocks on the stack (None: enough), rows behind the last token
    ([0], [1], 1, None, 0),
    ([63, 64, 65, 0], [1, 1, 1, 0], 4, None, 0),
    ([5, 0, 128, 700], [0, 0, 0, 0], 16, None, 3),
    ([0, 100, 64], [200, 1, 130], 6, None, 5),
    ([10, 20, 0], [300, 300, 300], 4, None, 0),         # beyond MB blocks
    ([0, 60, 0], [200, 200, 64], 6, 4, 7),              # the stack runs out
    ([0, 60, 0], [200, 200, 64], 6, 0, 0),              # an empty stack
    ([-5, 3], [4, -2], 2, None, 2),                     # negative lengths count as 0
    ([0, 0], [40, 40], 2, None, -30),                   # fewer rows than tokens
]


def run_extend(smla, ctx, new, MB, count, T, NB, seed=0, alias=False):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx, np.int32), np.asarray(new, np.int32)
    order = rng.permutation(NB).astype(np.int32)
    table = np.full((len(ctx), MB), -1, np.int32)
    at = 0
    for r, c in enumerate(ctx):
        n = min(ref.blocks(max(0, int(c))), MB)
        table[r, :n] = order[at:at + n]
        at += n
    stack = np.concatenate([order[at:], np.zeros(3, np.int32)])
    count = len(order) - at if count is None else count
    want = ref.extend(ctx, new, table, stack, count, T, NB)
    d_ctx, d_table, d_count = i32(ctx), i32(table), i32([count])
    out = None
    if alias:
        e = lambda n, t=torch.int32: torch.full((n,), -7, dtype=t, device="cuda")  # noqa: E731
        out = (e(len(ctx) + 1), d_ctx, e(T), e(T), e(T, torch.int64), d_count, e(1))
    got = smla.paged_blocks_extend(d_ctx, i32(new), d_table, i32(stack), d_count, T, NB, out=out)
    torch.cuda.synchronize()
    for name, a, b in zip(("table", "start", "lens", "req", "pos", "slot", "count", "missing"), (d_table,) + tuple(got), want):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1)), name
    if alias:
        assert got.seq_lens is d_ctx and got.free_count is d_count


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("case", EXTEND)
def test_extend(smla, case, alias):
    ctx, new, MB, count, pad = case
    T = sum(max(0, n) for n in new) + pad
    NB = sum(ref.blocks(max(0, c) + max(0, n)) for c, n in zip(ctx, new)) + 2
    run_extend(smla, ctx, new, MB, count, T, NB, alias=alias)


@pytest.mark.parametrize("R,most", [(255, 3), (257, 1), (1025, 9), (3000, 40), (8192, 2)])
def test_extend_many_requests(smla, R, most):
    rng = np.random.default_rng(R)
    ctx, new = rng.integers(0, 400, R), rng.integers(0, most + 1, R)
    NB = sum(ref.blocks(int(c + n)) for c, n in zip(ctx, new)) + 1
    run_extend(smla, ctx, new, 8, None, int(new.sum()) + 11, NB, alias=True)


def test_extend_without_requests(smla):
    torch = torch_mod()
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    got = smla.paged_blocks_extend(e, e, torch.empty((0, 4), dtype=torch.int32, device="cuda"), i32([3, 1]), i32([2]), 3, 8)
    assert got.query_start.tolist() == [0] and got.req_id_per_token.tolist() == [-1] * 3
    assert got.slot_mapping.tolist() == [-1] * 3 and got.free_count.tolist() == [2] and got.missing.tolist() == [0]


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("lens,gone,MB,count,F", [
    ([64], [1], 1, 0, 4), ([0, 1, 65, 700], [1, 0, 1, 1], 11, 3, 40), ([100, 100], [0, 0], 2, 5, 9),
    ([9999, 64], [1, 1], 3, 0, 9),            # longer than its table row
    ([300, 300, 300], [1, 1, 1], 5, 2, 10),   # more than the stack holds
    ([70000] * 3, [1, 0, 1], 1200, 1, 3000)])
def test_release(smla, lens, gone, MB, count, F, alias):
    torch = torch_mod()
    rng = np.random.default_rng(MB)
    R = len(lens)
    NB = R * MB + 2
    table = rng.permutation(NB)[:R * MB].reshape(R, MB).astype(np.int32)
    table[rng.random((R, MB)) < 0.1] = -1
    table[-1, MB // 2] = NB  # outside the cache
    stack = rng.integers(0, NB, F).astype(np.int32)
    want = ref.release(np.array(gone, bool), np.array(lens), table, stack, count, NB)
    d_lens, d_stack, d_count = i32(lens), i32(stack), i32([count])
    kw = dict(context_lens=d_lens, free_count_out=d_count) if alias else {}
    ctx, n = smla.paged_blocks_release(dev(np.array(gone, bool)), d_lens, i32(table), d_stack, d_count, NB, **kw)
    torch.cuda.synchronize()
    for a, b in zip((d_stack, ctx, n), want):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1))


def test_release_many_requests(smla):
    rng = np.random.default_rng(3)
    R, MB = 5000, 6
    lens, gone = rng.integers(0, 64 * MB + 1, R), rng.random(R) < 0.4
    table = rng.permutation(R * MB).reshape(R, MB).astype(np.int32)
    stack = np.zeros(R * MB, np.int32)
    want = ref.release(gone, lens, table, stack, 0, R * MB)
    d_stack = i32(stack)
    ctx, n = smla.paged_blocks_release(dev(gone), i32(lens), i32(table), d_stack, i32([0]), R * MB)
    for a, b in zip((d_stack, ctx, n), want):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1))


# ---------------------------------------------------------------- store

STORE = [
    # HK, D, context, new
    (1, 64, [0], [1]),
    (2, 128, [0, 1, 63, 64, 5], [1, 1, 1, 1, 0]),
    (3, 128, [0, 60, 127], [64, 5, 130]),
    (5, 64, [10, 0, 64, 33], [3, 200, 64, 31]),
    (9, 128, [7, 50], [9, 17]),
    (4, 64, [0, 3], [16, 8]),
]


def store_inputs(HK, D, ctx, new, seed):
    rng = np.random.default_rng(seed)
    lens = np.array([a + b for a, b in zip(ctx, new)], np.int32)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    need = [ref.blocks(int(n)) for n in lens]
    NB = sum(need) + 2
    table = np.full((len(ctx), max(need) + 1), -1, np.int32)
    order, at = rng.permutation(NB), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    T = int(start[-1])
    x = [ref.bf16_round(rng.standard_normal((T, HK, D)) * 2.0 ** rng.integers(-6, 7, (T, HK, 1))) for _ in range(2)]
    cache = [ref.e4m3_encode(rng.standard_normal((NB, HK, 64, D)) * 100) for _ in range(2)]
    scale = [(2.0 ** rng.integers(-8, 2, (NB, HK))).astype(np.float32) for _ in range(2)]
    return lens, start, table, NB, x, cache, scale


def run_store(smla, lens, start, table, x, cache, scale, k=None, v=None):
    torch = torch_mod()
    d_cache, d_scale = [dev(c) for c in cache], [dev(s) for s in scale]
    smla.kv_cache_store_fp8(bf16(x[0]) if k is None else k, bf16(x[1]) if v is None else v, i32(start), i32(lens),
                            i32(table), *d_cache, *d_scale)
    torch.cuda.synchronize()
    for i in range(2):
        c, s = ref.store(x[i], start, lens, table, cache[i], scale[i])
        assert np.array_equal(d_scale[i].cpu().numpy(), s)
        assert np.array_equal(d_cache[i].cpu().numpy(), c)


@pytest.mark.parametrize("case", STORE)
def test_store(smla, case):
    lens, start, table, _, x, cache, scale = store_inputs(*case, seed=4)
    run_store(smla, lens, start, table, x, cache, scale)


def test_store_special_values(smla):
    lens, start, table, _, x, cache, scale = store_inputs(2, 64, [3, 0, 10], [2, 70, 1], 5)
    x[0][0, 0, :4] = [np.inf, -np.inf, np.nan, 1.0]
    x[0][1, 1] = 0.0
    x[1][2, 0] = np.inf       # a row without a finite value
    x[1][3:, 1] = 0.0         # a zero block
    x[0][5, 1] = 1e-38        # below the smallest scale's reach
    x[0][6, 0, 0] = 3.3e38
    x[0], x[1] = ref.bf16_round(x[0]), ref.bf16_round(x[1])
    run_store(smla, lens, start, table, x, cache, scale)


@pytest.mark.parametrize("HK,D,ctx,new", [(3, 128, [5, 0], [130, 64]), (2, 64, [9, 0], [150, 30]),
                                          (2, 128, [3] + [40] * 5, [45] + [1] * 5), (2, 64, [0] * 6, [60, 1, 1, 1, 1, 1])])
def test_store_scattered_special_values(smla, HK, D, ctx, new):
    """Infinities and NaN in some blocks and heads and not in others, by one warp and by four."""
    lens, start, table, _, x, cache, scale = store_inputs(HK, D, ctx, new, 7)
    rng = np.random.default_rng(7)
    for y in x:
        where = (rng.random(y.shape) < 0.002) & (rng.random((1, HK, 1)) < 0.7)
        y[where] = rng.choice([np.inf, -np.inf, np.nan], where.sum())
        assert not np.isfinite(y).all()
    run_store(smla, lens, start, table, x, cache, scale)


def test_store_skips_what_has_no_block(smla):
    lens, start, table, NB, x, cache, scale = store_inputs(2, 128, [0, 100, 5, 64], [70, 40, 3, 9], 6)
    table[0, 1], table[1, 1], table[2, 0] = -1, NB, -5
    lens[3] = 4  # fewer tokens than new rows
    run_store(smla, lens, start, table[:, :2], x, cache, scale)  # and request 1's third block beyond the table


def test_store_slices_of_a_fused_projection(smla):
    lens, start, table, _, x, cache, scale = store_inputs(3, 64, [0, 40], [5, 60], 7)
    T = x[0].shape[0]
    torch = torch_mod()
    fused = torch.full((T, 12 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = (fused[:, a * 64:(a + 3) * 64].view(T, 3, 64) for a in (6, 9))
    k.copy_(bf16(x[0]))
    v.copy_(bf16(x[1]))
    run_store(smla, lens, start, table, x, cache, scale, k, v)


def test_store_in_steps_grows_the_scale(smla):
    """Rows of growing size appended one by one: each step's codes and scales."""
    torch = torch_mod()
    rng = np.random.default_rng(8)
    cache, scale = [np.full((2, 1, 64, 128), 0x7F, np.uint8)] * 2, [np.full((2, 1), np.nan, np.float32)] * 2
    d_cache, d_scale = [dev(c) for c in cache], [dev(s) for s in scale]
    table = np.array([[1, 0]], np.int32)
    for n in range(66):
        x = [ref.bf16_round(rng.standard_normal((1, 1, 128)) * 1.3 ** (n % 40)) for _ in range(2)]
        smla.kv_cache_store_fp8(bf16(x[0]), bf16(x[1]), i32([0, 1]), i32([n + 1]), i32(table), *d_cache, *d_scale)
        for i in range(2):
            cache[i], scale[i] = ref.store(x[i], [0, 1], [n + 1], table, cache[i], scale[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(d_scale[i].cpu().numpy(), scale[i]) and np.array_equal(d_cache[i].cpu().numpy(), cache[i])


# ---------------------------------------------------------------- attention

def attend(smla, b, q=None, **kw):
    torch = torch_mod()
    opt = dict(window=b.window, softcap=b.softcap, alibi_slopes=None if b.slopes is None else dev(b.slopes),
               prefix_lens=None if b.prefix is None else i32(b.prefix), doc_start=None if b.doc is None else i32(b.doc))
    opt.update(kw)
    ws = torch.zeros(max(smla.paged_attention_fp8_workspace_bytes(b.T, b.HK * b.G, b.HK, b.D, len(b.lens), m)
                         for m in (1, b.T, opt.get("max_query_len") or 1)), dtype=torch.uint8, device="cuda")
    out = torch.full((b.T, b.HK * b.G, b.D), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, b.HK * b.G), 77.0, dtype=torch.float32, device="cuda")
    smla.paged_attention_fp8(bf16(b.q) if q is None else q, *(dev(c) for c in b.caches), *(dev(s) for s in b.scales),
                             i32(b.table), i32(b.lens), i32(b.query_start), b.sm_scale, out=out, lse=lse, workspace=ws,
                             **opt)
    torch.cuda.synchronize()
    assert smla.read_device_status(ws) == 0
    return out.float().cpu().numpy(), lse.cpu().numpy()


def check(b, got, expected=None):
    out, lse = got
    want, want_lse, tol, ltol = expected or b.expected()
    mine = ~np.isnan(want_lse[:, 0])
    assert np.all(out[~mine] == 77.0) and np.all(lse[~mine] == 77.0), "rows of no request were written"
    out, lse, want, want_lse, tol, ltol = (x[mine] for x in (out, lse, want, want_lse, tol, ltol))
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(out[empty] == 0)
    err = np.abs(lse[~empty] - want_lse[~empty])
    assert np.all(err <= ltol[~empty]), f"lse off by {err.max():.3g}, allowed {ltol[~empty][err.argmax()]:.3g}"
    over = np.abs(out - want) - tol
    assert np.all(over <= 0), f"{(over > 0).sum()} of {over.size} outputs off, worst by {over.max():.3g} over {tol.flat[over.argmax()]:.3g}"


ATTENTION = [
    # HK, G, D, context, new tokens, options
    (1, 1, 64, [0], [1], {}),
    (1, 1, 128, [0, 63, 64, 65, 126, 127, 128, 129], [1] * 8, {}),
    (2, 4, 128, [1000], [1], {}),
    (3, 5, 64, [5, 700, 0, 64], [1, 1, 1, 1], {}),
    (1, 16, 128, [300, 20, 4000], [1, 1, 1], {}),
    (1, 17, 128, [300, 20], [1, 1], {}),
    (1, 128, 64, [130, 10], [1, 2], {}),
    (1, 128, 128, [130, 10], [1, 2], {}),
    (1, 40, 128, [200, 3], [1, 3], {}),
    (2, 3, 128, [20, 0, 200], [5, 9, 0], {}),
    (2, 8, 128, [0, 500], [70, 40], {}),
    (1, 4, 64, [0, 90], [150, 33], {}),
    (1, 2, 128, [0], [300], {}),
    (2, 1, 64, [260, 0], [200, 129], {}),
    (2, 6, 128, [40], [128], dict(softcap=3.0)),
    (2, 2, 64, [700, 3], [1, 1], dict(softcap=20.0)),
    (1, 8, 128, [900, 900, 2], [1, 4, 1], dict(window=1)),
    (2, 4, 64, [900, 100, 0], [3, 1, 100], dict(window=70)),
    (1, 4, 128, [400, 0], [90, 200], dict(window=64)),
    (2, 3, 64, [400, 10], [1, 2], dict(alibi=True)),
    (1, 12, 128, [100, 0], [60, 90], dict(alibi=True, softcap=10.0)),
    (1, 2, 128, [0, 50, 3], [150, 100, 2], dict(prefix=[100, 150, 0])),
    (2, 2, 64, [0, 130], [60, 3], dict(prefix=[60, 500], window=20, alibi=True)),
    # many segments a CTA, with one and with two filled halves of a query tile, in turn
    (60, 12, 64, [0, 400] * 4, [9, 30, 11, 1, 25, 4, 5, 40], {}),
    (48, 8, 128, [300, 0, 900] * 3, [16, 17, 33, 1, 32, 15, 40, 2, 20], dict(softcap=30.0)),
]


@pytest.mark.parametrize("power", [True, False])
@pytest.mark.parametrize("case", ATTENTION)
def test_attention(smla, case, power):
    HK, G, D, ctx, new, opt = case
    b = ref.Batch(11, HK, G, D, ctx, new, power_scales=power, **opt)
    check(b, attend(smla, b))


@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (20, 64)])
@pytest.mark.parametrize("most", [0, 1, 4, 1000])
def test_attention_whatever_the_estimate(smla, G, D, most):
    """max_query_len only chooses the work split."""
    b = ref.Batch(12, 2, G, D, [70, 0, 300], [1, 40, 7])
    check(b, attend(smla, b, max_query_len=most))


def test_attention_documents_and_empty_rows(smla):
    """Documents that start anywhere; tokens whose document starts behind them see nothing."""
    rng = np.random.default_rng(13)
    for HK, G, D, ctx, new in [(1, 4, 128, [0, 100], [200, 50]), (2, 2, 64, [500, 3], [1, 2]), (1, 1, 128, [0], [1])]:
        doc = []
        for c, n in zip(ctx, new):
            for p in range(c, c + n):
                doc.append(p + 1 if rng.random() < 0.2 else rng.integers(0, p + 1))
        doc[0] = ctx[0] + 5
        b = ref.Batch(14, HK, G, D, ctx, new, doc=doc)
        assert np.isneginf(b.expected()[1]).any()
        check(b, attend(smla, b))


@pytest.mark.parametrize("ctx,new", [([50, 90], [1, 1]), ([10, 0], [90, 40])])
def test_attention_padded_batch(smla, ctx, new):
    """Rows of no request before and behind the batch, a request without new
    tokens, and NaN queries there: left as they were."""
    b = ref.Batch(15, 2, 4, 128, ctx + [33], new + [0], pad=(3, 5))
    b.q[:3], b.q[-5:] = np.nan, np.nan
    check(b, attend(smla, b))


def test_attention_lengths_without_tokens(smla):
    """A request with fewer tokens than new rows: its first rows are at negative positions and see nothing."""
    b = ref.Batch(16, 1, 2, 64, [0, 100], [10, 1])
    b.lens[0] = 4
    check(b, attend(smla, b))
    b.lens[0] = 0
    check(b, attend(smla, b))


@pytest.mark.parametrize("new", [[1, 1], [80, 30]])
def test_attention_bad_pages(smla, new):
    """Keys of blocks outside the cache, or beyond the table, are not seen."""
    b = ref.Batch(17, 2, 4, 128, [400, 300], new)
    b.table[0, 1], b.table[0, 3], b.table[1, 0], b.table[1, 4] = -1, b.NB, -2 ** 31, 2 ** 31 - 1
    check(b, attend(smla, b))
    b.table = b.table[:, :3]
    check(b, attend(smla, b))
    b.table = np.full_like(b.table, -1)
    check(b, attend(smla, b))


def test_attention_large_values(smla):
    """Sharp rows: logits of hundreds, and scales 2^20 apart between K blocks."""
    b = ref.Batch(18, 1, 4, 128, [700, 10], [1, 30], q_size=60.0)
    check(b, attend(smla, b))
    b = ref.Batch(19, 1, 4, 128, [700, 10], [1, 30], q_size=1.0)
    b.scales[0] = b.scales[0] * np.where(np.arange(b.NB) % 2, 2.0 ** -20, 1.0)[:, None].astype(np.float32)
    check(b, attend(smla, b))


def test_attention_many_small_weights(smla):
    """One key far above 20 000 others that together still carry weight."""
    b = ref.Batch(20, 1, 2, 64, [20000], [1], q_size=0.0)
    b.q[:] = 1.0
    for c in b.caches[:1]:
        c[:] = np.where(c == ref.NAN_CODE, c, 0)
    blk, row = b.table[0, 5000 // 64], 5000 % 64
    b.caches[0][blk, 0, row] = ref.e4m3_encode(np.full(64, 120.0))
    b.scales[0][:] = np.float32(10.0 / (64 * 120 * b.sm_scale))
    check(b, attend(smla, b))


@pytest.mark.parametrize("new", [[1, 1], [30, 70]])
def test_attention_any_scales(smla, new):
    """Scales of either sign and of zero."""
    b = ref.Batch(29, 2, 4, 128, [700, 130], new)
    rng = np.random.default_rng(29)
    for s in b.scales:
        s *= rng.choice([-1.0, 1.0, 0.0], s.shape, p=[0.45, 0.45, 0.1]).astype(np.float32)
    check(b, attend(smla, b))


@pytest.mark.parametrize("top,rest", [(0, -13.6), (0, -15.4), (0, -17), (0, -18.3), (16, 0), (100, 84.5), (-5, -21.6),
                                      (-12, -23.4), (-40, -52.3)])
@pytest.mark.parametrize("HK,G,new", [(80, 1, 1), (40, 12, 1), (16, 16, 20)])
def test_attention_equal_small_weights(smla, HK, G, new, top, rest):
    """The newest block's keys weigh 2^top each, the 8000 before them 2^rest:
    rounding may not shift these to one side.  With V = 1 there and 0 in the
    newest block the result is their share of the sum.  Tolerance: weights
    within 2^-7 of their value, equal small ones within 2^-24 of the largest
    on average; in tiles of 256 rows within 2^-25, the sum being at least 2^-3
    (a sum below it is scaled up); the logits, as float32 products of magnitude
    |x|, within 2^-20 |x|; the bf16 result."""
    torch = torch_mod()
    R, D, n = 4, 64, 8000
    MB = n // 64 + 1
    NB = R * MB
    k = torch.full((NB, HK, 64, D), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    v = k.clone()
    table = torch.randperm(NB, device="cuda").to(torch.int32).view(R, MB)
    v[table[:, -1].long()] = 0
    ks = torch.full((NB, HK), rest / D * np.log(2), device="cuda")
    ks[table[:, -1].long()] = top / D * np.log(2)
    vs = torch.ones((NB, HK), device="cuda")
    lens = i32([n + 64] * R)
    out, lse = smla.paged_attention_fp8(
        torch.ones((R * new, HK * G, D), dtype=torch.bfloat16, device="cuda"), k, v, ks, vs, table, lens,
        i32(np.arange(R + 1) * new), 1.0, max_query_len=new, prefix_lens=lens)
    a, b = 64.0, n * 2.0 ** (rest - top)
    want, want_lse = b / (a + b), top * np.log(2) + np.log(a + b)
    dx = 2.0 ** -20 * max(abs(top), abs(rest))
    tol = (2.0 ** -7 + 2.0 ** -8 + 2 * dx) * want + n * 2.0 ** -24 / (a + b) + (n * 2.0 ** -22 if G * new > 48 else 0)
    assert (out.double() - want).abs().max().item() <= tol
    assert (lse.double() - want_lse).abs().max().item() <= dx + 2.0 ** -20 * abs(want_lse)


@pytest.mark.parametrize("HK,G,D,ctx,new,opt", [
    (1, 32, 64, [20, 3], [500, 90], dict(window=100)),
    (1, 128, 128, [0], [100], {}),
    (2, 16, 64, [0, 77], [400, 1], dict(doc=True)),
])
@pytest.mark.parametrize("most", [None, 1])
def test_attention_many_query_tiles(smla, HK, G, D, ctx, new, opt, most):
    """More than 32 query tiles a request, by either kernel."""
    if "doc" in opt:
        opt = dict(doc=[p - p % 90 for c, n in zip(ctx, new) for p in range(c, c + n)])
    b = ref.Batch(25, HK, G, D, ctx, new, **opt)
    check(b, attend(smla, b, max_query_len=most))


@pytest.mark.parametrize("G,new", [(2, [5, 9]), (16, [30, 5])])
def test_attention_fewer_tokens_than_rows(smla, G, new):
    """seq_lens below the number of new rows: the first of them have no position and see nothing."""
    b = ref.Batch(26, 1, G, 64, [0, 0], new)
    b.lens[:] = [3, 0]
    got = attend(smla, b)
    assert np.isneginf(got[1][:new[0] - 3]).all() and np.isneginf(got[1][new[0]:]).all()
    check(b, got)


@pytest.mark.parametrize("most", [1, 1000])
def test_attention_many_requests(smla, most):
    """8192 requests of a few tokens, some with a prefill chunk."""
    rng = np.random.default_rng(27)
    ctx, new = rng.integers(0, 140, 8192), np.where(rng.random(8192) < 0.01, rng.integers(0, 30, 8192), 1)
    b = ref.Batch(28, 1, 2, 64, ctx.tolist(), new.tolist())
    check(b, attend(smla, b, max_query_len=most))


@pytest.mark.parametrize("new", [[1, 1], [70, 1]])
def test_caches_beyond_32_bit_offsets(smla, new):
    """Store and attention in the last blocks of caches of 4.6 GB each."""
    torch = torch_mod()
    HK, G, D, NB = 8, 4, 128, 70000
    T = sum(new)
    k, v, q = (torch.randn((T, n, D), device="cuda").to(torch.bfloat16) for n in (HK, HK, HK * G))
    start = i32(np.cumsum([0] + new))
    got = []
    for first in (0, NB - 4):
        table = i32(first + np.array([[3, 1], [0, 2]]))
        cache = [torch.zeros((NB, HK, 64, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
        scale = [torch.zeros((NB, HK), device="cuda") for _ in range(2)]
        smla.kv_cache_store_fp8(k, v, start, i32(new), table, *cache, *scale)
        out, lse = smla.paged_attention_fp8(q, *cache, *scale, table, i32(new), start, 0.1, max_query_len=max(new))
        got.append([out, lse] + [x[first:first + 4].clone() for x in cache + scale])
        assert not cache[0][:NB - 4].any() or first == 0
        del cache, scale
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][2].any()


def test_graphs_in_turn(smla):
    """A prompt's and a decode step's attention, captured apart and replayed
    in turn and on two streams at once, on inputs that change in between."""
    torch = torch_mod()
    prep = []
    for seed, ctx, new, most in ((60, [30, 0], [90, 120], 120), (61, [900, 40, 3], [1, 1, 1], 1)):
        bs = [ref.Batch(seed + 10 * i, 2, 4, 128, ctx, new) for i in range(2)]
        ins = [[bf16(b.q), *(dev(c) for c in b.caches), *(dev(s) for s in b.scales), i32(b.table)] for b in bs]
        args = [x.clone() for x in ins[0]]
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        rest = (i32(bs[0].lens), i32(bs[0].query_start), bs[0].sm_scale)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = smla.paged_attention_fp8(*args, *rest, max_query_len=most)
        prep.append((bs, ins, args, graph, stream, out, rest))
    for i in (0, 1, 0):
        for bs, ins, args, *_ in prep:
            for a, x in zip(args, ins[i]):
                a.copy_(x)
        torch.cuda.synchronize()
        for _ in range(3):
            for p in prep:
                with torch.cuda.stream(p[4]):
                    p[3].replay()
        torch.cuda.synchronize()
        for bs, _, _, _, _, (out, lse), _ in prep:
            check(bs[i], (out.float().cpu().numpy(), lse.cpu().numpy()))


def test_attention_query_slices(smla):
    torch = torch_mod()
    b = ref.Batch(21, 2, 2, 64, [30, 200], [40, 1])
    fused = torch.full((b.T, 8 * 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = fused[:, 2 * 64:6 * 64].view(b.T, 4, 64)
    q.copy_(bf16(b.q))
    check(b, attend(smla, b, q=q))


def test_attention_nan_query_stays_in_its_row(smla):
    b = ref.Batch(22, 1, 4, 128, [100], [20])
    want = b.expected()
    b.q[3, 2, 5] = np.nan
    out, lse = attend(smla, b)
    assert np.isnan(out[3, 2]).all() and np.isnan(lse[3, 2])
    out[3, 2], lse[3, 2] = want[0][3, 2], want[1][3, 2]
    check(b, (out, lse), want)


@pytest.mark.parametrize("HK,G,new", [(8, 4, 1), (1, 1, 1), (3, 8, 4), (1, 2, 100)])
def test_attention_workspace_contents_do_not_matter(smla, HK, G, new):
    """Few key tiles for many CTAs; a workspace that holds NaN everywhere."""
    torch = torch_mod()
    b = ref.Batch(24, HK, G, 128, [1000, 130], [new, 1])
    n = smla.paged_attention_fp8_workspace_bytes(b.T, HK * G, HK, 128, 2, new)
    out, lse = smla.paged_attention_fp8(
        bf16(b.q), *(dev(c) for c in b.caches), *(dev(s) for s in b.scales), i32(b.table), i32(b.lens),
        i32(b.query_start), b.sm_scale, max_query_len=new,
        workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"))
    check(b, (out.float().cpu().numpy(), lse.cpu().numpy()))


def test_attention_is_deterministic(smla):
    b = ref.Batch(23, 2, 8, 128, [3000, 10, 900], [1, 60, 5])
    first = attend(smla, b)
    for _ in range(3):
        again = attend(smla, b)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


# ---------------------------------------------------------------- a serving step

def serve(smla, steps, table, stack, count, ctx, caches, scales, NB, HK, G, D, outs=None):
    """Each step: tables from lengths, store, attention over what is cached by then."""
    got = []
    for i, (new, q, k, v, T) in enumerate(steps):
        batch = smla.paged_blocks_extend(ctx, new, table, stack, count, T, NB)
        smla.kv_cache_store_fp8(k, v, batch.query_start, batch.seq_lens, table, *caches, *scales)
        out, lse = smla.paged_attention_fp8(q, *caches, *scales, table, batch.seq_lens, batch.query_start, D ** -0.5,
                                            max_query_len=T)
        ctx, count = batch.seq_lens, batch.free_count
        got.append((batch, out, lse))
    return got, ctx, count


def test_serving_steps(smla):
    """Prefill, then decode steps across block borders, then a request ends
    and another takes its blocks; eager, then the same captured and replayed
    on other inputs."""
    torch = torch_mod()
    HK, G, D, NB, MB = 2, 4, 128, 24, 6
    rng = np.random.default_rng(30)
    news = [[100, 3, 0], [1, 1, 1], [1, 62, 0], [30, 1, 5]]
    caches = [np.zeros((NB, HK, 64, D), np.uint8)] * 2
    scales = [np.zeros((NB, HK), np.float32)] * 2
    table, stack = np.full((3, MB), -1, np.int32), rng.permutation(NB).astype(np.int32)
    ctx, count = np.zeros(3, np.int32), NB
    steps, want = [], []
    for new in news:
        T = sum(new) + 2
        q, k, v = (ref.bf16_round(rng.standard_normal((T, n, D))) for n in (HK * G, HK, HK))
        steps.append((i32(new), bf16(q), bf16(k), bf16(v), T))
        table, start, ctx, _, _, slot, count, _ = ref.extend(ctx, new, table, stack, count, T, NB)
        for i, x in enumerate((k, v)):
            caches[i], scales[i] = ref.store(x, start, ctx, table, caches[i], scales[i])
        want.append((slot, ref.attention(q, *caches, *scales, table, ctx, start, D ** -0.5)))

    def state():
        z = lambda s, t: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        return dict(table=torch.full((3, MB), -1, dtype=torch.int32, device="cuda"), stack=i32(stack), count=i32([NB]),
                    ctx=i32([0, 0, 0]), caches=[z((NB, HK, 64, D), torch.uint8) for _ in range(2)],
                    scales=[z((NB, HK), torch.float32) for _ in range(2)], NB=NB, HK=HK, G=G, D=D)

    def compare(got):
        torch.cuda.synchronize()
        for (batch, out, lse), (slot, (o, l, tol, ltol)) in zip(got, want):
            assert np.array_equal(batch.slot_mapping.cpu().numpy(), slot)
            n = int(batch.query_start[-1])
            assert np.all(np.abs(out.float().cpu().numpy()[:n] - o[:n]) <= tol[:n])
            assert np.all(np.abs(lse.cpu().numpy()[:n] - l[:n]) <= ltol[:n])

    s = state()
    got, last, left = serve(smla, steps, **s)
    compare(got)
    assert np.array_equal(s["table"].cpu().numpy(), table) and int(left) == count
    for i in range(2):
        assert np.array_equal(s["caches"][i].cpu().numpy(), caches[i])
        assert np.array_equal(s["scales"][i].cpu().numpy(), scales[i])
    # request 1 ends: its two blocks come back
    gone = dev(np.array([False, True, False]))
    ctx2, left2 = smla.paged_blocks_release(gone, last, s["table"], s["stack"], left, NB)
    assert ctx2.tolist() == [int(ctx[0]), 0, int(ctx[2])] and int(left2) == count + ref.blocks(int(ctx[1]))

    # captured: the same steps from the same start, replayed twice
    s = state()
    first = {k: ([x.clone() for x in v] if isinstance(v, list) else v.clone()) for k, v in s.items() if not isinstance(v, int)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got, last, left = serve(smla, steps, **s)
    for _ in range(2):
        for k, v in first.items():
            for a, b in zip(s[k], v) if isinstance(v, list) else [(s[k], v)]:
                a.copy_(b)
        graph.replay()
        compare(got)


def test_tables_feed_the_latent_cache(smla):
    """The slot map and request ids of paged_blocks_extend with the store and
    the sparse decode over the 656-byte cache: every token attends to its
    request's whole context."""
    import oracle
    torch = torch_mod()
    rng = np.random.default_rng(31)
    NB, MB, H, K = 9, 3, 16, 192
    ctx, new = [0, 0], [130, 70]
    table = torch.full((2, MB), -1, dtype=torch.int32, device="cuda")
    batch = smla.paged_blocks_extend(i32(ctx), i32(new), table, i32(rng.permutation(NB)), i32([NB]), 200, NB)
    rows = ref.bf16_round(rng.standard_normal((200, 576)))
    cache = torch.zeros((NB, 64, 656), dtype=torch.uint8, device="cuda")
    smla.mla_cache_store_fp8(bf16(rows), batch.slot_mapping, cache)
    q = ref.bf16_round(rng.standard_normal((2, H, 576)))
    idx = np.where(np.arange(K)[None] < np.array(new)[:, None], np.arange(K)[None], -1).astype(np.int32)
    out, lse = smla.sparse_mla_decode_fp8(bf16(q), cache, dev(idx), table, i32([0, 1]), 0.05)
    torch.cuda.synchronize()
    bits = (q.view(np.uint32) >> 16).astype(np.uint16)
    want, want_lse = oracle.sparse_mla_decode(bits, cache.cpu().numpy(), idx, table.cpu().numpy(),
                                              np.array([0, 1], np.int32), 0.05)
    assert np.all(np.abs(out.float().cpu().numpy() - want) <= 1e-2 + 2e-2 * np.abs(want))
    assert np.all(np.abs(lse.cpu().numpy() - want_lse) <= 1e-3)


def test_two_streams_at_once(smla):
    """Calls on two streams, each with the workspace that it allocates."""
    torch = torch_mod()
    bs = [ref.Batch(40 + i, 2, 4, 128, [2000, 30], [1, 1]) for i in range(2)]
    ins = [(bf16(b.q), *(dev(c) for c in b.caches), *(dev(s) for s in b.scales), i32(b.table), i32(b.lens),
            i32(b.query_start), b.sm_scale) for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    got = [[] for _ in bs]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(smla.paged_attention_fp8(*ins[i], stream=s))
    torch.cuda.synchronize()
    for i, b in enumerate(bs):
        want = b.expected()
        for out, lse in got[i]:
            check(b, (out.float().cpu().numpy(), lse.cpu().numpy()), want)


def test_python_refusals(smla):
    torch = torch_mod()
    b = ref.Batch(50, 2, 2, 64, [3], [2])
    args = dict(q=bf16(b.q), k_cache=dev(b.caches[0]), v_cache=dev(b.caches[1]), k_scale=dev(b.scales[0]),
                v_scale=dev(b.scales[1]), block_table=i32(b.table), seq_lens=i32(b.lens), query_start=i32(b.query_start),
                sm_scale=0.1)
    bad = [dict(q=args["q"].float()), dict(q=args["q"][:, :, :32]), dict(q=args["q"].transpose(1, 2).contiguous().transpose(1, 2)),
           dict(k_cache=args["k_cache"].view(torch.int8)), dict(k_scale=args["k_scale"].half()),
           dict(v_cache=args["v_cache"][:, :1]), dict(seq_lens=args["seq_lens"].long()),
           dict(query_start=args["query_start"][:-1]), dict(alibi_slopes=torch.zeros(3, device="cuda")),
           dict(doc_start=torch.zeros(9, dtype=torch.int32, device="cuda")), dict(softcap=-1.0), dict(window=-2),
           dict(out=torch.empty((2, 4, 64), device="cuda")), dict(q=args["q"][:, :3]),
           dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(q=args["q"].cpu())]
    for kw in bad:
        with pytest.raises(smla.SmlaError):
            smla.paged_attention_fp8(**{**args, **kw})
