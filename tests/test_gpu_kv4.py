"""The paged 4-bit cache on the GPU against the 64-bit reference (kv4_reference.py).

Tolerance of an attention output, counted before the first run: k, v and their products are exact and q is exact in fp16,
so an output carries (a) the rounding of each p to fp16, 2^-11 of it, hence at most 2^-11 sum p |v| / sum p; (b) fp32 sums
of products and the exponential: dh / 16 tensor steps, each off by at most 2^-21 of the sum of magnitudes it met, twice
(two scores meet in a weight), and 2^-21 for exp and log; that is delta = 2 * (dh / 16) * 2^-21 * sum |q k| scale + 2^-21,
as a relative error of p; the sums over positions add 2^-17 at most; (c) partial rows of key splits rounded to fp16,
2^-11 of sum p |v| / sum p; (d) the output's own rounding, eps / 2 of it; (e) below 2^-14 fp16 numbers lie 2^-24 apart,
so a small p is off by up to 2^-25 of the largest p (which is 1, and sum p >= 1), hence the output by 2^-25 sum |v| over
the positions seen, and a small output or partial row in fp16 by 2^-25. lse: delta + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

import kv4_reference as R
from block_discrete_diffusion_b200 import dg

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def device(cuda_ok):
    torch.cuda.set_device(0)


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def make(n_kv, dh, lens, n_layers=1, spare=2, seed=0, max_pages=None):
    """A cache whose sequences have `lens` positions of random bytes, codes and finite scales, in pages in no order; everything
    behind a sequence's end, and every free page, holds NaN and infinite scales."""
    rng = np.random.default_rng(seed)
    need = [-(-n // 64) for n in lens]
    n_pages = sum(need) + spare
    c = dg.dg_kv4_cache(n_layers, n_kv, dh, n_pages, len(lens), max_pages or max(1, max(need)))
    pool = rng.integers(0, 256, (n_layers, n_pages, n_kv, 72 * dh), dtype=np.uint8)
    pool[..., 64 * dh:] = rng.integers(96, 136, pool[..., 64 * dh:].shape)      # scales 2^-3 .. 2^1.8
    order = list(rng.permutation(n_pages))
    table = np.full((len(lens), c.c.max_pages), -1, np.int32)
    for s, k in enumerate(need):
        for i in range(k):
            table[s, i] = order.pop()
    used = set(int(p) for p in table[table >= 0])
    for p in set(range(n_pages)) - used:
        pool[:, p, :, 64 * dh:] = rng.integers(248, 256, pool[:, p, :, 64 * dh:].shape)
    (_, _, ks), (_, _, vs) = R.grids(dh)
    for s, n in enumerate(lens):
        if n % 64:
            for g in (ks, vs):
                stale = np.unique(g[n % 64:])
                pool[:, table[s, n // 64], :, stale] = rng.integers(248, 256, (len(stale), n_layers, n_kv))
    c.pool.copy_(torch.from_numpy(pool.reshape(-1)))
    c.table.copy_(torch.from_numpy(table))
    c.lens.copy_(dev(lens))
    refs = np.zeros(n_pages, np.int32)
    refs[list(used)] = 1
    c.refs.copy_(torch.from_numpy(refs))
    return c


def blocks(c, layer, seq):
    """K, V float64 [n_kv, positions, dh] of a sequence's pages."""
    k = c.c
    pool = c.pool.cpu().numpy().reshape(k.n_layers, k.n_pages, k.n_kv, 72 * k.d_head)
    n = int(c.lens[seq])
    pages = c.table[seq, :-(-n // 64)].cpu().numpy()
    kk, vv = R.read_block(pool[layer, pages], k.d_head)      # [pages, n_kv, 64, dh]
    return (x.transpose(1, 0, 2, 3).reshape(k.n_kv, -1, k.d_head)[:, :n] for x in (kk, vv))


def check(c, layer, q, out, lse, rows, causal, scale, before=None):
    dh = c.c.d_head
    half = torch.finfo(q.dtype).eps / 2
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for s in range(c.c.n_seq):
        n, length = rows[s], int(c.lens[s])
        if before is not None:
            assert torch.equal(out[s, n:], before[s, n:]) and bool((lse[s, n:] == 7).all())
        if n == 0:
            continue
        k, v = blocks(c, layer, s)
        limits = [min(length, max(0, length - n + j + 1)) if causal else length for j in range(n)]
        o, want_lse, absum, reach, vsum = R.attention(q[s, :n].double().cpu().numpy(), k, v, limits, scale)
        delta = 2 * (dh / 16) * 2.0 ** -21 * reach + 2.0 ** -21
        tol = absum * (2 * 2.0 ** -11 + delta[..., None] + 2.0 ** -17) * (1 + half) + half * np.abs(o)
        tol += 2.0 ** -25 * (vsum + 2)
        err = np.abs(got[s, :n] - o)
        assert (err <= tol).all(), (s, float((err / tol).max()))
        seen = np.isfinite(want_lse)
        assert (got_lse[s, :n][~seen] == -np.inf).all()
        d = np.abs(got_lse[s, :n][seen] - want_lse[seen])
        assert (d <= delta[seen] + 2.0 ** -22 * np.abs(want_lse[seen])).all(), (s, float(d.max()))


def attend(c, n_q, T, dtype, rows=None, causal=False, seed=1, layer=0, scale=None, q_scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = c.c
    q = (torch.randn((k.n_seq, T, n_q, k.d_head), generator=g, device="cuda") * q_scale).to(dtype)
    out = torch.full_like(q, 3)
    before = out.clone()
    lse = torch.full((k.n_seq, T, n_q), 7.0, device="cuda")
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, n_q, T), dtype=torch.uint8, device="cuda")
    dg.dg_kv4_attend(c, layer, q, out, ws, rows=None if rows is None else dev(rows), lse=lse, causal=causal, scale=scale)
    assert dg.dg_kv4_error(c) == 0
    check(c, layer, q, out, lse, rows or [T] * k.n_seq, causal, scale or k.d_head ** -0.5, before)
    return q, out, lse


# pages of a sequence's table: as many as it has, or as many as a long context has. It decides how the work is divided and
# with few rows or short tables which form of the attention runs, and nothing else
TABLES = [None, 3000]
LENS = [[1], [0, 5, 64], [63, 64, 65], [127, 128, 129, 200], [700, 1, 257, 0, 513]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("n_q,n_kv,dh,dtype", [(16, 8, 128, BF16), (4, 2, 64, FP16), (4, 4, 128, FP16), (8, 1, 64, BF16)])
def test_single_tokens(lens, n_q, n_kv, dh, dtype):
    attend(make(n_kv, dh, lens), n_q, 1, dtype, causal=True)


@pytest.mark.parametrize("lens", [[1], [63, 64, 65], [700, 1, 257, 0, 513], [9000, 70, 4097], [300] * 40], ids=str)
@pytest.mark.parametrize("n_q,n_kv,dh,dtype", [(16, 8, 128, BF16), (4, 2, 64, FP16), (8, 1, 64, BF16)])
def test_single_tokens_that_may_have_long_contexts(lens, n_q, n_kv, dh, dtype):
    """The same in caches whose sequences may be long: the work is divided along all sequences and its parts are joined."""
    attend(make(n_kv, dh, lens, max_pages=3000), n_q, 1, dtype, causal=True)
    attend(make(n_kv, dh, lens, max_pages=3000), n_q, 2, dtype, rows=[min(2, n + 1) for n in range(len(lens))])


@pytest.mark.parametrize("n_seq", [33, 400])
def test_many_short_sequences(n_seq):
    lens = [(7 * i) % 90 for i in range(n_seq)]
    attend(make(1, 64, lens), 2, 1, FP16, causal=True)
    attend(make(1, 64, lens, max_pages=3000), 2, 1, FP16, causal=True)
    attend(make(1, 64, lens), 2, 9, FP16, causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,T,rows", [
    ([300], 256, None), ([256], 256, None), ([1], 1, None), ([100, 3, 0], 3, [3, 3, 2]), ([500, 129, 64], 130, [130, 65, 1]),
    ([5, 700], 40, [40, 0]), ([64, 128, 192, 320], 64, None), ([1000], 17, None), ([2], 256, None)], ids=str)
@pytest.mark.parametrize("n_q,n_kv,dh,dtype", [(16, 8, 128, BF16), (4, 2, 64, FP16), (3, 1, 128, FP16), (2, 2, 64, BF16)])
@pytest.mark.parametrize("table", TABLES)
def test_rows(lens, T, rows, causal, n_q, n_kv, dh, dtype, table):
    attend(make(n_kv, dh, lens, max_pages=table), n_q, T, dtype, rows=rows, causal=causal)


def test_many_query_heads():
    """More rows of a KV head than a tile has, from one position."""
    attend(make(1, 64, [100, 333], max_pages=3000), 40, 1, BF16)
    attend(make(1, 128, [100, 333]), 300, 1, FP16)
    attend(make(2, 128, [100, 333], max_pages=3000), 300, 3, FP16, causal=True)


@pytest.mark.parametrize("T", [1, 9, 200])
def test_long_ragged_lengths(T):
    attend(make(2, 128, [9000, 70, 4097]), 4, T, BF16, causal=True)


@pytest.mark.parametrize("q_scale,dtype", [(1e-30, BF16), (1e30, BF16), (1e-5, FP16), (500.0, FP16), (0.0, BF16)])
@pytest.mark.parametrize("T,table", [(1, None), (1, 3000), (130, 3000)])
def test_magnitudes_of_q(q_scale, dtype, T, table):
    c = make(1, 128, [200, 3], max_pages=table)
    attend(c, 2, T, dtype, q_scale=q_scale, scale=0.05 / max(q_scale, 1e-3) if q_scale else None)


@pytest.mark.parametrize("T,table", [(1, None), (33, None), (33, 3000)])
def test_strides(T, table):
    c = make(2, 64, [130, 77], max_pages=table)
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((2, T, 4 + 2 + 2, 64), generator=g, device="cuda").to(BF16)       # heads of a packed projection
    q = qkv[:, :, :4]
    wide = torch.full((4, 2, T, 72), 9.0, device="cuda").to(BF16)                       # head-major, padded channels
    out = wide[..., :64].permute(1, 2, 0, 3)
    lse = torch.full((2, T, 4), 7.0, device="cuda")
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 4, T), dtype=torch.uint8, device="cuda")
    dg.dg_kv4_attend(c, 0, q, out, ws, lse=lse, causal=True)
    check(c, 0, q, out, lse, [T, T], True, 0.125)
    assert bool((wide[..., 64:] == 9).all())


def test_pages_beyond_4_gib():
    layers, n_kv, dh = 1, 8, 128
    n_pages = 66000                                                                     # 4.9 GB
    c = dg.dg_kv4_cache(layers, n_kv, dh, n_pages, 1, 3000)
    small = make(n_kv, dh, [150], spare=0, max_pages=3000)
    top = [n_pages - 1, n_pages - 3, n_pages - 2]
    c.pool.view(n_pages, -1)[dev(top, torch.int64)] = small.pool.view(3, -1)[small.table[0, :3].long()]
    c.table[0, :3] = dev(top)
    c.lens[0] = 150
    for T in (1, 140):
        q = torch.randn((1, T, 16, dh), device="cuda").to(BF16)
        outs = []
        for cc in (c, small):
            out = torch.empty_like(q)
            ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(cc, 16, T), dtype=torch.uint8, device="cuda")
            dg.dg_kv4_attend(cc, 0, q, out, ws)
            outs.append(out)
        assert torch.equal(*outs)


@pytest.mark.parametrize("T,table", [(1, None), (40, None), (40, 3000)])
def test_non_finite_values(T, table):
    """A NaN among the cached values reaches the rows that see it; a row of q that is not finite makes its own row NaN only."""
    c = make(2, 64, [100, 100], max_pages=table)
    x = torch.zeros((2, 1, 2, 64), device="cuda").to(BF16)
    x[1, 0, 1, 5] = float("nan")
    dg.dg_kv4_append(c, 0, x, x)
    q = torch.randn((2, T, 4, 64), device="cuda").to(BF16)
    q[0, T - 1, 2, 9] = float("nan")
    out = torch.empty_like(q)
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 4, T), dtype=torch.uint8, device="cuda")
    dg.dg_kv4_attend(c, 0, q, out, ws)
    nan = out.isnan()
    assert bool(nan[1, :, 2:].any(-1).all()) and not bool(nan[1, :, :2].any())
    assert bool(nan[0, T - 1, 2].all()) and int(nan[0].sum()) == 64


# ---------------------------------------------------------------------------------------------
# rows in and out
# ---------------------------------------------------------------------------------------------
def rows_like(n, T, n_kv, dh, dtype, seed, mag):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((2, n, T, n_kv, dh), generator=g, device="cuda")
    if mag == "wide":
        x = x * torch.exp2(torch.randint(-20, 15, (2, n, T, n_kv, dh // 16), generator=g, device="cuda")
                           .float()).repeat_interleave(16, -1)
    elif mag == "ties":       # quotients on the borders of the codes, scales on the borders of their grid
        x = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5], device="cuda")[
            torch.randint(0, 8, x.shape, generator=g, device="cuda")] * x.sign()
        x[..., 0::16] = torch.tensor([6, 6.375, 3.1875, 0.0, 6144], device="cuda")[
            torch.randint(0, 5, x[..., 0::16].shape, generator=g, device="cuda")]
    elif mag == "odd":
        odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 6e4, 0.0, 2.0 ** -24], device="cuda")
        m = torch.rand(x.shape, generator=g, device="cuda") < 0.02
        x = torch.where(m, odd[torch.randint(0, 6, x.shape, generator=g, device="cuda")], x)
    x = x.to(dtype)
    return x[0], x[1]


@pytest.mark.parametrize("mag", ["unit", "wide", "ties", "odd"])
@pytest.mark.parametrize("dh,dtype", [(64, BF16), (64, FP16), (128, BF16), (128, FP16)])
@pytest.mark.parametrize("lens,T,rows", [([1, 64], 1, None), ([130, 65, 7], 66, [66, 1, 0]), ([200], 200, None)], ids=str)
def test_append_and_read(lens, T, rows, dh, dtype, mag):
    n_kv, n = 2, len(lens)
    c = make(n_kv, dh, lens, n_layers=2, seed=4)
    before = c.pool.cpu().numpy().reshape(2, -1, n_kv, 72 * dh)
    k, v = rows_like(n, T, n_kv, dh, dtype, 5, mag)
    want = before.copy()
    counts = rows or [T] * n
    xs = [x.double().cpu().numpy() for x in (k, v)]
    for s in range(n):
        for j in range(counts[s]):
            pos = lens[s] - counts[s] + j
            for h in range(n_kv):
                R.write_row(want[1, int(c.table[s, pos // 64]), h], pos % 64, xs[0][s, j, h], xs[1][s, j, h], dh)
    dg.dg_kv4_append(c, 1, k, v, rows=None if rows is None else dev(rows))
    assert dg.dg_kv4_error(c) == 0
    got = c.pool.cpu().numpy().reshape(2, -1, n_kv, 72 * dh)
    assert np.array_equal(got[0], before[0])
    # the bytes are those of the definition; a code may differ in the sign of a zero, or where its scale is NaN
    wk, wv = R.read_block(want[1], dh)
    gk, gv = R.read_block(got[1], dh)
    np.testing.assert_array_equal(gk, wk)
    np.testing.assert_array_equal(gv, wv)
    np.testing.assert_array_equal(got[1][..., 64 * dh:], want[1][..., 64 * dh:])
    # and read back exactly, into strided rows; those behind a sequence's count stay
    wide = torch.full((2, n, n_kv, T, dh + 8), 5.0, device="cuda").to(dtype)
    k2, v2 = (w[..., :dh].transpose(1, 2) for w in wide)
    dg.dg_kv4_read(c, 1, k2, v2, rows=None if rows is None else dev(rows))
    for s in range(n):
        kk, vv = blocks(c, 1, s)
        for x, ref in ((k2, kk), (v2, vv)):
            np.testing.assert_array_equal(x[s, :counts[s]].double().cpu().numpy(),
                                          ref[:, lens[s] - counts[s]:].transpose(1, 0, 2))
            assert bool((x[s, counts[s]:] == 5).all())
    assert bool((wide[..., dh:] == 5).all())


def test_append_takes_strided_rows():
    c = make(2, 64, [70, 3])
    qkv = torch.randn((2, 3, 8, 64), device="cuda").to(BF16)
    dg.dg_kv4_append(c, 0, qkv[:, :, 4:6], qkv[:, :, 6:])
    a = c.pool.clone()
    dg.dg_kv4_append(c, 0, qkv[:, :, 4:6].contiguous(), qkv[:, :, 6:].contiguous())
    assert torch.equal(a, c.pool)


def test_rows_that_do_not_fit_are_skipped():
    c = make(1, 64, [3, 70, 5])
    before = c.pool.clone()
    x = torch.randn((3, 4, 1, 64), device="cuda").to(BF16)
    dg.dg_kv4_append(c, 0, x, x, rows=dev([4, 0, -1]))      # longer than the sequence; nothing; negative
    assert dg.dg_kv4_error(c) == 8 and dg.dg_kv4_error(c) == 0
    dg.dg_kv4_append(c, 0, x, x, rows=dev([0, 5, 0]))       # more rows than there are
    assert dg.dg_kv4_error(c) == 8
    c.table[1, 1] = 77
    dg.dg_kv4_append(c, 0, x, x, rows=dev([0, 1, 0]))
    assert dg.dg_kv4_error(c) == 5
    c.refs[c.table[0, 0]] = 2
    dg.dg_kv4_append(c, 0, x, x, rows=dev([1, 0, 0]))       # a page with two owners
    assert dg.dg_kv4_error(c) == 5
    assert torch.equal(before, c.pool)
    q = torch.randn((3, 1, 2, 64), device="cuda").to(BF16)
    out = torch.zeros_like(q)
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 2, 1), dtype=torch.uint8, device="cuda")
    dg.dg_kv4_attend(c, 0, q, out, ws)
    assert dg.dg_kv4_error(c) == 5                          # sequence 1 has a page that is none
    c.lens[1] = 1 << 20
    dg.dg_kv4_attend(c, 0, q, out, ws)
    assert dg.dg_kv4_error(c) == 8
    ref = out.clone()
    dg.dg_kv4_attend(c, 0, q, out, ws)                      # the others are right all the same
    assert torch.equal(ref[[0, 2]], out[[0, 2]])


# ---------------------------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------------------------
def same(c, b):
    assert c.lens.tolist() == b.lens and c.refs.tolist() == b.refs and c.table.tolist() == b.table


@pytest.mark.parametrize("seed", range(6))
def test_page_calls_follow_the_rules(seed):
    rng = np.random.default_rng(seed)
    n_seq, n_pages, max_pages = int(rng.integers(2, 40)), int(rng.integers(20, 200)), int(rng.integers(3, 12))
    c = dg.dg_kv4_cache(2, 1, 64, n_pages, n_seq, max_pages)
    b = R.Book(n_seq, n_pages, max_pages)
    c.pool.random_(0, 256)
    content = c.pool.view(2, n_pages, -1).cpu().clone()
    refused = 0
    for _ in range(60):
        op = rng.choice(["extend", "extend", "fork", "free", "compact"])
        moves, code = [], 0
        if op == "extend":
            counts = (rng.integers(0, 100, n_seq) * (rng.random(n_seq) < 0.4)).tolist()
            free = b.refs.count(0)
            dg.dg_kv4_extend(c, dev(counts))
            fits = all(b.lens[s] + n <= max_pages * 64 for s, n in enumerate(counts))
            moves = b.extend(counts)
            code = 0 if moves is not None else 7 if fits else 8
            assert code != 7 or free < n_pages
        elif op == "fork":
            src = rng.integers(0, n_seq, int(rng.integers(1, 4))).tolist()
            dst = rng.permutation(n_seq)[:len(src)].tolist()
            if len(src) > n_seq:
                continue
            dg.dg_kv4_fork(c, dev(src), dev(dst))
            code = 0 if b.fork(src, dst) else 5
        elif op == "free":
            slots = rng.integers(0, n_seq, int(rng.integers(1, min(4, n_seq + 1)))).tolist()
            dg.dg_kv4_free(c, dev(slots))
            code = 0 if b.free(slots) else 5
        else:
            dg.dg_kv4_compact(c)
            moves = b.compact()
        assert dg.dg_kv4_error(c) == code
        refused += code != 0
        same(c, b)
        for a, d in moves or []:
            content[:, d] = content[:, a]
        assert torch.equal(c.pool.view(2, n_pages, -1).cpu(), content)
    assert refused


def test_many_pages():
    c = dg.dg_kv4_cache(1, 1, 64, 30000, 600, 64)
    b = R.Book(600, 30000, 64)
    rng = np.random.default_rng(1)
    counts = rng.integers(0, 64 * 64, 600).tolist()
    dg.dg_kv4_extend(c, dev(counts))
    assert b.extend(counts) == []
    same(c, b)
    gone = rng.permutation(600)[:300].tolist()
    dg.dg_kv4_free(c, dev(gone))
    assert b.free(gone)
    c.pool.view(torch.int32).view(30000, -1)[:] = torch.arange(30000, device="cuda", dtype=torch.int32)[:, None]
    at = c.table[c.table >= 0].clone()
    dg.dg_kv4_compact(c)
    live = c.table >= 0
    assert torch.equal(c.pool.view(torch.int32).view(30000, -1)[c.table[live].long(), 5], at)
    assert int(c.table.max()) + 1 == int(live.sum()) == int((c.refs > 0).sum())
    assert dg.dg_kv4_error(c) == 0


def test_bad_pairs_and_slots_change_nothing():
    c = make(1, 64, [100, 0, 30, 0], spare=3)
    state = c.book.clone()
    for call in (lambda: dg.dg_kv4_fork(c, dev([0]), dev([2])), lambda: dg.dg_kv4_fork(c, dev([0, 0]), dev([1, 1])),
                 lambda: dg.dg_kv4_fork(c, dev([0]), dev([4])), lambda: dg.dg_kv4_fork(c, dev([-1]), dev([1])),
                 lambda: dg.dg_kv4_fork(c, dev([1]), dev([1])), lambda: dg.dg_kv4_fork(c, dev([0, 1]), dev([1, 3])),
                 lambda: dg.dg_kv4_free(c, dev([0, 0])), lambda: dg.dg_kv4_free(c, dev([7]))):
        call()
        assert dg.dg_kv4_error(c) == 5
        assert torch.equal(state[4:], c.book[4:])
    for counts, code in (([0, 0, -1, 0], 8), ([0, 100000, 0, 0], 8), ([28, 0, 98, 1], 0), ([0, 65, 0, 63], 7)):
        dg.dg_kv4_extend(c, dev(counts))
        assert dg.dg_kv4_error(c) == code


# ---------------------------------------------------------------------------------------------
# a run of them
# ---------------------------------------------------------------------------------------------
def test_prompt_forks_and_grows():
    """A prompt goes in, two continuations share it and grow on their own, the prompt's slot is given back, the pool is closed
    up: every step's attention is that of a plain list of the quantised rows."""
    n_kv, dh, n_q, L = 2, 128, 4, 2
    c = dg.dg_kv4_cache(L, n_kv, dh, 12, 3, 5)
    g = torch.Generator(device="cuda").manual_seed(0)
    held = [[], [], []]                                # per sequence: (k, v) float64 [L, n_kv, dh] of every position

    def grow(counts):
        T = max(counts)
        dg.dg_kv4_extend(c, dev(counts))
        x = torch.randn((L, 2, 3, T, n_kv, dh), generator=g, device="cuda").to(BF16)
        for layer in range(L):
            dg.dg_kv4_append(c, layer, x[layer, 0], x[layer, 1], rows=dev(counts))
        code, byte = R.quantise(x.double().cpu().numpy())
        val = R.value(code, byte)
        for s, n in enumerate(counts):
            held[s] += [val[:, :, s, j] for j in range(n)]

    def see(T, causal):
        for layer in range(L):
            rows = [min(T, len(h)) for h in held]
            attend(c, n_q, T, BF16, rows=rows, causal=causal, layer=layer)
            for s in range(3):
                k, v = blocks(c, layer, s)
                for have, i in ((k, 0), (v, 1)):
                    if held[s]:
                        np.testing.assert_array_equal(have, np.stack([h[layer, i] for h in held[s]], 1))

    grow([100, 0, 0])
    see(100, True)
    dg.dg_kv4_fork(c, dev([0, 0]), dev([1, 2]))
    held[1], held[2] = list(held[0]), list(held[0])
    see(1, True)
    for counts in ([0, 1, 0], [1, 1, 1], [0, 40, 7]):
        grow(counts)
        see(1, True)
    dg.dg_kv4_free(c, dev([0]))
    held[0] = []
    dg.dg_kv4_compact(c)
    see(30, False)
    grow([0, 3, 60])
    see(30, True)
    assert dg.dg_kv4_error(c) == 0


def test_captured_step_replays_as_lengths_grow():
    n_kv, dh, n_q = 2, 128, 4
    c = make(n_kv, dh, [62, 130], spare=6, max_pages=4)
    e = make(n_kv, dh, [62, 130], spare=6, max_pages=4)
    ones = dev([1, 1])
    x = torch.randn((2, 1, n_kv, dh), device="cuda").to(BF16)
    q = torch.randn((2, 1, n_q, dh), device="cuda").to(BF16)
    outs = [torch.zeros_like(q), torch.zeros_like(q)]
    ws = [torch.empty(dg.dg_kv4_attend_workspace_bytes(c, n_q, 1), dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(cc, i):
        dg.dg_kv4_extend(cc, ones)
        dg.dg_kv4_append(cc, 0, x, x)
        dg.dg_kv4_attend(cc, 0, q, outs[i], ws[i], causal=True)

    step(e, 1)
    step(e, 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(c, 0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(c, 0)
        graph.replay()
    torch.cuda.current_stream().wait_stream(stream)
    for i in range(5):
        assert torch.equal(outs[0], outs[1]) and torch.equal(c.pool, e.pool) and torch.equal(c.lens, e.lens)
        x.normal_()
        q.normal_()
        step(e, 1)
        graph.replay()
        torch.cuda.synchronize()
    assert dg.dg_kv4_error(c) == 0


def test_side_stream_and_repeats_agree():
    c = make(8, 128, [3000, 77, 1500])
    q = torch.randn((3, 1, 16, 128), device="cuda").to(BF16)
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 16, 1), dtype=torch.uint8, device="cuda")
    out, again = torch.zeros_like(q), torch.zeros_like(q)
    dg.dg_kv4_attend(c, 0, q, out, ws, causal=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dg.dg_kv4_attend(c, 0, q, again, ws, causal=True, stream=s)
    s.synchronize()
    assert torch.equal(out, again)


def test_wrong_tensors_are_refused():
    c = make(2, 64, [5, 6])
    q = torch.zeros((2, 1, 4, 64), device="cuda", dtype=BF16)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for bad in (lambda: dg.dg_kv4_attend(c, 0, q.float(), q, ws), lambda: dg.dg_kv4_attend(c, 0, q, q.half(), ws),
                lambda: dg.dg_kv4_attend(c, 0, q[:1], q[:1], ws), lambda: dg.dg_kv4_attend(c, 0, q, q[:, :, :2], ws),
                lambda: dg.dg_kv4_attend(c, 0, q.cpu(), q, ws), lambda: dg.dg_kv4_attend(c, 0, q, q, ws, rows=dev([1])),
                lambda: dg.dg_kv4_attend(c, 0, q, q, ws, lse=torch.zeros((2, 1, 2), device="cuda")),
                lambda: dg.dg_kv4_attend(c, 0, q.transpose(2, 3), q, ws),
                lambda: dg.dg_kv4_attend(c, 0, q[0], q, ws),
                lambda: dg.dg_kv4_append(c, 0, q, q), lambda: dg.dg_kv4_extend(c, dev([1, 2], torch.int64)),
                lambda: dg.dg_kv4_fork(c, dev([0]), dev([0, 1])), lambda: dg.dg_kv4_cache(1, 1, 64, 4, 1, 4, pool=c.pool)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dg.DGError):
        dg.dg_kv4_attend(c, 0, q, q, ws[:16])
    with pytest.raises(dg.DGError):
        dg.dg_kv4_attend(c, 1, q, q, ws)


@pytest.mark.parametrize("causal", [False, True])
def test_long_lengths_with_few_and_many_rows(causal):
    """Sequences whose rows fill one 128-row tile, two, or part of one, long enough for many steps of each."""
    attend(make(2, 128, [5000, 3001, 4097, 2500]), 4, 256, BF16, rows=[40, 256, 64, 65], causal=causal)
    attend(make(1, 64, [4000, 6000]), 1, 130, FP16, rows=[129, 128], causal=causal)


# ---------------------------------------------------------------------------------------------
# a sequence set's prefixes
# ---------------------------------------------------------------------------------------------
def kv_views(seqs):
    """K [L, n_seq, n_kv, max_ctx, dh] and V transposed [L, n_seq, n_kv, dh, max_ctx] of a set's cache."""
    c, n = seqs.model.cfg, seqs.kv.numel() // 2
    shape = (c.n_layers, seqs.n_seq, c.n_kv)
    return (seqs.kv[:n].view(torch.bfloat16).view(*shape, seqs.max_ctx, c.d_head),
            seqs.kv[n:].view(torch.bfloat16).view(*shape, c.d_head, seqs.max_ctx))


@pytest.mark.parametrize("P", [1, 63, 130, 192])
def test_prefixes_wait_in_four_bits(P):
    """A prompt's prefix goes into the cache, is shared there, and comes back for two sequences of another set: its rows are the
    quantised ones, and a canvas step is the one that the same rows give when they are loaded directly."""
    import synthetic
    cfg = synthetic.TINY
    w = synthetic.make_model_weights(cfg, 0, device="cuda", gain_std=0.1)
    model = dg.dg_model_create(cfg, w)
    one = dg.dg_seqs_create(model, 2, 512)
    ids = synthetic.make_ids(P + 5, cfg.vocab, 1, device="cuda")
    dg.dg_prefill(one, ids, [P, 5])
    c = dg.dg_kv4_cache(cfg.n_layers, cfg.n_kv, cfg.d_head, 12, 3, 4)
    dg.dg_kv4_extend(c, dev([0, P, 0]))
    dg.dg_store_prefix_kv4(one, 0, c, 1)
    dg.dg_kv4_fork(c, dev([1]), dev([2]))
    assert dg.dg_kv4_error(c) == 0
    k, v = kv_views(one)
    rows = []
    for layer in range(cfg.n_layers):
        want = [R.value(*R.quantise(x.double().cpu().numpy())) for x in (k[layer, 0, :, :P],
                                                                        v[layer, 0, :, :, :P].transpose(1, 2).contiguous())]
        for got, x in zip(blocks(c, layer, 1), want):
            np.testing.assert_array_equal(got, x)
        rows.append([torch.tensor(x.transpose(1, 0, 2).copy(), device="cuda").to(torch.bfloat16) for x in want])
    back, direct = dg.dg_seqs_create(model, 2, 512), dg.dg_seqs_create(model, 2, 512)
    for seq, slot in ((0, 1), (1, 2)):
        dg.dg_load_prefix_kv4(back, seq, P, c, slot)
        dg.dg_load_prefix(direct, seq, P, [r[0] for r in rows], [r[1] for r in rows])
    assert dg.dg_kv4_error(c) == 0 and dg.dg_seqs_get_state(back)[0] == [P, P]
    assert torch.equal(back.kv, direct.kv)
    prm = dg.sampler_params(cfg.vocab, seed=3)
    logits = []
    for s in (back, direct):
        out = torch.empty(2 * 256, cfg.vocab, device="cuda")
        cids = torch.empty(512, dtype=torch.int32, device="cuda")
        commit = torch.empty(512, dtype=torch.uint8, device="cuda")
        dg.dg_canvas_init(s, prm, cids, commit)
        dg.dg_canvas_step(s, prm, cids, commit, torch.empty(512, device="cuda"),
                          torch.empty(2, dtype=torch.int32, device="cuda"), logits=out)
        assert dg.dg_device_error(s) == 0
        logits.append(out)
    assert torch.equal(*logits)


def test_prefixes_that_do_not_fit():
    import synthetic
    cfg = synthetic.TINY
    model = dg.dg_model_create(cfg, synthetic.make_model_weights(cfg, 0, device="cuda"))
    s = dg.dg_seqs_create(model, 1, 512)
    dg.dg_prefill(s, synthetic.make_ids(100, cfg.vocab, 1, device="cuda"), [100])
    c = dg.dg_kv4_cache(cfg.n_layers, cfg.n_kv, cfg.d_head, 4, 2, 4)
    dg.dg_kv4_extend(c, dev([99, 0]))
    before, kv = c.pool.clone(), s.kv.clone()
    dg.dg_store_prefix_kv4(s, 0, c, 0)                  # the slot has another length
    assert dg.dg_kv4_error(c) == 8 and torch.equal(before, c.pool)
    dg.dg_load_prefix_kv4(s, 0, 98, c, 0)
    assert dg.dg_kv4_error(c) == 8 and torch.equal(kv, s.kv)
    other = dg.dg_kv4_cache(cfg.n_layers + 1, cfg.n_kv, cfg.d_head, 4, 2, 4)
    short = dg.dg_kv4_cache(cfg.n_layers, cfg.n_kv, cfg.d_head, 4, 2, 1)
    for call in (lambda: dg.dg_store_prefix_kv4(s, 1, c, 0), lambda: dg.dg_store_prefix_kv4(s, 0, c, 2),
                 lambda: dg.dg_load_prefix_kv4(s, 0, 300, c, 0), lambda: dg.dg_load_prefix_kv4(s, 0, -1, c, 0),
                 lambda: dg.dg_store_prefix_kv4(s, 0, other, 0), lambda: dg.dg_load_prefix_kv4(s, 0, 80, short, 0)):
        with pytest.raises(dg.DGError):
            call()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n_q,n_kv,dh,dtype", [(16, 8, 128, BF16), (32, 8, 64, FP16)])
@pytest.mark.parametrize("lens,rows", [([700], None), ([1], None), ([2900], None), ([0, 300], [3, 256]), ([513, 40], [256, 0]),
                                       ([300, 1000, 5, 256, 64, 0, 700, 128], [256, 200, 129, 1, 0, 7, 128, 64])], ids=str)
def test_canvases_in_clusters(lens, rows, causal, n_q, n_kv, dh, dtype):
    """Canvases of one to eight sequences, which are shared out among clusters of six, four, two and single CTAs."""
    attend(make(n_kv, dh, lens), n_q, 256, dtype, rows=rows, causal=causal)


def test_dimensions_of_one_may_have_any_stride():
    c = make(1, 64, [70])
    q = torch.randn((1, 1, 1, 64), device="cuda").to(BF16)
    odd = q.as_strided((1, 1, 1, 64), (3, 5, 7, 1))
    outs = []
    for x in (q, odd):
        out = torch.empty_like(q)
        ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 1, 1), dtype=torch.uint8, device="cuda")
        dg.dg_kv4_attend(c, 0, x, out, ws)
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("T,table", [(1, None), (1, 3000), (256, None), (256, 3000)])
def test_output_over_the_queries(T, table):
    """The rows may be written over the queries that they come from."""
    c = make(8, 128, [900, 77], max_pages=table)
    q = torch.randn((2, T, 16, 128), device="cuda").to(BF16)
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 16, T), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    dg.dg_kv4_attend(c, 0, q, out, ws)
    dg.dg_kv4_attend(c, 0, q, q, ws)
    assert torch.equal(out, q)


@pytest.mark.parametrize("T,n_q,n_kv,dh", [(256, 16, 8, 128), (256, 10, 2, 64), (130, 7, 1, 128), (7, 16, 8, 128), (12, 15, 3, 64)])
@pytest.mark.parametrize("table", [None, 3000])
def test_queries_behind_the_last_row_do_not_matter(T, n_q, n_kv, dh, table):
    """Whatever the queries behind a sequence's last row hold, the rows before them are the same and theirs are left alone."""
    c, rows = make(n_kv, dh, [700, 300], max_pages=table), [T - 3, 2]
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, n_q, T), dtype=torch.uint8, device="cuda")
    q = torch.randn((2, T, n_q, dh), device="cuda").to(BF16)
    outs = []
    for x in (0.0, float("nan"), float("inf")):
        for s, n in enumerate(rows):
            q[s, n:] = x
        out = torch.full_like(q, 7.0)
        dg.dg_kv4_attend(c, 0, q, out, ws, rows=dev(rows))
        outs.append(out)
    for s, n in enumerate(rows):
        assert bool((outs[0][s, n:] == 7).all()) and bool(outs[0][s, :n].isfinite().all())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert dg.dg_kv4_error(c) == 0


@pytest.mark.parametrize("T", [1, 64, 256])
def test_captured_attention_is_repeatable_beside_another_stream(T):
    """Replays of a captured call give the same bits while another cache's calls run on another stream."""
    c, other = make(8, 128, [2000, 130], max_pages=3000), make(8, 128, [4000], seed=9)
    q = torch.randn((2, T, 16, 128), device="cuda").to(BF16)
    q2 = torch.randn((1, T, 16, 128), device="cuda").to(BF16)
    out, first, out2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q2)
    ws, ws2 = (torch.empty(dg.dg_kv4_attend_workspace_bytes(x, 16, T), dtype=torch.uint8, device="cuda") for x in (c, other))
    dg.dg_kv4_attend(c, 0, q, first, ws)
    dg.dg_kv4_attend(other, 0, q2, out2, ws2)
    want2 = out2.clone()
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            dg.dg_kv4_attend(c, 0, q, out, ws)
    for _ in range(20):
        with torch.cuda.stream(s):
            out.zero_()
            graph.replay()
        with torch.cuda.stream(s2):
            out2.zero_()
            dg.dg_kv4_attend(other, 0, q2, out2, ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(out2, want2)
    assert dg.dg_kv4_error(c) == 0 and dg.dg_kv4_error(other) == 0


@pytest.mark.parametrize("T,dh,lens", [(256, 128, [4000]), (256, 128, [3000, 700, 2900, 3000, 64, 2000, 1500, 3000]), (256, 64, [3000]),
                                       (64, 64, [700, 650]), (1, 128, [4000]), (1, 128, [32000]), (4, 128, [3000] * 8)])
def test_attention_is_repeatable_under_load(T, dh, lens):
    """A call gives the same bits beside calls that fill the memory system: its copies of pages come late and close together then,
    and must not meet values that are still being read."""
    c, busy = make(8, dh, lens), make(8, 128, [6000] * 8, seed=9)
    q = torch.randn((len(lens), T, 16, dh), device="cuda").to(BF16)
    out, lse = torch.empty_like(q), torch.empty((len(lens), T, 16), device="cuda")
    loads = []
    for rows in (256, 1):
        x = torch.randn((8, rows, 16, 128), device="cuda").to(BF16)
        loads.append((x, torch.empty_like(x),
                      torch.empty(dg.dg_kv4_attend_workspace_bytes(busy, 16, rows), dtype=torch.uint8, device="cuda")))
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 16, T), dtype=torch.uint8, device="cuda")
    dg.dg_kv4_attend(c, 0, q, out, ws, lse=lse)
    torch.cuda.synchronize()
    want, want_lse = out.clone(), lse.clone()
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(400):
        with torch.cuda.stream(s):
            dg.dg_kv4_attend(busy, 0, *loads[i % 2])
        with torch.cuda.stream(s2):
            out.zero_()
            dg.dg_kv4_attend(c, 0, q, out, ws, lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), i
    assert dg.dg_kv4_error(c) == 0 and dg.dg_kv4_error(busy) == 0
