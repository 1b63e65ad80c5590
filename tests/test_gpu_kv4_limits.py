"""The paged 4-bit cache on the GPU where it can go wrong: ends of the number ranges, calls that are refused on the device,
shares of work without pages.  The reference and the tolerance are those of test_gpu_kv4.py, where nothing else is said."""
import dataclasses

import numpy as np
import pytest
import torch

import kv4_reference as R
import synthetic
from block_discrete_diffusion_b200 import dg
from test_gpu_kv4 import BF16, FP16, attend, blocks, dev, kv_views, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def device(cuda_ok):
    torch.cuda.set_device(0)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[1], [64], [256], [300]], ids=str)
def test_canvas_with_fewer_pages_than_its_cluster_has_ctas(lens, causal):
    """A CTA without pages sends a row of weight 0 through the place of its queries: none of their bits may come with it.
    (Such bf16 queries, read as fp16, are infinities and NaN.)"""
    for seed in range(4):
        c = make(2, 128, lens, seed=seed)
        attend(c, 2, 256, BF16, causal=causal, seed=seed, q_scale=2.0 ** 122, scale=2.0 ** -124)
        attend(c, 2, 256, BF16, rows=[130], causal=causal, seed=seed, q_scale=2.0 ** 122, scale=2.0 ** -124)


@pytest.mark.parametrize("table", [None, 3000])
@pytest.mark.parametrize("n_q,n_kv,dh,dtype", [(4, 2, 128, BF16), (2, 2, 64, FP16)])
def test_whole_prompts(n_q, n_kv, dh, dtype, table):
    """Causal rows for every position, more than a tile has and more of one sequence than of another; and the last rows of it."""
    c = make(n_kv, dh, [1300, 517, 64], max_pages=table)
    attend(c, n_q, 1300, dtype, rows=[1300, 517, 64], causal=True)
    attend(c, n_q, 1300, dtype, rows=[700, 517, 1], causal=True)


# ---------------------------------------------------------------------------------------------
# attention at the ends of the number ranges
# ---------------------------------------------------------------------------------------------
# rows of a call and pages of a table: single tokens and canvases, each in clusters and along the line
FORMS = [(1, None), (1, 3000), (256, None), (256, 3000)]


def cache_of(k, v, table=None):
    """A cache with the rows k, v [positions, n_kv, dh] in one sequence, quantised; free pages before, between and behind."""
    n, n_kv, dh = k.shape
    pages = -(-n // 64)
    c = dg.dg_kv4_cache(1, n_kv, dh, pages + 2, 1, table or pages)
    c.pool.fill_(255)
    dg.dg_kv4_extend(c, dev([n]))
    dg.dg_kv4_append(c, 0, k[None], v[None])
    return c


def run(c, q, scale, rows=None, causal=False):
    T, n_q = q.shape[1:3]
    out, lse = torch.full_like(q, 3), torch.full(q.shape[:3], 7.0, device="cuda")
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, n_q, T), dtype=torch.uint8, device="cuda")
    dg.dg_kv4_attend(c, 0, q, out, ws, rows=rows, lse=lse, scale=scale, causal=causal)
    assert dg.dg_kv4_error(c) == 0
    return out, lse


def check_tails(c, q, out, lse, scale):
    """As check of test_gpu_kv4.py, with less room below: a weight is kept to 2^-32 of the row's largest, a joined part to 2^-39 of
    its row's largest magnitude."""
    dh, n = c.c.d_head, int(c.lens[0])
    half = torch.finfo(q.dtype).eps / 2
    k, v = blocks(c, 0, 0)
    o, want_lse, absum, reach, vsum = R.attention(q[0].double().cpu().numpy(), k, v, [n] * q.shape[1], scale)
    delta = 2 * (dh / 16) * 2.0 ** -21 * reach + 2.0 ** -21
    tol = absum * (2 * 2.0 ** -11 + delta[..., None] + 2.0 ** -17) * (1 + half) + half * np.abs(o) + 2.0 ** -32 * vsum
    tol += 2.0 ** -39 * absum.max(-1, keepdims=True)
    if q.dtype == FP16:
        tol += 2.0 ** -25              # steps of a small output
    err = np.abs(out[0].double().cpu().numpy() - o)
    assert (err <= tol).all(), float((err / tol).max())
    d = np.abs(lse[0].double().cpu().numpy() - want_lse)
    assert (d <= delta + 2.0 ** -22 * np.abs(want_lse)).all(), float(d.max())


@pytest.mark.parametrize("T,table", FORMS)
@pytest.mark.parametrize("dh,dtype", [(64, FP16), (128, BF16)])
@pytest.mark.parametrize("gap", [15.0, 20.0, 24.5, 25.5, 28.0])
@pytest.mark.parametrize("at", [0, 300, 699])
def test_a_long_tail_behind_one_dominant_key(T, table, dh, dtype, gap, at):
    """One position's weight is 2^gap of each other's, and its value is zero: the output is the tail's."""
    g = torch.Generator(device="cuda").manual_seed(int(gap))
    k, v = torch.zeros((700, 2, dh), device="cuda"), torch.rand((700, 2, dh), generator=g, device="cuda") * 5e4
    k[at, :, 0], v[at] = 6, 0
    q = torch.zeros((1, T, 4, dh), device="cuda").to(dtype)
    q[..., 0] = 1
    scale = float(np.float32(gap * np.log(2) / 6))
    c = cache_of(k.to(dtype), v.to(dtype), table)
    check_tails(c, q, *run(c, q, scale), scale)


@pytest.mark.parametrize("T,table", FORMS + [(200, None), (200, 3000)])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("power", [-40, -17, -14, -8, 13, "blocks"])
def test_values_of_any_magnitude(T, table, dh, power):
    """Outputs in bf16 keep their bits whatever the values' magnitude is, also where rows are joined from parts; values of one row
    whose blocks of channels are of different magnitudes too."""
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn((900, 2, dh), generator=g, device="cuda") for _ in range(2))
    if power == "blocks":
        v *= torch.exp2(torch.arange(dh // 16, device="cuda") % 5 * 4.0 - 12).repeat_interleave(16)
    else:
        v *= 2.0 ** power
    q = torch.randn((1, T, 4, dh), generator=g, device="cuda").to(BF16)
    c = cache_of(k.to(BF16), v.to(BF16), table)
    scale = float(np.float32(dh ** -0.5))
    check_tails(c, q, *run(c, q, scale), scale)


@pytest.mark.parametrize("T,table", FORMS)
@pytest.mark.parametrize("dh,dtype", [(64, FP16), (128, BF16)])
@pytest.mark.parametrize("power", [10, 17, 18, 20, 22, 24, 26, 27, 28, 30, 40, 100])
def test_scores_beyond_their_own_accuracy(T, table, dh, dtype, power):
    """Scores near 2^power, where fp32 numbers lie far apart, and further apart than they do: the largest one's value comes out, and
    rows beside it whose scores are small are what they are without it."""
    g = torch.Generator(device="cuda").manual_seed(power)
    n = 500
    k = torch.randint(-4, 5, (n, 2, dh), generator=g, device="cuda").float()
    v = torch.randn((n, 2, dh), generator=g, device="cuda")
    best, worst = 77, 401                       # 6 in channel 0, and -6; others are at most 4
    k[best, :, 0], k[worst, :, 0] = 6, -6
    c = cache_of(k.to(dtype), v.to(dtype), table)
    q = torch.zeros((1, T, 4, dh), device="cuda").to(dtype)
    up = 2.0 ** (power - 4)
    # heads 0 and 2 have large scores, 1 small ones beside those of 0, 3 none
    if dtype == BF16:
        q[..., 0, 0], q[..., 2, 0], q[..., 1, 0], scale = up, -up, 2.0 ** -3, 1.0
    else:
        q[..., 0, 0], q[..., 2, 0], q[..., 1, 0], scale = 2.0 ** 5, -2.0 ** 5, 2.0 ** -24, up / 2 ** 5
    out, lse = run(c, q, scale)
    _, vv = blocks(c, 0, 0)
    # The weight is rounded to fp16, by 2^-11, and the sum is not. A value has 6 bits, and a bf16 output's 8 are not reached by
    # that rounding (and a joined part's, 2^-11 too); an fp16 output is off by it and its own
    room = 0 if dtype == BF16 else 2.0 ** -10
    for h, pos in ((0, best), (2, worst)):
        want = np.broadcast_to(vv[h // 2, pos], (T, dh))
        assert (np.abs(out[0, :, h].double().cpu().numpy() - want) <= room * np.abs(want)).all()
        assert bool(((lse[0, :, h].double() - 6 * up).abs() <= 2.0 ** -22 * 6 * up).all())
    if dtype == BF16 or power <= 20:
        small = q.clone()
        small[..., 0::2, :] = 0
        alone, alone_lse = run(c, small, scale)
        check_tails(c, small, alone, alone_lse, scale)
        # (each is off by the tolerances above at most: a step of the output, and P's rounding of values up to 6)
        x, y = out[..., 1::2, :].float(), alone[..., 1::2, :].float()
        assert bool(((x - y).abs() <= torch.finfo(dtype).eps * y.abs() + 2 * 6 * 2.0 ** -11).all())


@pytest.mark.parametrize("dh,dtype", [(64, FP16), (128, BF16)])
@pytest.mark.parametrize("n_pages", [3, 300])
def test_rows_move_whole_or_not_at_all(dh, dtype, n_pages):
    """One page of several that has another owner, or is none, keeps all rows of its sequence where they are, in and out; the
    other sequences' rows move."""
    lens = [64 * n_pages - 10, 70, 64 * n_pages]
    T = 64 * n_pages - 30
    c = make(2, dh, lens, n_layers=2)
    rows = dev([T, 70, T])
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn((3, T, 2, dh), generator=g, device="cuda").to(dtype) for _ in range(2))
    table, refs, pool = c.table.clone(), c.refs.clone(), c.pool.clone()
    whole = c.pool.view(2, -1, 2 * 72 * dh)
    for at in (0, n_pages // 2, n_pages - 1):
        for kind in ("shared", "missing", "negative"):
            if kind == "shared":
                c.refs[table[0, at]] = 2
            else:
                c.table[0, at] = c.c.n_pages if kind == "missing" else -1
            c.pool.copy_(pool)
            dg.dg_kv4_append(c, 1, k, v, rows=rows)
            assert dg.dg_kv4_error(c) == 5
            mine = table[0, :n_pages].long()
            before = pool.view(2, -1, 2 * 72 * dh)
            assert torch.equal(whole[:, mine], before[:, mine]) and torch.equal(whole[0], before[0])
            c.refs.copy_(refs)
            c.pool.copy_(pool)
            dg.dg_kv4_append(c, 1, k, v, rows=rows * dev([0, 1, 1]))
            assert dg.dg_kv4_error(c) == 0
            want = c.pool.clone()
            c.pool.copy_(pool)
            if kind == "shared":
                c.refs[table[0, at]] = 2
            dg.dg_kv4_append(c, 1, k, v, rows=rows)     # the others' rows are those of a call without the first
            assert dg.dg_kv4_error(c) == 5 and torch.equal(want, c.pool)
            k2, v2 = torch.full_like(k, 3), torch.full_like(v, 3)
            dg.dg_kv4_read(c, 1, k2, v2, rows=rows)
            kk, vv = (x[2, :T] for x in (k2, v2))
            assert not bool((kk == 3).all()) and not bool((vv == 3).all())
            if kind == "shared":                        # (a shared page may be read)
                assert dg.dg_kv4_error(c) == 0 and not bool((k2[0] == 3).all())
            else:
                assert dg.dg_kv4_error(c) == 5 and bool((k2[0] == 3).all()) and bool((v2[0] == 3).all())
            c.table.copy_(table)
            c.refs.copy_(refs)


@pytest.mark.parametrize("page", [-1, 99])
def test_growth_behind_a_page_that_is_none(page):
    """The last page's table entry is out of range: nothing grows, and the code is that of an index (a count that does not fit, of
    another sequence, comes before it)."""
    c = make(1, 64, [70, 5, 64])
    c.table[0, 1] = page
    book, pool = c.book.clone(), c.pool.clone()
    for counts, code in (([1, 0, 0], 5), ([1, 2, 0], 5), ([1, -1, 0], 8), ([1, 0, 1 << 20], 8)):
        dg.dg_kv4_extend(c, dev(counts))
        assert dg.dg_kv4_error(c) == code
        assert torch.equal(c.book[16:], book[16:]) and torch.equal(c.pool, pool)
    dg.dg_kv4_extend(c, dev([0, 2, 0]))                 # what does not grow is not looked at
    assert dg.dg_kv4_error(c) == 0 and c.lens.tolist() == [70, 7, 64]


def test_expanded_outputs_are_refused():
    c = make(2, 64, [5, 6])
    x = torch.zeros((2, 3, 2, 64), device="cuda").to(BF16)
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 2, 3), dtype=torch.uint8, device="cuda")
    for wide in (x[:1].expand(2, 3, 2, 64), x[:, :1].expand(2, 3, 2, 64), x[:, :, :1].expand(2, 3, 2, 64)):
        for call in (lambda: dg.dg_kv4_attend(c, 0, x, wide, ws), lambda: dg.dg_kv4_read(c, 0, wide, x.clone()),
                     lambda: dg.dg_kv4_read(c, 0, x.clone(), wide)):
            with pytest.raises(dg.DGError):
                call()
        dg.dg_kv4_append(c, 0, wide, x)                 # what is read may be broadcast
        a = c.pool.clone()
        dg.dg_kv4_append(c, 0, wide.contiguous(), x)
        assert torch.equal(a, c.pool)


def test_both_kinds_of_error_are_told():
    """A wait that ran out and a count that does not fit, both recorded (here by hand): neither hides the other."""
    c = make(1, 64, [3])
    x = torch.zeros((1, 4, 1, 64), device="cuda").to(BF16)
    c.book[3] = 4
    dg.dg_kv4_append(c, 0, x, x)                        # four rows of three positions
    assert [dg.dg_kv4_error(c) for _ in range(3)] == [4, 8, 0]
    dg.dg_kv4_append(c, 0, x, x)
    c.book[3] = 4
    assert [dg.dg_kv4_error(c) for _ in range(3)] == [4, 8, 0]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,table", FORMS)
@pytest.mark.parametrize("page", [-1, 99])
@pytest.mark.parametrize("at", [0, 3, 10])
def test_rows_that_would_read_a_page_that_is_none_are_nan(T, table, dtype, page, at):
    """... beside other sequences' rows, which are what they are without it, and rows that end before it."""
    c = make(2, 128, [700, 700, 300], max_pages=table)
    q = torch.randn((3, T, 4, 128), device="cuda").to(dtype)
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 4, T), dtype=torch.uint8, device="cuda")
    outs = []
    for bad in (False, True):
        if bad:
            c.table[1, at] = page
        out, lse = torch.full_like(q, 3), torch.full(q.shape[:3], 7.0, device="cuda")
        dg.dg_kv4_attend(c, 0, q, out, ws, lse=lse)
        assert dg.dg_kv4_error(c) == (5 if bad else 0)
        outs.append((out, lse))
    for x, y in zip(*outs):
        assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2]) and bool(x.isfinite().all())
        assert bool(y[1].isnan().all())
    c.lens[1] = 64 * at                                 # a sequence that ends before that entry does not read it
    dg.dg_kv4_attend(c, 0, q, outs[0][0], ws)
    assert dg.dg_kv4_error(c) == 0 and bool(outs[0][0].isfinite().all())


@pytest.mark.parametrize("T,table", FORMS)
def test_calls_after_a_wait_ran_out(T, table):
    """Once the book says so (here by hand), waits that do not end at once are given up. The calls come to their end all the same,
    the code is told once, and the calls behind that are right."""
    c = make(8, 128, [3000, 700], max_pages=table)
    q = torch.randn((2, T, 16, 128), device="cuda").to(BF16)
    out, want = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(dg.dg_kv4_attend_workspace_bytes(c, 16, T), dtype=torch.uint8, device="cuda")
    dg.dg_kv4_attend(c, 0, q, want, ws)
    for _ in range(3):
        c.book[3] = 4
        for _ in range(5):
            dg.dg_kv4_attend(c, 0, q, out, ws)
        assert dg.dg_kv4_error(c) == 4 and dg.dg_kv4_error(c) == 0
        dg.dg_kv4_attend(c, 0, q, out, ws)
        assert dg.dg_kv4_error(c) == 0 and torch.equal(out, want)


# ---------------------------------------------------------------------------------------------
# a sequence set's prefixes
# ---------------------------------------------------------------------------------------------
def step_logits(s, cfg):
    """The logits of a canvas step behind the set's prefixes."""
    n, prm = s.n_seq * 256, dg.sampler_params(cfg.vocab, seed=3)
    out = torch.empty(n, cfg.vocab, device="cuda")
    ids, commit = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
    dg.dg_canvas_init(s, prm, ids, commit)
    dg.dg_canvas_step(s, prm, ids, commit, torch.empty(n, device="cuda"),
                      torch.empty(s.n_seq, dtype=torch.int32, device="cuda"), logits=out)
    return out


def test_a_refused_load_leaves_the_sequence_as_it_was():
    """A slot of another length, an empty one, one with a page that is none: neither the rows nor the length change, the steps
    go on behind the old prefix, and both objects tell."""
    cfg = synthetic.TINY
    model = dg.dg_model_create(cfg, synthetic.make_model_weights(cfg, 0, device="cuda"))
    s = dg.dg_seqs_create(model, 2, 512)
    dg.dg_prefill(s, synthetic.make_ids(107, cfg.vocab, 1, device="cuda"), [100, 7])
    c = dg.dg_kv4_cache(cfg.n_layers, cfg.n_kv, cfg.d_head, 6, 3, 4)
    dg.dg_kv4_extend(c, dev([99, 0, 130]))
    c.table[2, 1] = 6
    want = step_logits(s, cfg)
    kv, pool = s.kv.clone(), c.pool.clone()
    for P, slot, code in ((98, 0, 8), (100, 0, 8), (0, 0, 8), (64, 1, 8), (130, 2, 5)):
        dg.dg_load_prefix_kv4(s, 0, P, c, slot)
        assert dg.dg_seqs_get_state(s)[0] == [100, 7] and torch.equal(kv, s.kv)
        assert dg.dg_kv4_error(c) == code and dg.dg_kv4_error(c) == 0
        assert dg.dg_device_error(s) == code and dg.dg_device_error(s) == 0
    assert torch.equal(want, step_logits(s, cfg)) and dg.dg_device_error(s) == 0
    dg.dg_load_prefix_kv4(s, 0, 0, c, 1)                # a prefix without rows is one
    assert dg.dg_seqs_get_state(s)[0] == [0, 7]
    dg.dg_store_prefix_kv4(s, 0, c, 1)
    assert dg.dg_kv4_error(c) == 0 and dg.dg_device_error(s) == 0
    dg.dg_store_prefix_kv4(s, 0, c, 0)                  # ... that slot 0 does not hold
    assert dg.dg_kv4_error(c) == 8 and torch.equal(pool, c.pool)


@pytest.mark.parametrize("P", [1, 65, 1001, 4096])
@pytest.mark.parametrize("dh", [64, 128])
def test_prefixes_of_both_head_sizes_from_any_sequence(dh, P):
    """Prefixes of unequal lengths wait in the cache and come back to other sequences: their rows are the quantised ones, and what
    lies behind them is left alone."""
    cfg = dataclasses.replace(synthetic.TINY, d_head=dh)
    model = dg.dg_model_create(cfg, synthetic.make_model_weights(cfg, 0, device="cuda"))
    s, back = dg.dg_seqs_create(model, 3, 4608), dg.dg_seqs_create(model, 3, 4608)
    g = torch.Generator(device="cuda").manual_seed(P)
    lens = [P // 2 + 1, P, 200]
    for i, n in enumerate(lens):
        x = torch.randn((2, cfg.n_layers, n, cfg.n_kv, dh), generator=g, device="cuda").to(BF16)
        dg.dg_load_prefix(s, i, n, list(x[0]), list(x[1]))
    c = dg.dg_kv4_cache(cfg.n_layers, cfg.n_kv, dh, 150, 3, 64)
    dg.dg_kv4_extend(c, dev(lens[::-1]))
    back.kv.view(BF16).fill_(3)
    for i in range(3):
        dg.dg_store_prefix_kv4(s, i, c, 2 - i)
        dg.dg_load_prefix_kv4(back, (i + 1) % 3, lens[i], c, 2 - i)
    assert dg.dg_kv4_error(c) == 0 and dg.dg_seqs_get_state(back)[0] == [lens[2], lens[0], lens[1]]
    (k, v), (bk, bv) = kv_views(s), kv_views(back)
    for i, n in enumerate(lens):
        at = (i + 1) % 3
        for layer in range(cfg.n_layers):
            for x, got, held in zip((k[layer, i, :, :n], v[layer, i, :, :, :n].transpose(1, 2)),
                                    (bk[layer, at, :, :n], bv[layer, at, :, :, :n].transpose(1, 2)), blocks(c, layer, 2 - i)):
                want = R.value(*R.quantise(x.double().cpu().numpy()))
                np.testing.assert_array_equal(held, want)
                np.testing.assert_array_equal(got.double().cpu().numpy(), want)
        assert bool((bk[:, at, :, n:] == 3).all()) and bool((bv[:, at, :, :, n:] == 3).all())


def test_a_store_onto_shared_pages_changes_nothing():
    cfg = synthetic.TINY
    model = dg.dg_model_create(cfg, synthetic.make_model_weights(cfg, 0, device="cuda"))
    s = dg.dg_seqs_create(model, 1, 512)
    x = torch.randn((2, cfg.n_layers, 200, cfg.n_kv, cfg.d_head), device="cuda").to(BF16)
    dg.dg_load_prefix(s, 0, 200, list(x[0]), list(x[1]))
    c = dg.dg_kv4_cache(cfg.n_layers, cfg.n_kv, cfg.d_head, 8, 2, 4)
    dg.dg_kv4_extend(c, dev([100, 0]))
    dg.dg_kv4_fork(c, dev([0]), dev([1]))
    dg.dg_kv4_extend(c, dev([100, 0]))                  # its first page is still the other's too
    c.pool.random_(0, 256)
    before = c.pool.clone()
    dg.dg_store_prefix_kv4(s, 0, c, 0)
    assert dg.dg_kv4_error(c) == 5 and torch.equal(before, c.pool)
