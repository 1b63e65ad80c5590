"""The paged 4-bit cache's operators: what is measured, on which cases, and their plain forms.

A cache holds, for every layer, pages of 64 positions; a page holds one block of bytes per KV head (see `unpack`).
A value is code * scale: a 4-bit code (e2m1: sign, 0 0.5 1 1.5 2 3 4 6) and one scale byte for each 16 neighbouring
channels of one position (5 exponent bits, 3 mantissa bits: the upper byte of an fp16 below its sign bit).

  attend   softmax(scale q k^T) v over a sequence's cached positions: whole canvases, causal chunks, single tokens
  append   K / V rows quantised into a sequence's last positions, and read back as the values they then stand for
  fork     children share a parent's pages; each then grows, which copies its partly filled last page
  compact  live pages move to the lowest places, the tables follow

The book of a cache is one int32 buffer: 16 words of status, the sequences' lengths, the pages' reference counts, the
page tables [n_seq][max_pages] (-1: no page), scratch.
"""
import math
import random

import torch

own = False

PAGE = 64
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ----------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------
def _attend(name, n_seq, rows, length, n_q=16, n_kv=8, dh=128, ragged=False, causal=False, dtype="bf16"):
    return {"name": name, "op": "attend", "n_seq": n_seq, "rows": rows, "length": length, "n_q": n_q, "n_kv": n_kv,
            "dh": dh, "ragged": ragged, "causal": causal, "dtype": dtype}


def _append(name, n_seq, rows, length, n_kv=8, dh=128, ragged=False, dtype="bf16"):
    return {"name": name, "op": "append", "n_seq": n_seq, "rows": rows, "length": length, "n_kv": n_kv, "dh": dh,
            "ragged": ragged, "dtype": dtype}


def _pages(name, op, n_seq, length, layers, n_kv=8, dh=128, share=4):
    return {"name": name, "op": op, "n_seq": n_seq, "length": length, "layers": layers, "n_kv": n_kv, "dh": dh,
            "share": share}


def listed():
    return [
        # one canvas of 256 rows behind a 2048-token prompt: the batch-1 denoising step, where a call's latency counts
        _attend("canvas_1x2304", 1, 256, 2304),
        # eight canvases behind 32768-token prefixes of unequal lengths: the long-context serving step
        _attend("canvas_8x32k", 8, 256, 33024, ragged=True),
        # causal prompt chunks of a small model in fp16, ragged in rows and lengths
        _attend("chunk_5x1500_causal", 5, 256, 1500, n_q=4, n_kv=2, dh=64, ragged=True, causal=True, dtype="fp16"),
        # one token of one short conversation: the smallest call
        _attend("token_1x577", 1, 1, 577, causal=True),
        # one token of one long conversation: few rows, a long axis
        _attend("token_1x32k", 1, 1, 32768, causal=True),
        # one token each of 32 conversations up to 32768 positions
        _attend("token_32x32k", 32, 1, 32768, ragged=True, causal=True),
        # one new token for each of 32 sequences
        _append("append_32x1", 32, 1, 2048, ragged=True),
        # the finished canvases of 32 sequences go into the cache
        _append("append_32x256", 32, 256, 4096),
        # a long prompt goes in at once, at an odd length
        _append("append_1x32767", 1, 32767, 32767),
        # 8 prompts, each forked into 3 more continuations that then grow by a token: 30 layers
        _pages("fork_32x2k", "fork", 32, 2079, 30, share=4),
        # half of a small model's sequences have ended: their pages are given back and the pool closed up
        _pages("compact_16x1k", "compact", 16, 1000, 2, n_kv=2, dh=64),
        # the same for 30 layers of a large one
        _pages("compact_16x2k", "compact", 16, 2048, 30),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("canvas", "canvas", "token", "token", "append", "fork", "compact"))
    dh = rng.choice((64, 128))
    n_kv = rng.choice((2, 4, 8))
    if op in ("canvas", "token"):
        group = rng.choice((1, 2, 4))
        length = _log(rng, 1, 32768)
        rows = rng.choice((256, rng.randint(2, 256))) if op == "canvas" else rng.choice((1, 1, 1, 2, 3))
        n_seq = rng.randint(1, 32 if op == "token" else 8)
        if op == "canvas":  # no dearer than eight canvases of 16 heads behind 32768 positions
            while n_seq > 1 and n_seq * group * n_kv * rows * length * dh > 8 * 16 * 256 * 32768 * 128 // 2:
                n_seq -= 1
        c = _attend("", n_seq, rows, max(length, rows), n_q=group * n_kv, n_kv=n_kv, dh=dh, ragged=rng.random() < 0.6,
                    causal=op == "token" or rng.random() < 0.4, dtype=rng.choice(("bf16", "fp16")))
    elif op == "append":
        rows = _log(rng, 1, 8192)
        n_seq = max(1, min(rng.randint(1, 32), 32768 // rows))
        c = _append("", n_seq, rows, rows + rng.randint(0, 2048), n_kv=n_kv, dh=dh, ragged=rng.random() < 0.6,
                    dtype=rng.choice(("bf16", "fp16")))
    else:
        share = rng.randint(2, 4)
        c = _pages("", op, share * rng.randint(1, 8), _log(rng, 16, 2048), rng.randint(1, 30), n_kv=n_kv, dh=dh,
                   share=share)
    del c["name"]
    return c


def _lens(case):
    """Lengths and row counts of the sequences: part of the case, not of its seed."""
    r = random.Random("%d %d %d" % (case["n_seq"], case["length"], case.get("rows", 0)))
    n, length = case["n_seq"], case["length"]
    rows = [case.get("rows", 0)] * n
    lens = [length] * n
    if case.get("ragged"):
        rows = [r.randint(1, k) for k in rows]
        lens = [max(k, r.randint(max(1, length // 4), length)) for k in rows]
        lens[0], rows[0] = length, case["rows"]
    elif case["op"] == "compact":
        lens = [r.randint(max(1, length // 2), length) for _ in range(n)]
    elif case["op"] == "fork":
        lens = [max(1, length - 7 * i) if i < n // case["share"] else 0 for i in range(n)]
    return lens, rows


# ----------------------------------------------------------------------------------------------------------------
# layout
# ----------------------------------------------------------------------------------------------------------------
def _pad4(n):
    return (n + 3) // 4 * 4


def _sections(n_seq, n_pages, max_pages):
    """Offsets of the lengths, the reference counts, the tables and the scratch in the book, and its size (words)."""
    lens = 16
    refs = lens + _pad4(n_seq)
    table = refs + _pad4(n_pages)
    moves = table + _pad4(n_seq * max_pages)
    return lens, refs, table, moves, moves + 3 * _pad4(n_pages)


def _views(state):
    c = state["shape"]
    lens, refs, table, moves, _ = _sections(c["n_seq"], c["n_pages"], c["max_pages"])
    b = state["book"]
    return (b[lens:lens + c["n_seq"]], b[refs:refs + c["n_pages"]],
            b[table:table + c["n_seq"] * c["max_pages"]].view(c["n_seq"], c["max_pages"]))


def _split(raw, dh):
    """One page's block of a head: codes of K, codes of V, scales of K, scales of V."""
    k, s = PAGE * dh // 2, PAGE * dh // 16
    return raw[..., :k], raw[..., k:2 * k], raw[..., 2 * k:2 * k + s], raw[..., 2 * k + s:]


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), dim=-1)


def unpack(raw, dh):
    """Codes and scale bytes of blocks `raw` uint8 [..., 72 dh] in the order of positions and channels: [..., 64, dh] and
    [..., 64, dh / 16], of K and of V."""
    kc, vc, ks, vs = _split(raw, dh)
    lead = raw.shape[:-1]
    p = len(lead)

    def order(x, shape, axes, to):
        x = x.reshape(lead + shape)
        return x.permute(tuple(range(p)) + tuple(p + a for a in axes)).reshape(lead + to)

    h = dh // 64
    # K: [16-position tile][h][position % 8][t][j][pair of channels][position // 8 % 2][channel % 2];
    # channel = dh/4 t + 16 h + 4 j + 2 pair + nibble
    kc = order(_nibbles(kc), (4, h, 8, 4, 4, 2, 2, 2), (0, 6, 2, 3, 1, 4, 5, 7), (PAGE, dh))
    # V: [16-position tile][h][channel group of dh/8][t][j][upper 8 positions][channel % 2][position % 2];
    # position = 16 tile + 8 upper + 2 t + nibble, channel = dh/8 group + 8 h + 2 j + channel % 2
    vc = order(_nibbles(vc), (4, h, 8, 4, 4, 2, 2, 2), (0, 5, 3, 7, 2, 1, 4, 6), (PAGE, dh))
    # scales of K: [position % 8][t][position // 8][block % h], block = h t + ...; of V: [block][t][tile][upper][nibble]
    ks = order(ks, (8, 4, 8, h), (2, 0, 1, 3), (PAGE, dh // 16))
    vs = order(vs, (dh // 16, 4, 4, 2, 2), (2, 3, 1, 4, 0), (PAGE, dh // 16))
    return kc, ks, vc, vs


def pack(kc, ks, vc, vs, dh):
    """The inverse of `unpack`."""
    lead = kc.shape[:-2]
    p, h = len(lead), dh // 64

    def back(x, shape, axes):
        x = x.reshape(lead + tuple(shape[a] for a in axes))
        inv = [0] * len(axes)
        for i, a in enumerate(axes):
            inv[a] = i
        return x.permute(tuple(range(p)) + tuple(p + a for a in inv)).contiguous()

    def join(x):
        return (x[..., 0] | (x[..., 1] << 4)).reshape(lead + (-1,))

    kc = join(back(kc, (4, h, 8, 4, 4, 2, 2, 2), (0, 6, 2, 3, 1, 4, 5, 7)))
    vc = join(back(vc, (4, h, 8, 4, 4, 2, 2, 2), (0, 5, 3, 7, 2, 1, 4, 6)))
    ks = back(ks, (8, 4, 8, h), (2, 0, 1, 3)).reshape(lead + (-1,))
    vs = back(vs, (dh // 16, 4, 4, 2, 2), (2, 3, 1, 4, 0)).reshape(lead + (-1,))
    return torch.cat((kc, vc, ks, vs), dim=-1)


def quantise(x):
    """Codes uint8 [..., dh] and scale bytes uint8 [..., dh / 16] of rows x, in 32 bits. Every comparison is decided as in
    exact arithmetic: a quotient of such short numbers is either on a border or well off it."""
    b = x.float().reshape(x.shape[:-1] + (-1, 16))
    amax = b.abs().amax(-1)
    a = (amax / 6).clamp(max=10240.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -14))).clamp(min=-14)
    e = torch.where(torch.exp2(e) > a, e - 1, e).clamp(min=-14)   # log2 may round up to the next power
    m = torch.round(a * torch.exp2(3 - e))                        # 0 .. 16 steps of 2^(e - 3), ties to even
    byte = torch.where(a < 2.0 ** -14, m, (e + 15) * 8 + m - 8)
    byte = torch.where(torch.isnan(amax), torch.full_like(byte, 255.0), byte).to(torch.uint8)
    s = (byte.to(torch.int16) << 7).view(torch.float16).float()[..., None]
    y = torch.where(s > 0, b.abs() / s, torch.zeros_like(b))
    code = (y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int()
    code = code + (y > 2.5).int() + (y >= 3.5).int() + (y > 5).int()
    code = (code + 8 * (b < 0).int()).to(torch.uint8)
    return code.reshape(x.shape), byte


def values(code, scale):
    """code * scale in fp32."""
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=code.device)
    s = (scale.to(torch.int16) << 7).view(torch.float16).float()
    v = levels[code.int()].reshape(s.shape + (16,)) * s[..., None]
    return v.reshape(code.shape)


# ----------------------------------------------------------------------------------------------------------------
# what a user's program has in hand
# ----------------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n, n_kv, dh = case["n_seq"], case["n_kv"], case["dh"]
    layers = case.get("layers", 1)
    lens, rows = _lens(case)
    need = [-(-k // PAGE) for k in lens]
    grow = 1 if case["op"] == "fork" else 0
    max_pages = max(need) + grow
    n_pages = sum(need) + (2 * n if grow else 3)
    shape = {"n_seq": n, "n_pages": n_pages, "max_pages": max_pages, "layers": layers, "n_kv": n_kv, "dh": dh}
    book = torch.zeros(_sections(n, n_pages, max_pages)[-1], dtype=torch.int32, device="cuda")
    state = {"case": case, "shape": shape, "book": book}
    lens_v, refs_v, table_v = _views(state)
    # the pages of a cache in use lie in no order
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int64)[:sum(need)]
    table = torch.full((n, max_pages), -1, dtype=torch.int32)
    at, place = 0, order.int().cpu()
    for i, k in enumerate(need):
        table[i, :k] = place[at:at + k]
        at += k
    table_v.copy_(table)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lens_v.copy_(lens_t)
    refs_v[order] = 1
    # what a page held before stays in it: bytes of no meaning, infinite and NaN scales among them
    pool = torch.randint(0, 256, (layers, n_pages, n_kv, 72 * dh), generator=g, device="cuda", dtype=torch.uint8)
    state["pool"] = pool
    if case["op"] in ("attend", "append"):
        for i in range(0, n_pages, 256):  # K and V ~ N(0, 1), quantised; the last page's unused positions keep their bytes
            k, v = (torch.randn((min(256, n_pages - i), n_kv, PAGE, dh), generator=g, device="cuda") for _ in range(2))
            kc, ks = quantise(k)
            vc, vs = quantise(v)
            pool[0, i:i + 256] = pack(kc, ks, vc, vs, dh)
        last = torch.tensor([table[i, k - 1] for i, k in enumerate(need) if k], device="cuda", dtype=torch.int64)
        left = torch.tensor([k % PAGE or PAGE for k in lens if k], device="cuda")
        kc, ks, vc, vs = unpack(pool[0, last], dh)
        behind = (torch.arange(PAGE, device="cuda")[None] >= left[:, None])[:, None, :, None]
        junk = torch.randint(0, 256, vs.shape, generator=g, device="cuda", dtype=torch.uint8)
        pool[0, last] = pack(kc, torch.where(behind, junk, ks), vc, torch.where(behind, junk, vs), dh)
        state["rows"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
    if case["op"] == "attend":
        t = TYPES[case["dtype"]]
        state["q"] = torch.randn((n, case["rows"], case["n_q"], dh), generator=g, device="cuda").to(t)
        state["out"] = torch.zeros_like(state["q"])
        state["lse"] = torch.zeros((n, case["rows"], case["n_q"]), device="cuda")
        state["scale"] = dh ** -0.5
    elif case["op"] == "append":
        t = TYPES[case["dtype"]]
        k, v = (torch.randn((n, case["rows"], n_kv, dh), generator=g, device="cuda") for _ in range(2))
        k[..., 3] *= 8  # a loud channel, as keys have
        state["k"], state["v"] = k.to(t), v.to(t)
        state["k_read"], state["v_read"] = torch.zeros_like(state["k"]), torch.zeros_like(state["v"])
    elif case["op"] == "fork":
        parents = n // case["share"]
        state["src"] = torch.arange(parents, n, device="cuda", dtype=torch.int32) % parents
        state["dst"] = torch.arange(parents, n, device="cuda", dtype=torch.int32)
        state["grow"] = torch.ones(n, dtype=torch.int32, device="cuda")
    else:
        ended = torch.randperm(n, generator=g, device="cuda")[:n // 2]
        state["ended"] = ended.int()
    state["book0"] = book.clone()
    return state


# ----------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    return {"attend": _run_attend, "append": _run_append, "fork": _run_fork, "compact": _run_compact}[op](state)


def _cache(state):
    from block_discrete_diffusion_b200 import dg
    if "cache" not in state:
        c = state["shape"]
        state["cache"] = dg.dg_kv4_cache(c["layers"], c["n_kv"], c["dh"], c["n_pages"], c["n_seq"], c["max_pages"],
                                         pool=state["pool"], book=state["book"])
        if state["case"]["op"] == "attend":
            state["ws"] = torch.empty(dg.dg_kv4_attend_workspace_bytes(state["cache"], state["case"]["n_q"],
                                                                       state["case"]["rows"]),
                                      dtype=torch.uint8, device="cuda")
    return dg, state["cache"]


def _cached(state):
    """The sequences' cached K and V in fp32, [n_seq, n_kv, positions, dh], and which positions exist."""
    lens, _, table = _views(state)
    dh = state["shape"]["dh"]
    raw = state["pool"][0][table.clamp(min=0).int()]                     # [n_seq, pages, n_kv, bytes]
    kc, ks, vc, vs = unpack(raw, dh)
    n, p, h = raw.shape[:3]
    there = torch.arange(p * PAGE, device="cuda")[None] < lens[:, None]
    out = []
    for code, scale in ((kc, ks), (vc, vs)):
        x = values(code, scale).transpose(1, 2).reshape(n, h, p * PAGE, dh)
        out.append(torch.where(there[:, None, :, None], x, torch.zeros((), device="cuda")))
        del x
    return out[0], out[1], there


def _run_attend(state):
    case = state["case"]
    if own:
        dg, cache = _cache(state)
        dg.dg_kv4_attend(cache, 0, state["q"], state["out"], state["ws"], rows=state["rows"], lse=state["lse"],
                         scale=state["scale"], causal=case["causal"])
        return state["out"], state["lse"]
    lens, _, _ = _views(state)
    k, v, there = _cached(state)
    n, rows, n_q, dh = state["q"].shape
    n_kv, keys = k.shape[1], k.shape[2]
    q = state["q"].float().reshape(n, rows, n_kv, n_q // n_kv, dh).permute(0, 2, 3, 1, 4).reshape(n, n_kv, -1, dh)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(state["scale"])
    del k
    seen = there[:, None, :].expand(n, rows, keys)
    if case["causal"]:
        place = lens[:, None] - state["rows"][:, None] + torch.arange(rows, device="cuda")
        seen = seen & (torch.arange(keys, device="cuda") <= place[:, :, None])
    seen = seen[:, None, None].expand(n, n_kv, n_q // n_kv, rows, keys).reshape(n, n_kv, -1, keys)
    s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.log(total) + top
    o = o.reshape(n, n_kv, -1, rows, dh).permute(0, 3, 1, 2, 4).reshape(n, rows, n_q, dh)
    lse = lse.reshape(n, n_kv, -1, rows).permute(0, 3, 1, 2).reshape(n, rows, n_q)
    there = (torch.arange(rows, device="cuda")[None] < state["rows"][:, None])[:, :, None]
    return (torch.where(there[..., None], o.to(state["out"].dtype), state["out"]),
            torch.where(there, lse, state["lse"]))


def _run_append(state):
    if own:
        dg, cache = _cache(state)
        dg.dg_kv4_append(cache, 0, state["k"], state["v"], rows=state["rows"])
        dg.dg_kv4_read(cache, 0, state["k_read"], state["v_read"], rows=state["rows"])
        return state["k_read"], state["v_read"]
    lens, _, table = _views(state)
    n, rows, n_kv, dh = state["k"].shape
    place = (lens - state["rows"])[:, None] + torch.arange(rows, device="cuda")
    there = torch.arange(rows, device="cuda")[None] < state["rows"][:, None]
    p = (place // PAGE).clamp(0, table.shape[1] - 1).long()
    page = torch.gather(table, 1, p.int().long())[there].long()         # [written rows]
    slot = (place % PAGE)[there].long()
    pool = state["pool"][0]
    touched, where = torch.unique(page, return_inverse=True)
    parts = list(unpack(pool[touched], dh))
    new = quantise(state["k"][there]) + quantise(state["v"][there])     # [written rows, n_kv, ...]
    parts[0][where, :, slot], parts[1][where, :, slot] = new[0], new[1]
    parts[2][where, :, slot], parts[3][where, :, slot] = new[2], new[3]
    pool[touched] = pack(*parts, dh)
    kc, ks, vc, vs = unpack(pool[touched], dh)
    state["k_read"][there] = values(kc[where, :, slot], ks[where, :, slot]).to(state["k"].dtype)
    state["v_read"][there] = values(vc[where, :, slot], vs[where, :, slot]).to(state["v"].dtype)
    return state["k_read"], state["v_read"]


def _run_fork(state):
    state["book"].copy_(state["book0"])  # the pass starts from the same sequences every time
    lens, refs, table = _views(state)
    if own:
        dg, cache = _cache(state)
        dg.dg_kv4_fork(cache, state["src"], state["dst"])
        dg.dg_kv4_extend(cache, state["grow"])
        return lens, refs, table, state["pool"]
    src, dst, max_pages = state["src"].long(), state["dst"].long(), table.shape[1]
    table[dst] = table[src]
    lens[dst] = lens[src]
    shared = table[dst].reshape(-1)
    shared = shared[shared >= 0].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    # growth: a copy of a shared, partly filled last page, then new pages, from the lowest free places on
    old, new = lens.long(), (lens + state["grow"]).long()
    last = torch.gather(table, 1, (old // PAGE).clamp(max=max_pages - 1)[:, None])[:, 0].long()
    copy = (state["grow"] > 0) & (old % PAGE > 0) & (refs[last.clamp(min=0)] > 1)
    have = (old + PAGE - 1) // PAGE
    first = have - copy.long()
    where = torch.arange(max_pages, device="cuda")[None]
    fresh = (where >= first[:, None]) & (where < ((new + PAGE - 1) // PAGE)[:, None])
    free = torch.nonzero(refs == 0)[:, 0]
    place = free[:int(fresh.sum())]
    from_ = last[copy]
    table[fresh] = place.int()
    refs[place] = 1
    refs.index_add_(0, from_, torch.full_like(from_, -1, dtype=torch.int32))
    to = torch.gather(table, 1, (have - 1).clamp(min=0)[:, None])[:, 0].long()[copy]
    state["pool"][:, to] = state["pool"][:, from_]
    lens.copy_(new)
    return lens, refs, table, state["pool"]


def _run_compact(state):
    state["book"].copy_(state["book0"])
    lens, refs, table = _views(state)
    if own:
        dg, cache = _cache(state)
        dg.dg_kv4_free(cache, state["ended"])
        dg.dg_kv4_compact(cache)
        return lens, refs, table, state["pool"]
    ended = state["ended"].long()
    gone = table[ended].reshape(-1)
    gone = gone[gone >= 0].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[ended] = -1
    lens[ended] = 0
    live = refs > 0
    n_live = int(live.sum())
    src = torch.nonzero(live[n_live:])[:, 0] + n_live
    dst = torch.nonzero(~live[:n_live])[:, 0]
    state["pool"][:, dst] = state["pool"][:, src]
    now = torch.arange(len(refs), device="cuda", dtype=torch.int32)
    now[src] = dst.int()
    table.copy_(torch.where(table >= 0, now[table.clamp(min=0).long()], table))
    refs[dst] = refs[src]
    refs[src] = 0
    return lens, refs, table, state["pool"]


# ----------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------
def work(case):
    lens, rows = _lens(case)
    n_kv, dh = case["n_kv"], case["dh"]
    value = 0.5625  # bytes of a cached value, its share of the scale included
    if case["op"] == "attend":
        n_q = case["n_q"]
        seen = [sum(max(0, min(k, k - r + j + 1 if case["causal"] else k)) for j in range(r)) for k, r in zip(lens, rows)]
        return {"bytes": 2 * n_kv * dh * value * sum(lens) + sum(rows) * n_q * (4 * dh + 4),
                "flops": 4 * n_q * dh * sum(seen)}
    if case["op"] == "append":  # rows in, 4 bits out and in again, rows out
        return {"bytes": 2 * n_kv * dh * sum(rows) * (2 + value + value + 2), "flops": 0}
    page = 72 * dh * n_kv * case["layers"]
    if case["op"] == "fork":
        parents = case["n_seq"] // case["share"]
        copies = sum(case["share"] for k in lens[:parents] if k % PAGE)
        return {"bytes": 2 * copies * page + 8 * sum(-(-k // PAGE) for k in lens) * case["share"], "flops": 0}
    # half of the sequences' pages are free: half of the live pages lie above the others' end
    live = sum(-(-k // PAGE) for k in lens) / 2
    return {"bytes": 2 * (live / 2) * page + 4 * sum(-(-k // PAGE) for k in lens), "flops": 0}


# ----------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------------
def _exact_block(raw, dh):
    """K and V [64, dh] in 64 bits of blocks `raw` [..., 72 dh], gathered value by value from where each lies."""
    pos = torch.arange(PAGE, device=raw.device)[:, None]
    ch = torch.arange(dh, device=raw.device)[None]
    quarter, h = dh // 4, dh // 64

    def value(byte, upper, scale):
        c = torch.where(upper, raw[..., byte] >> 4, raw[..., byte] & 15).long()
        size = (c & 7).double()
        size = torch.where(size < 2, size / 2, torch.where(size < 4, size / 2, torch.where(size < 6, size - 2, 2 * size - 8)))
        b = raw[..., scale].long()
        e, m = (b >> 3).double(), (b & 7).double()
        s = torch.where(e > 0, (8 + m) * torch.exp2(e - 18), m * torch.exp2(torch.full_like(e, -17)))
        return size * (1 - 2 * (c >> 3).double()) * s

    t, rest = ch // quarter, ch % quarter
    word = ((pos // 16 * h + rest // 16) * 32 + pos % 8 * 4 + t) * 4 + rest % 16 // 4
    byte = 4 * word + 2 * (rest % 4 // 2) + pos // 8 % 2
    scale = PAGE * dh + (pos % 8 * 4 + t) * 8 * h + pos // 8 * h + rest // 16
    k = value(byte, (ch % 2 == 1).expand(PAGE, dh), scale)
    eighth = dh // 8
    t, rest = pos % 8 // 2, ch % eighth
    word = ((pos // 16 * h + rest // 8) * 32 + ch // eighth * 4 + t) * 4 + rest % 8 // 2
    byte = PAGE * dh // 2 + 4 * word + 2 * (pos // 8 % 2) + ch % 2
    scale = PAGE * dh + PAGE * dh // 16 + ((ch // 16 * 4 + t) * 4 + pos // 16) * 4 + 2 * (pos // 8 % 2) + pos % 2
    return k, value(byte, (pos % 2 == 1).expand(PAGE, dh), scale)


def _exact_quantised(x):
    """The values in 64 bits that rows x stand for once they are held in 4 bits: nearest scale, nearest level, ties to even."""
    b = x.double().reshape(x.shape[:-1] + (-1, 16))
    a = b.abs().amax(-1, keepdim=True) / 6
    grid = torch.arange(31 * 8, device=x.device)
    e, m = (grid // 8).double(), (grid % 8).double()
    scales = torch.where(e > 0, (8 + m) * torch.exp2(e - 18), m * 2.0 ** -17)
    scales = scales[scales <= 10240]
    s = scales[_nearest(a, scales)]
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    y = torch.where(s > 0, b.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b))
    v = levels[_nearest(y, levels)] * s
    return torch.where(b < 0, -v, v).reshape(x.shape)


def _nearest(x, grid):
    up = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    low, high = x - grid[up - 1], grid[up] - x
    return torch.where((low < high) | ((low == high) & (up % 2 == 1)), up - 1, up)


def exact(case, seed):
    if case["op"] not in ("attend", "append"):
        return None
    lens, rows = _lens(case)
    state = prepare(case, seed)
    if case["op"] == "append":
        out = []
        for name in ("k", "v"):
            x = torch.zeros(state[name].shape, dtype=torch.float64, device="cuda")
            for i, r in enumerate(rows):
                x[i, :r] = _exact_quantised(state[name][i, :r])
            out.append(x)
        return tuple(out)
    _, _, table = _views(state)
    group = case["n_q"] // case["n_kv"]
    o = torch.zeros(state["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(state["lse"].shape, dtype=torch.float64, device="cuda")
    for i, (length, r) in enumerate(zip(lens, rows)):
        pages = table[i, :-(-length // PAGE)].long()
        for head in range(case["n_kv"]):
            k, v = _exact_block(state["pool"][0, pages, head], case["dh"])
            k, v = k.reshape(-1, case["dh"])[:length], v.reshape(-1, case["dh"])[:length]
            for q in range(head * group, (head + 1) * group):
                s = state["q"][i, :r, q].double() @ k.T * case["dh"] ** -0.5
                if case["causal"]:
                    hidden = torch.arange(length, device="cuda") > (length - r + torch.arange(r, device="cuda"))[:, None]
                    s = s.masked_fill(hidden, -math.inf)
                lse[i, :r, q] = torch.logsumexp(s, -1)
                o[i, :r, q] = torch.softmax(s, -1) @ v
    return o, lse
