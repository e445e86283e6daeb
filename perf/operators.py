"""Measured cases of the paged 8-bit key/value cache: attention over it (dense and over selected keys), appending
to it, and the operations on its pages.

The cache holds FP8 e4m3 codes `k`, `v` [pages, kv_heads, page_size, head_dim] with one UE8M0 exponent byte per page
and head (`k_exps`, `v_exps` [pages, kv_heads], value 2^(e - 127)).  Sequence s holds positions [0, seq_lens[s]) in
the pages page_table[s, 0 .. ceil(len / page_size)).  The rows of a call belong to sequences by `row_starts`; the n
rows of a sequence are its last n positions.
"""
import math
import random

import torch

own = False  # false: the plain forms below; true: the framework's own operators

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------- cases
def listed():
    a = {"op": "attention", "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16", "select": 0, "mix": 1}
    return [
        # one user's next token over a short conversation: latency alone
        dict(a, name="decode_1x777", seqs=1, rows=1, length=777),
        # a serving batch of single tokens, contexts from a few thousand to 64K tokens: the cache is read once
        dict(a, name="decode_32x64k_ragged", seqs=32, rows=1, length=65536),
        # verifying five drafted tokens per sequence of a smaller model: odd lengths, half precision, head size 64
        dict(a, name="verify_16x5_fp16_d64", seqs=16, rows=5, length=8191, heads=16, kv_heads=4, dim=64, page=32,
             dtype="fp16"),
        # a 2,048-token chunk of a long prompt whose first 30K tokens are cached
        dict(a, name="prefill_2048_of_32k", seqs=1, rows=2048, length=32768),
        # several prompts of different, odd lengths prefilled from their first token
        dict(a, name="prefill_ragged_5x1531", seqs=5, rows=1531, length=1531, heads=16, kv_heads=2, page=16, mix=5),
        # single tokens that read the 2,048 keys the indexer chose from 64K-token contexts
        dict(a, name="select_decode_32x2048", seqs=32, rows=1, length=65536, select=2048),
        # a prompt chunk whose rows each read their own 512 chosen keys; 32 query heads share two key heads
        dict(a, name="select_prefill_1023x512", seqs=3, rows=1023, length=32768, kv_heads=2, select=512, mix=3),
        # writing a prompt batch's keys and values into the cache
        dict(op="append", name="append_prefill_4x4000", seqs=4, rows=4000, length=9000, kv_heads=8, dim=128, page=64,
             dtype="bf16", mix=2),
        # one new token for each of 128 sequences: partly filled blocks whose scale may have to grow
        dict(op="append", name="append_decode_128", seqs=128, rows=1, length=1500, kv_heads=8, dim=128, page=64,
             dtype="bf16", mix=4),
        # 48 samples forked from 4 prompts: whole pages shared, the last partial page copied
        dict(op="fork", name="fork_48", pages=8192, seqs=64, length=6000, count=48, kv_heads=8, dim=128, page=64, mix=6),
        # finished requests give their pages back
        dict(op="free", name="free_200", pages=65536, seqs=512, length=1500, count=200, kv_heads=2, dim=64, page=16,
             mix=7),
        # a half-empty pool packed to its front
        dict(op="compact", name="compact_16k_pages", pages=16384, seqs=96, length=8000, count=40, kv_heads=8, dim=128,
             page=64, mix=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "select", "select", "append", "append", "fork", "free",
                     "compact", "copy", "reserve"))
    mix = rng.randrange(1, 1 << 20)
    page = rng.choice((16, 32, 64, 128))
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    if op in ("attention", "select"):
        group = rng.choice((1, 2, 4, 5, 8, 16, 32) if kv_heads <= 2 else (1, 3, 4, 7, 8))
        dtype = rng.choice(("bf16", "bf16", "fp16"))
        base = dict(op="attention", heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, mix=mix)
        if op == "select":
            rows = _log(rng, 1, 512)
            seqs = rng.randrange(1, 5) if rows > 16 else rng.randrange(1, 33)
            return dict(base, seqs=seqs, rows=rows, length=_log(rng, max(rows, 1000), 65536),
                        select=rng.choice((512, 1024, 2048)))
        if rng.random() < 0.5:  # single tokens and short runs of them
            return dict(base, seqs=_log(rng, 1, 48), rows=rng.randrange(1, 9), length=_log(rng, 8, 32768), select=0)
        seqs, length = rng.randrange(1, 4), _log(rng, 64, 16384)  # prompts and their chunks
        rows = min(length, 2048, (1 << 31) // (seqs * length * kv_heads * group))
        return dict(base, seqs=seqs, rows=_log(rng, 9, rows), length=length, select=0)
    base = dict(op=op, kv_heads=kv_heads, dim=dim, page=page, mix=mix)
    if op == "append":
        seqs = _log(rng, 1, 200)
        rows = rng.choice((1, 2, _log(rng, 1, 4000)))
        rows = min(rows, 16000 // seqs)
        return dict(base, seqs=seqs, rows=rows, length=rows + _log(rng, 1, 2000),
                    dtype=rng.choice(("bf16", "fp16", "fp32")))
    seqs = rng.randrange(8, 128)
    pages = max(8 * seqs, _log(rng, 256, 16384))
    length = max(page, pages * page // seqs)
    return dict(base, pages=pages, seqs=seqs, length=length, count=rng.randrange(1, seqs))


# ------------------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """Each sequence's length and its rows in the call (host lists, from the case alone)."""
    r = random.Random(case["mix"])
    lens, rows = [], []
    for s in range(case["seqs"]):
        n = case["rows"] if s == 0 or case["rows"] <= 8 else r.randrange(max(1, case["rows"] // 3), case["rows"] + 1)
        n = min(n, case["length"])
        extra = case["length"] - case["rows"]
        lens.append(n + (extra if s == 0 else r.randrange(extra // 8, extra + 1)) if extra > 0 else n)
        rows.append(n)
    return lens, rows


def _pow2(e):
    """2^e in 32 bits, from its bit pattern."""
    return ((e.int().clamp(-126, 127) + 127) << 23).view(torch.float32)


def _need(amax):
    """The least exponent byte whose scale brings amax to 448 or below."""
    f, e = torch.frexp(amax)  # f in [0.5, 1); 448 = 0.875 * 2^9
    return torch.where(amax > 0, torch.where(f <= 0.875, e - 9, e - 8) + 127, 7).clamp(7, 247)


def _codes(gen, pages, heads, page, dim):
    """Normal values of varying size, rounded block by block to e4m3 codes under power-of-two scales."""
    codes = torch.empty((pages, heads, page, dim), dtype=torch.uint8, device="cuda")
    exps = torch.empty((pages, heads), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (heads * page * dim))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn((n, heads, page, dim), generator=gen, device="cuda")
        size = torch.randint(-1, 2, (n, heads, 1, 1), generator=gen, device="cuda")
        x = x * _pow2(size)
        e = _need(x.abs().amax((2, 3)))
        codes[i:i + n] = (x * _pow2(127 - e)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        exps[i:i + n] = e.to(torch.uint8)
    return codes, exps


def _table(gen, lens, page, pages, extra=0):
    """A page table over distinct pages in random order, and each page's count of users."""
    need = [-(-n // page) for n in lens]
    width = max(max(need, default=1), 1) + extra
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    start = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
    count = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    have = col[None, :] < count[:, None]
    table[have] = order[(start[:, None] + col[None, :])[have]]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:sum(need)].long()] = 1
    return table, refs


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    st = {"case": case}
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    if case["op"] in ("attention", "append"):
        lens, rows = _lengths(case)
        pages = sum(-(-n // page) for n in lens) + 3
        st["table"], st["refs"] = _table(gen, lens, page, pages)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        total = sum(rows)
        st["starts"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device="cuda")
        st["max_len"], st["max_rows"], st["rows"] = max(lens), max(rows), total
        dt = DTYPES[case["dtype"]]
        if case["op"] == "attention":
            st["q"] = (1.5 * torch.randn((total, case["heads"], d), generator=gen, device="cuda")).to(dt)
            if case["select"]:
                st["selected"] = _selection(gen, st, case["select"])
        else:
            st["new_k"] = (1.5 * torch.randn((total, hk, d), generator=gen, device="cuda")).to(dt)
            st["new_v"] = (1.5 * torch.randn((total, hk, d), generator=gen, device="cuda")).to(dt)
    else:
        pages = case["pages"]
        r = random.Random(case["mix"])
        lens, left = [], pages * 3 // 4
        for _ in range(case["seqs"]):
            n = r.randrange(1, 2 * case["length"])
            n = min(n, left * page)
            left -= -(-n // page)
            lens.append(n)
        empty = set(r.sample(range(case["seqs"]), case["count"]))
        if case["op"] in ("fork", "compact"):  # the listed sequences are gone: their pages are holes
            lens = [0 if s in empty else n for s, n in enumerate(lens)]
        st["table"], st["refs"] = _table(gen, lens, page, pages, extra=8)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        if case["op"] == "fork":
            full = [s for s, n in enumerate(lens) if n][:4]
            kids = sorted(empty) if full else []
            st["children"] = ints(kids)
            st["parents"] = ints([full[i % len(full)] for i in range(len(kids))])
        elif case["op"] == "free":
            st["gone"] = ints(sorted(empty))
        elif case["op"] == "reserve":
            st["counts"] = ints([r.randrange(1, 2 * page) if s in empty else 0 for s in range(case["seqs"])])
        elif case["op"] == "copy":
            n = max(1, min(case["count"] * 8, pages // 4))
            pick = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
            st["src"], st["dst"] = pick[:n].clone(), pick[n:2 * n].clone()
    st["k"], st["k_exps"] = _codes(gen, pages, hk, page, d)
    st["v"], st["v_exps"] = _codes(gen, pages, hk, page, d)
    if own:  # the handle that a program keeps beside its tensors
        import sparse_attention_indexer_relu_gb300 as mqa
        st["cache"] = mqa.KVCache(st["k"], st["v"], st["k_exps"], st["v_exps"], st["table"], st["lens"], st["refs"])
        if case["op"] == "attention":
            st["workspace"] = mqa.alloc_kv_workspace(st["cache"], st["rows"], case["heads"])
    return st


def _row_of(st):
    """Each row's sequence and the number of positions it sees."""
    at = torch.arange(st["rows"], dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(st["starts"], at, right=True) - 1
    starts = st["starts"].long()
    sees = st["lens"].long()[seq] - (starts[seq + 1] - at)  # position of the row, from 0
    return seq, at - starts[seq], sees + 1


def _selection(gen, st, k):
    """The indexer's answer: k distinct visible positions of each row in no order, then -1 where fewer are visible."""
    _, _, sees = _row_of(st)
    sees = sees[:, None]
    j = torch.arange(k, device="cuda")[None, :]
    # one position from each of k equal stretches of the visible range, in an order of its own
    part = torch.rand((st["rows"], k), generator=gen, device="cuda")
    lo, hi = j * sees // k, (j + 1) * sees // k
    pos = torch.where(sees > k, lo + (part * (hi - lo)).long().clamp(max=(hi - lo - 1)), j)
    order = torch.rand((1, k), generator=gen, device="cuda").argsort(1).expand(st["rows"], k)
    pos = torch.where(sees > k, pos.gather(1, order), pos)
    return torch.where(pos < sees, pos, -1).to(torch.int32).contiguous()


# ------------------------------------------------------------------------------------------------- plain forms
def _values(codes, exps):
    """Codes [..., n, d] under exponents [...] in 32 bits."""
    return codes.view(torch.float8_e4m3fn).float() * _pow2(exps.int() - 127)[..., None, None]


def _softmax_sum(scores, mask, v):
    """Rows of scores [..., n, t] over v [..., t, d]; a row whose mask leaves nothing gives zeros."""
    scores = scores.masked_fill(~mask, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _attention(st):
    case, q = st["case"], st["q"]
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    g = case["heads"] // hk
    seq, i, sees = _row_of(st)
    scale = 1.0 / math.sqrt(d)
    if case["select"]:
        pos = st["selected"].long()
        mask = (pos >= 0) & (pos < sees[:, None])
        pos = torch.where(mask, pos, 0)
        at = st["table"][seq[:, None], pos // page].long()
        code = lambda c: c[at, :, pos % page].view(torch.float8_e4m3fn).float()  # noqa: E731  [rows, k, hk, d]
        size = lambda e: _pow2(e[at].int() - 127)[..., None]  # noqa: E731
        kf = (code(st["k"]) * size(st["k_exps"])).transpose(1, 2)
        vf = (code(st["v"]) * size(st["v_exps"])).transpose(1, 2)
        scores = torch.matmul(q.float().view(-1, hk, g, d), kf.transpose(-1, -2)) * scale
        return _softmax_sum(scores, mask[:, None, None, :], vf).reshape(q.shape).to(q.dtype)
    s, n, width = case["seqs"], st["max_rows"], -(-st["max_len"] // page)
    at = st["table"][:, :width].clamp(min=0).long()
    flat = lambda c, e: _values(c[at], e[at]).permute(0, 2, 1, 3, 4).reshape(s, hk, width * page, d)  # noqa: E731
    qf = q.new_zeros((s, n, hk, g, d), dtype=torch.float32)
    qf[seq, i] = q.float().view(-1, hk, g, d)
    qf = qf.permute(0, 2, 3, 1, 4).reshape(s, hk, g * n, d)
    scores = torch.matmul(qf, flat(st["k"], st["k_exps"]).transpose(-1, -2)) * scale
    limit = torch.zeros((s, n), dtype=torch.int64, device="cuda")
    limit[seq, i] = sees
    mask = torch.arange(width * page, device="cuda") < limit[:, :, None]
    mask = mask[:, None].expand(s, g, n, width * page).reshape(s, 1, g * n, width * page)
    o = _softmax_sum(scores, mask, flat(st["v"], st["v_exps"]))
    return o.view(s, hk, g, n, d).permute(0, 3, 1, 2, 4)[seq, i].reshape(q.shape).to(q.dtype)


def _append(st):
    page = st["case"]["page"]
    seq, _, sees = _row_of(st)
    pos = sees - 1
    pages, slot = st["table"][seq, pos // page].long(), pos % page
    first = (st["lens"].long() - (st["starts"][1:] - st["starts"][:-1]))[seq]  # first new position of the sequence
    held = first - pos // page * page  # tokens that the row's page held before
    for codes, exps, x in ((st["k"], st["k_exps"], st["new_k"]), (st["v"], st["v_exps"], st["new_v"])):
        x = x.float()
        need = _need(x.abs().amax(-1)).to(torch.int32)  # [rows, heads]
        old = torch.where(held[:, None] > 0, exps[pages].int(), 0)
        new = torch.zeros(exps.shape, dtype=torch.int32, device="cuda")
        where = pages[:, None].expand_as(need)
        new.scatter_reduce_(0, where, torch.maximum(need, old), "amax")
        grown = new[pages]
        # the page's earlier tokens under the larger scale
        lead = (pos == first) & (held > 0)
        again, grow = pages[lead], (old - grown)[lead]
        kept = torch.arange(page, device="cuda")[None, :] < held[lead][:, None]
        was = codes[again]
        now = was.view(torch.float8_e4m3fn).float() * _pow2(grow)[:, :, None, None]
        now = now.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[again] = torch.where(kept[:, None, :, None], now, was)
        y = (x * _pow2(127 - grown)[..., None]).clamp(-448.0, 448.0)
        codes[pages, :, slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        exps[pages] = grown.to(torch.uint8)


def _move(st, src, dst):
    """Pages src to pages dst of every pool."""
    st["k"][dst], st["v"][dst] = st["k"][src], st["v"][src]
    st["k_exps"][dst], st["v_exps"][dst] = st["k_exps"][src], st["v_exps"][src]


def _fork(st, table, lens, refs):
    page = st["case"]["page"]
    mum, kid = st["parents"].long(), st["children"].long()
    n = lens[mum].long()
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    row = torch.where(col < -(-n // page)[:, None], table[mum], -1)
    part = n % page != 0
    src = row.gather(1, (n // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0][part].long()
    dst = torch.nonzero(refs == 0)[:, 0][:src.shape[0]]
    shared = row[col < (n // page)[:, None]].long()
    refs.scatter_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    refs[dst] = 1
    row[part, (n // page)[part]] = dst.int()
    table[kid], lens[kid] = row, n.int()
    _move(st, src, dst)


def _free(st, table, lens, refs):
    gone = st["gone"].long()
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    held = table[gone][col < -(-lens[gone] // st["case"]["page"])[:, None]].long()
    refs.scatter_add_(0, held, -torch.ones_like(held, dtype=torch.int32))
    table[gone], lens[gone] = -1, 0


def _compact(st, table, lens, refs):
    at = torch.arange(refs.shape[0], device="cuda")
    live = (refs > 0).sum()
    src, dst = torch.nonzero((refs > 0) & (at >= live))[:, 0], torch.nonzero((refs == 0) & (at < live))[:, 0]
    to = at.int()
    to[src] = dst.int()
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    table.copy_(torch.where(col < -(-lens // st["case"]["page"])[:, None], to[table.clamp(min=0).long()], table))
    refs[dst] = refs[src]
    refs[src] = 0
    _move(st, src, dst)


def _reserve(st, table, lens, refs):
    page = st["case"]["page"]
    now = lens + st["counts"]
    have, want = -(-lens // page), -(-now // page)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    new = (col >= have[:, None]) & (col < want[:, None])
    pages = torch.nonzero(refs == 0)[:, 0]
    table[new] = pages[:int(new.sum())].int()
    refs[table[new].long()] = 1
    lens.copy_(now)


PAGES = {"fork": _fork, "free": _free, "compact": _compact, "reserve": _reserve}


def run(st):
    op = st["case"]["op"]
    if own:
        import sparse_attention_indexer_relu_gb300 as mqa
    if op == "attention":
        if own:
            return mqa.kv_attention(st["q"], st["cache"], st["starts"], selected=st.get("selected"),
                                    max_rows=st["max_rows"], workspace=st["workspace"])
        return _attention(st)
    if op == "append":
        if own:
            mqa.kv_append(st["cache"], st["new_k"], st["new_v"], st["starts"])
        else:
            _append(st)
        return _pools(st)
    if op == "copy":
        if own:
            mqa.kv_copy_pages(st["cache"], st["src"], st["dst"])
        else:
            _move(st, st["src"].long(), st["dst"].long())
        return _pools(st)
    # each pass starts from the same tables: what it changes is a copy
    table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
    if own:
        cache = st["cache"].replace(page_table=table, seq_lens=lens, refcounts=refs)
        if op == "fork":
            mqa.kv_fork(cache, st["parents"], st["children"])
        elif op == "free":
            mqa.kv_free(cache, st["gone"])
        elif op == "reserve":
            mqa.kv_reserve(cache, st["counts"])
        else:
            mqa.kv_compact(cache)
    else:
        PAGES[op](st, table, lens, refs)
    return dict(_pools(st), table=table, lens=lens, refs=refs) if op in ("fork", "compact") else (table, lens, refs)


def _pools(st):
    """The cache's own buffers: code values (to be multiplied by 2^(exponent - 127)) and exponents."""
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn),
            "k_exps": st["k_exps"], "v_exps": st["v_exps"]}


# ------------------------------------------------------------------------------------------------- cost
def work(case):
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    if case["op"] == "attention":
        lens, rows = _lengths(case)
        total, width = sum(rows), 2
        io = 2 * total * case["heads"] * d * width
        if case["select"]:
            seen = [[min(case["select"], n - r + i + 1) for i in range(r)] for n, r in zip(lens, rows)]
            pairs = sum(map(sum, seen))
            # a sequence's rows together need each of its keys once at most
            keys = sum(min(n, sum(v)) for n, v in zip(lens, seen))
            return {"bytes": io + keys * hk * 2 * d + 4 * total * case["select"],
                    "flops": 4 * d * case["heads"] * pairs}
        pairs = sum(r * (n - r) + r * (r + 1) // 2 for n, r in zip(lens, rows))
        return {"bytes": io + sum(lens) * hk * 2 * d, "flops": 4 * d * case["heads"] * pairs}
    if case["op"] == "append":
        total = sum(_lengths(case)[1])
        width = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * total * hk * d * (width + 1), "flops": 4 * total * hk * d}
    data = 2 * hk * page * d + 2 * hk  # one page of every pool
    each = case["length"] // page + 1  # pages of a sequence, about
    if case["op"] == "fork":
        return {"bytes": case["count"] * (2 * data + 16 * each), "flops": 0}
    if case["op"] == "free":
        return {"bytes": case["count"] * 16 * each, "flops": 0}
    if case["op"] == "reserve":
        return {"bytes": 4 * case["pages"] + 12 * case["seqs"] + 16 * case["count"], "flops": 0}
    if case["op"] == "copy":
        return {"bytes": max(1, min(case["count"] * 8, case["pages"] // 4)) * (2 * data + 8), "flops": 0}
    live = min(case["pages"] * 3 // 4, case["seqs"] * each) * (case["seqs"] - case["count"]) / case["seqs"]
    return {"bytes": int(2 * data * live * (1 - live / case["pages"])) + 8 * case["pages"], "flops": 0}


# ------------------------------------------------------------------------------------------------- in 64 bits
def _pow2d(e):
    """2^e in 64 bits, from its bit pattern."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(codes):
    """What a code stands for, from its fields: sign, four exponent bits of bias 7, three of mantissa."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    size = torch.where(e == 0, m / 512.0, (8.0 + m) * _pow2d(e - 10))
    return torch.where(c >= 128, -size, size)


def exact(case, seed):
    if case["op"] != "attention":
        return _exact_append(case, seed) if case["op"] == "append" else None
    st = prepare(case, seed)
    lens, rows = _lengths(case)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    g = case["heads"] // hk
    pairs = sum(r * n for n, r in zip(lens, rows)) * case["heads"]
    if not case["select"] and 4.0 * d * pairs > 8e12:
        return None
    out = torch.zeros((st["rows"], case["heads"], d), dtype=torch.float64, device="cuda")
    r0 = 0
    for s, (n, r) in enumerate(zip(lens, rows)):
        used = st["table"][s, :-(-n // page)].long()
        for h in range(hk):
            two = lambda c, e: (_e4m3(c[used, h]) * _pow2d(e[used, h].long() - 127)[:, None, None]  # noqa: E731
                                ).reshape(-1, d)[:n]
            kd, vd = two(st["k"], st["k_exps"]), two(st["v"], st["v_exps"])
            for a in range(0, r, 512):
                b = min(r, a + 512)
                qd = st["q"][r0 + a:r0 + b, h * g:(h + 1) * g].double()
                last = torch.arange(n - r + a, n - r + b, device="cuda")  # the rows' own positions
                if case["select"]:
                    sel = st["selected"][r0 + a:r0 + b].long()
                    weight = torch.zeros((b - a, n + 1), dtype=torch.float64, device="cuda")
                    ok = (sel >= 0) & (sel <= last[:, None])
                    weight.scatter_add_(1, torch.where(ok, sel, n), torch.ones_like(sel, dtype=torch.float64))
                    weight = weight[:, :n]
                else:
                    weight = (torch.arange(n, device="cuda")[None, :] <= last[:, None]).double()
                score = torch.einsum("rgd,td->rgt", qd, kd) / math.sqrt(d)
                score = torch.where(weight[:, None] > 0, score, -math.inf)
                score = score - score.max(-1, keepdim=True).values.clamp(min=-1e300)
                p = score.exp_() * weight[:, None]
                o = torch.einsum("rgt,td->rgd", p, vd)
                norm = p.sum(-1, keepdim=True)
                out[r0 + a:r0 + b, h * g:(h + 1) * g] = torch.where(norm > 0, o / norm, 0.0)
        r0 += r
    return out


def _round_e4m3(x):
    """The nearest e4m3 value of x (64 bits), ties to even, at most 448."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4  # spacing 2^e: three mantissa bits, down to 2^-9
    return (torch.round(x * _pow2d(-e)) * _pow2d(e)).clamp(-448.0, 448.0)


def _exact_append(case, seed):
    st = prepare(case, seed)
    lens, rows = _lengths(case)
    page = case["page"]
    got = {}
    for name in ("k", "v"):
        value, exps, r0 = _e4m3(st[name]), st[name + "_exps"].clone(), 0
        for s, (n, r) in enumerate(zip(lens, rows)):
            x = st["new_" + name][r0:r0 + r].double()
            first, r0 = n - r, r0 + r
            for c in range(first // page, (n - 1) // page + 1):
                p = int(st["table"][s, c])
                lo, hi = max(first, c * page), min(n, (c + 1) * page)
                part = x[lo - first:hi - first].transpose(0, 1)  # [heads, tokens, d]
                amax = part.abs().amax((1, 2))
                e = torch.ceil(torch.log2(amax / 448.0)).long()
                e = torch.where(amax > 448.0 * _pow2d(e), e + 1, e)
                e = torch.where(amax <= 224.0 * _pow2d(e), e - 1, e) + 127
                e = torch.where(amax > 0, e, 7).clamp(7, 247)
                if lo > c * page:
                    was = exps[p].long()
                    e = torch.maximum(e, was)
                    old = value[p, :, :lo - c * page]
                    value[p, :, :lo - c * page] = _round_e4m3(old * _pow2d(was - e)[:, None, None])
                value[p, :, lo - c * page:hi - c * page] = _round_e4m3(part * _pow2d(127 - e)[:, None, None])
                exps[p] = e.to(torch.uint8)
        got[name], got[name + "_exps"] = value, exps
    return got
