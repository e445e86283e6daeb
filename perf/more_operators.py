"""Measured cases of what a step of serving needs around the paged 8-bit cache: the norm and rotation of query and key
heads, attention with a sliding window and first positions that stay visible, attention for a tree of drafted tokens
with the tree's masks, and taking over the drafted tokens that were accepted.

The cache holds FP8 e4m3 codes `k`, `v` [pages, kv_heads, page_size, head_dim] with one UE8M0 exponent byte per page
and head (value 2^(e - 127)).  Sequence s holds positions [0, seq_lens[s]) in the pages page_table[s, ...].  The rows
of a call belong to sequences by `row_starts`; the n rows of a sequence are its last n positions.
"""
import math
import random

import torch

own = False  # false: the plain forms below; true: the framework's own operators

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------- cases
def listed():
    r = {"op": "rotate", "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128, "dtype": "bf16", "pairs": "halves",
         "far": 32768}
    a = {"op": "window", "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16", "sinks": 4, "mix": 1}
    t = {"op": "tree", "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16", "mix": 1}
    m = {"op": "mask", "kv_heads": 2, "dim": 64, "page": 64, "mix": 3}
    c = {"op": "accept", "kv_heads": 8, "dim": 128, "page": 64, "mix": 4}
    return [
        # one user's next token: latency alone
        dict(r, name="rotate_1", rows=1),
        # a prompt batch of a layer: the rows of a fused projection are read and written once
        dict(r, name="rotate_16k", rows=16384),
        # one user's next token in a layer that sees the last 1,024 tokens and the first 4
        dict(a, name="window_1x5000", seqs=1, rows=1, length=5000, window=1024),
        # a serving batch over contexts of up to 32K tokens, of which a window layer reads 4K each
        dict(a, name="window_128x32k", seqs=128, rows=1, length=32768, window=4096),
        # a 2,048-token chunk of a long prompt in a window layer
        dict(a, name="window_chunk_2048", seqs=1, rows=2048, length=32768, window=4096),
        # prompts of odd lengths from their first token, small heads, half precision, a window that ends inside tiles
        dict(a, name="window_ragged_5x1531", seqs=5, rows=1531, length=1531, heads=16, kv_heads=4, dim=64, page=16,
             dtype="fp16", window=301, sinks=17, mix=5),
        # one user's draft of 13 tokens
        dict(t, name="tree_1x13", seqs=1, rows=13, length=3001),
        # a serving batch that verifies drafts of up to 64 tokens over contexts of up to 32K
        dict(t, name="tree_16x64", seqs=16, rows=64, length=32768),
        # the masks and positions of one small draft, and of a large batch's drafts
        dict(m, name="mask_1x13", seqs=1, rows=13, length=700),
        dict(m, name="mask_256x64", seqs=256, rows=64, length=900),
        # one user's accepted tokens, and those of a large batch
        dict(c, name="accept_1x13", seqs=1, rows=13, length=3001),
        dict(c, name="accept_256x64", seqs=256, rows=64, length=2000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "window", "window", "tree", "mask", "accept"))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 5, 8, 16) if kv_heads <= 2 else (1, 3, 4, 7))
    dim = rng.choice((64, 128, 128))
    if op == "rotate":
        dim = rng.choice((64, 128, 128, 256))
        rows = _log(rng, 1, 16384 * 40 * 128 // ((kv_heads * (group + 1)) * dim * 2) // 2)
        return dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, rows=min(rows, 30000),
                    rotary=rng.choice((dim, dim, dim // 2, 16 * rng.randrange(1, dim // 16 + 1))),
                    dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")), pairs=rng.choice(("halves", "neighbours")),
                    far=_log(rng, 1000, 1 << 24))
    base = dict(op=op, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 32, 64, 128)), mix=rng.randrange(1, 1 << 20))
    if op in ("mask", "accept"):
        seqs = _log(rng, 1, 256)
        rows = _log(rng, 1, min(256, 16384 // seqs))
        return dict(base, seqs=seqs, rows=rows, length=rows + _log(rng, 1, 2000))
    base.update(heads=kv_heads * group, dtype=rng.choice(("bf16", "bf16", "fp16")))
    if op == "tree":
        seqs, rows = _log(rng, 1, 24), _log(rng, 2, 200)
        most = max(rows + 1, min(32768, (1 << 28) // (seqs * rows * kv_heads * group)))
        return dict(base, seqs=seqs, rows=rows, length=_log(rng, rows + 1, most))
    window, sinks = _log(rng, 16, 8192), rng.choice((0, 1, 4, 4, rng.randrange(0, 200)))
    if rng.random() < 0.5:  # single tokens and short runs of them
        seqs = _log(rng, 1, 128)
        rows = rng.randrange(1, 9) if seqs <= 32 else 1
        return dict(base, seqs=seqs, rows=rows, length=_log(rng, 8, 32768), window=window, sinks=sinks)
    seqs, length = rng.randrange(1, 4), _log(rng, 64, 16384)  # prompts and their chunks
    rows = min(length, 2048, max(16, (1 << 28) // (seqs * kv_heads * group * min(length, window + sinks + 2048))))
    return dict(base, seqs=seqs, rows=_log(rng, 9, rows), length=length, window=window, sinks=sinks)


# ------------------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """Each sequence's length and its rows in the call (host lists, from the case alone)."""
    r = random.Random(case["mix"])
    lens, rows = [], []
    extra = case["length"] - case["rows"]
    for s in range(case["seqs"]):
        n = case["rows"] if s == 0 or case["rows"] <= 8 else r.randrange(max(1, case["rows"] // 3), case["rows"] + 1)
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


def _table(gen, lens, page, pages):
    """A page table over distinct pages in random order, and each page's count of users."""
    need = [-(-n // page) for n in lens]
    width = max(max(need), 1) + 2
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


def _inv_freq(case):
    """Angle per position of each rotated pair, in 64 bits."""
    i = torch.arange(0, case["rotary"], 2, dtype=torch.float64, device="cuda")
    return 500000.0 ** (-i / case["rotary"])


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "rotate":
        rows, h, hk, d = case["rows"], case["heads"], case["kv_heads"], case["dim"]
        dt = DTYPES[case["dtype"]]
        st["qkv"] = (1.5 * torch.randn((rows, h + 2 * hk, d), generator=gen, device="cuda")).to(dt)
        st["wq"], st["wk"] = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt) for _ in range(2))
        st["positions"] = torch.randint(0, case["far"], (rows,), generator=gen, device="cuda").int()
        st["inv_freq"] = _inv_freq(case)
        if own:  # the frequencies as a program lays them out once
            import sparse_attention_indexer_relu_gb300 as mqa
            st["turns"] = mqa.rope_turns(st["inv_freq"])
        return st
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    lens, rows = _lengths(case)
    pages = sum(-(-n // page) for n in lens) + 3
    total = sum(rows)
    st["table"], st["refs"] = _table(gen, lens, page, pages)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["starts"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device="cuda")
    st["max_len"], st["max_rows"], st["rows"] = max(lens), max(rows), total
    if case["op"] in ("window", "tree"):
        st["q"] = (1.5 * torch.randn((total, case["heads"], d), generator=gen, device="cuda")).to(DTYPES[case["dtype"]])
    if case["op"] in ("tree", "mask"):
        # each drafted token hangs on an earlier one of its sequence, the earliest on the sequence's last token
        i = _row_of(st)[1]
        pick = torch.rand(total, generator=gen, device="cuda", dtype=torch.float64) ** 0.5
        st["parents"] = (pick * (i + 1)).long().clamp(max=i).sub(1).int()
    if case["op"] == "tree":
        st["mask"] = _mask(st)[0]
    if case["op"] == "accept":
        # a random part of each sequence's rows, in order: as many as verification accepts, sometimes none
        seq, i, _ = _row_of(st)
        n = (st["starts"][1:] - st["starts"][:-1]).long()
        share = torch.rand(case["seqs"], generator=gen, device="cuda", dtype=torch.float64) ** 2
        st["counts"] = (share * (n + 1)).long().clamp(max=n).int()
        order = torch.argsort(seq.double() + torch.rand(total, generator=gen, device="cuda", dtype=torch.float64))
        keep = torch.zeros(total, dtype=torch.bool, device="cuda")
        keep[order] = i < st["counts"][seq]
        at = torch.argsort(seq * 2 + (~keep).long(), stable=True)  # the kept rows of a sequence first
        st["accepted"] = i[at].int()
    st["k"], st["k_exps"] = _codes(gen, pages, hk, page, d)
    st["v"], st["v_exps"] = _codes(gen, pages, hk, page, d)
    if own:  # the handle that a program keeps beside its tensors
        import sparse_attention_indexer_relu_gb300 as mqa
        st["cache"] = mqa.KVCache(st["k"], st["v"], st["k_exps"], st["v_exps"], st["table"], st["lens"], st["refs"])
        if "q" in st:
            st["workspace"] = mqa.alloc_kv_workspace(st["cache"], st["rows"], case["heads"])
    return st


def _row_of(st):
    """Each row's sequence, its number among the sequence's rows, and the number of positions up to its own."""
    at = torch.arange(st["rows"], dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(st["starts"], at, right=True) - 1
    starts = st["starts"].long()
    return seq, at - starts[seq], st["lens"].long()[seq] - (starts[seq + 1] - at) + 1


# ------------------------------------------------------------------------------------------------- plain forms
def _values(codes, exps):
    """Codes [..., n, d] under exponents [...] in 32 bits."""
    return codes.view(torch.float8_e4m3fn).float() * _pow2(exps.int() - 127)[..., None, None]


def _rotate(st):
    case = st["case"]
    h, hk, r = case["heads"], case["kv_heads"], case["rotary"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def head(x, w):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = (y[..., :r // 2], y[..., r // 2:r]) if case["pairs"] == "halves" else (y[..., :r:2], y[..., 1:r:2])
        pair = (a * cos - b * sin, b * cos + a * sin)
        turned = torch.cat(pair, -1) if case["pairs"] == "halves" else torch.stack(pair, -1).flatten(-2)
        return torch.cat((turned, y[..., r:]), -1).to(st["qkv"].dtype)

    return {"q": head(st["qkv"][:, :h], st["wq"]), "k": head(st["qkv"][:, h:h + hk], st["wk"])}


def _mask(st):
    """The rows of its own draft that each row sees (itself and what it hangs on), as bits, and its position."""
    n, words = st["max_rows"], -(-st["max_rows"] // 32)
    seq, i, _ = _row_of(st)
    up = torch.zeros((st["starts"].shape[0] - 1, n, n), dtype=torch.float32, device="cuda")
    up[seq, i, i] = 1.0
    has = st["parents"] >= 0
    up[seq[has], i[has], st["parents"][has].long()] = 1.0
    for _ in range(max(1, (n - 1).bit_length())):  # paths of twice the length each time
        up = (torch.matmul(up, up) > 0).float()
    sees = up[seq, i].bool()
    bits = torch.nn.functional.pad(sees, (0, words * 32 - n)).view(-1, words, 32).long()
    bits = (bits << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
    start = st["lens"].long() - (st["starts"][1:] - st["starts"][:-1])
    return mask, (start[seq] + sees.sum(-1) - 1).int()


def _softmax_sum(scores, mask, v):
    """Rows of scores [..., n, t] over v [..., t, d]; a row whose mask leaves nothing gives zeros."""
    scores = scores.masked_fill(~mask, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _attention(st):
    """Rows of each sequence side by side, over the positions that any of them sees."""
    case, q = st["case"], st["q"]
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    g = case["heads"] // hk
    seq, i, upto = _row_of(st)
    s, n = case["seqs"], st["max_rows"]
    first = st["lens"].long() - (st["starts"][1:] - st["starts"][:-1])  # position of a sequence's first row
    own_pos = torch.full((s, n), -1, dtype=torch.int64, device="cuda")
    own_pos[seq, i] = upto - 1
    if case["op"] == "window":
        w, sinks = case["window"], min(case["sinks"], st["max_len"])
        lo = (first - w + 1).clamp(min=sinks)  # behind the first positions, from where the first row's window begins
        width = min(w + n, st["max_len"])
        pos = torch.cat((torch.arange(sinks, device="cuda").expand(s, sinks),
                         lo[:, None] + torch.arange(width, device="cuda")), 1)
        at, me = pos[:, None, :], own_pos[:, :, None]
        mask = (at <= me) & ((at > me - w) | (at < sinks))
    else:
        pos = torch.arange(st["max_len"], device="cuda").expand(s, -1)
        at, me = pos[:, None, :], own_pos[:, :, None]
        rel = (pos - first[:, None]).clamp(0, n - 1)  # number of the drafted row at a position
        words = torch.zeros((s, n, st["mask"].shape[1]), dtype=torch.int32, device="cuda")
        words[seq, i] = st["mask"]
        bit = words.gather(2, (rel >> 5)[:, None, :].expand(s, n, -1)) >> (rel & 31)[:, None, :] & 1
        mask = (me >= 0) & (at < st["lens"][:, None, None]) & ((at < first[:, None, None]) | (bit != 0))
    held = pos < st["lens"][:, None]
    where = torch.where(held, st["table"].gather(1, torch.where(held, pos // page, 0)), 0).long()
    slot = pos % page

    def read(codes, exps):
        x = codes[where, :, slot].view(torch.float8_e4m3fn).float() * _pow2(exps[where].int() - 127)[..., None]
        return x.transpose(1, 2)  # [s, hk, t, d]

    qf = q.new_zeros((s, n, hk, g, d), dtype=torch.float32)
    qf[seq, i] = q.float().view(-1, hk, g, d)
    qf = qf.permute(0, 2, 3, 1, 4).reshape(s, hk, g * n, d)
    scores = torch.matmul(qf, read(st["k"], st["k_exps"]).transpose(-1, -2)) / math.sqrt(d)
    mask = mask[:, None].expand(s, g, n, -1).reshape(s, 1, g * n, -1)
    o = _softmax_sum(scores, mask, read(st["v"], st["v_exps"]))
    return o.view(s, hk, g, n, d).permute(0, 3, 1, 2, 4)[seq, i].reshape(q.shape).to(q.dtype)


def _accept(st, table, lens, refs):
    """Kept rows take their places as if they had been written there: the scale of a page is the least that holds what
    comes in, and no less than it was where earlier positions stay in it."""
    page = st["case"]["page"]
    seq, i, _ = _row_of(st)
    first = st["lens"].long() - (st["starts"][1:] - st["starts"][:-1])
    kept = i < st["counts"][seq]
    moved = kept & (st["accepted"] != i)
    seq, to, src = seq[moved], (first[seq] + i)[moved], (first[seq] + st["accepted"])[moved]
    begin = torch.full_like(st["lens"], 1 << 30).long()
    begin.scatter_reduce_(0, seq, to, "amin")  # the first place that a sequence's moved rows take
    src_page, src_slot = table[seq, src // page].long(), src % page
    to_page, to_slot = table[seq, to // page].long(), to % page
    held = (begin[seq] - to // page * page).clamp(min=0)  # positions of the page that stay
    lead = (to == torch.maximum(begin[seq], to // page * page)) & (held > 0)
    for codes, exps in ((st["k"], st["k_exps"]), (st["v"], st["v_exps"])):
        x = codes[src_page, :, src_slot].view(torch.float8_e4m3fn).float() * _pow2(exps[src_page].int() - 127)[..., None]
        need = _need(x.abs().amax(-1)).to(torch.int32)
        old = torch.where(held[:, None] > 0, exps[to_page].int(), 0)
        new = torch.zeros(exps.shape, dtype=torch.int32, device="cuda")
        new.scatter_reduce_(0, to_page[:, None].expand_as(need), torch.maximum(need, old), "amax")
        grown = new[to_page]
        again, grow = to_page[lead], (old - grown)[lead]
        stays = torch.arange(page, device="cuda")[None, :] < held[lead][:, None]
        was = codes[again]
        now = was.view(torch.float8_e4m3fn).float() * _pow2(grow)[:, :, None, None]
        now = now.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[again] = torch.where(stays[:, None, :, None], now, was)
        y = (x * _pow2(127 - grown)[..., None]).clamp(-448.0, 448.0)
        codes[to_page, :, to_slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        exps[to_page] = grown.to(torch.uint8)
    now = first + st["counts"]
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    gone = (col >= -(-now // page)[:, None]) & (col < -(-lens.long() // page)[:, None])
    freed = table[gone].long()
    refs.scatter_add_(0, freed, -torch.ones_like(freed, dtype=torch.int32))
    table[gone] = -1
    lens.copy_(now)


def run(st):
    op = st["case"]["op"]
    if own:
        import sparse_attention_indexer_relu_gb300 as mqa
    if op == "rotate":
        h, hk = st["case"]["heads"], st["case"]["kv_heads"]
        if own:
            q, k = mqa.qk_norm_rope(st["qkv"][:, :h], st["qkv"][:, h:h + hk], st["turns"], st["positions"],
                                    q_weight=st["wq"], k_weight=st["wk"], eps=1e-6,
                                    interleaved=st["case"]["pairs"] != "halves")
            return {"q": q, "k": k}
        return _rotate(st)
    if op == "window":
        if own:
            return mqa.kv_attention(st["q"], st["cache"], st["starts"], window=st["case"]["window"],
                                    sinks=st["case"]["sinks"], max_rows=st["max_rows"], workspace=st["workspace"])
        return _attention(st)
    if op == "tree":
        if own:
            return mqa.kv_attention(st["q"], st["cache"], st["starts"], tree=st["mask"], max_rows=st["max_rows"],
                                    workspace=st["workspace"])
        return _attention(st)
    if op == "mask":
        if own:
            mask, positions = mqa.kv_tree_mask(st["cache"], st["parents"], st["starts"], st["max_rows"])
        else:
            mask, positions = _mask(st)
        return {"mask": mask, "positions": positions}
    # each pass starts from the same tables: what it changes is a copy
    table, lens, refs = st["table"].clone(), st["lens"].clone(), st["refs"].clone()
    if own:
        cache = st["cache"].replace(page_table=table, seq_lens=lens, refcounts=refs)
        mqa.kv_accept(cache, st["starts"], st["counts"], st["accepted"])
    else:
        _accept(st, table, lens, refs)
    # the cache's own buffers: code values (to be multiplied by 2^(exponent - 127)) and exponents
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn), "k_exps": st["k_exps"],
            "v_exps": st["v_exps"], "table": table, "lens": lens, "refs": refs}


# ------------------------------------------------------------------------------------------------- cost
def work(case):
    hk, d = case["kv_heads"], case["dim"]
    if case["op"] == "rotate":
        width = 4 if case["dtype"] == "fp32" else 2
        n = case["rows"] * (case["heads"] + hk) * d
        return {"bytes": 2 * n * width + 4 * case["rows"], "flops": 8 * n}
    lens, rows = _lengths(case)
    total = sum(rows)
    if case["op"] == "mask":
        return {"bytes": total * (8 + 4 * -(-max(rows) // 32)), "flops": 0}
    if case["op"] == "accept":  # about a third of the rows is kept, and read and written once
        return {"bytes": total // 3 * 4 * hk * d + 12 * case["seqs"] + 4 * total, "flops": 0}
    io = 4 * total * case["heads"] * d
    if case["op"] == "tree":
        # the positions before the draft; of the draft itself a few each
        pairs = sum(r * (n - r) + r * min(r, 8) for n, r in zip(lens, rows))
        return {"bytes": io + sum(lens) * hk * 2 * d, "flops": 4 * d * case["heads"] * pairs}
    w, sinks = case["window"], case["sinks"]
    seen = [[min(n - r + i + 1, w) + min(sinks, max(0, n - r + i + 1 - w)) for i in range(r)] for n, r in zip(lens, rows)]
    keys = sum(min(n, min(sinks, max(0, n - r + 1 - w)) + w + r - 1) for n, r in zip(lens, rows))
    return {"bytes": io + keys * hk * 2 * d, "flops": 4 * d * case["heads"] * sum(map(sum, seen))}


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


def _round_e4m3(x):
    """The nearest e4m3 value of x (64 bits), ties to even, at most 448."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4  # spacing 2^e: three mantissa bits, down to 2^-9
    return (torch.round(x * _pow2d(-e)) * _pow2d(e)).clamp(-448.0, 448.0)


def exact(case, seed):
    if case["op"] == "rotate":
        return _exact_rotate(case, seed)
    if case["op"] in ("window", "tree"):
        return _exact_attention(case, seed)
    return _exact_accept(case, seed) if case["op"] == "accept" else None


def _exact_rotate(case, seed):
    st = prepare(case, seed)
    h, hk, r = case["heads"], case["kv_heads"], case["rotary"]
    got = {}
    for name, x, w in (("q", st["qkv"][:, :h], st["wq"]), ("k", st["qkv"][:, h:h + hk], st["wk"])):
        y = x.double()
        y = y / (y.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * w.double()
        out = y.clone()
        for j in range(r // 2):
            angle = st["positions"].double() * st["inv_freq"][j]
            c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            a, b = (j, j + r // 2) if case["pairs"] == "halves" else (2 * j, 2 * j + 1)
            out[..., a] = y[..., a] * c - y[..., b] * s
            out[..., b] = y[..., a] * s + y[..., b] * c
        got[name] = out
    return got


def _exact_attention(case, seed):
    st = prepare(case, seed)
    lens, rows = _lengths(case)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    g = case["heads"] // hk
    if 4.0 * d * sum(r * n for n, r in zip(lens, rows)) * case["heads"] > 8e12:
        return None
    out = torch.zeros((st["rows"], case["heads"], d), dtype=torch.float64, device="cuda")
    r0 = 0
    for s, (n, r) in enumerate(zip(lens, rows)):
        used = st["table"][s, :-(-n // page)].long()
        t = torch.arange(n, device="cuda")
        if case["op"] == "tree":
            sees = torch.zeros((r, n), dtype=torch.bool, device="cuda")
            sees[:, :n - r] = True
            for j in range(r):
                sees[:, n - r + j] = (st["mask"][r0:r0 + r, j // 32].long() >> (j % 32)) & 1 == 1
        for k in range(hk):
            two = lambda c, e: (_e4m3(c[used, k]) * _pow2d(e[used, k].long() - 127)[:, None, None]  # noqa: E731
                                ).reshape(-1, d)[:n]
            kd, vd = two(st["k"], st["k_exps"]), two(st["v"], st["v_exps"])
            for a in range(0, r, 512):
                b = min(r, a + 512)
                qd = st["q"][r0 + a:r0 + b, k * g:(k + 1) * g].double()
                if case["op"] == "tree":
                    ok = sees[a:b]
                else:
                    back = torch.arange(n - r + a, n - r + b, device="cuda")[:, None] - t  # how far behind the row
                    ok = (back >= 0) & ((back < case["window"]) | (t < case["sinks"]))
                score = torch.einsum("rgd,td->rgt", qd, kd) / math.sqrt(d)
                score = torch.where(ok[:, None], score, -math.inf)
                p = (score - score.max(-1, keepdim=True).values.clamp(min=-1e300)).exp_()
                norm = p.sum(-1, keepdim=True)
                out[r0 + a:r0 + b, k * g:(k + 1) * g] = torch.where(norm > 0, torch.einsum("rgt,td->rgd", p, vd) / norm,
                                                                   0.0)
        r0 += r
    return out


def _exact_accept(case, seed):
    st = prepare(case, seed)
    lens, rows = _lengths(case)
    page = case["page"]
    counts, accepted, table = st["counts"].tolist(), st["accepted"].tolist(), st["table"].tolist()
    got = {"table": None, "lens": None, "refs": None}
    for name in ("k", "v"):
        value, exps, r0 = _e4m3(st[name]), st[name + "_exps"].clone(), 0
        for s, (n, r) in enumerate(zip(lens, rows)):
            first, keep = n - r, accepted[r0:r0 + counts[s]]
            r0 += r
            stay = next((j for j, x in enumerate(keep) if x != j), len(keep))
            lo = first + stay
            while lo < first + len(keep):  # page by page
                hi = min(first + len(keep), (lo // page + 1) * page)
                src = torch.tensor([first + keep[p - first] for p in range(lo, hi)], device="cuda")
                src_page = torch.tensor([table[s][(first + keep[p - first]) // page] for p in range(lo, hi)], device="cuda")
                x = value[src_page, :, src % page] * _pow2d(exps[src_page].long() - 127)[..., None]  # [t, heads, d]
                amax = x.abs().amax((0, 2))
                e = torch.ceil(torch.log2(amax / 448.0)).nan_to_num(neginf=-120.0).long()
                e = torch.where(amax > 448.0 * _pow2d(e), e + 1, e)
                e = torch.where(amax <= 224.0 * _pow2d(e), e - 1, e) + 127
                e = torch.where(amax > 0, e, 7).clamp(7, 247)
                p, slot = table[s][lo // page], lo % page
                if slot:
                    was = exps[p].long()
                    e = torch.maximum(e, was)
                    value[p, :, :slot] = _round_e4m3(value[p, :, :slot] * _pow2d(was - e)[:, None, None])
                value[p, :, slot:slot + hi - lo] = _round_e4m3(x.transpose(0, 1) * _pow2d(127 - e)[:, None, None])
                exps[p] = e.to(torch.uint8)
                lo = hi
        got[name], got[name + "_exps"] = value, None
    return got
