"""Measured cases of the operators around the keys and values of a decode step:
rotary positions, a paged cache in 4-bit floats with its attention, and the
forking, growing, freeing and compacting of the pages of a cache.

The 4-bit cache holds u8 codes [pages, heads, page, D/2] and u8 scales
[pages, heads, page, D/32] of keys and of values.  A code is a float of 1 sign,
2 exponent and 1 mantissa bits (0, 0.5, 1, 1.5, 2, 3, 4, 6); a scale byte e
stands for 2^(e - 127), 255 for NaN; value = code * scale.  Channel 32 b + 2 j + i
of a token's row is nibble i (low first) of byte j * D/32 + b of the row for keys;
for values four tokens of a page share 2 D bytes, and the byte is
(4 j + token % 4) * D/32 + b of them.

    write      per 32 channels x: s = the smallest power of two from 2^-125 on with
               max|x| <= 7 s, at most 2^125; code = x / s to the nearest float, ties
               to the even code, at most 6 (a block that holds an infinity or a NaN: NaN)
    read       code * s, rounded once to the wanted type
    keep       new token keep[b, a] of sequence b moves to the place of its new token a
    attend     out[t, h] = sum_j softmax_j(alpha q[t, h] . k[j, h // g]) v[j, h // g]
               over the tokens j that row t sees (causal, or a tree of drafts)
    fork       children take over their parents' rows of the page table, and every
               page's count of owners grows; then the children grow: a shared last
               page is replaced by a copy, new pages are the lowest free ones
    compact    used pages move into free ones so that they come to lie at the front
    rope       channel pairs of a row at position p turn by p * frequency
"""

import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
DEVICE = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _case(name, kind, type_="f32", seqs=1, new=1, length=1, q_heads=8, kv_heads=8, dim=128, page=64, tree=False,
          ragged=0, children=0, mx4=True, rot=128, layout="half", scaling="none", base=10000.0, factor=1.0,
          inverse=False):
    return {"name": name, "kind": kind, "type": type_, "seqs": seqs, "new": new, "length": length, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "tree": tree, "ragged": ragged, "children": children,
            "mx4": mx4, "rot": rot, "layout": layout, "scaling": scaling, "base": base, "factor": factor,
            "inverse": inverse}


def listed():
    return [
        # one user's next token after a short talk: latency is all
        _case("attend_one_f32", "attend", "f32", 1, 1, 1023, 32, 8, 128, 64),
        # a serving batch with requests of all ages, one of them a book
        _case("attend_batch_bf16", "attend", "bf16", 32, 1, 32768, 32, 8, 128, 64, ragged=1),
        # wide draft trees over long contexts
        _case("attend_tree_f16", "attend", "f16", 8, 64, 8192, 32, 8, 128, 64, tree=True),
        # the second piece of two prompts taken in pieces, every head its own keys
        _case("attend_chunk_f32", "attend", "f32", 2, 509, 4093, 16, 16, 64, 32),
        # the drafts of a batch's trees go in, the accepted ones are kept and read
        _case("rows_step_f32", "rows", "f32", 64, 24, 2000, 32, 8, 128, 64, tree=True, ragged=3),
        # a batch of prompts goes in, and what the cache now holds comes back for the prompts' own attention
        _case("rows_prompts_bf16", "rows", "bf16", 4, 8192, 8192, 32, 8, 128, 64, ragged=4),
        # one prompt is sampled four ways: its pages are shared and the last one is copied
        _case("fork_one", "fork", "f32", 1, 1, 1001, kv_heads=8, page=64, children=4),
        # a batch of searches goes one step on: most last pages are shared
        _case("fork_batch", "fork", "bf16", 64, 3, 8192, kv_heads=8, page=32, ragged=5, children=512, mx4=False),
        # a small pool after some requests left
        _case("compact_small", "compact", "f32", 24, 1, 900, kv_heads=8, page=16, ragged=6),
        # a large pool, half of it freed
        _case("compact_large", "compact", "bf16", 256, 1, 4096, kv_heads=2, page=16, ragged=7, mx4=False),
        # a decode step's queries and keys, positions far into a long context
        _case("rope_step_f32", "rope", "f32", 64, 1, 100000, 32, 8, 128, layout="interleaved", scaling="turns",
              base=500000.0, factor=8.0, ragged=8),
        # prompts, part of the head
        _case("rope_prompts_bf16", "rope", "bf16", 4, 8192, 8192, 32, 8, 128, rot=64, scaling="linear", factor=4.0),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        kind = rng.choice(("attend", "attend", "attend", "rows", "fork", "compact", "rope"))
        kv_heads = rng.choice((1, 2, 4, 8, 16))
        group = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
        tree = (kind in ("attend", "rows")) and rng.random() < 0.4
        seqs = _log(rng, 1, 64)
        children, dim, page = 0, rng.choice((64, 128, 128, 256)), rng.choice((16, 32, 64, 128))
        rot = dim
        if kind == "attend":
            new = _log(rng, 2, 130) if tree else rng.choice((1, 1, _log(rng, 2, 600)))
            length = new + _log(rng, 1, 131072)
        elif kind == "rows":
            new = _log(rng, 2, 130) if tree else _log(rng, 1, 8192)
            length = new + _log(rng, 1, 8192) if tree or rng.random() < 0.5 else new
        elif kind == "fork":
            new, length, children = _log(rng, 1, 200), _log(rng, 1, 8192), _log(rng, 1, 1024)
        elif kind == "compact":
            new, length, seqs = 1, _log(rng, 1, 8192), _log(rng, 1, 512)
        else:
            new = rng.choice((1, _log(rng, 1, 8192)))
            length = new + _log(rng, 1, 1 << 20)
            dim = rng.choice((64, 80, 96, 128, 128, 256))
            rot = rng.choice((dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)))
        scaling = rng.choice(("none", "linear", "base", "turns", "index"))
        if scaling == "base" and rot < 4:
            scaling = "none"
        c = _case("", kind, rng.choice(("f32", "bf16", "f16")), seqs, new, length, kv_heads * group, kv_heads, dim, page,
                  tree, rng.choice((0, rng.randrange(1, 1 << 20))), children, kind in ("attend", "rows") or rng.random() < 0.5, rot,
                  rng.choice(("half", "interleaved")), scaling, rng.choice((10000.0, 500000.0, 1000000.0)),
                  rng.choice((2.0, 4.0, 8.0, 32.0)) if scaling != "none" else 1.0, rng.random() < 0.3)
        del c["name"]
        held = seqs * length * kv_heads * dim if kind != "rope" else 0
        scores = seqs * new * kv_heads * group * length if kind == "attend" else 0
        owned = children * (-(-length // page) + -(-new // page) + 2) * page * kv_heads * dim
        w = work(c)
        if held <= 1 << 28 and scores <= 1 << 27 and owned <= 1 << 29 and w["bytes"] <= 3e8 and w["flops"] <= 3e10:
            return c


def _sizes(case):
    """(lengths, new tokens) of the sequences: all alike, or spread below the largest, which the first one has."""
    n, new, length = case["seqs"], case["new"], case["length"]
    if not case["ragged"]:
        return [length] * n, [new] * n
    r = random.Random(case["ragged"])
    lengths, news = [length], [new]
    while len(lengths) < n:
        m = r.randint(max(1, new // 4), new)
        if case["kind"] in ("fork", "compact"):
            lengths.append(r.randint(1, length))
        else:
            whole = case["kind"] == "rows" and new == length
            lengths.append(m if whole else m + r.randint(0, max(0, length - new)))
        news.append(m)
    return lengths, news


def _children(case):
    """Each child's parent, and the tokens it grows by."""
    r = random.Random(case["ragged"] + 77)
    n = case["seqs"]
    return ([r.randrange(n) for _ in range(case["children"])],
            [r.randint(1, case["new"]) for _ in range(case["children"])])


def _token_bytes(case):
    """Of a token's key and value, codes and scales, in the cache."""
    d = case["dim"]
    return case["kv_heads"] * (d // 2 + d // 32 if case["mx4"] else d + d // 8) * 2


def _tail(case):
    """Tokens of a sequence that are read back to show what was copied."""
    return min(8, case["length"])


def work(case):
    lengths, news = _sizes(case)
    rows, e, page = sum(news), BYTES[case["type"]], case["page"]
    kind = case["kind"]
    if kind == "rope":
        elements = rows * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * elements * e + 4 * rows, "flops": 3 * rows * (case["q_heads"] + case["kv_heads"]) * case["rot"]}
    per_token = _token_bytes(case)
    per_row = case["kv_heads"] * case["dim"] * 2 * e
    if kind == "fork":
        parents, grown = _children(case)
        total = 0
        for p, g in zip(parents, grown):
            held, want = -(-lengths[p] // page), -(-(lengths[p] + g) // page)
            total += 4 * (3 * held + 3 * want)              # a row in and out, counts in and out, and the same on leaving
            total += 2 * page * per_token if lengths[p] % page else 0
            total += min(_tail(case), lengths[p]) * (per_token + per_row)
        return {"bytes": total, "flops": total // 4}
    if kind == "compact":
        used = sum(-(-n // page) for n in lengths)
        moved = used // 2                                   # half of a pool of twice as many pages, thereabouts
        tail = sum(min(_tail(case), n) for n in lengths)
        return {"bytes": 4 * 2 * used * 2 + 4 * 2 * used + 8 * moved + 2 * moved * page * per_token + tail * (per_token + per_row),
                "flops": 4 * used}
    elements = rows * case["kv_heads"] * case["dim"] * 2
    if kind == "rows":      # rows in, codes and scales out; codes and scales in, rows out; the kept ones once more
        kept = sum(len(_kept(n)) for n in news) if case["tree"] else 0
        return {"bytes": 2 * rows * (per_row + per_token) + 2 * kept * per_token, "flops": 6 * elements}
    pairs = 0
    for length, n in zip(lengths, news):
        pairs += n * (length - n) + (_tree_pairs(n) if case["tree"] else n * (n + 1) // 2)
    qo = 2 * rows * case["q_heads"] * case["dim"] * e
    return {"bytes": sum(lengths) * per_token + qo, "flops": 4 * pairs * case["q_heads"] * case["dim"]}


def _parents(n):
    """A draft tree of n tokens: token j hangs under token (j - 1) // 3, the first one under the context."""
    return [(j - 1) // 3 if j else -1 for j in range(n)]


def _tree_pairs(n):
    depth = []
    for p in _parents(n):
        depth.append(1 if p < 0 else depth[p] + 1)
    return sum(depth)


def _kept(n):
    """The accepted tokens of a tree of n: from the first one always to the last child."""
    path = [0]
    while 3 * path[-1] + 1 < n:
        path.append(min(3 * path[-1] + 3, n - 1))
    return path


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _starts(news):
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    return starts


def _cache_of(case, pages, g):
    """Codes and scales of about unit values."""
    shape = (pages, case["kv_heads"], case["page"])
    s = {}
    for name in ("k", "v"):
        if case["mx4"]:
            s[name] = torch.randint(0, 256, shape + (case["dim"] // 2,), generator=g, device=DEVICE, dtype=torch.uint8)
            s[name + "_scale"] = torch.randint(124, 128, shape + (case["dim"] // 32,), generator=g, device=DEVICE,
                                               dtype=torch.uint8)
        else:
            s[name] = torch.randint(-127, 128, shape + (case["dim"],), generator=g, device=DEVICE, dtype=torch.int8)
            s[name + "_scale"] = torch.empty(shape + (case["dim"] // 32,), device=DEVICE).uniform_(
                0.5 / 73, 1.5 / 73, generator=g)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    lengths, news = _sizes(case)
    kind, dtype = case["kind"], TYPES[case["type"]]
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    starts = _starts(news)
    s = {"kind": kind, "type": dtype, "page": page, "mx4": case["mx4"], "rows": starts[-1],
         "lengths": _int(lengths), "offsets": _int(starts)}

    def rows(h):
        return torch.randn((sum(news), h, dim), generator=g, device=DEVICE).to(dtype)

    if kind == "rope":
        s["q"], s["k"] = rows(case["q_heads"]), rows(heads)
        s.update(rot=case["rot"], interleaved=case["layout"] == "interleaved", inverse=case["inverse"],
                 amplitude=_amplitude(case))
        s["frequencies"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=DEVICE)
        if own:
            from quantized_decode_gemv_q8_amd import binding
            s["rope"] = binding.Rope.scaled(case["rot"], case["base"], case["scaling"], case["factor"],
                                            length=8192, interleaved=s["interleaved"], device=DEVICE)
        return s

    need = [-(-length // page) for length in lengths]
    if kind == "compact":
        pages = 2 * sum(need) + 5
    elif kind == "fork":
        parents, grown = _children(case)
        pages = sum(need) + sum(-(-n // page) + 1 for n in grown) + 7
    else:
        pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((len(need), max(need) + (1 if kind in ("fork", "compact") else 0)), -1, dtype=torch.int32,
                       device=DEVICE)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s.update(_cache_of(case, pages, g))
    if kind in ("fork", "compact"):
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEVICE)
        s["refs"][order[:at].long()] = 1
        s["held"] = [min(_tail(case), n) for n in (lengths if kind == "compact" else [lengths[p] for p in parents])]
        s["tail"] = _int(_starts(s["held"]))
        s["tail_rows"] = sum(s["held"])
    if kind == "fork":
        n = len(parents)
        s["parent"] = _int(parents)
        s["grown"] = _int([lengths[p] + m for p, m in zip(parents, grown)])
        columns = max([table.shape[1]] + [-(-(lengths[p] + m) // page) for p, m in zip(parents, grown)])
        s["child_table"] = torch.full((n, columns), -1, dtype=torch.int32, device=DEVICE)
        s["child_lengths"], s["none"] = _int([0] * n), _int([0] * n)
    if kind in ("rows", "attend"):
        s.update(longest=max(lengths), most_new=max(news), alpha=1 / math.sqrt(dim), tree=None)
    if kind == "attend":
        s["q"] = rows(case["q_heads"])
    if kind == "rows":
        s["new_k"], s["new_v"] = rows(heads), rows(heads)
        if case["tree"]:
            s["keep"] = torch.full((len(news), max(len(_kept(n)) for n in news)), -1, dtype=torch.int32)
            for b, n in enumerate(news):
                s["keep"][b, :len(_kept(n))] = torch.tensor(_kept(n), dtype=torch.int32)
            s["keep"] = s["keep"].to(DEVICE)
    if kind == "attend" and case["tree"]:
        n, words = max(news), -(-max(news) // 64)
        bits = []                   # token j sees itself and what its parent sees
        for j, p in enumerate(_parents(n)):
            bits.append((bits[p] if p >= 0 else 0) | 1 << j)
        signed = [[((b >> 64 * w) + (1 << 63)) % (1 << 64) - (1 << 63) for w in range(words)] for b in bits]
        whole = torch.tensor(signed, dtype=torch.int64, device=DEVICE)
        s["tree"] = torch.cat([whole[:m] for m in news])
    return s


# ---------------------------------------------------------------- rotary frequencies

def _frequencies(case):
    """Radians per position of each channel pair.  Contexts are stretched from 8192
    tokens: all frequencies alike (linear), by a larger base (base), or the slow ones
    only: those that make at most 1 turn in the 8192 are divided, those that make 4
    (turns) or 32 (index) stay, between them a blend that is linear in the turns or in
    the pair's index."""
    rot, base, f, length = case["rot"], case["base"], case["factor"], 8192
    if case["scaling"] == "base":
        base *= f ** (rot / (rot - 2))
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / f for x in freq]
    if case["scaling"] in ("none", "base"):
        return freq

    def index(turns):
        return rot * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))

    out = []
    for i, x in enumerate(freq):
        if case["scaling"] == "turns":
            w = (length * x / (2 * math.pi) - 1.0) / (4.0 - 1.0)
        else:
            first, last = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rot - 1)
            w = 1.0 - (i - first) / max(last - first, 1e-3)
        w = min(max(w, 0.0), 1.0)
        out.append(x * w + x / f * (1.0 - w))
    return out


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "index" else 1.0


# ---------------------------------------------------------------- the plain forms

def _places(s, table, lengths, offsets, rows):
    """For each row its sequence, its index among the sequence's new tokens, its page and its place there."""
    row = torch.arange(rows, device=DEVICE)
    offsets = offsets.long()
    seq = torch.searchsorted(offsets, row, right=True) - 1
    index = row - offsets[seq]
    position = lengths.long()[seq] - (offsets[seq + 1] - offsets[seq]) + index
    return seq, index, table.long()[seq, position // s["page"]], position % s["page"]


def _floats(bytes_, scale):
    """f32 values [..., D] of rows of bytes [..., 16, D/32] and scales [..., D/32]."""
    grid = torch.tensor(GRID + tuple(-x for x in GRID), device=DEVICE)
    nibbles = torch.stack((bytes_ & 15, bytes_ >> 4), -1).long()                     # [..., 16, NB, 2]
    e = scale.float() - 127
    step = torch.where(scale == 255, torch.nan, torch.ldexp(torch.ones_like(e), e))  # [..., NB]
    return (grid[nibbles] * step[..., None, :, None]).transpose(-3, -2).flatten(-3)


def _rows_of_values(v):
    """The values' codes, [pages, heads, page, D/2], as [pages, heads, page / 4, 16, 4, D/32]."""
    pages, heads, page, half = v.shape
    return v.view(pages, heads, page // 4, 16, 4, half // 16)


def _held_values(s, name, page, at):
    """f32 values [n, heads, D] of tokens `at` of pages `page`."""
    codes, scale = s[name], s[name + "_scale"][page, :, at]
    if not s["mx4"]:
        x = codes[page, :, at]
        x = x.reshape(*x.shape[:-1], 16, x.shape[-1] // 32, 2).transpose(-3, -2).float()
        return (x * scale[..., None, None]).flatten(-3)
    if name == "v":
        return _floats(_rows_of_values(codes)[page, :, at // 4, :, at % 4], scale)
    x = codes[page, :, at]
    return _floats(x.reshape(*x.shape[:-1], 16, -1), scale)


def _plain_write(s, name, x, page, at):
    x = x.float().reshape(*x.shape[:2], -1, 32)
    top = x.abs().amax(-1)
    fine = torch.isfinite(top)
    # 7 s is reached where the mantissa is 1.75: its bits then are 0x600000
    e = (((top.view(torch.int32) + 0x1fffff) >> 23) - 2).clamp(2, 252)
    y = torch.ldexp(x, (127 - e).float()[..., None]).abs()
    code = torch.zeros(x.shape, dtype=torch.uint8, device=DEVICE)
    for k in range(7):
        middle = (GRID[k] + GRID[k + 1]) / 2
        code += (y >= middle) if k % 2 else (y > middle)
    code |= torch.signbit(x).to(torch.uint8) << 3
    code = torch.where(fine[..., None], code, 0)
    code = code.reshape(*code.shape[:3], 16, 2)
    bytes_ = (code[..., 0] | code[..., 1] << 4).transpose(-2, -1)                     # [rows, heads, 16, NB]
    if name == "v":
        _rows_of_values(s[name])[page, :, at // 4, :, at % 4] = bytes_
    else:
        s[name][page, :, at] = bytes_.flatten(-2)
    s[name + "_scale"][page, :, at] = torch.where(fine, e, 255).to(torch.uint8)


def _plain_keep(s):
    keep, offsets, lengths = s["keep"].long(), s["offsets"].long(), s["lengths"].long()
    first = (lengths - (offsets[1:] - offsets[:-1]))[:, None]
    last = lengths[:, None] - 1
    to = first + torch.arange(keep.shape[1], device=DEVICE)
    source = torch.where(keep >= 0, first + keep, torch.minimum(to, last))   # a place that keeps nothing: itself
    to = torch.minimum(to, last)
    size, table = s["page"], s["table"].long()
    pf, pt = torch.gather(table, 1, source // size), torch.gather(table, 1, to // size)
    for name in ("k", "k_scale", "v_scale"):
        s[name][pt, :, to % size] = s[name][pf, :, source % size]
    v = _rows_of_values(s["v"])
    v[pt, :, to % size // 4, :, to % 4] = v[pf, :, source % size // 4, :, source % 4]


def _plain_read(s, table, lengths, offsets, rows):
    _, _, page, at = _places(s, table, lengths, offsets, rows)
    return {name: _held_values(s, name, page, at).to(s["type"]) for name in ("k", "v")}


def _gathered(s, name):
    """[seqs, heads, longest, D] values of all sequences, padded."""
    size = s["page"]
    pages = s["table"].long().clamp(min=0)
    codes, scale = s[name][pages], s[name + "_scale"][pages]        # [seqs, pages, heads, page, ..]
    if name == "v":
        seqs, n, heads, _, half = codes.shape
        codes = codes.view(seqs, n, heads, size // 4, 16, 4, half // 16).transpose(4, 5)
        codes = codes.reshape(seqs, n, heads, size, 16, half // 16)
    else:
        codes = codes.unflatten(-1, (16, -1))
    x = _floats(codes, scale)
    x = x.transpose(1, 2).reshape(x.shape[0], x.shape[2], -1, x.shape[-1])
    return x[:, :, :s["longest"]]


def _plain_attention(s):
    q, heads = s["q"].float(), s["k"].shape[1]
    seqs, n, longest = s["lengths"].shape[0], s["most_new"], s["longest"]
    group, dim = q.shape[1] // heads, q.shape[2]
    offsets, lengths = s["offsets"].long(), s["lengths"].long()
    count = offsets[1:] - offsets[:-1]
    i = torch.arange(n, device=DEVICE)
    row = (offsets[:-1, None] + i).clamp(max=s["rows"] - 1)                            # [seqs, n]
    x = q[row].reshape(seqs, n, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(seqs, heads, n * group, dim)
    score = torch.matmul(x, _gathered(s, "k").transpose(-1, -2)) * s["alpha"]
    j = torch.arange(longest, device=DEVICE)
    behind = j - (lengths - count)[:, None]                                            # index among the new ones
    if s["tree"] is None:
        sees = behind[:, None, :] <= i[None, :, None]
    else:
        at = behind.clamp(0, 64 * s["tree"].shape[1] - 1)
        words = torch.gather(s["tree"][row], 2, (at // 64)[:, None, :].expand(-1, n, -1))
        sees = (behind < 0)[:, None, :] | ((words >> (at % 64)[:, None, :]) & 1).bool()
    sees = sees & (j < lengths[:, None])[:, None, :]
    sees = sees[:, None, :, None, :].expand(-1, -1, -1, group, -1).reshape(seqs, 1, n * group, longest)
    score = torch.where(sees, score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(sees, torch.exp(score - top), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, _gathered(s, "v")) / total.clamp(min=1e-30)
    out = out.reshape(seqs, heads, n, group, dim).permute(0, 2, 1, 3, 4).reshape(seqs, n, heads * group, dim)
    seq, index, _, _ = _places(s, s["table"], s["lengths"], s["offsets"], s["rows"])
    return out[seq, index].to(s["type"])


def _plain_release(refs, table, held):
    """Every page of the rows loses one owner."""
    mine = torch.arange(table.shape[1], device=DEVICE) < held[:, None]
    refs.index_add_(0, table[mine].long(), torch.full((1,), -1, dtype=torch.int32, device=DEVICE).expand(int(mine.sum())))
    table[mine] = -1


def _plain_fork(s):
    refs, page = s["refs"], s["page"]
    table, lengths = s["child_table"], s["child_lengths"]
    _plain_release(refs, table, -(-lengths.long() // page))      # the last step's children leave
    parent = s["parent"].long()
    lengths.copy_(s["lengths"][parent])
    table.fill_(-1)
    held = -(-lengths.long() // page)
    mine = torch.arange(s["table"].shape[1], device=DEVICE) < held[:, None]
    table[:, :s["table"].shape[1]] = torch.where(mine, s["table"][parent], -1)
    refs.index_add_(0, s["table"][parent][mine].long(), torch.ones((), dtype=torch.int32, device=DEVICE).expand(int(mine.sum())))
    # growing: a shared last page that is written to is replaced, then come new ones
    want = -(-s["grown"].long() // page)
    last = torch.gather(table, 1, (held - 1).clamp(min=0)[:, None])[:, 0].long()
    replaced = (lengths % page != 0) & (refs[last.clamp(min=0)] > 1)
    need = want - held + replaced.long()
    free = torch.nonzero(refs <= 0)[:, 0].to(torch.int32)
    upto = torch.cumsum(need, 0)
    missing = torch.where(upto <= free.shape[0], 0, need).to(torch.int32)
    column = torch.arange(table.shape[1], device=DEVICE)
    first = held - replaced.long()
    takes = (column >= first[:, None]) & (column < want[:, None]) & (missing == 0)[:, None]
    rank = (upto - need)[:, None] + column - first[:, None]
    given = free[rank[takes].clamp(max=free.shape[0] - 1)]
    replaced = replaced & (missing == 0)
    table[takes] = given
    refs[given.long()] = 1
    refs.index_add_(0, last[replaced], torch.full((), -1, dtype=torch.int32, device=DEVICE).expand(int(replaced.sum())))
    moves = torch.full((len(parent), 2), -1, dtype=torch.int32, device=DEVICE)
    moves[:, 0] = torch.where(replaced, last, -1).to(torch.int32)
    moves[:, 1] = torch.where(replaced, torch.gather(table, 1, (held - 1).clamp(min=0)[:, None])[:, 0], -1)
    _plain_copy(s, moves)
    read = _plain_read(s, table, lengths, s["tail"], s["tail_rows"])
    lengths.copy_(s["grown"])
    return {"refs": refs, "table": table, "lengths": lengths, "moves": moves, "missing": missing, **read}


def _plain_copy(s, moves):
    moves = moves[moves[:, 0] >= 0].long()
    for name in ("k", "k_scale", "v", "v_scale"):
        s[name][moves[:, 1]] = s[name][moves[:, 0]]


def _plain_compact(s):
    refs, page = s["refs"], s["page"]
    used = refs > 0
    n = int(used.sum())
    pages = refs.shape[0]
    moves = torch.full((pages // 2, 2), -1, dtype=torch.int32, device=DEVICE)
    source = torch.nonzero(used[n:])[:, 0] + n
    to = torch.nonzero(~used[:n])[:, 0]
    moves[:len(source), 0], moves[:len(source), 1] = source.to(torch.int32), to.to(torch.int32)
    where = torch.arange(pages, device=DEVICE)
    where[source] = to
    where = torch.where(used, where, -1).to(torch.int32)
    out = torch.zeros_like(refs)
    out[where[used].long()] = refs[used]
    held = -(-s["lengths"].long() // page)
    mine = (torch.arange(s["table"].shape[1], device=DEVICE) < held[:, None]) & (s["table"] >= 0)
    table = torch.where(mine, where[s["table"].long().clamp(min=0)], -1)
    _plain_copy(s, moves)
    read = _plain_read(s, table, s["lengths"], s["tail"], s["tail_rows"])
    return {"refs": out, "table": table, "moves": moves, "used": torch.tensor([n], dtype=torch.int32, device=DEVICE), **read}


def _plain_rope(s):
    row = torch.arange(s["rows"], device=DEVICE)
    offsets = s["offsets"].long()
    seq = torch.searchsorted(offsets, row, right=True) - 1
    position = s["lengths"].long()[seq] - offsets[seq + 1] + row
    angle = position.double()[:, None] * s["frequencies"]           # 32 bits lose far positions' angles
    c, t = (torch.cos(angle) * s["amplitude"]).float()[:, None], (torch.sin(angle) * s["amplitude"]).float()[:, None]
    if s["inverse"]:
        t = -t
    out, rot = {}, s["rot"]
    for name in ("q", "k"):
        x = s[name].float()
        if s["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack((a * c - b * t, a * t + b * c), -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat((a * c - b * t, a * t + b * c), -1)
        out[name] = torch.cat((turned, x[..., rot:]), -1).to(s["type"])
    return out


def _plain(s):
    if s["kind"] == "attend":
        return _plain_attention(s)
    if s["kind"] == "rope":
        return _plain_rope(s)
    if s["kind"] == "fork":
        return _plain_fork(s)
    if s["kind"] == "compact":
        return _plain_compact(s)
    held = (s["table"], s["lengths"], s["offsets"])
    _, _, page, at = _places(s, *held, s["rows"])
    _plain_write(s, "k", s["new_k"], page, at)
    _plain_write(s, "v", s["new_v"], page, at)
    if "keep" in s:
        _plain_keep(s)
    return _plain_read(s, *held, s["rows"])


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    from quantized_decode_gemv_q8_amd import binding

    if s["kind"] == "rope":
        q, k = binding.q8_rope((s["q"], s["k"]), s["rope"], lengths=s["lengths"], offsets=s["offsets"],
                               inverse=s["inverse"])
        return {"q": q, "k": k}
    make, copy, read = ((binding.Mx4Cache, binding.q8_mx4_copy, binding.q8_mx4_read) if s["mx4"] else
                        (binding.Q8Cache, binding.q8_cache_copy, binding.q8_cache_read))
    cache = make(s["k"], s["k_scale"], s["v"], s["v_scale"])
    if s["kind"] == "fork":
        refs, table, lengths = s["refs"], s["child_table"], s["child_lengths"]
        binding.q8_pages_resize(refs, table, lengths, s["none"], s["page"])             # the last step's children leave
        binding.q8_pages_fork(refs, s["table"], s["lengths"], s["parent"], s["page"], table_out=table,
                              lengths_out=lengths)
        moves, missing = binding.q8_pages_resize(refs, table, lengths, s["grown"], s["page"])
        copy(cache, moves)
        k, v = read(cache, table, lengths, s["tail"], s["tail_rows"], dtype=s["type"])
        lengths.copy_(s["grown"])
        return {"refs": refs, "table": table, "lengths": lengths, "moves": moves, "missing": missing, "k": k, "v": v}
    if s["kind"] == "compact":
        refs, table, moves, used = binding.q8_pages_compact(s["refs"], s["table"], s["lengths"], s["page"])
        copy(cache, moves)
        k, v = read(cache, table, s["lengths"], s["tail"], s["tail_rows"], dtype=s["type"])
        return {"refs": refs, "table": table, "moves": moves, "used": used, "k": k, "v": v}
    held = (s["table"], s["lengths"], s["offsets"])
    if s["kind"] == "attend":
        return binding.q8_mx4_attention(s["q"], cache, *held, tree=s["tree"], alpha=s["alpha"])
    binding.q8_mx4_write(cache, s["new_k"], s["new_v"], *held)
    if "keep" in s:
        binding.q8_mx4_keep(cache, *held, s["keep"])
    k, v = binding.q8_mx4_read(cache, *held, s["rows"], dtype=s["type"])
    return {"k": k, "v": v}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_value(name, case, codes, scale, at):
    """[heads, n, D] values in 64 bits of tokens `at` (of the sequence's own pages, which follow one another)."""
    dim, page = case["dim"], case["page"]
    blocks = dim // 32
    channel = torch.arange(dim, device=DEVICE)
    b, j, i = channel // 32, channel % 32 // 2, channel % 2
    inside = at % page
    sc = scale[at // page, :, inside].transpose(0, 1)[..., b]                # [heads, n, D]
    if not case["mx4"]:
        place = j * 2 * blocks + 2 * b + i
        return codes[at // page, :, inside].transpose(0, 1)[..., place].double() * sc.double()
    flat = codes.flatten(2)                                                   # [pages, heads, page * D / 2]
    if name == "v":
        byte = (inside // 4)[:, None] * 2 * dim + (4 * j[None, :] + (inside % 4)[:, None]) * blocks + b[None, :]
    else:
        byte = inside[:, None] * (dim // 2) + (j * blocks + b)[None, :]
    taken = torch.gather(flat[at // page], 2, byte[:, None, :].expand(-1, flat.shape[1], -1)).transpose(0, 1)
    nibble = (taken >> (4 * i).to(torch.uint8)) & 15
    m, e = (nibble & 1).double(), ((nibble >> 1) & 3).double()
    size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
    return torch.where(nibble >= 8, -size, size) * torch.exp2(sc.double() - 127)


def _exact_rounded(x):
    """Rows [n, heads, D] as the 4-bit cache holds them."""
    x = x.double()
    blocks = x.reshape(*x.shape[:2], -1, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(top / 7)))         # no block of normal numbers is all zeros, or at a border
    y = blocks.abs() / s
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return (torch.round(y / step) * step).clamp(max=6).mul(s).copysign(blocks).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    lengths, news = _sizes(case)
    kind, page, heads, dim = case["kind"], case["page"], case["kv_heads"], case["dim"]
    if kind == "rope":
        return _exact_rope(case, s, lengths, news)
    if kind in ("fork", "compact"):
        return _exact_pages(case, s, lengths)
    table = s["table"].cpu()
    group = case["q_heads"] // heads
    outs, start = {"k": [], "v": [], "o": []}, 0
    for b, (length, n) in enumerate(zip(lengths, news)):
        owned = table[b, :-(-length // page)].long().to(DEVICE)
        if kind == "rows":
            for name in ("k", "v"):
                x = _exact_rounded(s["new_" + name][start:start + n])
                if case["tree"]:
                    x = x.clone()
                    for a, j in enumerate(_kept(n)):
                        x[a] = x[j]
                outs[name].append(x)
        else:
            sees = torch.ones((n, length), dtype=torch.bool, device=DEVICE)
            block = torch.zeros((n, n), dtype=torch.bool)
            parent = _parents(n)
            for i in range(n):
                if case["tree"]:
                    j = i
                    while j >= 0:
                        block[i, j] = True
                        j = parent[j]
                else:
                    block[i, :i + 1] = True
            sees[:, length - n:] = block.to(DEVICE)
            q = s["q"][start:start + n].double()
            o = torch.zeros((n, heads * group, dim), dtype=torch.float64, device=DEVICE)
            at = torch.arange(length, device=DEVICE)
            for h in range(heads):
                k, v = (_exact_value(x, case, s[x][owned, h:h + 1], s[x + "_scale"][owned, h:h + 1], at)[0]
                        for x in ("k", "v"))
                for f in range(h * group, (h + 1) * group):
                    z = (q[:, f] @ k.T) * s["alpha"]
                    z = z.masked_fill(~sees, -math.inf)
                    w = torch.exp(z - z.max(dim=1, keepdim=True).values)
                    o[:, f] = (w @ v) / w.sum(dim=1, keepdim=True)
            outs["o"].append(o)
        start += n
    if kind == "attend":
        return torch.cat(outs["o"])
    return {"k": torch.cat(outs["k"]), "v": torch.cat(outs["v"])}


def _exact_rope(case, s, lengths, news):
    rot = case["rot"]
    positions = torch.cat([torch.arange(length - n, length, device=DEVICE) for length, n in zip(lengths, news)])
    # whole turns are taken off before the sine: 64 bits hold the rest to some 1e-10
    turns = positions.double()[:, None] * (torch.tensor(_frequencies(case), dtype=torch.float64, device=DEVICE) / (2 * math.pi))
    angle = 2 * math.pi * (turns - torch.round(turns)) * (-1 if case["inverse"] else 1)
    w = torch.polar(torch.full_like(angle, _amplitude(case)), angle)[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        head = x[..., :rot]
        pairs = head.unflatten(-1, (-1, 2)) if s["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-2, -1)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        y = x.clone()
        y[..., :rot] = (z if s["interleaved"] else z.transpose(-2, -1)).flatten(-2)
        out[name] = y
    return out


def _exact_pages(case, s, lengths):
    page = case["page"]
    refs, table = s["refs"].tolist(), s["table"].tolist()
    pages = len(refs)
    if case["kind"] == "compact":
        used = [p for p in range(pages) if refs[p] > 0]
        n = len(used)
        empty = iter([p for p in range(n) if refs[p] <= 0])
        where = {p: p if p < n else next(empty) for p in used}
        moves = [[p, where[p]] for p in used if p >= n]
        out = [0] * pages
        for p in used:
            out[where[p]] = refs[p]
        new = [[where[p] if c < -(-length // page) else -1 for c, p in enumerate(row)]
               for row, length in zip(table, lengths)]
        result = {"refs": out, "table": new, "moves": moves + [[-1, -1]] * (pages // 2 - len(moves)), "used": [n]}
        old, read_lengths = table, lengths
    else:
        parents, grown = _children(case)
        columns = s["child_table"].shape[1]
        new, moves, need = [], [], []
        for p in parents:
            held = table[p][:-(-lengths[p] // page)]
            for x in held:
                refs[x] += 1
            new.append(held + [-1] * (columns - len(held)))
        old = [list(row) for row in new]
        empty = iter([p for p in range(pages) if refs[p] <= 0])
        shared = [refs[row[-(-lengths[p] // page) - 1]] > 1 and lengths[p] % page != 0 for row, p in zip(new, parents)]
        for row, p, m, again in zip(new, parents, grown, shared):
            held = -(-lengths[p] // page)
            moves.append([-1, -1])
            if again:
                moves[-1] = [row[held - 1], next(empty)]
                refs[moves[-1][0]] -= 1
                row[held - 1] = moves[-1][1]
                refs[row[held - 1]] = 1
            for c in range(held, -(-(lengths[p] + m) // page)):
                row[c] = next(empty)
                refs[row[c]] = 1
        result = {"refs": refs, "table": new, "lengths": [lengths[p] + m for p, m in zip(parents, grown)], "moves": moves,
                  "missing": [0] * len(parents)}
        read_lengths = [lengths[p] for p in parents]
    result = {name: _int(x).reshape(-1, 2) if name == "moves" else _int(x) for name, x in result.items()}
    first = max(len(row) for row in old)
    held = torch.tensor([row + [0] * (first - len(row)) for row in old], device=DEVICE)
    at = [[held_length - n + i for i in range(n)] for held_length, n in zip(read_lengths, s["held"])]
    seq = torch.tensor([b for b, row in enumerate(at) for _ in row], device=DEVICE)
    place = torch.tensor([x for row in at for x in row], device=DEVICE)
    source = held[seq, place // page]                   # the pages as they were: a copy holds the same
    for name in ("k", "v"):
        # each token's page as one of its own
        rows = []
        for part in torch.arange(len(place), device=DEVICE).split(2048):
            pages_of = source[part]
            at_ = torch.arange(len(part), device=DEVICE) * page + place[part] % page
            rows.append(_exact_value(name, case, s[name][pages_of], s[name + "_scale"][pages_of], at_).transpose(0, 1))
        result[name] = torch.cat(rows)
    return result
