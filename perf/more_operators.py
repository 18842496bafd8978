"""The pages of the 8-bit key/value cache in serving, and attention of sequences that share some of them, as
workloads: copying pages in every layer, forking sequences and reserving the pages of their next tokens, moving the
pages in use together, and attention of a batch whose sequences begin with the same tokens.

run() is one pass through an operator, in its plain form (elementary torch operations, scores in 32 bits)
or, with `own`, through the library's entry points; exact() is the definition in 64 bits.
"""
import math

import torch

own = False

PAGES = (16, 32, 64, 128)
QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------ cases
def _shared(name, B, groups, H, HK, N, d, page, fmt, dtype, plo, phi, lo, hi):
    """B sequences of `groups` groups with prefixes of plo to phi tokens; lo to hi tokens of their own behind them."""
    return {"name": name, "op": "shared", "B": B, "groups": groups, "H": H, "HK": HK, "N": N, "d": d, "page": page,
            "fmt": fmt, "dtype": dtype, "plo": plo, "phi": phi, "lo": lo, "hi": hi}


def _copy(name, layers, pages, moves, HK, d, page, fmt):
    return {"name": name, "op": "copy", "layers": layers, "pages": pages, "moves": moves, "HK": HK, "d": d, "page": page,
            "fmt": fmt}


def _grow(name, layers, HK, d, page, fmt, prompts, samples, decoding, admitted, lo, hi, new):
    """A step of a serving batch: `samples` sequences forked from each of `prompts`, `decoding` sequences
    that drop rejected drafts, `admitted` prompts that take the rows of finished ones; then the pages of the next
    `new` tokens (of the whole prompt, where it is admitted). Sequences hold lo to hi tokens."""
    return {"name": name, "op": "grow", "layers": layers, "HK": HK, "d": d, "page": page, "fmt": fmt, "prompts": prompts,
            "samples": samples, "decoding": decoding, "admitted": admitted, "lo": lo, "hi": hi, "new": new}


def _compact(name, layers, pages, used, rows, HK, d, page, fmt):
    """`used` percent of the pages are in use, by `rows` sequences, anywhere in the pool."""
    return {"name": name, "op": "compact", "layers": layers, "pages": pages, "used": used, "rows": rows, "HK": HK, "d": d,
            "page": page, "fmt": fmt}


def listed():
    return [
        # The smallest: four samples of one prompt of 1000 tokens, GPT-2 small's heads, one token each.
        _shared("shared_samples", 4, 1, 12, 12, 1, 64, 16, "int8", "bf16", 1000, 1000, 9, 64),
        # A serving batch behind one long instruction: 64 sequences, four query heads to a K/V head.
        _shared("shared_batch", 64, 1, 32, 8, 1, 128, 64, "e4m3", "bf16", 8192, 8192, 50, 2000),
        # Several prompts of unequal length, 16 samples of each, their rows mixed in the batch.
        _shared("shared_groups", 96, 6, 16, 4, 1, 128, 32, "int8", "fp16", 2000, 16000, 100, 1500),
        # Drafted tokens checked by one pass, five for each of 16 sequences behind one prompt.
        _shared("shared_drafts", 16, 1, 16, 2, 5, 128, 16, "e4m3", "fp16", 4000, 4000, 100, 1000),
        # The largest: 256 sequences that ask about one document of 32K tokens.
        _shared("shared_document", 256, 1, 32, 8, 1, 128, 128, "e4m3", "bf16", 32768, 32768, 256, 2048),
        # Three small pages of one layer (latency).
        _copy("copy_few", 1, 64, 3, 12, 64, 16, "int8"),
        # Sequences moved elsewhere in the pools of eight layers.
        _copy("copy_many", 8, 1100, 500, 8, 128, 64, "e4m3"),
        # Four samples forked from each of two prompts, twelve layers of GPT-2 small's heads.
        _grow("fork_samples", 12, 12, 64, 16, "int8", 2, 4, 0, 0, 500, 1000, 1),
        # A beam search's batch: 15 sequences forked from each of 16, eight layers.
        _grow("fork_beams", 8, 8, 128, 64, "e4m3", 16, 15, 0, 0, 1000, 4000, 1),
        # A step of a batch in flight: 128 sequences decode with drafts, 32 prompts are admitted.
        _grow("step_admit", 4, 4, 64, 16, "e4m3", 0, 0, 128, 32, 1000, 8000, 4),
        # A small pool moved together.
        _compact("compact_small", 2, 256, 50, 8, 2, 64, 16, "int8"),
        # Half-empty pools of four layers.
        _compact("compact_large", 4, 2048, 45, 48, 8, 128, 64, "e4m3"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    c = _drawn(rng)
    del c["name"]
    return c


def _drawn(rng):
    op = rng.choice(("shared", "shared", "shared", "copy", "grow", "grow", "compact"))
    d, page, fmt = rng.choice((64, 128)), rng.choice(PAGES), rng.choice(("e4m3", "int8"))
    HK = rng.choice((1, 2, 3, 4, 5, 8, 12, 16))
    if op == "shared":
        G, N = rng.choice((1, 2, 4, 7, 8, 16)), rng.choice((1, 1, 1, _between(rng, 2, 8)))
        B = _between(rng, 2, 256)
        groups = min(rng.choice((1, 1, 2, _between(rng, 1, 16))), B)
        hi = _between(rng, N, max(N, min(4096, (1 << 28) // (B * HK * d))))
        phi = _between(rng, 16, max(16, min(32768, (1 << 28) // (B * HK * G * N), (1 << 27) // (groups * HK * d))))
        return _shared("", B, groups, HK * G, HK, N, d, page, fmt, rng.choice(("bf16", "fp16")), _between(rng, max(1, phi // 8), phi),
                       phi, _between(rng, N, hi), hi)
    layers = rng.choice((1, 2, 4, 8, 12))
    room = (1 << 29) // (layers * HK * d * page)  # pages, so that all layers' pools stay within 1 GB
    if op == "copy":
        pages = _between(rng, 3, max(3, min(4096, room)))
        return _copy("", layers, pages, _between(rng, 1, pages // 2), HK, d, page, fmt)
    if op == "compact":
        pages = _between(rng, 4, max(4, min(16384, room)))
        return _compact("", layers, pages, rng.randrange(5, 100), _between(rng, 1, 64), HK, d, page, fmt)
    prompts = rng.choice((0, 1, _between(rng, 1, 16)))
    samples = _between(rng, 1, 16) if prompts else 0
    decoding = rng.choice((0, _between(rng, 1, 128)))
    admitted = rng.choice((0, _between(rng, 1, 32))) if prompts or decoding else _between(rng, 1, 32)
    sequences = prompts + prompts * samples // 8 + 1 + decoding + 2 * admitted
    hi = _between(rng, 1, max(1, min(16384, room * page // (2 * sequences))))
    return _grow("", layers, HK, d, page, fmt, prompts, samples, decoding, admitted, _between(rng, 1, hi), hi, _between(rng, 1, 8))


def _spread(n, lo, hi):
    """n lengths from lo to hi in equal steps."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _tokens(c):
    """shared: per sequence its group, the whole pages' tokens that the group shares, and all its tokens."""
    pre = _spread(c["groups"], c["plo"], c["phi"])
    mine = _spread(c["B"], c["lo"], c["hi"])
    of = [b % c["groups"] for b in range(c["B"])]
    return of, [x // c["page"] * c["page"] for x in pre], [pre[g] + x for g, x in zip(of, mine)], pre


def _batch(c):
    """grow: per row its kind, the tokens it holds, its parent, and start and count of the tokens to come."""
    kind = ["prompt"] * c["prompts"] + ["sample"] * (c["prompts"] * c["samples"]) + ["decode"] * c["decoding"] + ["admit"] * c["admitted"]
    T, S = c["prompts"], len(kind)
    length = _spread(T, c["lo"], c["hi"]) if T else []
    parent = list(range(S))
    for i in range(T * c["samples"]):  # neighbours are of different prompts
        parent[T + i] = i % T
        length.append(length[i % T])
    for n in (c["decoding"], c["admitted"]):
        length += _spread(n, c["lo"], c["hi"]) if n else []
    start, count = list(length), [c["new"]] * S
    for b, k in enumerate(kind):
        if k == "prompt":
            count[b] = 0
        if k == "admit":
            parent[b], start[b], count[b] = -1, 0, length[b]
    return kind, length, parent, start, count


def _page_bytes(c):
    """Codes and scales of one page, K and V, in every layer."""
    return c["layers"] * 2 * c["HK"] * (c["page"] * c["d"] + 4)


def work(c):
    page = c["page"]
    if c["op"] == "shared":
        of, shared, total, _ = _tokens(c)
        held = sum(shared) + sum(n - shared[g] for g, n in zip(of, total))
        pages = sum(shared) // page + sum(-(-(n - shared[g]) // page) for g, n in zip(of, total))
        N = c["N"]
        seen = sum(N * n - N * (N - 1) // 2 for n in total)
        return {"bytes": 2 * held * c["HK"] * c["d"] + pages * (8 * c["HK"] + 4) + c["B"] * c["H"] * N * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["H"] * seen}
    if c["op"] == "copy":
        return {"bytes": 2 * c["moves"] * _page_bytes(c) + 8 * c["moves"], "flops": c["moves"]}
    if c["op"] == "compact":
        used = c["pages"] * c["used"] // 100
        moved = used * (c["pages"] - used) // c["pages"]  # in a random order
        return {"bytes": 2 * moved * _page_bytes(c) + 8 * c["pages"] + 8 * used, "flops": 2 * c["pages"]}
    kind, length, parent, start, count = _batch(c)
    entries = sum(-(-n // page) for n, k in zip(length, kind) if k in ("sample", "admit"))
    looked = sum(-(-(s + n) // page) - s // page for s, n in zip(start, count) if n)
    copied = sum(k == "sample" and s % page != 0 for k, s in zip(kind, start))
    return {"bytes": 2 * copied * _page_bytes(c) + 12 * entries + 12 * looked, "flops": 2 * entries + 4 * looked}


# ------------------------------------------------------------------ inputs
def _scale_of(amax, qmax):
    """The smallest power of two s with amax <= qmax * s, exactly."""
    m, e = torch.frexp(amax)
    qm, qe = math.frexp(qmax)
    return torch.ldexp(torch.ones_like(amax), e - qe + (m > qm).to(e.dtype))


def _pool(c, pages, g, spread):
    """Codes and scales of `pages` pages; some channels are much larger than the rest for spread > 1."""
    HK, d, page, fmt = c["HK"], c["d"], c["page"], c["fmt"]
    x = torch.randn((pages, HK, page, d), generator=g, device="cuda", dtype=torch.float16)
    x = x * torch.exp2(torch.randn((HK, 1, d), generator=g, device="cuda") * (spread - 1.0)).to(x.dtype)
    s = _scale_of(x.abs().amax(dim=(2, 3)).float(), QMAX[fmt])
    x = (x / s[:, :, None, None].to(x.dtype)).clamp(-QMAX[fmt], QMAX[fmt])
    return (torch.round(x) if fmt == "int8" else x).to(CODES[fmt]), s


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _layers(c, s, pages, g):
    """The pools of every layer: names k0, ks0, v0, vs0, k1, ..."""
    for i in range(c["layers"]):
        for n, spread in (("k", 2.0), ("v", 1.0)):
            s[f"{n}{i}"], s[f"{n}s{i}"] = _pool(c, pages, g, spread)
    s["names"] = [f"{n}{i}" for i in range(c["layers"]) for n in ("k", "ks", "v", "vs")]


def _rows_of_pages(need, order, width):
    """A page table whose rows take need[b] pages each from `order`, -1 behind them."""
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def _prepare_shared(c, s, g, order):
    page = c["page"]
    of, shared, total, pre = _tokens(c)
    first, at = [], 0
    for x in shared:
        first.append(at)
        at += x // page
    width = max(-(-n // page) for n in total) + 1
    need = [-(-(n - shared[gr]) // page) for gr, n in zip(of, total)]
    pages = at + sum(need) + 3
    order = order(pages)
    table = torch.full((c["B"], width), -1, dtype=torch.int32)
    for b, gr in enumerate(of):
        n = shared[gr] // page
        table[b, :n] = order[first[gr]:first[gr] + n]
        table[b, n:n + need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"], s["len"], s["of"], s["prefix"] = table.cuda(), _ints(total), _ints(of), _ints(pre)
    (s["k0"], s["ks0"]), (s["v0"], s["vs0"]) = _pool(c, pages, g, 2.0), _pool(c, pages, g, 1.0)
    q = torch.randn((c["B"], c["N"], c["H"], c["d"]), generator=g, device="cuda")  # as a projection leaves it
    s["q"] = q.to(DTYPES[c["dtype"]]).transpose(1, 2)


def _prepare_grow(c, s, g, order):
    page = c["page"]
    kind, length, parent, start, count = _batch(c)
    # finished sequences, whose rows are taken, were as long as the prompts that come; drafts reached into one page more
    need = [0 if k == "sample" else -(-n // page) + (k == "decode") for k, n in zip(kind, length)]
    fresh = sum(-(-(a + n) // page) - a // page for a, n in zip(start, count))
    pages = sum(need) + fresh + 5
    s["table"] = _rows_of_pages(need, order(pages), max(-(-(a + n) // page) for a, n in zip(start, count)) + 2).cuda()
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["refs"][s["table"][s["table"] >= 0].long()] = 1
    s["parent"], s["start"], s["count"] = _ints(parent), _ints(start), _ints(count)
    s["keep"] = _ints(length)
    _layers(c, s, pages, g)


def _prepare_compact(c, s, g, order):
    pages, used = c["pages"], max(1, c["pages"] * c["used"] // 100)
    need = [used // c["rows"] + (b < used % c["rows"]) for b in range(c["rows"])]
    s["table0"] = _rows_of_pages(need, order(pages), max(need) + 1).cuda()
    s["refs0"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["refs0"][s["table0"][s["table0"] >= 0].long()] = 1
    s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
    _layers(c, s, pages, g)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": c}

    def order(pages):
        return torch.randperm(pages, generator=host).to(torch.int32)

    if c["op"] == "shared":
        _prepare_shared(c, s, g, order)
    elif c["op"] == "grow":
        _prepare_grow(c, s, g, order)
    elif c["op"] == "compact":
        _prepare_compact(c, s, g, order)
    else:
        pages = order(c["pages"])
        s["src"], s["dst"] = pages[:c["moves"]].cuda(), pages[c["moves"]:2 * c["moves"]].cuda()
        _layers(c, s, c["pages"], g)
    if own:
        import exact_io_aware_11_gb300 as fa
        s["caches"] = [fa.KVCache(s[f"k{i}"], s[f"v{i}"], s[f"ks{i}"], s[f"vs{i}"]) for i in range(c.get("layers", 1))]
        if c["op"] == "shared":
            need = fa.cache_attention_shared_workspace_bytes(s["caches"][0], c["B"], c["H"], c["N"], s["table"].shape[1], c["groups"])
        elif c["op"] == "grow":
            need = fa.cache_reserve_workspace_bytes(s["caches"][0], *s["table"].shape)
        elif c["op"] == "compact":
            need = fa.cache_compact_workspace_bytes(s["caches"][0])
        else:
            need = 0
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _move(s, src, dst):
    """Pages src of every layer's pools to dst."""
    for n in s["names"]:
        x = s[n].view(torch.uint8) if s[n].dtype == torch.float8_e4m3fn else s[n]
        x[dst] = x[src]


def _plain_fork(s):
    c, old, refs = s["case"], s["table"], s["refs"]
    S, W = old.shape
    row, col = torch.arange(S, device="cuda"), torch.arange(W, device="cuda")
    parent, keep = s["parent"].long(), s["keep"].long()
    new = old[parent.clamp(min=0)]
    stay = (parent >= 0)[:, None] & (col < ((keep + c["page"] - 1) // c["page"])[:, None])
    new = torch.where(stay, new, -1)
    for t, by in ((new, 1), (old, -1)):
        refs.scatter_add_(0, t.clamp(min=0).long().flatten(), torch.where(t >= 0, by, 0).to(torch.int32).flatten())
    old.copy_(new)


def _plain_reserve(s):
    c, table, refs = s["case"], s["table"], s["refs"]
    S, W = table.shape
    page = c["page"]
    col = torch.arange(W, device="cuda")
    start, count = s["start"].long(), s["count"].long()
    inside = (col >= (start // page)[:, None]) & (col < ((start + count + page - 1) // page)[:, None]) & (count > 0)[:, None]
    at = table.clamp(min=0).long()
    b, k = (inside & ((table < 0) | (refs[at] > 1))).nonzero(as_tuple=True)  # in the order of rows, then columns
    p = table[b, k].long()
    # the how-manieth of this call's users of its page each is: the last one of all keeps the page
    by_page, perm = torch.sort(p, stable=True)
    first = torch.searchsorted(by_page, by_page)
    rank = torch.empty_like(p)
    rank[perm] = torch.arange(p.numel(), device="cuda") - first
    take = (p < 0) | (rank < refs[p.clamp(min=0)].long() - 1)
    free = (refs == 0).nonzero(as_tuple=True)[0]
    n = torch.cumsum(take, 0)  # pages taken up to here
    fail = torch.where(take & (n > free.numel()), b, S).amin() if b.numel() else torch.tensor(S, device="cuda")
    go = take & (b < fail)
    bt, kt, pt = b[go], k[go], p[go]
    dst = free[n[go] - 1]
    refs.scatter_add_(0, pt.clamp(min=0), torch.where(pt >= 0, -1, 0).to(torch.int32))
    refs[dst] = 1
    table[bt, kt] = dst.to(torch.int32)
    held = (pt >= 0) & (kt == start[bt] // page) & (start[bt] % page != 0)
    _move(s, pt[held], dst[held])
    # once a row's pages are not there any more, the rows that need none are served alone
    return (~(inside & ((table < 0) | (refs[table.clamp(min=0).long()] > 1))).any(1)).to(torch.int32)


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    P = refs.numel()
    used = refs != 0
    live = used.sum()
    at = torch.arange(P, device="cuda")
    src, dst = (used & (at >= live)).nonzero(as_tuple=True)[0], (~used & (at < live)).nonzero(as_tuple=True)[0]
    _move(s, src, dst)
    where = torch.where(used, at, -1)
    where[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, where[table.clamp(min=0).long()].to(torch.int32), table))
    return where.to(torch.int32), live.to(torch.int32).view(1)


def _rows32(s, n, at):
    """Pages `at` [..., m] of K or V in 32 bits: [..., HK, m * page, d]."""
    x = s[n + "0"].view(torch.uint8)[at].view(s[n + "0"].dtype).float() * s[n + "s0"][at][..., None, None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _plain_shared(s):
    c = s["case"]
    B, H, HK, N, d, page = c["B"], c["H"], c["HK"], c["N"], c["d"], c["page"]
    of, shared, total, _ = _tokens(c)
    o = torch.empty((B, H, N, d), dtype=s["q"].dtype, device="cuda")
    lse = torch.empty((B, H, N), dtype=torch.float32, device="cuda")
    for g in range(c["groups"]):
        members = [b for b in range(B) if of[b] == g]
        cols = shared[g] // page
        if cols:
            at = s["table"][members[0], :cols].long()
            pk, pv = _rows32(s, "k", at), _rows32(s, "v", at)  # [HK, Lp, d]
        wide = max(-(-total[b] // page) - cols for b in members)
        step = max(1, (1 << 29) // (H * N * (shared[g] + wide * page) + 2 * HK * wide * page * d))
        for i in range(0, len(members), step):
            m = torch.tensor(members[i:i + step], device="cuda")
            n = m.numel()
            q = s["q"][m].float().reshape(n, HK, H // HK * N, d)
            length = s["len"][m].long()[:, None, None] - shared[g]
            at = s["table"][m, cols:cols + wide].long().clamp(min=0)
            k, v = _rows32(s, "k", at), _rows32(s, "v", at)  # [n, HK, Lo, d]
            j = torch.arange(k.shape[2], device="cuda")
            see = (j < length) & (j <= length - N + torch.arange(N, device="cuda")[:, None])
            v = torch.where((j < length[:, 0])[:, None, :, None], v, 0.0)
            x = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5).view(n, HK, H // HK, N, -1)
            x = x.masked_fill_(~see[:, None, None], -math.inf).view(n, HK, H // HK * N, -1)
            top = x.amax(-1, keepdim=True)
            if cols:
                y = torch.matmul(q.transpose(0, 1).reshape(HK, -1, d), pk.transpose(1, 2)).mul_(d ** -0.5)
                y = y.view(HK, n, H // HK * N, -1).transpose(0, 1)
                top = torch.maximum(top, y.amax(-1, keepdim=True))
            x = x.sub_(top).exp_()
            l, a = x.sum(-1, keepdim=True), torch.matmul(x, v)
            if cols:
                y = y.sub_(top).exp_()
                l = l + y.sum(-1, keepdim=True)
                z = torch.matmul(y.transpose(0, 1).reshape(HK, n * (H // HK) * N, -1), pv)
                a = a + z.view(HK, n, H // HK * N, d).transpose(0, 1)
            o[m] = (a / l).reshape(n, H, N, d).to(o.dtype)
            lse[m] = (top + torch.log(l)).reshape(n, H, N)
    return [o, lse]


# ------------------------------------------------------------------ one pass
def _with_pools(s, out):
    return out | {n: s[n] for n in s["names"]}


def run(s):
    c = s["case"]
    if own:
        import exact_io_aware_11_gb300 as fa
    if c["op"] == "shared":
        if own:
            return list(fa.cache_attention_shared(s["q"], s["caches"][0], s["table"], s["len"], s["of"], s["prefix"], workspace=s["ws"]))
        return _plain_shared(s)
    if c["op"] == "copy":
        if own:
            fa.cache_copy(s["caches"], s["src"], s["dst"])
        else:
            _move(s, s["src"].long(), s["dst"].long())
        return _with_pools(s, {})
    if c["op"] == "grow":
        if own:
            fa.cache_fork(s["table"], s["refs"], c["page"], s["parent"], keep=s["keep"])
            ok = fa.cache_reserve(s["caches"], s["table"], s["refs"], s["start"], s["count"], workspace=s["ws"])
        else:
            _plain_fork(s)
            ok = _plain_reserve(s)
        return _with_pools(s, {"table": s["table"], "refs": s["refs"], "ok": ok})
    # what sequences that came and went since have left, each time
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    if own:
        where, live = fa.cache_compact(s["caches"], s["table"], s["refs"], workspace=s["ws"])
    else:
        where, live = _plain_compact(s)
    return _with_pools(s, {"table": s["table"], "refs": s["refs"], "where": where, "live": live})


# ------------------------------------------------------------------ definitions in 64 bits
def _exact_pools(s, moves):
    out = {}
    for n in s["names"]:
        x = s[n].double()
        if moves:
            src, dst = (torch.tensor(t, device="cuda") for t in zip(*moves))
            x[dst] = x[src]
        out[n] = x
    return out


def _exact_grow(c, s):
    """Row by row and column by column, as the definitions read."""
    page = c["page"]
    _, length, parent, start, count = _batch(c)
    old, refs = s["table"].tolist(), s["refs"].tolist()
    W = len(old[0])
    table = []
    for b, p in enumerate(parent):
        keep = -(-length[b] // page) if p >= 0 else 0
        table.append([old[p][k] if k < keep else -1 for k in range(W)])
    for rows, by in ((table, 1), (old, -1)):
        for row in rows:
            for p in row:
                if p >= 0:
                    refs[p] += by
    free = [p for p, n in enumerate(refs) if n == 0]
    moves = []
    for b in range(len(table)):
        for k in range(start[b] // page, min(W, -(-(start[b] + count[b]) // page)) if count[b] else 0):
            p = table[b][k]
            if p >= 0 and refs[p] == 1:
                continue
            new = free.pop(0)
            refs[new] = 1
            table[b][k] = new
            if p >= 0:
                refs[p] -= 1
                if k == start[b] // page and start[b] % page:
                    moves.append((p, new))
    return {"table": _ints(table), "refs": _ints(refs), "ok": _ints([1] * len(table))} | _exact_pools(s, moves)


def _exact_compact(c, s):
    refs, table = s["refs0"].tolist(), s["table0"].tolist()
    live = sum(n != 0 for n in refs)
    where = [p if n else -1 for p, n in enumerate(refs)]
    moves, hole = [], 0
    for p in range(live, len(refs)):
        if refs[p]:
            while refs[hole]:
                hole += 1
            moves.append((p, hole))
            where[p], refs[hole], refs[p] = hole, refs[p], 0
    table = [[where[p] if p >= 0 else p for p in row] for row in table]
    return {"table": _ints(table), "refs": _ints(refs), "where": _ints(where), "live": _ints([live])} | _exact_pools(s, moves)


def _exact_shared(c, s):
    """Each K/V head of each sequence by itself, over its whole row of the page table."""
    B, H, HK, N, d, page = c["B"], c["H"], c["HK"], c["N"], c["d"], c["page"]
    total = _tokens(c)[2]
    if 4 * H * N * d * sum(total) > 3e11 or B * HK > 4096:
        return None  # too long in 64 bits
    o = torch.empty((B, H, N, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, H, N), dtype=torch.float64, device="cuda")
    for b, L in enumerate(total):
        at = s["table"][b, :-(-L // page)].long()
        k, v = ((s[n + "0"].view(torch.uint8)[at].view(s[n + "0"].dtype).double() * s[n + "s0"][at].double()[:, :, None, None])
                .transpose(0, 1).flatten(1, 2)[:, :L] for n in ("k", "v"))
        hidden = torch.arange(L, device="cuda") > (L - N + torch.arange(N, device="cuda"))[:, None]
        x = torch.einsum("hgnd,hld->hgnl", s["q"][b].double().view(HK, H // HK, N, d), k) / math.sqrt(d)
        x = x.masked_fill(hidden, -math.inf)
        z = torch.logsumexp(x, -1)
        lse[b] = z.reshape(H, N)
        o[b] = torch.einsum("hgnl,hld->hgnd", torch.exp(x - z[..., None]), v).reshape(H, N, d)
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "copy":
        return _exact_pools(s, list(zip(s["src"].tolist(), s["dst"].tolist())))
    return {"shared": _exact_shared, "grow": _exact_grow, "compact": _exact_compact}[c["op"]](c, s)
