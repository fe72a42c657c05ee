"""What is measured of beam search over the paged cache: the cases, their inputs and the plain forms.

The operators are beam_select (the best continuations over a lane's beams and the vocabulary), kv_pages_fork (beams
continue from their parents' pages: tables permuted, shared, trimmed and freed in place), kv_pages_reserve (pages for
the next tokens, a part-filled page that others share replaced), kv_pages_copy (the moves that a reserve or a
compaction asks for, in one layer's cache) and kv_pages_compact (live pages into the lowest places).

Pages are counted: refs[p] is the number of table entries (and outside holders) that name page p, 0 for a free one.
Row b of the table holds n_pages[b] entries, of which ceil(seq_lens[b] / page) are in use; entries behind those are
left as they are. A page handed out is the lowest free one, rows in order, so every result follows from the inputs.
"""
import math
import random

import numpy as np
import torch

own = False

FMTS = ("bf16", "fp8", "nvfp4")


# ------------------------------------------------------------------ cases
def _beam(name, dtype, lanes, beams, vocab, n_out, finished=0.0, dead=False, apart=0):
    c = {"op": "beam", "dtype": dtype, "lanes": lanes, "beams": beams, "vocab": vocab, "n_out": n_out,
         "finished": finished, "dead": dead, "apart": apart}
    if name:
        c["name"] = name
    return c


def _pages(name, op, rows, beams, ctx, page, pool=1.0, new=1, moves=0, ragged=False):
    """`pool`: pages of the pool for each page in use."""
    c = {"op": op, "rows": rows, "beams": beams, "ctx": ctx, "page": page, "pool": pool, "new": new, "moves": moves,
         "ragged": ragged}
    if name:
        c["name"] = name
    return c


def _copy(name, fmt, moves, tokens, page=64, kv_heads=4, dim=128):
    """`tokens` of each page are moved (0: the whole page)."""
    c = {"op": "copy", "fmt": fmt, "moves": moves, "tokens": tokens, "page": page, "kv_heads": kv_heads, "dim": dim}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one prompt searched with eight beams, the eight lanes of a decode step: latency
        _beam("beam-bf16-step", "bf16", 1, 8, 65536, 8),
        # several prompts, an odd vocabulary, twice as many candidates as beams, some of them finished
        _beam("beam-fp32-odd", "fp32", 4, 4, 100003, 8, finished=0.2),
        # the first step after the prompts: one row of each, 32 beams to open
        _beam("beam-bf16-first", "bf16", 8, 1, 131072, 32),
        # many prompts at once: bound by the logits' bytes
        _beam("beam-fp32-wide", "fp32", 64, 8, 131072, 8),
        # one step of eight beams after 16,421 tokens: latency
        _pages("fork-step", "fork", 8, 8, 16421, 64),
        # the largest table, small pages
        _pages("fork-wide", "fork", 1024, 16, 32768, 16, ragged=True),
        # the page of the next token for eight beams, half of them on a page that they share
        _pages("reserve-step", "reserve", 8, 8, 16421, 64, pool=4.0),
        # prompts of up to 8,192 tokens into small pages of a large pool, little of it free
        _pages("reserve-prompts", "reserve", 64, 4, 60000, 16, pool=1.45, new=8192, ragged=True),
        # the part-filled last pages of eight beams
        _copy("copy-fp8-tails", "fp8", 8, 37),
        # whole pages moved by a compaction
        _copy("copy-bf16-pages", "bf16", 2048, 0, kv_heads=8),
        # a few pages of a small pool moved between two steps
        _pages("compact-step", "compact", 8, 8, 16421, 64, pool=2.0, moves=64),
        # a large pool, half of it free, all at once
        _pages("compact-pool", "compact", 64, 4, 60000, 16, pool=2.0, moves=200000, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("beam", "beam", "beam", "fork", "reserve", "copy", "copy", "compact"))
    if op == "beam":
        lanes, beams = _log(rng, 1, 64), rng.choice((1, 2, 3, 4, 5, 6, 8, 12, 16))
        vocab = min(_log(rng, 300, 262144), (64 * 8 * 131072) // (lanes * beams))
        return _beam("", rng.choice(("bf16", "fp32")), lanes, beams, vocab, rng.choice((beams, 2 * beams, _log(rng, 1, 64))),
                     finished=rng.choice((0.0, 0.0, 0.2)), dead=rng.random() < 0.25, apart=rng.choice((0, 0, 8, 13)))
    if op == "copy":
        fmt, page = rng.choice(FMTS), rng.choice((16, 32, 48, 64, 128, 256))
        kv_heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 128, 256))
        most = max(1, (2048 * 64 * 8 * 128) // (page * kv_heads * dim))
        return _copy("", fmt, _log(rng, 1, min(8192, most)), rng.choice((0, rng.randrange(1, page + 1))), page, kv_heads, dim)
    page = rng.choice((16, 32, 48, 64, 128, 256))
    beams = rng.choice((1, 2, 3, 4, 5, 8, 16))
    rows = beams * _log(rng, 1, 1024 // beams)
    most = {"fork": 1024 * 32768 // 16, "reserve": 64 * 60000 // 16, "compact": 64 * 60000 // 16}[op]
    ctx = _log(rng, 2, min(60000, page * most // rows))
    return _pages("", op, rows, beams, ctx, page, pool=rng.choice((1.5, 2.0, 3.0)),
                  new=rng.choice((1, 1, _log(rng, 1, max(1, min(8192, ctx // 4))))), moves=_log(rng, 1, 20000),
                  ragged=rng.random() < 0.6)


def _tokens(case):
    """Tokens of every move: part-filled pages differ."""
    most = case["tokens"]
    return [most - (i * 5) % most if most else case["page"] for i in range(case["moves"])]


def _row_bytes(case):
    """Bytes of one token's codes and scales of one head, keys or values."""
    return {"bf16": 2 * case["dim"], "fp8": case["dim"] + 1, "nvfp4": case["dim"] // 2 + case["dim"] // 16}[case["fmt"]]


def _lens(case):
    """Tokens of every row: beams of one prompt alike but for those that ended earlier, ragged prompts shorter."""
    rows, beams, ctx = case["rows"], case["beams"], case["ctx"]
    groups = rows // beams
    out = []
    for b in range(rows):
        g, i = divmod(b, beams)
        top = ctx - (g * ctx) // (2 * groups) - (g * 7) % max(1, ctx // 3) if case["ragged"] and g else ctx
        out.append(max(0, top - (1 if i % 5 == 3 else 0)))
    return np.array(out, dtype=np.int64)


def _new(case):
    """Tokens to come of every row: ragged prompts shorter, and a row of every seven without any."""
    b = np.arange(case["rows"])
    n = np.maximum(1, case["new"] - (b * case["new"]) // (2 * case["rows"])) if case["ragged"] else np.full(case["rows"], case["new"])
    return np.where(b % 7 == 6, 0, n)


def work(case):
    op = case["op"]
    if op == "beam":
        rows = case["lanes"] * case["beams"]
        live = rows * (1 - case["finished"]) - (case["lanes"] * (case["beams"] // 2) if case["dead"] else 0)
        values = max(case["lanes"], live) * case["vocab"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": values * size + rows * 5 + case["lanes"] * case["n_out"] * 13, "flops": 4 * values}
    if op == "copy":
        return {"bytes": sum(_tokens(case)) * 2 * case["kv_heads"] * _row_bytes(case) * 2 + 16 * case["moves"], "flops": 0}
    lens, page = _lens(case), case["page"]
    held = int((-(-lens // page)).sum())
    if op == "fork":
        # half of the rows go on from another row: its entries read and written, and the counts of the pages that
        # no other beam shares changed
        shared = int(_shared(case, lens).sum()) * case["beams"]
        return {"bytes": held // 2 * 8 + (held - shared) * 8 + 12 * case["rows"], "flops": 0}
    pool = _pool_pages(case)
    if op == "reserve":
        fresh = int((-(-(lens + _new(case)) // page) - -(-lens // page)).sum())
        return {"bytes": pool * 4 + fresh * 8 + 16 * case["rows"], "flops": 0}
    return {"bytes": pool * 8 + held * 4 + min(case["moves"], pool // 4) * 28, "flops": 0}


# ------------------------------------------------------------------ inputs
def _shared(case, lens):
    """Columns that the beams of a prompt share: all but the last few pages."""
    need = (-(-lens // case["page"])).reshape(-1, case["beams"]).min(1)
    return np.maximum(0, need - 3)


def _pool_pages(case):
    lens, beams = _lens(case), case["beams"]
    used = -(-lens // case["page"])
    held = used + (np.arange(len(lens)) % 3 == 1)
    shared = np.repeat(_shared(case, lens), beams)
    pages = int((held - shared).sum() + shared[::beams].sum())
    return max(16, int(case["pool"] * pages) + (-(-case["new"] // case["page"]) + 2) * case["rows"] // (1 if case["op"] == "reserve" else 8) + 8)


def _roots(case):
    """The rows that beams go on from: the first of every two keeps its own, the other follows a row of its prompt."""
    b = np.arange(case["rows"])
    first = b - b % case["beams"]
    return np.where((b - first) % 2 == 0, b, first + 2 * (((b - first) * 5 // 2) % ((case["beams"] + 1) // 2)))


def prepare_pages(case, seed):
    dev = torch.device("cuda")
    rng = np.random.default_rng(seed)
    rows, beams, page = case["rows"], case["beams"], case["page"]
    lens = _lens(case)
    used = -(-lens // page)
    held = used + (np.arange(rows) % 3 == 1)               # a third of the rows hold a page ahead
    pool = _pool_pages(case)
    wide = int(held.max()) + -(-case["new"] // page) + 2
    wide += -wide % 4
    shared = np.repeat(_shared(case, lens), beams)
    cols = np.arange(wide)[None]
    inside = cols < held[:, None]
    first = (np.arange(rows) % beams == 0)[:, None]
    mine = inside & ((cols >= shared[:, None]) | first)
    rank = (np.cumsum(mine) - 1).reshape(rows, wide)
    owner = np.where(cols < shared[:, None], (np.arange(rows) - np.arange(rows) % beams)[:, None], np.arange(rows)[:, None])
    ids = rng.permutation(pool)
    table = np.where(inside, ids[np.clip(rank[owner, cols], 0, pool - 1)], 0)
    parent = _roots(case)
    if case["op"] == "fork":
        parent = np.where(np.arange(rows) % 11 == 10, -1, parent)             # some are done with
        parent = np.where((parent >= 0) & (parent % 11 == 10), -1, parent)
    if case["op"] == "reserve":                            # as a fork leaves them
        table, lens = table[parent], lens[parent]
        held = -(-lens // page)
        inside = cols < held[:, None]
    refs = np.bincount(table[inside], minlength=pool)
    taken = rng.integers(0, pool, max(1, pool // 64))      # pages that a prefix store holds besides
    refs[taken] += (refs[taken] > 0) | (case["op"] != "reserve")
    sizes = [rows * wide, rows, rows, pool]
    at = np.concatenate([[0], np.cumsum([n + -n % 4 for n in sizes])])
    start = np.zeros(at[-1], dtype=np.int32)
    for i, part in enumerate((table, lens, held, refs)):
        start[at[i]:at[i] + sizes[i]] = part.reshape(-1)
    start = torch.from_numpy(start).to(dev)
    now = start.clone()
    part = [now[at[i]:at[i] + sizes[i]] for i in range(4)]
    s = {"case": case, "start": start, "now": now, "table": part[0].view(rows, wide), "lens": part[1], "held": part[2],
         "refs": part[3], "page": page, "parent": torch.from_numpy(parent.astype(np.int32)).to(dev),
         "new": torch.from_numpy(_new(case).astype(np.int32)).to(dev)}
    cap = max(case["moves"], rows)
    s["moves"] = torch.full((cap, 4), -1, dtype=torch.int32, device=dev)
    s["count"] = torch.zeros(1, dtype=torch.int32, device=dev)
    s["left"] = torch.zeros(1, dtype=torch.int32, device=dev)
    s["limit"] = case["moves"]
    s["map"] = torch.zeros(pool, dtype=torch.int32, device=dev)
    return s


def prepare(case, seed):
    if case["op"] not in ("beam", "copy"):
        return prepare_pages(case, seed)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 2 + 1)
    rng = random.Random(seed)
    if case["op"] == "copy":
        n, H, page, dim, fmt = case["moves"], case["kv_heads"], case["page"], case["dim"], case["fmt"]
        pages = 2 * n + 3
        row = {"bf16": dim, "fp8": dim, "nvfp4": dim // 2}[fmt]
        s = {"case": case, "parts": []}
        for _ in range(2):
            if fmt == "bf16":
                s["parts"].append(torch.randn((pages, H, page, row), generator=gen, device=dev, dtype=torch.bfloat16))
                continue
            s["parts"].append(torch.randint(0, 120 if fmt == "fp8" else 256, (pages, H, page, row), generator=gen, device=dev,
                                            dtype=torch.uint8))
            s["parts"].append(torch.randint(1, 23, (pages, H, page) + (() if fmt == "fp8" else (dim // 16,)), generator=gen,
                                            device=dev, dtype=torch.uint8))
        ids = list(range(pages))
        rng.shuffle(ids)                                   # pages lie anywhere in the pool
        moves = torch.tensor([ids[:n], ids[n:2 * n], _tokens(case), [0] * n], dtype=torch.int32).T.contiguous()
        s["moves"], s["count"] = moves.to(dev), torch.tensor([n], dtype=torch.int32, device=dev)
        return s
    L, B, V = case["lanes"], case["beams"], case["vocab"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    wide = torch.empty((L * B, V + case["apart"]), dtype=dt, device=dev).normal_(0.0, 2.5, generator=gen)
    logits = wide[:, :V]
    # a few likely tokens, as a model gives them
    hot = torch.randint(0, V // 12, (L * B, 12), generator=gen, device=dev) + torch.arange(12, device=dev) * (V // 12)
    peaks = 8.0 + 4.0 * torch.rand((L * B, 12), generator=gen, device=dev)
    logits.scatter_(1, hot, peaks.to(dt))
    scores = -20.0 * torch.rand((L, B), generator=gen, device=dev) ** 2
    scores = scores.sort(1, descending=True).values
    if case["dead"]:
        scores[:, B - B // 2:] = -math.inf
    finished = torch.rand((L, B), generator=gen, device=dev) < case["finished"]
    out = (L, case["n_out"])
    return {"case": case, "logits": logits, "scores": scores, "finished": finished, "eos": V // 2, "pad": 0,
            "out": (torch.empty(out, device=dev), torch.empty(out, dtype=torch.int32, device=dev),
                    torch.empty(out, dtype=torch.int32, device=dev), torch.empty(out, dtype=torch.bool, device=dev))}


# ------------------------------------------------------------------ plain forms
def _beam_plain(s):
    case = s["case"]
    L, B, V, N = case["lanes"], case["beams"], case["vocab"], case["n_out"]
    x = s["logits"].float()
    finished, scores = s["finished"].view(-1), s["scores"].view(-1)
    live = (scores > -math.inf) & ~finished
    top = x.amax(1, keepdim=True)
    lse = top[:, 0].double() + torch.log(torch.exp((x - top).double()).sum(1))
    # a row's best tokens by value, ties to the lowest token: one whole number orders both
    bits = x.view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = order * (1 << 25) + (V - 1 - torch.arange(V, device=x.device))
    k = min(N, V)
    token = torch.topk(key, k, 1).indices                                          # [L * B, k]
    value = scores.double()[:, None] + (x.gather(1, token).double() - lse[:, None])
    value = torch.where(live[:, None], value, torch.full_like(value, -math.inf))
    value[:, 0] = torch.where(finished, scores.double(), value[:, 0])
    token = torch.where(finished[:, None], torch.full_like(token, s["pad"]), token)
    value, token = value.view(L, B * k), token.view(L, B * k)
    best = torch.sort(value, stable=True, dim=1, descending=True)
    got, at = best.values[:, :N], best.indices[:, :N]
    if got.shape[1] < N:
        more = N - got.shape[1]
        got = torch.cat([got, torch.full((L, more), -math.inf, dtype=got.dtype, device=got.device)], 1)
        at = torch.cat([at, torch.zeros((L, more), dtype=at.dtype, device=at.device)], 1)
    some = got > -math.inf
    first = torch.arange(L, device=x.device)[:, None] * B
    parent = torch.where(some, first + at // k, first)
    token = torch.where(some, token.gather(1, at), torch.full_like(at, s["pad"]))
    done = some & (finished[parent] | (token == s["eos"]))
    for o, v in zip(s["out"], (got, token, parent, done)):
        o.copy_(v)
    return list(s["out"])


def _fork_plain(s):
    table, lens, held, refs, page = s["table"].long(), s["lens"].long(), s["held"].long(), s["refs"], s["page"]
    parent = s["parent"].long()
    n, wide = table.shape
    cols = torch.arange(wide, device=table.device)[None]
    alive = parent >= 0
    src = parent.clamp_min(0)
    new_len = torch.where(alive, lens[src], torch.zeros_like(lens))
    keep = (new_len + page - 1) // page
    from_row = torch.where(cols < keep[:, None], table[src], table)
    change = torch.zeros(refs.shape[0] + 1, dtype=torch.int64, device=table.device)
    none = refs.shape[0]
    change.scatter_add_(0, torch.where(cols < keep[:, None], from_row, none).view(-1), torch.ones(n * wide, dtype=torch.int64, device=table.device))
    change.scatter_add_(0, torch.where(cols < held[:, None], table, none).view(-1), -torch.ones(n * wide, dtype=torch.int64, device=table.device))
    s["refs"].add_(change[:none].int())
    s["table"].copy_(from_row)
    s["lens"].copy_(new_len)
    s["held"].copy_(keep)
    return [s["table"], s["lens"], s["held"], s["refs"]]


def _reserve_plain(s):
    table, lens, held, refs, page = s["table"].long(), s["lens"].long(), s["held"].long(), s["refs"].long(), s["page"]
    new = s["new"].long()
    n, wide = table.shape
    dev = table.device
    rows, cols = torch.arange(n, device=dev), torch.arange(wide, device=dev)[None]
    active = new > 0
    first, last = lens // page, (lens + new + page - 1) // page
    part = active & (lens % page != 0)
    tail = table[rows, first.clamp_max(wide - 1)]
    spot = torch.where(part, tail, refs.shape[0])
    sharing = torch.zeros(refs.shape[0] + 1, dtype=torch.int64, device=dev).scatter_add_(0, spot, torch.ones_like(spot))
    lowest = torch.full((refs.shape[0] + 1,), n, dtype=torch.int64, device=dev).scatter_reduce_(0, spot, rows, "amin")
    count = refs[tail]
    keeps = (count == 1) | ((sharing[spot] == count) & (lowest[spot] == rows))
    copied = part & ~keeps
    need = (active[:, None] & (cols >= held[:, None]) & (cols < last[:, None])) | (copied[:, None] & (cols == first[:, None]))
    free = torch.nonzero(refs == 0)[:, 0]
    total = need.sum()
    s["left"].copy_((free.shape[0] - total).view(1))
    s["count"].zero_()
    if int(total) <= free.shape[0]:
        rank = torch.cumsum(need.view(-1), 0).view(n, wide) - 1
        page_of = torch.cat([free, free.new_zeros(1)])[rank.clamp(0, free.shape[0])]
        table_new = torch.where(need, page_of, table)
        refs.scatter_add_(0, torch.where(copied, tail, 0), -copied.long())
        refs[free[:int(total)]] = 1
        who = torch.nonzero(copied)[:, 0]
        s["moves"][:who.shape[0]] = torch.stack([tail[who], table_new[who, first[who]], lens[who] % page, 0 * who], 1).int()
        s["count"].fill_(who.shape[0])
        s["table"].copy_(table_new)
        s["refs"].copy_(refs)
        s["held"].copy_(torch.where(active, torch.maximum(held, last), held))
    return [s["table"], s["held"], s["refs"], s["moves"], s["count"], s["left"]]


def _compact_plain(s):
    table, held, refs = s["table"].long(), s["held"].long(), s["refs"].long()
    dev, pool = refs.device, refs.shape[0]
    at = torch.arange(pool, device=dev)
    live = refs != 0
    total = int(live.sum())
    holes = torch.nonzero(~live & (at < total))[:, 0]
    movers = torch.nonzero(live & (at >= total))[:, 0].flip(0)                       # the highest first
    m = min(holes.shape[0], s["limit"])
    holes, movers = holes[:m], movers[:m]
    page_map = torch.where(live, at, torch.full_like(at, -1))
    page_map[movers] = holes
    s["moves"][:m] = torch.stack([movers, holes, torch.full_like(holes, s["page"]), 0 * holes], 1).int()
    s["count"].fill_(m)
    s["left"].fill_(total)
    refs[holes] = refs[movers]
    refs[movers] = 0
    inside = torch.arange(table.shape[1], device=dev)[None] < held[:, None]
    s["table"].copy_(torch.where(inside, page_map[table], table))
    s["refs"].copy_(refs)
    s["map"].copy_(page_map)
    return [s["table"], s["refs"], s["map"], s["moves"], s["count"], s["left"]]


def _copy_plain(s):
    page = s["case"]["page"]
    src, dst, tokens = (s["moves"][:, i].long() for i in range(3))
    if s["case"]["tokens"] == 0:
        for part in s["parts"]:
            part[dst] = part[src]
        return list(s["parts"])
    move, off = torch.nonzero(torch.arange(page, device=src.device)[None] < tokens[:, None]).unbind(1)
    for part in s["parts"]:
        part[dst[move], :, off] = part[src[move], :, off]
    return list(s["parts"])


# ------------------------------------------------------------------ the framework's calls
def _handles(s):
    """The pages, moves and workspace, which a program makes once and keeps."""
    if "handle" not in s:
        import bit_quantized_weight_gb300 as qg
        case = s["case"]
        if case["op"] == "beam":
            need = qg.beam_select_workspace_size(case["lanes"], case["beams"], case["vocab"], case["n_out"])
            s["handle"] = torch.empty(need, dtype=torch.uint8, device=s["logits"].device)
        elif case["op"] == "copy":
            s["handle"] = qg.KVCache(case["fmt"], s["parts"][0], s["parts"][len(s["parts"]) // 2],
                                     *([] if case["fmt"] == "bf16" else [s["parts"][1], s["parts"][3]]))
            s["list"] = qg.KVMoves(s["moves"], s["count"])
        else:
            s["handle"] = qg.KVPages(s["table"], s["lens"], s["held"], s["refs"], s["page"])
            s["list"] = qg.KVMoves(s["moves"][:s["limit"]] if case["op"] == "compact" else s["moves"], s["count"])
    return s["handle"]


def run(s):
    op = s["case"]["op"]
    if op in ("reserve", "compact"):
        s["now"].copy_(s["start"])                         # the same step again
    if not own:
        return {"beam": _beam_plain, "fork": _fork_plain, "reserve": _reserve_plain, "compact": _compact_plain,
                "copy": _copy_plain}[op](s)
    import bit_quantized_weight_gb300 as qg
    handle = _handles(s)
    if op == "beam":
        qg.beam_select(s["logits"], s["scores"], *s["out"], finished=s["finished"], eos=s["eos"], pad=s["pad"],
                       workspace=handle)
        return list(s["out"])
    if op == "copy":
        qg.kv_pages_copy(handle, s["list"])
        return list(s["parts"])
    if op == "fork":
        qg.kv_pages_fork(handle, s["parent"])
        return [s["table"], s["lens"], s["held"], s["refs"]]
    if op == "reserve":
        qg.kv_pages_reserve(handle, s["new"], s["list"], n_free=s["left"])
        return [s["table"], s["held"], s["refs"], s["moves"], s["count"], s["left"]]
    qg.kv_pages_compact(handle, s["list"], s["map"], n_live=s["left"])
    return [s["table"], s["refs"], s["map"], s["moves"], s["count"], s["left"]]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """The selection's scores by sorting every candidate of a lane, and moved values one move after another; what
    else the page calls give is whole numbers."""
    if case["op"] not in ("beam", "copy") or case.get("fmt") in ("fp8", "nvfp4"):
        return None
    s = prepare(case, seed)
    if case["op"] == "copy":
        parts = [part.double() for part in s["parts"]]
        for src, dst, n, _ in s["moves"].tolist():
            for part in parts:
                part[dst, :, :n] = part[src, :, :n]
        return parts
    L, B, V, N = case["lanes"], case["beams"], case["vocab"], case["n_out"]
    out = [torch.full((L, N), -math.inf, dtype=torch.float64), torch.full((L, N), s["pad"], dtype=torch.int32),
           torch.zeros((L, N), dtype=torch.int32), torch.zeros((L, N), dtype=torch.bool)]
    done = s["finished"].cpu()
    for lane in range(L):
        out[2][lane] = lane * B
        z = s["logits"][lane * B:(lane + 1) * B].double()
        z = s["scores"][lane].double()[:, None] + z - torch.logsumexp(z, 1, keepdim=True)
        for b in range(B):
            if bool(done[lane, b]):
                z[b] = -math.inf
                z[b, s["pad"]] = s["scores"][lane, b].double()
        value, at = torch.sort(z.view(-1), stable=True, dim=0, descending=True)
        n = min(N, int((value > -math.inf).sum()))
        at = at[:n].cpu()
        out[0][lane, :n] = value[:n].cpu()
        out[1][lane, :n] = (at % V).int()
        out[2][lane, :n] = (lane * B + at // V).int()
        out[3][lane, :n] = (at % V == s["eos"]) | done[lane][at // V]
    return out
