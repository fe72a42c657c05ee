"""What is measured of the decode cache and its attention: the cases, their inputs and the plain forms.

The operators are kv_cache_append (quantise a step's or a prompt's keys and values as they are written into a
paged cache), kv_cache_read (the stored tokens as values again), kv_cache_accept (keep the accepted path of a
drafted tree) and tree_attention (drafted tokens, each seeing the whole context and its own ancestors, over the
cache as it is stored).

The cache: pages of `page` tokens, key/value heads apart, codes [pages][kv_heads][page][row].
  bf16   row = dim values
  fp8    row = dim E4M3 codes; one byte s per token and head, 1..22: value = code * 2^(s-15) * g
  nvfp4  row = dim/2 bytes of two E2M1 codes (low nibble = even index), one E4M3 scale per 16: code * scale * g
Quantising (y = x / g in 32 bits): fp8 takes the smallest s with max|y| <= 448 * 2^(s-15); nvfp4 takes
scale = E4M3(max|y| / 6) and code = E2M1(y / scale), 0 for scale 0; each to nearest, ties to even, saturating.
"""
import math
import random

import torch

own = False

FMTS = ("bf16", "fp8", "nvfp4")


# ------------------------------------------------------------------ cases
def _case(name, op, fmt, lanes, ctx, tree, heads=48, kv_heads=4, dim=128, page=64, ragged=False, g=1.0, lse=False):
    c = {"op": op, "fmt": fmt, "lanes": lanes, "ctx": ctx, "tree": tree, "heads": heads, "kv_heads": kv_heads,
         "dim": dim, "page": page, "ragged": ragged, "g": g, "lse": lse}
    if name:
        c["name"] = name
    return c


def listed():
    # 6144 query rows and 512 key rows of the fused QKV projection as 48 and 4 heads of 128 (or 24 and 2 of 256);
    # 32 and 4 heads for a hidden size of 2048. Eight lanes are the most a decode step batches.
    return [
        # one step of eight lanes with three drafts each: latency
        _case("append-fp8-step", "append", "fp8", 8, 4096, 4),
        # prompts of several lanes, packed and ragged, quantised and read back as the prompt's own attention would
        _case("append-nvfp4-prompt", "append", "nvfp4", 5, 0, 7680, page=16, ragged=True, g=0.75),
        # one long prompt into an unquantised cache
        _case("append-bf16-prompt", "append", "bf16", 1, 37, 32768, kv_heads=8),
        # a shared prefix fetched as bf16
        _case("read-fp8-prefix", "read", "fp8", 3, 0, 24576, kv_heads=8, ragged=True),
        # the last tokens of each lane
        _case("read-nvfp4-tail", "read", "nvfp4", 8, 16001, 33, page=32),
        # the accepted path of small trees, eight lanes
        _case("accept-fp8-step", "accept", "fp8", 8, 4096, 8),
        # the same for large trees of many lanes
        _case("accept-bf16-wide", "accept", "bf16", 96, 700, 64, kv_heads=8, ragged=True),
        # one token of one lane after a short context: latency
        _case("attend-bf16-one", "attend", "bf16", 1, 1000, 1, lse=True),
        # a decode step of eight lanes, ragged, up to 16,384 tokens of context
        _case("attend-fp8-decode", "attend", "fp8", 8, 16384, 1, ragged=True),
        # drafted trees of seven on 4-bit caches
        _case("attend-nvfp4-tree", "attend", "nvfp4", 8, 16384, 7, g=0.75, ragged=True),
        # one long prompt of 260,096 tokens, a window of 16 drafts
        _case("attend-fp8-long", "attend", "fp8", 1, 260096, 16, lse=True),
        # the widest trees: bound by arithmetic
        _case("attend-bf16-wide", "attend", "bf16", 8, 16384, 64, heads=32, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "read", "accept", "attend", "attend", "attend"))
    fmt = rng.choice(FMTS)
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    page = rng.choice((16, 32, 48, 64, 128, 256))
    lanes = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, _log(rng, 1, 64)))
    ragged = rng.random() < 0.6
    g = rng.choice((1.0, 0.75, 1.375))
    if op in ("append", "read"):
        most = max(1, (32768 * 8 * 128) // (lanes * kv_heads * dim))
        return _case("", op, fmt, lanes, rng.choice((0, _log(rng, 1, 20000 // lanes))), _log(rng, 1, min(24576, most)),
                     kv_heads=kv_heads, dim=dim, page=page, ragged=ragged, g=g)
    if op == "accept":
        return _case("", op, fmt, lanes, rng.choice((0, _log(rng, 1, 4096))), _log(rng, 1, 64), kv_heads=kv_heads,
                     dim=dim, page=page, ragged=ragged, g=g)
    group = rng.choice((1, 2, 4, 6, 7, 8, 12, 16))
    tree = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 1, 64)))
    # no more products than the widest tree, no more stored values than the longest prompt
    most = min((4 * 16384 * 64 * 32 * 128) // (lanes * tree * group * kv_heads * dim),
               (260096 * 4 * 128) // (lanes * kv_heads * dim))
    ctx = rng.choice((0, _log(rng, 1, max(2, min(2000, most)))) + (_log(rng, 1, max(2, min(200000, most))),) * 4)
    return _case("", op, fmt, lanes, ctx, tree, heads=group * kv_heads, kv_heads=kv_heads, dim=dim, page=page,
                 ragged=ragged, g=g, lse=rng.random() < 0.4)


def _lens(case):
    """Tokens already in the cache, by lane: the first lane has them all, ragged ones fewer and odd."""
    n, ctx = case["lanes"], case["ctx"]
    return [ctx - (b * ctx) // (2 * n) - (b * 7) % max(1, ctx // 3) if case["ragged"] and b and ctx else ctx for b in range(n)]


def _counts(case):
    n, tree = case["lanes"], case["tree"]
    return [max(1, tree - (b * tree) // (2 * n)) if case["ragged"] else tree for b in range(n)]


def work(case):
    row = {"bf16": 2 * case["dim"], "fp8": case["dim"] + 1, "nvfp4": case["dim"] // 2 + case["dim"] // 16}[case["fmt"]]
    tokens = sum(_counts(case))
    stored = 2 * case["kv_heads"] * row                    # a token's keys and values as they are held
    plain = 2 * case["kv_heads"] * 2 * case["dim"]         # and as bf16
    if case["op"] == "append":
        back = plain if case["fmt"] == "nvfp4" else 0
        return {"bytes": tokens * (plain + stored) + (tokens * (stored + back) if back else 0), "flops": 0}
    if case["op"] == "read":
        return {"bytes": tokens * (plain + stored), "flops": 0}
    if case["op"] == "accept":
        kept = sum((t + 1) // 2 for t in _counts(case))
        return {"bytes": kept * 2 * stored, "flops": 0}
    keys = [length + t for length, t in zip(_lens(case), _counts(case))]
    rows = tokens * case["heads"]
    flops = sum(4 * case["dim"] * k * t * case["heads"] for k, t in zip(keys, _counts(case)))
    return {"bytes": sum(keys) * stored + rows * case["dim"] * 4 + (rows * 4 if case["lse"] else 0), "flops": flops}


# ------------------------------------------------------------------ inputs
def _pool(case, pages, gen, dev):
    """Pages of quantised normal values."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    codes, scales = _quantise(x, case["fmt"], case["g"])
    return {"codes": codes, "scales": scales, "g": case["g"] if case["fmt"] != "bf16" else 1.0}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 2 + 1)
    rng = random.Random(seed)
    n, page, D = case["lanes"], case["page"], case["dim"]
    lens, counts = _lens(case), _counts(case)
    max_pages = max((length + t + page - 1) // page for length, t in zip(lens, counts)) + 1
    used = [(length + t + page - 1) // page for length, t in zip(lens, counts)]
    ids = list(range(sum(used) + 2))
    rng.shuffle(ids)                                       # pages lie anywhere in the pool
    table = torch.zeros((n, max_pages), dtype=torch.int32)
    at = 0
    for b in range(n):
        table[b, :used[b]] = torch.tensor(ids[at:at + used[b]], dtype=torch.int32)
        at += used[b]
    start = [0]
    for t in counts:
        start.append(start[-1] + t)
    total = start[-1]
    s = {"case": case, "fmt": case["fmt"], "page": page, "kv_heads": case["kv_heads"], "dim": D, "total": total,
         "table": table.to(dev), "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "start": torch.tensor(start, dtype=torch.int32, device=dev),
         "k": _pool(case, len(ids), gen, dev), "v": _pool(case, len(ids), gen, dev)}
    if case["op"] == "append":
        # k and v are columns of the fused projection's output
        qkv = torch.randn((total, (case["heads"] + 2 * case["kv_heads"]) * D), generator=gen, device=dev,
                          dtype=torch.bfloat16)
        qkv = qkv.view(total, -1, D)
        s["new_k"], s["new_v"] = qkv[:, case["heads"]:case["heads"] + case["kv_heads"]], qkv[:, case["heads"] + case["kv_heads"]:]
        s["qkv"] = qkv
    if case["op"] in ("read", "append", "accept"):
        s["k_out"] = torch.zeros((total, case["kv_heads"], D), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    if case["op"] == "accept":
        path = torch.zeros(total, dtype=torch.int32)
        kept = [(t + 1) // 2 for t in counts]              # half of the drafts, an ascending path from the root
        for b in range(n):                                 # through late drafts: a repeated pass moves the same rows
            chosen = [0] + sorted(rng.sample(range(kept[b], counts[b]), kept[b] - 1))
            path[start[b]:start[b] + kept[b]] = torch.tensor(chosen, dtype=torch.int32)
        s["path"], s["kept"] = path.to(dev), torch.tensor(kept, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.zeros(n, dtype=torch.int32, device=dev)
    if case["op"] == "attend":
        s["q"] = torch.randn((total, case["heads"], D), generator=gen, device=dev, dtype=torch.bfloat16)
        masks = []
        for t in counts:                                   # a random tree: each draft sees its ancestors and itself
            m = []
            for i in range(t):
                m.append((m[rng.randrange(max(0, i - 4), i)] if i else 0) | (1 << i))
            masks += m
        s["mask"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=dev)
        s["max_tree"] = max(counts)
        s["out"] = torch.zeros((total, case["heads"], D), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros((total, case["heads"]), dtype=torch.float32, device=dev) if case["lse"] else None
    return s


# ------------------------------------------------------------------ plain forms
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _two_to(e):
    """2^e for a tensor of whole e in [-126, 127], in 32 bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x, fmt, g):
    """Codes and scales of x[..., dim]."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    y = x.float() / g
    if fmt == "fp8":
        m, e = torch.frexp(y.abs().amax(-1))
        s = (e - 9 + (m > 0.875)).clamp(-14, 7)            # 448 = 0.875 * 2^9
        s = torch.where(m == 0, torch.full_like(s, -14), s)
        return _e4m3(y * _two_to(-s)[..., None]).view(torch.uint8), (s + 15).to(torch.uint8)
    blocks = y.unflatten(-1, (-1, 16))
    scale = _e4m3(blocks.abs().amax(-1) / 6.0)
    f = scale.float()[..., None]
    r = torch.where(f > 0, blocks / f, torch.zeros_like(blocks))
    a = r.abs()
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code + 8 * torch.signbit(r).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _values(codes, scales, fmt, g):
    """The values in 32 bits that codes and scales stand for."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * _two_to(scales.to(torch.int32) - 15)[..., None] * g
    lut = torch.tensor(_E2M1, device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    return (lut[pair].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2) * g


def _rows(s):
    """Lane and position in the lane's drafts of every packed token."""
    i = torch.arange(s["total"], device=s["start"].device)
    lane = torch.searchsorted(s["start"][1:].contiguous(), i.to(torch.int32), right=True)
    return lane, i - s["start"].long()[lane]


def _slots(s, lane, pos):
    page = s["table"].long()[lane, pos // s["page"]]
    return page, pos % s["page"]


def _gather(part, page, off, fmt):
    codes = part["codes"][page, :, off]
    return _values(codes, None if part["scales"] is None else part["scales"][page, :, off], fmt, part["g"])


def _stored(s):
    """The pools as outputs: E4M3 codes as such, scale exponents as whole numbers."""
    if s["fmt"] == "bf16":
        return [s["k"]["codes"], s["v"]["codes"]]
    return [s["k"]["codes"].view(torch.float8_e4m3fn), s["k"]["scales"],
            s["v"]["codes"].view(torch.float8_e4m3fn), s["v"]["scales"]]


def _read_plain(s):
    lane, j = _rows(s)
    page, off = _slots(s, lane, s["lens"].long()[lane] + j)
    s["k_out"].copy_(_gather(s["k"], page, off, s["fmt"]))
    s["v_out"].copy_(_gather(s["v"], page, off, s["fmt"]))
    return [s["k_out"], s["v_out"]]


def _append_plain(s):
    lane, j = _rows(s)
    page, off = _slots(s, lane, s["lens"].long()[lane] + j)
    ck, sk = _quantise(s["new_k"], s["fmt"], s["k"]["g"])
    cv, sv = _quantise(s["new_v"], s["fmt"], s["v"]["g"])
    s["k"]["codes"][page, :, off] = ck
    s["v"]["codes"][page, :, off] = cv
    if sk is not None:
        s["k"]["scales"][page, :, off] = sk
        s["v"]["scales"][page, :, off] = sv


def _accept_plain(s):
    lane, j = _rows(s)
    keep = torch.nonzero(j < s["kept"].long()[lane])[:, 0]
    lane, j = lane[keep], j[keep]
    base = s["lens"].long()[lane]
    page, off = _slots(s, lane, base + s["path"].long()[keep])
    to_page, to_off = _slots(s, lane, base + j)
    s["k"]["codes"][to_page, :, to_off] = s["k"]["codes"][page, :, off]
    s["v"]["codes"][to_page, :, to_off] = s["v"]["codes"][page, :, off]
    if s["k"]["scales"] is not None:
        s["k"]["scales"][to_page, :, to_off] = s["k"]["scales"][page, :, off]
        s["v"]["scales"][to_page, :, to_off] = s["v"]["scales"][page, :, off]
    s["new_lens"].copy_(s["lens"] + s["kept"])


def _attend_plain(s):
    case = s["case"]
    n, H, G, D, T = case["lanes"], case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], s["max_tree"]
    dev = s["q"].device
    lens, count = s["lens"].long(), (s["start"][1:] - s["start"][:-1]).long()
    L = case["ctx"] + T
    pos = torch.arange(L, device=dev)
    stored = pos[None] < (lens + count)[:, None]                                   # [n, L]
    page, off = _slots(s, torch.arange(n, device=dev)[:, None], torch.where(stored, pos[None], 0))
    k, v = _gather(s["k"], page, off, s["fmt"]), _gather(s["v"], page, off, s["fmt"])   # [n, L, H, D]
    lane, j = _rows(s)
    q = torch.zeros((n, T, H, G, D), device=dev)
    q[lane, j] = s["q"].float().view(-1, H, G, D)
    mask = torch.zeros((n, T), dtype=torch.int64, device=dev)
    mask[lane, j] = s["mask"]
    draft = pos[None] - lens[:, None]                                              # [n, L]
    bit = (mask[:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1
    seen = ((draft < 0)[:, None] | (bit == 1)) & stored[:, None]                   # [n, T, L]
    score = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(n, H, T * G, D), k.permute(0, 2, 3, 1)) / math.sqrt(D)
    score = score.view(n, H, T, G, L).masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(n, H, T * G, L), v.permute(0, 2, 1, 3)).view(n, H, T, G, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    s["out"].copy_(out.permute(0, 2, 1, 3, 4)[lane, j].reshape(-1, H * G, D))
    if s["lse"] is None:
        return [s["out"]]
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3)                      # [n, T, H, G]
    s["lse"].copy_(lse[lane, j].reshape(-1, H * G))
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------ the framework's calls
def _handles(s):
    """The cache, the batch and the workspace, which a program makes once and keeps."""
    if "cache" not in s:
        import bit_quantized_weight_gb300 as qg
        s["cache"] = qg.KVCache(s["fmt"], s["k"]["codes"], s["v"]["codes"], s["k"]["scales"], s["v"]["scales"],
                                k_gscale=s["k"]["g"], v_gscale=s["v"]["g"])
        s["batch"] = qg.KVBatch(s["table"], s["lens"], s["start"], s["total"])
        if "q" in s:
            need = qg.tree_attention_workspace_size(s["cache"], s["q"].shape[1], s["max_tree"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=s["q"].device)
    return s["cache"], s["batch"]


def run(s):
    op = s["case"]["op"]
    if own:
        import bit_quantized_weight_gb300 as qg
        cache, batch = _handles(s)
        if op == "attend":
            qg.tree_attention(cache, batch, s["q"], s["out"], s["max_tree"], tree_mask=s["mask"], lse=s["lse"],
                              workspace=s["workspace"])
            return [s["out"]] if s["lse"] is None else [s["out"], s["lse"]]
        if op == "append":
            qg.kv_cache_append(cache, batch, s["new_k"], s["new_v"])
        elif op == "accept":
            qg.kv_cache_accept(cache, batch, s["path"], s["kept"], new_lens=s["new_lens"])
        if op == "read" or s["fmt"] == "nvfp4":
            qg.kv_cache_read(cache, batch, s["k_out"], s["v_out"])
    else:
        if op == "attend":
            return _attend_plain(s)
        if op == "append":
            _append_plain(s)
        elif op == "accept":
            _accept_plain(s)
        if op == "read" or s["fmt"] == "nvfp4":
            _read_plain(s)
    outs = [s["k_out"], s["v_out"]] if op == "read" or s["fmt"] == "nvfp4" else _stored(s)
    return outs + [s["new_lens"]] if op == "accept" else outs


# ------------------------------------------------------------------ the definition in 64 bits
def _decode64(codes, scales, fmt, g):
    """Values of codes [..., row] in 64 bits, from tables of every code."""
    dev = codes.device
    if fmt == "bf16":
        return codes.double()
    e4m3 = []
    for c in range(256):
        e, m, sign = (c >> 3) & 15, c & 7, -1.0 if c & 128 else 1.0
        e4m3.append(math.nan if c & 127 == 127 else sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)))
    e4m3 = torch.tensor(e4m3, dtype=torch.float64, device=dev)
    if fmt == "fp8":
        two = torch.tensor([2.0 ** (b - 15) for b in range(256)], dtype=torch.float64, device=dev)
        return e4m3[codes.long()] * two[scales.long()].unsqueeze(-1) * g
    value = torch.tensor([(-1.0 if c & 8 else 1.0) * (0, 0.5, 1, 1.5, 2, 3, 4, 6)[c & 7] for c in range(16)],
                         dtype=torch.float64, device=dev)
    both = torch.empty(codes.shape + (2,), dtype=torch.float64, device=dev)
    both[..., 0], both[..., 1] = value[(codes & 15).long()], value[(codes >> 4).long()]
    flat = both.reshape(codes.shape[:-1] + (-1,))
    return flat * e4m3[scales.long()].repeat_interleave(16, -1) * g


def _nearest(x, grid):
    """Each x as the index of the nearest value of the ascending `grid`, ties to the even index, by bisection."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def _pack64(x, fmt, g):
    """Codes, scales of x in 64 bits. The quotients x / g, max / 6 and y / scale are 32-bit numbers by definition."""
    if fmt == "bf16":
        return x, None
    grid = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]
    y = (x.double() / g).float().double()
    if fmt == "fp8":
        top = y.abs().amax(-1)
        steps = torch.tensor([448.0 * 2.0 ** e for e in range(-14, 7)], dtype=torch.float64, device=x.device)
        s = torch.searchsorted(steps, top) - 14
        r = y * torch.exp2(-s.double()).unsqueeze(-1)
        code = _nearest(r.abs().clamp_max(448.0), grid) + 128 * torch.signbit(r)
        return code.to(torch.uint8), (s + 15).to(torch.uint8)
    blocks = y.view(y.shape[:-1] + (-1, 16))
    scale = _nearest((blocks.abs().amax(-1) / 6.0).float().double().clamp_max(448.0), grid)
    f = torch.tensor(grid, dtype=torch.float64, device=x.device)[scale].unsqueeze(-1)
    r = torch.where(f > 0, (blocks / f.clamp_min(1e-30)).float().double(), torch.zeros_like(blocks))
    code = _nearest(r.abs().clamp_max(6.0), [0, 0.5, 1, 1.5, 2, 3, 4, 6]) + 8 * torch.signbit(r)
    code = code.view(y.shape).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    fmt, page, H, D = case["fmt"], case["page"], case["kv_heads"], case["dim"]
    lens, counts = _lens(case), _counts(case)
    table = s["table"].cpu().long()
    dev = s["table"].device

    def where(b, first, n):
        p = torch.arange(first, first + n)
        return table[b, p // page].to(dev), (p % page).to(dev)

    def take(part, at):
        pg, off = at
        return part["codes"][pg, :, off], None if part["scales"] is None else part["scales"][pg, :, off]

    def put(part, at, codes, scales):
        pg, off = at
        part["codes"][pg, :, off] = codes
        if scales is not None:
            part["scales"][pg, :, off] = scales

    if case["op"] != "attend":
        first, outs = 0, ([], [])
        path = s["path"].cpu().tolist() if case["op"] == "accept" else None
        for b, (length, t) in enumerate(zip(lens, counts)):
            for name, new, out in (("k", "new_k", outs[0]), ("v", "new_v", outs[1])):
                at = where(b, length, t)
                if case["op"] == "append":
                    put(s[name], at, *_pack64(s[new][first:first + t], fmt, s[name]["g"]))
                elif case["op"] == "accept":
                    chosen = path[first:first + (t + 1) // 2]
                    codes, scales = take(s[name], at)
                    put(s[name], where(b, length, len(chosen)), codes[chosen], None if scales is None else scales[chosen])
                out.append(_decode64(*take(s[name], at), fmt, s[name]["g"]))
            first += t
        if case["op"] == "read" or fmt == "nvfp4":
            outs = [torch.cat(outs[0]), torch.cat(outs[1])]
        elif fmt == "bf16":
            outs = [s["k"]["codes"].double(), s["v"]["codes"].double()]
        else:
            unit = torch.full((1,), 15, dtype=torch.uint8, device=dev)
            outs = [_decode64(s["k"]["codes"], unit, fmt, 1.0), s["k"]["scales"],
                    _decode64(s["v"]["codes"], unit, fmt, 1.0), s["v"]["scales"]]
        return outs + [s["lens"] + s["kept"]] if case["op"] == "accept" else outs
    out = torch.zeros((s["total"], case["heads"], D), dtype=torch.float64, device=dev)
    lse = torch.full((s["total"], case["heads"]), -math.inf, dtype=torch.float64, device=dev)
    G, first = case["heads"] // H, 0
    for b, (length, t) in enumerate(zip(lens, counts)):
        k = _decode64(*take(s["k"], where(b, 0, length + t)), fmt, s["k"]["g"])
        v = _decode64(*take(s["v"], where(b, 0, length + t)), fmt, s["v"]["g"])
        bits = s["mask"][first:first + t].cpu().tolist()
        seen = torch.ones((t, length + t), dtype=torch.bool)
        for i in range(t):
            seen[i, length:] = torch.tensor([bool((bits[i] >> j) & 1) for j in range(t)])
        for h in range(H):
            q = s["q"][first:first + t, h * G:(h + 1) * G].double()                  # [t, G, D]
            z = (q.reshape(t * G, D) @ k[:, h].T).view(t, G, -1) * D ** -0.5
            z = torch.where(seen.to(dev)[:, None], z, -math.inf)
            sums = torch.logsumexp(z, -1)
            w = torch.exp(z - torch.where(sums > -math.inf, sums, 0.0)[..., None])
            out[first:first + t, h * G:(h + 1) * G] = (w.view(t * G, -1) @ v[:, h]).view(t, G, D)
            lse[first:first + t, h * G:(h + 1) * G] = sums
        first += t
    return [out, lse] if case["lse"] else [out]
