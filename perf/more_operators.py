"""Cases of the operators that keep long contexts in less memory: the latent cache held in 4 bits
(insert, gather, attention), latent attention with a sliding window and first tokens that stay
visible, and the paged caches' bookkeeping (free and grow, fork, compact). Each has a plain form
in elementary torch operations, which also runs where the library is not built, and an exact form
in 64 bits."""
import math

import torch

own = False

BLOCK = 256                       # tokens of one page
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
BASE = 10000.0
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
GROUP = 16                        # latent values that share a block scale


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a few short prompts enter a 4-bit cache and their rows are read back for the
        # projections of the expanded form: latency
        dict(name="q4_prompt_short", op="prompt", dtype="bf16", latent=512, rope=64, seqs=5,
             len_lo=3, len_hi=900, new_lo=1, new_hi=700, layout="pairs"),
        # ragged prompt chunks behind long prefixes, every cached row read back
        dict(name="q4_prompt_long", op="prompt", dtype="bf16", latent=512, rope=64, seqs=6,
             len_lo=9000, len_hi=130000, new_lo=700, new_hi=8192, layout="half"),
        # the smallest decode step of the fp32 layer on a 4-bit cache
        dict(name="q4_tiny_fp32", op="attn", cache="fp4", dtype="fp32", heads=8, latent=128,
             rope=32, seqs=3, len_lo=5, len_hi=1024, new_lo=1, new_hi=1),
        # the decode batch of the library's headline, 64 heads, from 4 bits
        dict(name="q4_decode", op="attn", cache="fp4", dtype="bf16", heads=64, latent=512, rope=64,
             seqs=32, len_lo=32768, len_hi=32768, new_lo=1, new_hi=1),
        # mixed decode lengths, 128 heads
        dict(name="q4_mixed", op="attn", cache="fp4", dtype="bf16", heads=128, latent=512, rope=64,
             seqs=16, len_lo=4096, len_hi=131072, new_lo=1, new_hi=1),
        # chunks of drafted or newly arrived tokens over cached contexts, few heads
        dict(name="q4_chunk", op="attn", cache="fp4", dtype="bf16", heads=16, latent=512, rope=64,
             seqs=7, len_lo=900, len_hi=21000, new_lo=2, new_hi=130),
        # the smallest windowed decode, fp32
        dict(name="window_tiny_fp32", op="attn", cache="plain", dtype="fp32", heads=8, latent=128,
             rope=32, seqs=3, len_lo=5, len_hi=1024, new_lo=1, new_hi=1, window=128, sinks=4),
        # long contexts of which only the sinks' and the window's pages are kept
        dict(name="window_decode", op="attn", cache="plain", dtype="bf16", heads=64, latent=512,
             rope=64, seqs=64, len_lo=9000, len_hi=1 << 20, new_lo=1, new_hi=1, window=4096,
             sinks=4),
        # prompt chunks under a short window, 4-bit cache
        dict(name="window_chunk", op="attn", cache="fp4", dtype="bf16", heads=16, latent=512,
             rope=64, seqs=4, len_lo=3000, len_hi=60000, new_lo=200, new_hi=2100, window=1024,
             sinks=130),
        # sequences end and others take their rows of the block table: latency
        dict(name="pages_turnover", op="turnover", seqs=64, blocks=512, pages=16384, share=0.25),
        # a prompt's children (beams, samples): full pages shared, the cut page copied
        dict(name="pages_fork", op="fork", seqs=64, blocks=40, parents=3, children=45, pages=1024,
             plain=4, packed=4),
        # a fragmented pool is drawn together
        dict(name="pages_compact", op="compact", seqs=48, blocks=32, pages=1500, plain=4, packed=2,
             share=0.3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["prompt", "attn", "attn", "attn", "window", "window", "turnover", "fork",
                     "compact"])
    if op == "prompt":
        new = _log(rng, 1, 4000)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), latent=512, rope=64,
                    seqs=rng.randint(1, 8), len_lo=new, len_hi=_log(rng, 8192, 60000),
                    new_lo=max(1, new // 3), new_hi=new, layout=rng.choice(["pairs", "half"]))
    if op == "turnover":
        blocks = _log(rng, 3, 512)
        return dict(op=op, seqs=rng.randint(2, 200), blocks=blocks, pages=_log(rng, 700, 30000),
                    share=rng.choice([0.1, 0.3, 0.8]))
    if op == "fork":
        children = rng.randint(1, 40)
        return dict(op=op, seqs=children + rng.randint(1, 9), blocks=rng.randint(1, 60),
                    parents=1, children=children, pages=rng.randint(600, 1100),
                    plain=rng.randint(0, 3), packed=rng.randint(1, 4))
    if op == "compact":
        return dict(op=op, seqs=rng.randint(1, 40), blocks=rng.randint(2, 30),
                    pages=rng.randint(90, 1200), plain=rng.randint(0, 3),
                    packed=rng.randint(1, 3), share=rng.choice([0.1, 0.4, 0.9]))
    more, cache = {}, "fp4"
    if op == "window":
        more = dict(window=_log(rng, 1, 6000), sinks=rng.choice([0, 1, 4, 64, 300]))
        cache = rng.choice(["plain", "fp4"])
    if rng.random() < 0.2:                           # the small fp32 layer
        new = _log(rng, 1, 16)
        return dict(op="attn", cache=cache, dtype="fp32", heads=rng.randint(1, 8), latent=128,
                    rope=32, seqs=rng.randint(1, 4), len_lo=new, len_hi=_log(rng, 30, 1024),
                    new_lo=1, new_hi=new, **more)
    heads = rng.choice([1, 5, 8, 16, 24, 32, 40, 64, 96, 128])
    if rng.random() < 0.6:                           # decode
        hi = _log(rng, 20, 24000)
        return dict(op="attn", cache=cache, dtype="bf16", heads=heads, latent=512, rope=64,
                    seqs=_log(rng, 1, 40), len_lo=max(1, hi // rng.randint(1, 16)), len_hi=hi,
                    new_lo=1, new_hi=1, **more)
    new, hi = _log(rng, 2, 150), _log(rng, 300, 16000)
    return dict(op="attn", cache=cache, dtype="bf16", heads=heads, latent=512, rope=64,
                seqs=rng.randint(1, 6), len_lo=max(new, hi // 10), len_hi=max(new, hi), new_lo=1,
                new_hi=new, **more)


def _spread(n, lo, hi, shift=0.0):
    """n whole numbers spread over [lo, hi], evenly in their logarithm, in a mixed order."""
    u = [((b + 1) * 0.6180339887498949 + shift) % 1.0 for b in range(n)]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** x)))) for x in u]


def _lengths(case):
    """(whole lengths, new tokens) of the case's sequences."""
    total = _spread(case["seqs"], case["len_lo"], case["len_hi"])
    new = _spread(case["seqs"], case["new_lo"], case["new_hi"], 0.4)
    return [max(t, n) for t, n in zip(total, new)], new


def _seen(case, p):
    """Keys that a token at position p sees."""
    w, s = case.get("window", p + 1), case.get("sinks", 0)
    first = max(0, p + 1 - w)
    return p + 1 - first + min(s, first)


def _read(case, t, n):
    """Cached rows that n new tokens of a sequence of t read at least once."""
    first = max(0, t - n + 1 - case.get("window", t))
    return t - first + min(case.get("sinks", 0), first)


def _row_bytes(case):
    c, r = case["latent"], case["rope"]
    if case.get("cache", "fp4") == "fp4":            # codes, rotary part, block scales, row scale
        return c // 2 + 2 * r + c // GROUP + 4
    return (c + r) * (2 if case["dtype"] == "bf16" else 4)


def work(case):
    if case["op"] == "turnover":
        # the table and the counts are read, what changes is written
        freed, _ = _turnover(case)
        return {"bytes": 4 * (case["seqs"] * case["blocks"] + case["pages"] + 8 * sum(freed)),
                "flops": case["pages"]}
    if case["op"] == "fork":
        _, length, _ = _family(case)
        rows = sum(n % BLOCK for n in length)
        moved = rows * (case["plain"] * 1152 + case["packed"] * 420)
        return {"bytes": 2 * moved + 4 * (case["pages"] + 4 * sum(-(-n // BLOCK) for n in length)),
                "flops": case["pages"]}
    if case["op"] == "compact":
        # a page at or behind the number of used ones moves if it is used: a share 1 - share does
        used = int(case["pages"] * (1 - case["share"]))
        moved = (case["pages"] - used) * (1 - case["share"])
        page = BLOCK * (case["plain"] * 1152 + case["packed"] * 420)
        return {"bytes": 2 * moved * page + 8 * (case["pages"] + case["seqs"] * case["blocks"]),
                "flops": case["pages"]}
    es = 2 if case["dtype"] == "bf16" else 4
    total, new = _lengths(case)
    w = case["latent"] + case["rope"]
    put = sum(new) * (w * es + _row_bytes(case))
    if case["op"] == "prompt":
        return {"bytes": put + sum(total) * (_row_bytes(case) + w * es),
                "flops": sum(new) * 12 * w + sum(total) * 2 * w}
    h, c = case["heads"], case["latent"]
    pairs = sum(_seen(case, p) for t, n in zip(total, new) for p in range(t - n, t))
    rows = sum(_read(case, t, n) for t, n in zip(total, new))
    return {"bytes": put + rows * _row_bytes(case) + sum(new) * h * (w + c) * es,
            "flops": 2 * pairs * h * (w + c)}


# ------------------------------------------------------------------------------ inputs
def _turnover(case):
    """(blocks that each row of the table gives back and takes again, blocks that it keeps)."""
    n, blocks = case["seqs"], case["blocks"]
    have = _spread(n, 1, blocks)
    most = int(case["pages"] * 0.9)
    if sum(have) > most:                             # the pool holds what the table names
        have = [max(1, h * most // (sum(have) + n)) for h in have]
    if sum(have) > most:
        have = [1 if b < most else 0 for b in range(n)]
    goes = [((b + 1) * 0.7548776662466927) % 1.0 < case["share"] for b in range(n)]
    return [h if g else 0 for h, g in zip(have, goes)], [0 if g else h for h, g in zip(have, goes)]


def _family(case):
    """(parent of each child, positions that it takes over, blocks of each parent)."""
    parents = [b % case["parents"] for b in range(case["children"])]
    length = _spread(case["children"], 1, case["blocks"] * BLOCK)
    return parents, length, [case["blocks"]] * case["parents"]


def _rand(g, dt, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dt)


def _pools(case, g):
    """The layers' pools: bf16 latent rows and 4-bit ones (any bytes: pages are moved as they
    are), 512 + 64 values a token."""
    rows = case["pages"] * BLOCK
    plain = [_rand(g, torch.bfloat16, rows, 576) for _ in range(case["plain"])]
    packed = [(torch.randint(0, 256, (rows, 416), generator=g, device="cuda", dtype=torch.uint8),
               torch.rand(rows, generator=g, device="cuda")) for _ in range(case["packed"])]
    return plain, packed


def _blocks(rows, blocks, g, pages):
    """A block table whose row b holds rows[b] blocks on shuffled pages, and the pages' counts."""
    have = torch.tensor(rows, device="cuda")
    at = torch.arange(blocks, device="cuda")[None] < have[:, None]
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(rows), blocks), -1, dtype=torch.int32, device="cuda")
    bt[at] = perm[:sum(rows)]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[perm[:sum(rows)].long()] = 1
    return bt, refs


def _page_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"], "case": case}

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device="cuda")
    if case["op"] == "turnover":
        freed, kept = _turnover(case)
        have = [a + b for a, b in zip(freed, kept)]
        s["bt"], s["refs"] = _blocks(have, case["blocks"], g, case["pages"])
        s["first"], s["last"] = ints([0] * len(have)), ints(freed)
        return s
    s["plain"], s["packed"] = _pools(case, g)
    if case["op"] == "fork":
        parents, length, have = _family(case)
        rows = have + [0] * (case["seqs"] - len(have))
        s["bt"], s["refs"] = _blocks(rows, case["blocks"] + 1, g, case["pages"])
        k = case["seqs"] - case["children"]
        s["src"], s["dst"] = ints(parents), ints(list(range(k, case["seqs"])))
        s["length"] = ints(length, torch.int64)
        # the children's rows are given back before they are forked again
        s["first"] = ints([0] * case["seqs"])
        s["last"] = ints([case["blocks"] + 1 if b >= k else 0 for b in range(case["seqs"])])
        return s
    # fragments: a share of the pool is free, spread all over it
    used = torch.rand(case["pages"], generator=g, device="cuda") >= case["share"]
    refs = used.to(torch.int32)
    cells = case["seqs"] * case["blocks"]
    order = torch.randperm(case["pages"], generator=g, device="cuda")
    bt = torch.full((cells,), -1, dtype=torch.int32, device="cuda")
    n = min(cells, case["pages"])
    named = torch.where(used[order[:n]], order[:n], torch.full_like(order[:n], -1)).to(torch.int32)
    bt[torch.randperm(cells, generator=g, device="cuda")[:n]] = named
    s["bt0"], s["refs0"] = bt.view(case["seqs"], case["blocks"]), refs
    s["bt"], s["refs"] = s["bt0"].clone(), refs.clone()
    return s


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    if case["op"] in ("turnover", "fork", "compact"):
        return _page_inputs(case, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]
    s = {"op": case["op"], "case": case, "fp4": case.get("cache", "fp4") == "fp4"}
    total, new = _lengths(case)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["total"], s["new"], s["cu_host"] = total, new, cu
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["start"] = torch.tensor([t - n for t, n in zip(total, new)], dtype=torch.int64, device="cuda")
    w = case["latent"] + case["rope"]
    # the blocks that a sequence still needs: the sinks' and those from its window on
    need = torch.zeros(len(total), max(-(-t // BLOCK) for t in total), dtype=torch.bool)
    for b, (t, n) in enumerate(zip(total, new)):
        first = max(0, t - n + 1 - case.get("window", t))
        need[b, first // BLOCK:-(-t // BLOCK)] = True
        need[b, :-(-min(case.get("sinks", 0), t) // BLOCK)] = True
    need = need.cuda()
    pages = int(need.sum())
    s["bt"] = torch.full(need.shape, -1, dtype=torch.int32, device="cuda")
    s["bt"][need] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["x"] = _rand(g, dt, cu[-1], w)                 # the down-projection's output
    s["gamma"] = 1 + 0.1 * torch.randn(case["latent"], generator=g, device="cuda")
    if s["fp4"]:
        rows = torch.randn(pages * BLOCK, w, generator=g, device="cuda")
        s["pool"], s["scale"] = _encode(rows[:, :case["latent"]], rows[:, case["latent"]:], None)
    else:
        s["pool"], s["scale"] = _rand(g, dt, pages * BLOCK, w), None
    if case["op"] == "prompt":
        tot = torch.tensor([0] + total, device="cuda").cumsum(0)
        s["cu_rows"] = tot.to(torch.int32)
        s["zeros"] = torch.zeros(len(total), dtype=torch.int64, device="cuda")
        s["rows"] = sum(total)
    else:
        s["q"] = _rand(g, dt, cu[-1], case["heads"], w)
        s["softmax"] = (128 + case["rope"]) ** -0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import compressed_sparse_long_gb300 as v4a
    from compressed_sparse_long_gb300.layer import PagedPool
    if case["op"] in ("turnover", "fork", "compact"):
        from compressed_sparse_long_gb300.pages import PageTable
        pools = [PagedPool(d, None, s["bt"], BLOCK) for d in s.get("plain", [])]
        pools += [PagedPool(d, e, s["bt"], BLOCK) for d, e in s.get("packed", [])]
        s["table"] = PageTable(pools, s["bt"], s["refs"])
        return s
    from compressed_sparse_long_gb300.latent import LatentLayer
    layout = v4a.ROPE_HALF if case.get("layout") == "half" else v4a.ROPE_INTERLEAVED
    cfg = v4a.latent_cfg(v4a.BF16 if case["dtype"] == "bf16" else v4a.FP32, case.get("heads", 1),
                         case["latent"], v4a.rope_cfg(case["rope"], layout=layout, base=BASE),
                         rms_eps=EPS, cache_format=v4a.LATENT_FP4 if s["fp4"] else v4a.LATENT_PLAIN)
    s["layer"] = LatentLayer(cfg, PagedPool(s["pool"], s["scale"], s["bt"], BLOCK), gamma=s["gamma"])
    s["max_pos"] = max(s["total"]) - 1
    return s


# -------------------------------------------------------------------------- plain forms
def _encode(z, k, r):
    """4-bit rows of values r z (r: one factor a row, or None) and rotary parts k, both fp32:
    (bytes [codes | rotary part in f16 | block scales in e4m3 | up to 16 bytes], row scales)."""
    n, c = z.shape
    if r is None:
        r = torch.ones(n, 1, device=z.device)
    u = z.abs().amax(1, keepdim=True) * (1.0 / 2688.0)
    scale = r * u
    least = (k.abs().amax(1, keepdim=True) * (1.0 / 32768.0)).clamp_min(2.0 ** -100)
    small = scale < least
    u, scale = torch.where(small, least / r, u), torch.where(small, least, scale)
    t = (z * (1.0 / u)).view(n, c // GROUP, GROUP)
    block = (t.abs().amax(2) * (1.0 / 6.0)).to(torch.float8_e4m3fn)
    b = block.float()[..., None]
    t = torch.where(b > 0, t * (1.0 / b), torch.zeros_like(t))
    a = t.abs()
    code = sum((a > m if up else a >= m).to(torch.uint8) for m, up in
               ((0.25, 1), (0.75, 0), (1.25, 1), (1.75, 0), (2.5, 1), (3.5, 0), (5.0, 1)))
    code = (code + 8 * (t < 0).to(torch.uint8)).view(n, c)
    code = code[:, 0::2] + 16 * code[:, 1::2]
    half = (k * (1.0 / scale)).half().view(torch.uint8)
    raw = torch.cat([code, half, block.view(torch.uint8)], 1)
    pad = torch.zeros(n, -raw.shape[1] % 16, dtype=torch.uint8, device=z.device)
    return torch.cat([raw, pad], 1), scale[:, 0].contiguous()


def _decode(raw, scale, c, r):
    """Values of 4-bit rows, fp32."""
    table = torch.tensor(LEVELS + [-v for v in LEVELS], device=raw.device)
    lead = raw.shape[:-1]
    code = torch.stack([raw[..., :c // 2] & 15, raw[..., :c // 2] >> 4], -1).flatten(-2)
    block = raw[..., c // 2 + 2 * r:c // 2 + 2 * r + c // GROUP].contiguous().view(torch.float8_e4m3fn).float()
    lat = table[code.int()].view(*lead, c // GROUP, GROUP) * block[..., None]
    pe = raw[..., c // 2:c // 2 + 2 * r].contiguous().view(torch.float16).float()
    return torch.cat([lat.flatten(-2), pe], -1) * scale[..., None]


def _rotate(x, pos, layout):
    """x [n, d] fp32 rotated at pos [n]; the angles in 64 bits."""
    half = x.shape[-1] // 2
    rate = BASE ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    ang = pos.double()[:, None] * rate
    c, s = ang.cos().float(), ang.sin().float()
    a, b = (x[..., :half], x[..., half:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    y0, y1 = a * c - b * s, a * s + b * c
    return torch.cat([y0, y1], -1) if layout == "half" else torch.stack([y0, y1], -1).flatten(-2)


def _of_token(cu, start, n):
    """(sequence, position, place in its sequence) of every row of a packed batch."""
    cu = cu.long()
    seq = torch.repeat_interleave(cu.diff(), output_size=n)
    at = torch.arange(n, device="cuda") - cu[seq]
    return seq, start[seq] + at, at


def _slots(s, seq, pos):
    """Pool rows of positions (of page 0 where a block has no page: those are masked)."""
    return s["bt"][seq, pos // BLOCK].long().clamp_min(0) * BLOCK + pos % BLOCK


def _plain_insert(s, case):
    x, c = s["x"].float(), case["latent"]
    seq, pos, _ = _of_token(s["cu"], s["start"], s["cu_host"][-1])
    z = x[:, :c] * s["gamma"]
    r = torch.rsqrt(x[:, :c].double().square().mean(-1, keepdim=True) + EPS).float()
    pe = _rotate(x[:, c:], pos, case.get("layout", "pairs"))
    slot = _slots(s, seq, pos)
    if s["fp4"]:
        s["pool"][slot], s["scale"][slot] = _encode(z, pe, r)
    else:
        s["pool"][slot] = torch.cat([z * r, pe], -1).to(s["pool"].dtype)


def _values(s, slot):
    if s["fp4"]:
        return _decode(s["pool"][slot], s["scale"][slot], s["case"]["latent"], s["case"]["rope"])
    return s["pool"][slot].float()


def _plain_attn(s, case):
    """Every sequence at once, its new tokens and keys padded to the longest."""
    h, c, n_seq, most = case["heads"], case["latent"], len(s["total"]), max(s["new"])
    window, sinks = case.get("window"), case.get("sinks", 0)
    total = torch.tensor(s["total"], device="cuda")
    if window is None:
        key = torch.arange(max(s["total"]), device="cuda").expand(n_seq, -1)
        there = key < total[:, None]
    else:                                            # the sinks, then what any token's window holds
        first = (s["start"] + 1 - window).clamp_min(sinks)
        span = min(window - 1 + most, max(s["total"]))
        key = torch.cat([torch.arange(sinks, device="cuda").expand(n_seq, -1),
                         first[:, None] + torch.arange(span, device="cuda")], 1)
        there = key < total[:, None]
    key = torch.where(there, key, torch.zeros_like(key))
    rows = _values(s, _slots(s, torch.arange(n_seq, device="cuda")[:, None], key))
    seq, pos, at = _of_token(s["cu"], s["start"], s["cu_host"][-1])
    q = torch.zeros(n_seq, most, h, rows.shape[-1], device="cuda")
    q[seq, at] = s["q"].float()
    sc = torch.bmm(q.flatten(1, 2), rows.transpose(1, 2)) * s["softmax"]
    sc = sc.view(n_seq, most, h, -1)
    last = s["start"][:, None] + torch.arange(most, device="cuda")
    see = there[:, None] & (key[:, None] <= last[..., None])
    if window is not None:
        see &= (key[:, None] > last[..., None] - window) | (key[:, None] < sinks)
    sc.masked_fill_(~see[:, :, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    o = torch.bmm(p.flatten(1, 2), rows[..., :c]) / p.sum(-1).flatten(1, 2)[..., None]
    return o.view(n_seq, most, h, c)[seq, at].to(s["q"].dtype)


def _plain_free(s):
    blk = torch.arange(s["bt"].shape[1], device="cuda")[None]
    goes = (blk >= s["first"][:, None]) & (blk < s["last"][:, None]) & (s["bt"] >= 0)
    s["refs"].index_add_(0, s["bt"].clamp_min(0).long().flatten(), -goes.int().flatten())
    s["bt"].masked_fill_(goes, -1)


def _lowest_free(refs):
    """Page number by rank among the free pages, lowest first."""
    free = refs == 0
    out = torch.zeros(refs.numel() + 1, dtype=torch.int64, device="cuda")
    page = torch.arange(refs.numel(), device="cuda")
    out.scatter_(0, torch.where(free, free.long().cumsum(0) - 1, refs.numel()), page)
    return out


def _plain_grow(s):
    blk = torch.arange(s["bt"].shape[1], device="cuda")[None]
    takes = (blk >= s["first"][:, None]) & (blk < s["last"][:, None]) & (s["bt"] < 0)
    rank = takes.flatten().long().cumsum(0).view(takes.shape) - 1
    page = _lowest_free(s["refs"])[rank.clamp(0, s["refs"].numel())]
    s["refs"].index_add_(0, torch.where(takes, page, 0).flatten(), takes.int().flatten())
    s["bt"].copy_(torch.where(takes, page.int(), s["bt"]))


def _plain_fork(s):
    length, src, dst = s["length"], s["src"].long(), s["dst"].long()
    blk = torch.arange(s["bt"].shape[1], device="cuda")[None]
    whole, cut = length // BLOCK, length % BLOCK
    old = s["bt"][src]
    shared = (blk < whole[:, None]) & (old >= 0)
    s["refs"].index_add_(0, old.clamp_min(0).long().flatten(), shared.int().flatten())
    part = cut > 0
    page = _lowest_free(s["refs"])[(part.long().cumsum(0) - 1).clamp_min(0)]
    s["refs"].index_add_(0, torch.where(part, page, 0), part.int())
    new = torch.where(shared, old, torch.full_like(old, -1))
    new = torch.where((blk == whole[:, None]) & part[:, None], page[:, None].int(), new)
    s["bt"][dst] = new
    row = torch.arange(BLOCK, device="cuda")[None]
    source = old.gather(1, whole.clamp_max(old.shape[1] - 1)[:, None]).long() * BLOCK + row
    move = row < cut[:, None]
    a, b = source[move], (page[:, None] * BLOCK + row)[move]
    pairs = list(s["plain"]) + [t for p in s["packed"] for t in p]
    [t.index_copy_(0, b, t[a]) for t in pairs]


def _plain_compact(s):
    used = s["refs"] > 0
    count, page = used.sum(), torch.arange(s["refs"].numel(), device="cuda")
    high, low = used & (page >= count), ~used & (page < count)
    a, b = page[high], page[low]                     # as many of one as of the other
    where = page.clone()
    where[a] = b
    s["bt"].copy_(torch.where(s["bt"] >= 0, where[s["bt"].clamp_min(0).long()].int(), s["bt"]))
    s["refs"][b] = s["refs"][a]
    s["refs"][a] = 0
    pairs = list(s["plain"]) + [t for p in s["packed"] for t in p]
    [t.view(page.numel(), -1).index_copy_(0, b, t.view(page.numel(), -1)[a]) for t in pairs]
    return count.to(torch.int32).view(1)


def _written(s):
    """What an insert changes, as far as it is numbers: the row scales of a 4-bit pool, a plain one."""
    return s["scale"] if s["fp4"] else s["pool"]


def _page_outputs(s, *more):
    return [s["bt"], s["refs"], *more, s.get("plain", []), s.get("packed", [])]


def _plain(s, case):
    if s["op"] == "turnover":
        _plain_free(s)
        _plain_grow(s)
        return _page_outputs(s)
    if s["op"] == "fork":
        _plain_free(s)
        _plain_fork(s)
        return _page_outputs(s)
    if s["op"] == "compact":
        s["bt"].copy_(s["bt0"])
        s["refs"].copy_(s["refs0"])
        return _page_outputs(s, _plain_compact(s))
    _plain_insert(s, case)
    if s["op"] == "prompt":
        seq, pos, _ = _of_token(s["cu_rows"], s["zeros"], s["rows"])
        return _values(s, _slots(s, seq, pos)).to(s["x"].dtype)
    return [_plain_attn(s, case), _written(s)]


def run(s):
    case = s["case"]
    if not own:
        return _plain(s, case)
    if s["op"] == "turnover":
        s["table"].free(s["first"], s["last"])
        s["table"].grow(s["first"], s["last"])
        return _page_outputs(s)
    if s["op"] == "fork":
        s["table"].free(s["first"], s["last"])
        s["table"].fork(s["src"], s["dst"], s["length"])
        return _page_outputs(s)
    if s["op"] == "compact":
        s["bt"].copy_(s["bt0"])
        s["refs"].copy_(s["refs0"])
        return _page_outputs(s, s["table"].compact())
    lay, c = s["layer"], case["latent"]
    lay.insert(s["cu"], s["start"], s["x"][:, :c], s["x"][:, c:])
    if s["op"] == "prompt":
        return lay.gather(s["cu_rows"], s["zeros"], s["rows"])
    out = lay.attention(s["cu"], s["start"], s["max_pos"], s["q"], window=case.get("window"),
                        sinks=case.get("sinks", 0))
    return [out, _written(s)]


# -------------------------------------------------------------------------- exact forms
def _exact_rows(x, k, factor):
    """What 4-bit rows of x * factor and rotary parts k stand for, in 64 bits: the nearest
    level of each value over its block's scale."""
    n, c = x.shape
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    top = x.abs().max(1).values * factor / 2688
    s = torch.maximum(top, torch.clamp(k.abs().max(1).values / 32768, min=2.0 ** -100))[:, None]
    y = (x * factor[:, None] / s).reshape(n, -1, GROUP)
    b = (y.abs().max(2).values / 6).to(torch.float32).to(torch.float8_e4m3fn).double()[..., None]
    v = torch.where(b > 0, y / b.clamp_min(1e-300), torch.zeros_like(y))
    near = torch.bucketize(v.abs(), (level[1:] + level[:-1]) / 2)
    v = torch.copysign(level[near], v) * b
    half = (k / s).to(torch.float16).double()
    return torch.cat([v.reshape(n, c), half], 1) * s


def _exact_pool(s, case):
    """(seq, position) -> cached values in 64 bits, the new tokens' among them."""
    c = case["latent"]
    if s["fp4"]:
        raw, r = s["pool"], case["rope"]
        level = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
        pool = torch.empty(raw.shape[0], c + r, dtype=torch.float64, device="cuda")
        for odd in (0, 1):
            nib = (raw[:, :c // 2].int() >> (4 * odd)) & 15
            pool[:, odd:c:2] = level[(nib & 7).long()] * (1 - 2 * (nib >> 3)).double()
        b = raw[:, c // 2 + 2 * r:c // 2 + 2 * r + c // GROUP].contiguous().view(torch.float8_e4m3fn).double()
        pool[:, :c] *= b.repeat_interleave(GROUP, 1)
        pool[:, c:] = raw[:, c // 2:c // 2 + 2 * r].contiguous().view(torch.float16).double()
        pool *= s["scale"].double()[:, None]
    else:
        pool = s["pool"].double()
    for b in range(case["seqs"]):
        lo, hi = s["cu_host"][b], s["cu_host"][b + 1]
        p = int(s["start"][b]) + torch.arange(hi - lo, device="cuda")
        x = s["x"][lo:hi].double()
        f = 1 / torch.sqrt((x[:, :c] ** 2).sum(1) / c + EPS)
        d = case["rope"]
        z = (torch.complex(x[:, c:c + d // 2].contiguous(), x[:, c + d // 2:].contiguous())
             if case.get("layout") == "half"
             else torch.view_as_complex(x[:, c:].reshape(-1, d // 2, 2).contiguous()))
        i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
        ang = p.double()[:, None] * torch.exp(-2.0 * i / d * math.log(BASE))
        z = z * torch.polar(torch.ones_like(ang), ang)
        pe = (torch.cat([z.real, z.imag], 1) if case.get("layout") == "half"
              else torch.view_as_real(z).flatten(1))
        lat = x[:, :c] * s["gamma"].double()
        slot = s["bt"][b].long()[p // BLOCK] * BLOCK + p % BLOCK
        if s["fp4"]:
            pool[slot] = _exact_rows(lat, pe, f)
        else:
            # attention reads the rows as they are stored
            pool[slot] = torch.cat([lat * f[:, None], pe], 1).to(s["pool"].dtype).double()
    return pool


def exact(case, seed):
    if case["op"] in ("turnover", "fork", "compact") or work(case)["flops"] > 2.5e12:
        return None
    s = _inputs(case, seed)
    pool = _exact_pool(s, case)
    outs = []
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        p = torch.arange(t, device="cuda")
        if case["op"] == "attn" and "window" in case:
            p = p[(p < case["sinks"]) | (p > t - n - case["window"])]
        keys = pool[s["bt"][b].long()[p // BLOCK] * BLOCK + p % BLOCK]
        if case["op"] == "prompt":
            outs.append(keys)
            continue
        lo = s["cu_host"][b]
        for i in range(0, n, 256):
            q = s["q"][lo + i:lo + min(n, i + 256)].double()
            at = (t - n + i + torch.arange(q.shape[0], device="cuda"))[:, None, None]
            logit = s["softmax"] * torch.einsum("thd,kd->thk", q, keys)
            hidden = p > at
            if "window" in case:
                hidden = hidden | ((p <= at - case["window"]) & (p >= case["sinks"]))
            logit = logit.masked_fill(hidden, -math.inf)
            wt = torch.exp(logit - torch.logsumexp(logit, 2, keepdim=True))
            outs.append(torch.einsum("thk,kd->thd", wt, keys[:, :case["latent"]]))
    return torch.cat(outs) if case["op"] == "prompt" else [torch.cat(outs), None]
