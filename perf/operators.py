"""Cases of the paged latent-attention operators: rotary positions, the latent cache's insert
and gather, and attention over it in the absorbed form (decode and chunks) and the expanded
form (prompts). Each has a plain form in elementary torch operations, which also runs where
the library is not built, and an exact form in 64 bits."""
import math

import torch

own = False

BLOCK = 256                       # tokens of one page
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ROPE = {"base": 10000.0, "factor": 8.0, "orig": 4096, "low": 1.0, "high": 32.0, "amp": 1.1}
EPS = 1e-6


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's query heads, 32 sequences of a 64-head layer: latency
        dict(name="rope_decode", op="rope", dtype="bf16", n=32, heads=64, dim=64, layout="pairs",
             scaling="none", inverse=False, span=32768),
        # the gradient of the rotation over a prompt chunk, long-context frequencies, fp32
        dict(name="rope_prompt_inverse", op="rope", dtype="fp32", n=8192, heads=64, dim=64,
             layout="half", scaling="yarn", inverse=True, span=1 << 20),
        # one decode step's new cache rows: latency
        dict(name="insert_decode", op="insert", dtype="bf16", latent=512, rope=64, seqs=32,
             len_lo=4096, len_hi=32768, new_lo=1, new_hi=1, layout="pairs", scaling="none"),
        # the new rows of ragged prompt chunks
        dict(name="insert_prompt", op="insert", dtype="bf16", latent=512, rope=64, seqs=6,
             len_lo=2000, len_hi=130000, new_lo=700, new_hi=8192, layout="half", scaling="yarn"),
        # the cached prefix of a few short prompts, for the expanded form
        dict(name="gather_short", op="gather", dtype="bf16", latent=512, rope=64, seqs=8,
             len_lo=1, len_hi=700),
        # the cached prefixes of long contexts
        dict(name="gather_long", op="gather", dtype="bf16", latent=512, rope=64, seqs=4,
             len_lo=9000, len_hi=122880),
        # the smallest decode of the fp32 layer: a few short sequences
        dict(name="attn_tiny_fp32", op="attn", dtype="fp32", heads=8, latent=128, rope=32,
             seqs=3, len_lo=5, len_hi=1024, new_lo=1, new_hi=1),
        # the decode batch of the library's headline: 32 sequences of 32,768 tokens, 64 heads
        dict(name="attn_decode", op="attn", dtype="bf16", heads=64, latent=512, rope=64,
             seqs=32, len_lo=32768, len_hi=32768, new_lo=1, new_hi=1),
        # mixed decode lengths, 128 heads
        dict(name="attn_mixed", op="attn", dtype="bf16", heads=128, latent=512, rope=64,
             seqs=16, len_lo=4096, len_hi=131072, new_lo=1, new_hi=1),
        # chunks of drafted or newly arrived tokens over cached contexts, few heads
        dict(name="attn_chunk", op="attn", dtype="bf16", heads=16, latent=512, rope=64, seqs=7,
             len_lo=900, len_hi=21000, new_lo=2, new_hi=130),
        # a prompt of 8,192 tokens
        dict(name="expanded_prompt", op="expanded", dtype="bf16", heads=64, nope=128, rope=64,
             v=128, seqs=1, len_lo=8192, len_hi=8192, new_lo=8192, new_hi=8192, causal=True),
        # ragged chunks whose prefixes were gathered from the cache
        dict(name="expanded_chunk", op="expanded", dtype="bf16", heads=16, nope=128, rope=64,
             v=128, seqs=5, len_lo=1500, len_hi=20000, new_lo=300, new_hi=2100, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["rope", "insert", "gather", "attn", "attn", "attn", "expanded", "expanded"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    layout = rng.choice(["pairs", "half"])
    scaling = rng.choice(["none", "linear", "parts", "yarn"])
    if op == "rope":
        n, heads = _log(rng, 1, 8192), rng.randint(1, 64)
        return dict(op=op, dtype=dtype, n=n, heads=heads, dim=rng.choice([32, 64]), layout=layout,
                    scaling=scaling, inverse=rng.random() < 0.5, span=_log(rng, 100, 1 << 20))
    if op == "insert":
        new = _log(rng, 1, 4000)
        return dict(op=op, dtype=dtype, latent=512, rope=64, seqs=rng.randint(1, 8), len_lo=new,
                    len_hi=_log(rng, 8192, 130000), new_lo=max(1, new // 3), new_hi=new,
                    layout=layout, scaling=scaling)
    if op == "gather":
        hi = _log(rng, 3, 90000)
        return dict(op=op, dtype=dtype, latent=512, rope=64, seqs=rng.randint(1, 4),
                    len_lo=max(1, hi // rng.randint(1, 30)), len_hi=hi)
    if op == "attn" and dtype == "fp32":
        new = _log(rng, 1, 16)
        return dict(op=op, dtype=dtype, heads=rng.randint(1, 8), latent=128, rope=32,
                    seqs=rng.randint(1, 4), len_lo=new, len_hi=_log(rng, 30, 1024), new_lo=1,
                    new_hi=new)
    heads = rng.choice([1, 5, 8, 16, 24, 32, 40, 64, 96, 128])
    if op == "attn":
        if rng.random() < 0.6:                       # decode
            seqs, hi = _log(rng, 1, 40), _log(rng, 20, 24000)
            return dict(op=op, dtype="bf16", heads=heads, latent=512, rope=64, seqs=seqs,
                        len_lo=max(1, hi // rng.randint(1, 16)), len_hi=hi, new_lo=1, new_hi=1)
        new, hi = _log(rng, 2, 150), _log(rng, 300, 16000)
        return dict(op=op, dtype="bf16", heads=heads, latent=512, rope=64, seqs=rng.randint(1, 6),
                    len_lo=max(new, hi // 10), len_hi=max(new, hi), new_lo=1, new_hi=new)
    new = _log(rng, 3, 4000)
    hi = _log(rng, new, 12000)
    return dict(op=op, dtype="bf16", heads=rng.choice([3, 8, 16, 20, 32]), nope=128, rope=64, v=128,
                seqs=rng.randint(1, 4), len_lo=max(new, hi // 5), len_hi=hi,
                new_lo=max(1, new // 4), new_hi=new, causal=rng.random() < 0.8)


def _spread(n, lo, hi, shift=0.0):
    """n whole numbers spread over [lo, hi], evenly in their logarithm, in a mixed order."""
    out = []
    for b in range(n):
        u = ((b + 1) * 0.6180339887498949 + shift) % 1.0
        out.append(max(lo, min(hi, int(round(lo * (hi / lo) ** u)))))
    return out


def _lengths(case):
    """(whole lengths, new tokens) of the case's sequences."""
    total = _spread(case["seqs"], case["len_lo"], case["len_hi"])
    if "new_lo" not in case:
        return total, total
    new = _spread(case["seqs"], case["new_lo"], case["new_hi"], 0.4)
    return [max(t, n) for t, n in zip(total, new)], new


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        e = case["n"] * case["heads"] * case["dim"]
        return {"bytes": 2 * e * es + 8 * case["n"], "flops": 3 * e}
    total, new = _lengths(case)
    if case["op"] in ("insert", "gather"):
        w = case["latent"] + case["rope"]
        norm = 4 * w if case["op"] == "insert" else 0
        return {"bytes": sum(new) * 2 * w * es, "flops": sum(new) * norm}
    pairs = 0                                        # (query token, visible key) pairs
    for t, n in zip(total, new):
        pairs += n * t - (n * (n - 1) // 2 if case.get("causal", True) else 0)
    h = case["heads"]
    if case["op"] == "attn":
        c, w = case["latent"], case["latent"] + case["rope"]
        return {"bytes": (sum(total) * w + sum(new) * h * (w + c)) * es,
                "flops": 2 * pairs * h * (w + c)}
    dk, dv = case["nope"] + case["rope"], case["v"]
    return {"bytes": (sum(new) * h * (dk + dv) + sum(total) * (h * (case["nope"] + dv) + case["rope"])) * es,
            "flops": 2 * pairs * h * (dk + dv)}


# ------------------------------------------------------------------------------ inputs
def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    s = {"op": case["op"], "case": case}
    if case["op"] == "rope":
        n, h, d = case["n"], case["heads"], case["dim"]
        width = 576 if d == 64 else 160              # the rotated dims end a wider query head
        s["q"] = rand(n, h, width)
        s["pos"] = torch.randint(0, case["span"], (n,), generator=g, device="cuda")
        return s
    total, new = _lengths(case)
    cu, start = [0], []
    for t, n in zip(total, new):
        cu.append(cu[-1] + n)
        start.append(t - n)
    s["total"], s["new"], s["cu_host"], s["start_host"] = total, new, cu, start
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["start"] = torch.tensor(start, dtype=torch.int64, device="cuda")
    if case["op"] == "expanded":
        h = case["heads"]
        cuk = [0]
        for t in total:
            cuk.append(cuk[-1] + t)
        s["cuk_host"] = cuk
        s["cuk"] = torch.tensor(cuk, dtype=torch.int32, device="cuda")
        s["q"] = rand(cu[-1], h, case["nope"] + case["rope"])
        s["kv"] = rand(cuk[-1], h, case["nope"] + case["v"])   # one projection's output
        s["k_pe"] = rand(cuk[-1], case["rope"])
        return s
    w = case["latent"] + case["rope"]
    # block tables: logical blocks of a sequence on a shuffled pool; an insert needs only the
    # blocks that it writes, a reader all of them
    blocks = []
    for t, n in zip(total, new):
        first = (t - n) // BLOCK if case["op"] == "insert" else 0
        blocks.append((first, (t + BLOCK - 1) // BLOCK))
    pages = sum(b - a for a, b in blocks)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(total), max(b for _, b in blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, (a, b) in enumerate(blocks):
        bt[i, a:b] = perm[at:at + b - a]
        at += b - a
    s["bt"] = bt
    s["pool"] = rand(pages * BLOCK, w)
    if case["op"] == "insert":
        s["x"] = rand(cu[-1], w)                     # the down-projection's output
        s["gamma"] = 1 + 0.1 * torch.randn(case["latent"], generator=g, device="cuda")
    if case["op"] == "attn":
        s["q"] = rand(cu[-1], case["heads"], w)
        s["scale"] = (128 + case["rope"]) ** -0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import compressed_sparse_long_gb300 as v4a
    from compressed_sparse_long_gb300.latent import LatentLayer
    from compressed_sparse_long_gb300.layer import PagedPool
    layout = v4a.ROPE_HALF if case.get("layout") == "half" else v4a.ROPE_INTERLEAVED
    kinds = {"none": v4a.ROPE_SCALE_NONE, "linear": v4a.ROPE_SCALE_LINEAR,
             "parts": v4a.ROPE_SCALE_BY_PARTS, "yarn": v4a.ROPE_SCALE_YARN}
    scaling = case.get("scaling", "none")
    more = {} if scaling == "none" else {"factor": ROPE["factor"]}
    if scaling in ("parts", "yarn"):
        more.update(orig_max_pos=ROPE["orig"], low=ROPE["low"], high=ROPE["high"],
                    amplitude=ROPE["amp"])
    s["rope"] = v4a.rope_cfg(case.get("rope", case.get("dim")), layout=layout, base=ROPE["base"],
                             scaling=kinds[scaling], **more)
    if case["op"] == "rope":
        return s
    dtype = v4a.BF16 if case["dtype"] == "bf16" else v4a.FP32
    cfg = v4a.latent_cfg(dtype, case.get("heads", 1), case.get("latent", 512), s["rope"],
                         nope_dim=case.get("nope", 128), v_dim=case.get("v", 128), rms_eps=EPS)
    pool = PagedPool(s["pool"], None, s["bt"], BLOCK) if "pool" in s else None
    s["layer"] = LatentLayer(cfg, pool, gamma=s.get("gamma"))
    s["max_pos"] = max(s["total"]) - 1
    return s


# -------------------------------------------------------------------------- plain forms
def _frequencies(dim, scaling):
    """Turning rate of each pair (radians a position) and the factor on cos and sin."""
    base, f = ROPE["base"], ROPE["factor"]
    rate = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == "none":
        return rate, 1.0
    if scaling == "linear":
        return [r / f for r in rate], 1.0
    lo, hi, orig = ROPE["low"], ROPE["high"], ROPE["orig"]
    if scaling == "parts":
        keep = [(orig * r / (2 * math.pi) - lo) / (hi - lo) for r in rate]
    else:
        def pair_of(turns):
            return dim * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        a = max(math.floor(pair_of(hi)), 0)
        b = min(math.ceil(pair_of(lo)), dim - 1)
        keep = [1.0 - (i - a) / max(b - a, 1e-3) for i in range(dim // 2)]
    keep = [min(max(k, 0.0), 1.0) for k in keep]
    return [r * (k + (1 - k) / f) for r, k in zip(rate, keep)], ROPE["amp"]


def _rotate(x, pos, layout, scaling, inverse=False):
    """x [n, ..., d] fp32 rotated at pos [n]; the angles in 64 bits."""
    rate, amp = _frequencies(x.shape[-1], scaling)
    ang = pos.double()[:, None] * torch.tensor(rate, dtype=torch.float64, device=x.device)
    c, s = (amp * ang.cos()).float(), (amp * ang.sin()).float()
    if inverse:
        s = -s
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (x.shape[-1] // 2,)
    c, s = c.view(shape), s.view(shape)
    half = x.shape[-1] // 2
    a, b = (x[..., :half], x[..., half:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    y0, y1 = a * c - b * s, a * s + b * c
    if layout == "half":
        return torch.cat([y0, y1], -1)
    return torch.stack([y0, y1], -1).flatten(-2)


def _positions(s):
    """(sequence, position) of every new token."""
    n = s["cu_host"][-1]
    cu = s["cu"].long()
    seq = torch.repeat_interleave(cu.diff(), output_size=n)
    return seq, s["start"][seq] + torch.arange(n, device="cuda") - cu[seq]


def _rows(s, b, n):
    """The first n cached rows of sequence b."""
    pages = s["bt"][b, :(n + BLOCK - 1) // BLOCK].long()
    return s["pool"].view(-1, BLOCK, s["pool"].shape[1])[pages].flatten(0, 1)[:n]


def _softmax_rows(sc, mask):
    if mask is not None:
        sc = sc.masked_fill(~mask, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    return p, p.sum(-1, keepdim=True)


def _plain_attn(s, case):
    h, c = case["heads"], case["latent"]
    out = torch.empty(s["cu_host"][-1], h, c, dtype=s["q"].dtype, device="cuda")
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        keys = _rows(s, b, t).float()
        at = s["cu_host"][b]
        step = max(1, (1 << 28) // (h * t))
        for i in range(0, n, step):
            j = min(n, i + step)
            q = s["q"][at + i:at + j].float().flatten(0, 1)
            sc = (q @ keys.t()) * s["scale"]
            mask = None
            if n > 1:
                last = torch.arange(t - n + i, t - n + j, device="cuda").repeat_interleave(h)
                mask = torch.arange(t, device="cuda")[None, :] <= last[:, None]
            p, l = _softmax_rows(sc, mask)
            o = (p @ keys[:, :c]) / l
            out[at + i:at + j] = o.view(j - i, h, c).to(out.dtype)
    return out


def _plain_expanded(s, case):
    h, dn, dv = case["heads"], case["nope"], case["v"]
    scale = (dn + case["rope"]) ** -0.5
    out = torch.empty(s["cu_host"][-1], h, dv, dtype=s["q"].dtype, device="cuda")
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        qa, ka = s["cu_host"][b], s["cuk_host"][b]
        step = max(1, min(h, (1 << 29) // (n * t)))
        mask = None
        if case["causal"]:
            mask = (torch.arange(t, device="cuda")[None, :] <=
                    torch.arange(t - n, t, device="cuda")[:, None])
        pe = s["k_pe"][ka:ka + t].float()
        for i in range(0, h, step):
            q = s["q"][qa:qa + n, i:i + step].float().transpose(0, 1)
            kv = s["kv"][ka:ka + t, i:i + step].float().transpose(0, 1)
            sc = (q[..., :dn] @ kv[..., :dn].transpose(1, 2) + q[..., dn:] @ pe.t()) * scale
            p, l = _softmax_rows(sc, mask)
            out[qa:qa + n, i:i + step] = ((p @ kv[..., dn:]) / l).transpose(0, 1).to(out.dtype)
    return out


def _plain(s):
    case = s["case"]
    if s["op"] == "rope":
        x = s["q"][..., -case["dim"]:]
        return _rotate(x.float(), s["pos"], case["layout"], case["scaling"],
                       case["inverse"]).to(x.dtype)
    if s["op"] == "insert":
        x, c = s["x"].float(), case["latent"]
        lat = x[:, :c] * torch.rsqrt(x[:, :c].square().mean(-1, keepdim=True) + EPS) * s["gamma"]
        seq, pos = _positions(s)
        pe = _rotate(x[:, c:], pos, case["layout"], case["scaling"])
        slot = s["bt"][seq, pos // BLOCK].long() * BLOCK + pos % BLOCK
        s["pool"][slot] = torch.cat([lat, pe], -1).to(s["pool"].dtype)
        return s["pool"]
    if s["op"] == "gather":
        return torch.cat([_rows(s, b, t) for b, t in enumerate(s["total"])])
    return _plain_attn(s, case) if s["op"] == "attn" else _plain_expanded(s, case)


def run(s):
    if not own:
        return _plain(s)
    case = s["case"]
    if s["op"] == "rope":
        from compressed_sparse_long_gb300.latent import rope
        return rope(s["rope"], s["q"][..., -case["dim"]:], s["pos"], inverse=case["inverse"])
    lay = s["layer"]
    if s["op"] == "insert":
        c = case["latent"]
        lay.insert(s["cu"], s["start"], s["x"][:, :c], s["x"][:, c:])
        return s["pool"]
    if s["op"] == "gather":
        return lay.gather(s["cu"], s["start"], s["cu_host"][-1])
    if s["op"] == "attn":
        return lay.attention(s["cu"], s["start"], s["max_pos"], s["q"])
    dn = case["nope"]
    return lay.attention_expanded(s["cu"], s["cuk"], s["q"], s["kv"][..., :dn], s["k_pe"],
                                  s["kv"][..., dn:], causal=case["causal"])


# -------------------------------------------------------------------------- exact forms
def _exact_rotation(x, pos, case, inverse=False):
    """Complex form in 64 bits: a pair is one number, turned by exp(i pos theta)."""
    d = x.shape[-1]
    x = x.double()
    z = (torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous())
         if case["layout"] == "half"
         else torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous()))
    i = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    theta = torch.exp(-2.0 * i / d * math.log(ROPE["base"]))
    amp = 1.0
    if case["scaling"] == "linear":
        theta = theta / ROPE["factor"]
    elif case["scaling"] != "none":
        amp = ROPE["amp"]
        if case["scaling"] == "parts":
            turns = ROPE["orig"] * theta / (2 * math.pi)
            keep = ((turns - ROPE["low"]) / (ROPE["high"] - ROPE["low"])).clamp(0, 1)
        else:
            edge = [d / 2 * math.log(ROPE["orig"] / (2 * math.pi * t)) / math.log(ROPE["base"])
                    for t in (ROPE["high"], ROPE["low"])]
            first, last = max(0, math.floor(edge[0])), min(d - 1, math.ceil(edge[1]))
            keep = 1 - ((i - first) / max(last - first, 1e-3)).clamp(0, 1)
        theta = theta * keep + theta / ROPE["factor"] * (1 - keep)
    ang = pos.double().view(-1, *([1] * (x.dim() - 2)), 1) * theta
    z = z * torch.polar(torch.full_like(ang, amp), -ang if inverse else ang)
    if case["layout"] == "half":
        return torch.cat([z.real, z.imag], -1)
    return torch.view_as_real(z).flatten(-2)


def exact(case, seed):
    if work(case)["flops"] > 1.2e13:
        return None
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(s["q"][..., -case["dim"]:], s["pos"], case, case["inverse"])
    if case["op"] == "gather":
        out = []
        for b, t in enumerate(s["total"]):
            p = torch.arange(t, device="cuda")
            out.append(s["pool"][s["bt"][b].long()[p // BLOCK] * BLOCK + p % BLOCK].double())
        return torch.cat(out)
    if case["op"] == "insert":
        pool, c = s["pool"].double(), case["latent"]
        for b in range(case["seqs"]):
            lo, hi = s["cu_host"][b], s["cu_host"][b + 1]
            p = s["start_host"][b] + torch.arange(hi - lo, device="cuda")
            x = s["x"][lo:hi].double()
            norm = torch.sqrt((x[:, :c] ** 2).sum(1, keepdim=True) / c + EPS)
            slot = s["bt"][b].long()[p // BLOCK] * BLOCK + p % BLOCK
            pool[slot, :c] = x[:, :c] / norm * s["gamma"].double()
            pool[slot, c:] = _exact_rotation(x[:, c:], p, case)
        return pool
    outs = []
    for b in range(case["seqs"]):
        t, n, h = s["total"][b], s["new"][b], case["heads"]
        lo = s["cu_host"][b]
        keys = None
        if case["op"] == "attn":
            p = torch.arange(t, device="cuda")
            keys = s["pool"][s["bt"][b].long()[p // BLOCK] * BLOCK + p % BLOCK].double()
        per_seq = []
        for head in range(h) if n > 1 else [slice(0, h)]:
            q = s["q"][lo:lo + n, head].double().reshape(-1, s["q"].shape[-1])
            if case["op"] == "attn":
                k, v, scale = keys, keys[:, :case["latent"]], s["scale"]
            else:
                ka = s["cuk_host"][b]
                kv = s["kv"][ka:ka + t, head].double().reshape(t, -1, case["nope"] + case["v"])
                pe = s["k_pe"][ka:ka + t].double()
                scale = (case["nope"] + case["rope"]) ** -0.5
                if n == 1:                           # one query token: its heads one by one
                    per_seq.append(torch.stack([
                        torch.softmax(scale * (torch.cat([kv[:, g, :case["nope"]], pe], 1) @ q[g]), 0)
                        @ kv[:, g, case["nope"]:] for g in range(h)])[None])
                    continue
                k = torch.cat([kv[:, 0, :case["nope"]], pe], 1)
                v = kv[:, 0, case["nope"]:]
            part = []
            for i in range(0, q.shape[0], 4096):
                logit = scale * torch.einsum("rd,kd->rk", q[i:i + 4096], k)
                if n > 1 and case.get("causal", True):
                    row = torch.arange(i, i + logit.shape[0], device="cuda")[:, None] + (t - n)
                    logit = torch.where(torch.arange(t, device="cuda")[None] <= row, logit,
                                        torch.full_like(logit, -math.inf))
                part.append(torch.exp(logit - torch.logsumexp(logit, 1, keepdim=True)) @ v)
            o = torch.cat(part)
            per_seq.append(o.view(1, h, -1) if n == 1 else o.view(n, 1, -1))
        outs.append(torch.cat(per_seq, 1) if len(per_seq) > 1 else per_seq[0])
    return torch.cat(outs)
