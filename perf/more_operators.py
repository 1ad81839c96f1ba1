"""Cases of the operators that bring a prompt into a latent pool, with their plain forms in torch.

* ``rope``: one layer's projections made ready for attention: the latent key of each token normalised, its RoPE
  dims rotated, the row put into its slot of the pool (bf16, or the 4-bit format), and each query head normalised and rotated;
* ``prompt``: causal attention of whole prompts, or of their next chunks, over keys of 128 dims a head and 64 RoPE
  dims that all heads share, sequences packed one behind the other.

A row is 512 latent dims and 64 RoPE dims. The 4-bit row is 416 bytes: 512 e2m1 codes (two to a byte, the even dim in
the low four bits), 32 e4m3 scales (one to 16 dims), 64 RoPE dims in bf16.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DL, DR = 512, 64                    # latent dims, RoPE dims
DK = DL + DR
DN, DV = 128, 128                   # a head's own dims of a key, and of a value
BLOCK = 16                          # latent dims to a scale of the 4-bit row
CODE_BYTES, SCALES = DL // 2, DL // BLOCK
ROW = CODE_BYTES + SCALES + 2 * DR  # 416 bytes
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
MAX_POS = 131072


# ---------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step of 61 requests, 64 heads: the query heads' RoPE dims go behind the absorbed ones
        {"name": "rope_token", "op": "rope", "rows": 61, "heads": 64, "dim": 64, "width": 2112, "pool": "bf16", "norm": True, "halves": False, "skip": 0},
        # a step of 32 draft trees of 8 nodes into the 4-bit pool; the projection's rows are normalised already
        {"name": "rope_tree", "op": "rope", "rows": 256, "heads": 16, "dim": 64, "width": 576, "pool": "kv4", "norm": False, "halves": False, "skip": 0},
        # a prompt's chunk with norms of the latent rows and of the query heads
        {"name": "rope_prompt", "op": "rope", "rows": 16384, "heads": 64, "dim": 192, "width": 2112, "pool": "bf16", "norm": True, "halves": False, "skip": 0},
        # a 64k prompt's rows into the 4-bit pool, padding rows among them, no queries in the same call
        {"name": "rope_64k", "op": "rope", "rows": 65536, "heads": 0, "dim": 64, "width": 576, "pool": "kv4", "norm": False, "halves": True, "skip": 7},
        # an odd number of tokens, a few heads, pairs half a head apart
        {"name": "rope_odd", "op": "rope", "rows": 2111, "heads": 5, "dim": 192, "width": 584, "pool": "bf16", "norm": True, "halves": True, "skip": 19},
        # a short chat message, where latency counts
        {"name": "prompt_chat", "op": "prompt", "seqs": 1, "lo": 61, "hi": 61, "ctx": 0, "heads": 8, "group": 1, "causal": True},
        # the next message of a long chat: a few new tokens over all that went before
        {"name": "prompt_turn", "op": "prompt", "seqs": 1, "lo": 17, "hi": 17, "ctx": 16384, "heads": 64, "group": 1, "causal": True},
        # single new tokens of a batch over contexts of different lengths, four query heads to a key head
        {"name": "prompt_token", "op": "prompt", "seqs": 61, "lo": 1, "hi": 1, "ctx": 4096, "heads": 16, "group": 4, "causal": True},
        # prompts of different lengths packed into one call
        {"name": "prompt_pack", "op": "prompt", "seqs": 24, "lo": 61, "hi": 2048, "ctx": 0, "heads": 16, "group": 1, "causal": True},
        # the last chunk of a 64k prompt
        {"name": "prompt_chunk", "op": "prompt", "seqs": 1, "lo": 2048, "hi": 2048, "ctx": 63488, "heads": 8, "group": 1, "causal": True},
        # a prompt with all heads on one card
        {"name": "prompt_8k", "op": "prompt", "seqs": 1, "lo": 8192, "hi": 8192, "ctx": 0, "heads": 64, "group": 1, "causal": True},
        # a long prompt, the heads shared out over cards
        {"name": "prompt_32k", "op": "prompt", "seqs": 1, "lo": 32768, "hi": 32768, "ctx": 0, "heads": 8, "group": 1, "causal": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    if rng.random() < 0.4:
        pool = rng.choice(["bf16", "bf16", "kv4"])
        dim = rng.choice([64, 64, 128, 192, 192, 256, 72])
        heads = rng.choice([0, 8, 16, 64, rng.randint(1, 128)])
        rows = min(_log(rng, 1, 65536), (16384 * 64 * 192) // max(1, heads * max(dim, 192)))
        return {"op": "rope", "rows": rows, "heads": heads, "dim": dim, "width": rng.choice([576, 584, 2112]), "pool": pool,
                "norm": pool == "bf16" and rng.random() < 0.8, "halves": rng.random() < 0.4, "skip": rng.choice([0, 2, 19])}
    group = rng.choice([1, 1, 2, 4, 8])
    heads = group * max(1, rng.choice([8, 16, 64, rng.randint(1, 40)]) // group)
    seqs = rng.choice([1, _log(rng, 1, 64)])
    hi = rng.choice([_log(rng, 100, 32768), _log(rng, 1, 32768), _log(rng, 1, 64)])
    ctx = rng.choice([0, 0, _log(rng, 1, 100000)])
    causal = rng.random() < 0.9
    most = 8e9 if causal and not ctx else 4e9
    while seqs * hi * (hi + ctx) * heads > most or seqs * ctx * heads > 2e7:
        if ctx > hi:
            ctx //= 2
        else:
            hi = (hi + 1) // 2
    return {"op": "prompt", "seqs": seqs, "lo": rng.randint(max(1, hi // 30), hi), "hi": hi, "ctx": ctx, "heads": heads,
            "group": group, "causal": causal}


def lengths(case):
    """(new tokens, keys) of a case's sequences: spread over their logarithm from lo to hi, contexts from ctx / seqs to ctx."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    new = [hi if n == 1 else int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    return new, [m + case["ctx"] * (i + 1) // n for i, m in enumerate(new)]


def _kept(case):
    return case["rows"] - (case["rows"] // case["skip"] if case["skip"] else 0)


def work(case):
    if case["op"] == "rope":
        n, kept = case["rows"], _kept(case)
        out = 2 * DK if case["pool"] == "bf16" else ROW
        # rows in, normalised rows out, the kept ones into the pool, a table row, position and slot; query heads in and out
        b = n * (2 * DK + 2 * DK + 4 * 2 * (DR // 2) + 8) + kept * out + n * case["heads"] * 4 * case["dim"]
        if case["pool"] == "kv4":  # read back as values
            b += kept * ROW + n * (2 * DK + 4)
        return {"bytes": b, "flops": 0}
    new, keys = lengths(case)
    pairs = sum(m * (k - m) + m * (m + 1) // 2 if case["causal"] else m * k for m, k in zip(new, keys))
    h, hk = case["heads"], case["heads"] // case["group"]
    return {"bytes": sum(new) * h * (2 * (DN + DR) + 2 * DV + 4) + sum(keys) * (2 * hk * (DN + DV) + 2 * DR),
            "flops": 2 * pairs * h * (DN + DR + DV)}


# ------------------------------------------------------------------------------------------ the inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def _cos_sin():
    """float32 [MAX_POS, 64]: the cosines of a position's 32 angles, then their sines."""
    f = 10000.0 ** (-torch.arange(DR // 2, dtype=torch.float64, device=DEVICE) / (DR // 2))
    a = torch.arange(MAX_POS, dtype=torch.float64, device=DEVICE)[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=DEVICE, generator=g)

    if case["op"] == "rope":
        n, heads, dim = case["rows"], case["heads"], case["dim"]
        x = normal(n, case["width"])
        x[:, :DL] *= torch.linspace(0.3, 2.0, DL, device=DEVICE)
        slots = torch.randperm(n + n // 8 + 1, device=DEVICE, generator=g)[:n].to(torch.int32)
        if case["skip"]:
            slots[torch.arange(n, device=DEVICE) % case["skip"] == case["skip"] - 1] = -1
        if n < 4096:  # tokens of many requests
            pos = torch.randint(0, MAX_POS, (n,), device=DEVICE, generator=g, dtype=torch.int32)
        else:         # a prompt, from some token on
            pos = torch.arange(n, device=DEVICE, dtype=torch.int32) + seed % (MAX_POS - n)
        s = {"op": "rope", "rows": x.to(torch.bfloat16)[:, :DK], "slots": slots, "pos": pos, "table": _cos_sin(), "halves": case["halves"],
             "weight": (1.0 + 0.2 * normal(DL)).to(torch.bfloat16) if case["norm"] else None, "q": None, "q_weight": None, "q_out": None}
        many = n + n // 8 + 1
        if case["pool"] == "bf16":
            s["pool"] = torch.zeros(many, DK, dtype=torch.bfloat16, device=DEVICE)
        else:
            s["pool"] = torch.zeros(many, ROW, dtype=torch.uint8, device=DEVICE)
        if heads and dim == DR:  # the RoPE dims of whole heads, into the last dims of absorbed queries
            s["q"] = normal(n, heads, DN + DR).to(torch.bfloat16)[:, :, DN:]
            s["q_out"] = torch.zeros(n, heads, DK, dtype=torch.bfloat16, device=DEVICE)[:, :, DL:]
        elif heads:
            s["q"] = normal(n, heads, dim).to(torch.bfloat16)
            s["q_weight"] = (1.0 + 0.2 * normal(dim)).to(torch.bfloat16)
        return s
    new, keys = lengths(case)
    order = torch.randperm(len(new), device=DEVICE, generator=g).tolist()
    new, keys = [new[i] for i in order], [keys[i] for i in order]
    heads, hk = case["heads"], case["heads"] // case["group"]
    cu = lambda v: _ints([sum(v[:i]) for i in range(len(v) + 1)])
    kv = normal(sum(keys), hk, DN + DV).to(torch.bfloat16)  # one projection gives a head's key dims and its values
    rows = normal(sum(keys), DK).to(torch.bfloat16)
    return {"op": "prompt", "q": normal(sum(new), heads, DN + DR).to(torch.bfloat16), "k": kv[:, :, :DN], "v": kv[:, :, DN:],
            "k_rope": rows[:, DL:], "cu_q": cu(new), "cu_k": cu(keys), "max_q": max(new), "max_k": max(keys), "causal": case["causal"]}


# ------------------------------------------------------------------------------------- the plain forms

def _rotate(x, table, halves):
    """The last 64 dims of x [n, ..., d] (float32) turned by the angles of table [n, 64]."""
    shape = [x.shape[0]] + [1] * (x.dim() - 2) + [DR // 2]
    c, s = table[:, :DR // 2].view(shape), table[:, DR // 2:].view(shape)
    head, r = x[..., :-DR], x[..., -DR:]
    a, b = (r[..., :DR // 2], r[..., DR // 2:]) if halves else (r[..., 0::2], r[..., 1::2])
    a, b = a * c - b * s, b * c + a * s
    r = torch.cat([a, b], -1) if halves else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([head, r], -1)


def _normed(x, weight):
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _quantise(rows):
    """bf16 rows [n, 576] as 416-byte rows: a block's scale is its largest magnitude / 6 in e4m3, a code the nearest e2m1
    value of x / scale (ties to the even code)."""
    n = rows.shape[0]
    x = rows[:, :DL].float().view(n, SCALES, BLOCK)
    scale = (x.abs().amax(2, keepdim=True) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    y = torch.where(s > 0, x / s, 0.0)
    m = y.abs()
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int()
            + (m >= 3.5).int() + (m > 5.0).int()) + 8 * (y < 0).int()
    code = code.view(n, CODE_BYTES, 2).to(torch.uint8)
    rope = rows[:, DL:].contiguous().view(torch.uint8)
    return torch.cat([code[:, :, 0] | (code[:, :, 1] << 4), scale.view(n, SCALES).view(torch.uint8), rope], 1)


def _values(rows):
    """416-byte rows [n, 416] as float32 rows [n, 576]."""
    code = rows[:, :CODE_BYTES]
    code = torch.stack([code & 15, code >> 4], -1).flatten(1)
    e, m = (code >> 1) & 3, (code & 1).float()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.float() - 1))
    v = torch.where(code >= 8, -v, v)
    scale = rows[:, CODE_BYTES:CODE_BYTES + SCALES].contiguous().view(torch.float8_e4m3fn).float()
    v = (v.unflatten(1, (SCALES, BLOCK)) * scale[..., None]).flatten(1)
    return torch.cat([v, rows[:, CODE_BYTES + SCALES:].contiguous().view(torch.bfloat16).float()], 1)


def _plain_rope(s):
    x, table, slots = s["rows"].float(), s["table"][s["pos"].long()], s["slots"].long()
    y = _rotate(torch.cat([_normed(x[:, :DL], s["weight"]), x[:, DL:]], 1), table, s["halves"]).to(torch.bfloat16)
    kept = slots >= 0
    out = {"rows": y}
    if s["pool"].dtype == torch.bfloat16:
        s["pool"][slots[kept]] = y[kept]
        out["pool"] = s["pool"]
    else:
        s["pool"][slots[kept]] = _quantise(y[kept])
        out["pool"] = torch.where(kept[:, None], _values(s["pool"][slots.clamp(min=0)]), 0.0).to(torch.bfloat16)
    if s["q"] is not None:
        q = _rotate(_normed(s["q"].float(), s["q_weight"]), table, s["halves"]).to(torch.bfloat16)
        out["q"] = q if s["q_out"] is None else s["q_out"].copy_(q)
    return out


def _plain_prompt(s):
    q, cu_q, cu_k, max_q, max_k = s["q"].float(), s["cu_q"].long(), s["cu_k"].long(), s["max_q"], s["max_k"]
    seqs, heads, group = len(cu_q) - 1, q.shape[1], q.shape[1] // s["k"].shape[1]
    new, keys = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, t = torch.arange(max_q, device=q.device), torch.arange(max_k, device=q.device)
    qi = (cu_q[:-1, None] + i).clamp(max=q.shape[0] - 1)              # the padded batch's rows
    ki = (cu_k[:-1, None] + t).clamp(max=s["k"].shape[0] - 1)
    k = torch.cat([s["k"].float(), s["k_rope"].float()[:, None, :].expand(-1, s["k"].shape[1], -1)], 2)
    k = k[ki].repeat_interleave(group, 2).transpose(1, 2)              # [seqs, heads, max_k, 192]
    v = s["v"].float()[ki].repeat_interleave(group, 2).transpose(1, 2)
    seen = (t < keys[:, None])[:, None, :].expand(-1, max_q, -1)
    if s["causal"]:
        seen = seen & (t <= (i + (keys - new)[:, None])[:, :, None])
    x = torch.matmul(q[qi].transpose(1, 2), k.transpose(2, 3)).mul_(SCALE).masked_fill_(~seen[:, None], -math.inf)
    top = x.amax(3, keepdim=True)
    x.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    z = x.sum(3, keepdim=True)
    out = torch.matmul(x, v)
    out = torch.where(z > 0, out / z, 0.0).transpose(1, 2)              # [seqs, max_q, heads, 128]
    lse = (top + torch.log(z))[..., 0].transpose(1, 2)
    real = i < new[:, None]
    return {"out": out[real].to(torch.bfloat16), "lse": lse[real]}


def run(state):
    s = state
    if own:
        import speculative_decode_mla_gb300 as m
        if s["op"] == "rope":
            rows, q = m.rope_append(s["pool"], s["rows"], s["slots"], s["pos"], s["table"], weight=s["weight"], eps=EPS, q=s["q"],
                                    q_weight=s["q_weight"], q_out=s["q_out"], halves=s["halves"])
            pool = s["pool"] if s["pool"].dtype == torch.bfloat16 else m.kv4_gather(s["pool"], s["slots"])
            return {"rows": rows, "pool": pool} if q is None else {"rows": rows, "pool": pool, "q": q}
        out, lse = m.prompt_attn(s["q"], s["k"], s["k_rope"], s["v"], s["cu_q"], s["cu_k"], max_q_len=s["max_q"],
                                 max_k_len=s["max_k"], causal=s["causal"])
        return {"out": out, "lse": lse}
    return _plain_rope(s) if s["op"] == "rope" else _plain_prompt(s)


# ------------------------------------------------------------------------------ the definition in 64 bits

def _nearest(x, grid):
    """The nearest value of an ascending grid (even index at a tie) to each x >= 0, in float64."""
    i = torch.searchsorted(grid, x.contiguous(), right=True).clamp(1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 0))
    return torch.where(up, hi, lo)


def _complex_turn(r, table, halves):
    """RoPE dims r [n, ..., 64] in float64, their pairs taken as complex numbers and turned."""
    pairs = r.unflatten(-1, (2, DR // 2)).transpose(-1, -2) if halves else r.unflatten(-1, (DR // 2, 2))
    z = torch.view_as_complex(pairs.contiguous())
    w = torch.complex(table[:, :DR // 2].double(), table[:, DR // 2:].double())
    z = torch.view_as_real(z * (w if r.dim() == 2 else w[:, None]))
    return (z.transpose(-1, -2) if halves else z).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        table, x, slots = s["table"][s["pos"].long()], s["rows"].double(), s["slots"].long()
        lat = x[:, :DL]
        if s["weight"] is not None:
            lat = lat / (lat.pow(2).sum(1, keepdim=True) / DL + EPS).sqrt() * s["weight"].double()
        y = torch.cat([lat, _complex_turn(x[:, DL:], table, s["halves"])], 1)
        kept = slots >= 0
        out = {"rows": y}
        if case["pool"] == "bf16":
            pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device=x.device)
            pool[slots[kept]] = y[kept]
        else:
            f8 = torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127],
                              device=x.device, dtype=torch.float64)
            f4 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device, dtype=torch.float64)
            b = lat.reshape(-1, SCALES, BLOCK)
            scale = _nearest(b.abs().amax(2) / 6, f8)[:, :, None]
            code = _nearest((b.abs() / torch.where(scale > 0, scale, 1.0)).clamp(max=6.0), f4)
            pool = torch.cat([(torch.sign(b) * code * scale).reshape(-1, DL), y[:, DL:]], 1)
            pool[~kept] = 0
        out["pool"] = pool
        if s["q"] is not None:
            q = s["q"].double()
            if s["q_weight"] is not None:
                q = q / (q.pow(2).sum(2, keepdim=True) / q.shape[2] + EPS).sqrt() * s["q_weight"].double()
            out["q"] = torch.cat([q[..., :-DR], _complex_turn(q[..., -DR:], table, s["halves"])], 2)
        return out
    cu_q, cu_k, heads = s["cu_q"].tolist(), s["cu_k"].tolist(), case["heads"]
    out = torch.zeros(cu_q[-1], heads, DV, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((cu_q[-1], heads), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b in range(case["seqs"]):
        m, n = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        kr = s["k_rope"][cu_k[b]:cu_k[b + 1]].double()
        for h in range(case["heads"] // case["group"]):
            k, v = s["k"][cu_k[b]:cu_k[b + 1], h].double(), s["v"][cu_k[b]:cu_k[b + 1], h].double()
            mine = slice(h * case["group"], (h + 1) * case["group"])
            for i in range(0, m, 2048):
                e = min(m, i + 2048)
                end = min(n, e + n - m) if case["causal"] else n
                q = s["q"][cu_q[b] + i:cu_q[b] + e, mine].double()
                x = (torch.einsum("ihd,td->iht", q[..., :DN], k[:end]) + torch.einsum("ihd,td->iht", q[..., DN:], kr[:end])) * SCALE
                if case["causal"]:
                    late = torch.arange(end, device=x.device) > torch.arange(i, e, device=x.device)[:, None] + n - m
                    x.masked_fill_(late[:, None, :], -math.inf)
                l = torch.logsumexp(x, 2)
                lse[cu_q[b] + i:cu_q[b] + e, mine] = l
                out[cu_q[b] + i:cu_q[b] + e, mine] = torch.einsum("iht,td->ihd", torch.exp(x - l[:, :, None]), v[:end])
    return {"out": out, "lse": lse}
