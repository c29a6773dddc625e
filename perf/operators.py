"""Measured cases of the paged key/value cache: appending rows with the position
rotation, attention over the pages, and attention of a batch that shares a prefix.

``run`` computes a case in plain torch operations (fp32, angles in 64 bits), or,
with ``own``, through the framework's PagedKV.  ``exact`` is the operator's
definition in 64 bits, one sequence at a time.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = dict(op=op, type="bf16", Hq=32, Hkv=32, D=128, page=64, slots_first=False, seqs=1, rows=1,
             ragged=False, len_min=256, len_max=256, mask="none", pruned=False, groups=0,
             prefix_min=0, prefix_max=0, lse=False, mix=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoded token of one sequence: latency
        _case("append_one_token", "append", Hq=28, Hkv=4, page=16, len_min=513, len_max=513),
        # a decode block of every sequence of a batch with many key/value heads
        _case("append_blocks", "append", seqs=16, rows=32, len_min=512, len_max=1280),
        # prompts of different lengths entering the cache, in fp16, slots before heads
        _case("append_prompts", "append", type="f16", Hq=28, Hkv=4, seqs=8, rows=2048, ragged=True,
              len_min=2048, len_max=8192, page=128, slots_first=True),
        # a short context of one sequence, one block: latency
        _case("attn_short_block", "attn", Hq=28, Hkv=4, rows=32, len_min=544, len_max=544),
        # one token of each sequence of a ragged batch, small pages
        _case("attn_tokens", "attn", Hq=28, Hkv=4, seqs=32, len_min=61, len_max=9216, page=16, lse=True),
        # one token against one long context, fp16
        _case("attn_long_token", "attn", type="f16", Hq=28, Hkv=4, len_min=131001, len_max=131001,
              page=128, slots_first=True),
        # a decode block of every sequence of a ragged batch
        _case("attn_blocks", "attn", seqs=16, rows=32, len_min=768, len_max=1280),
        # long contexts whose suffix is pruned to a window and the trailing position
        _case("attn_pruned", "attn", Hq=28, Hkv=4, seqs=4, rows=64, len_min=8256, len_max=9216, pruned=True),
        # chunks of two prompts entering under a block-causal mask
        _case("attn_prompt_chunks", "attn", Hq=28, Hkv=4, seqs=2, rows=1024, len_min=2048, len_max=4096,
              mask="blocks", page=32),
        # samples of one long prompt, one token each
        _case("shared_tokens", "shared", Hq=28, Hkv=4, seqs=32, len_min=1, len_max=300, groups=1,
              prefix_min=8192, prefix_max=8192, page=16),
        # samples of a few prompts, a decode block each
        _case("shared_blocks", "shared", type="f16", seqs=12, rows=32, len_min=32, len_max=256, groups=3,
              prefix_min=512, prefix_max=1024, lse=True),
        # many samples of one long system prompt, a decode block each: the largest
        _case("shared_many_blocks", "shared", Hq=28, Hkv=4, seqs=32, rows=32, len_min=32, len_max=512,
              groups=1, prefix_min=8192, prefix_max=8192),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "shared", "shared"])
    hq, hkv = rng.choice([(32, 32), (28, 4), (28, 4), (7, 1), (32, 8)])
    kw = dict(Hq=hq, Hkv=hkv, D=rng.choice([128, 128, 128, 64, 32]), type=rng.choice(["bf16", "f16"]),
              page=rng.choice([16, 32, 64, 128, 256]), slots_first=rng.random() < 0.5,
              lse=op != "append" and rng.random() < 0.5, mix=rng.randrange(1 << 30))
    if op == "append":
        seqs = _log(rng, 1, 64)
        rows = _log(rng, 1, 4096 // seqs)
        hi = rows + _log(rng, 1, 8192)
        return _case(None, op, seqs=seqs, rows=rows, ragged=rng.random() < 0.5, len_min=rows, len_max=hi, **kw)
    if op == "attn":
        seqs = _log(rng, 1, 64)
        rows = rng.choice([1, 1, _log(rng, 1, 64), _log(rng, 1, 64), _log(rng, 1, 1024)])
        rows = max(1, min(rows, 2048 // seqs))
        hi = rows + _log(rng, 1, max(2, min(65536, 400000 // (seqs * hkv))))
        hi = max(rows, min(hi, 4_000_000 // (seqs * rows) + rows))
        mask = rng.choice(["none", "none", "causal", "blocks"])
        return _case(None, op, seqs=seqs, rows=rows, ragged=rng.random() < 0.5, len_min=max(rows, hi // 4),
                     len_max=hi, mask=mask, pruned=mask == "none" and rng.random() < 0.3, **kw)
    groups = _log(rng, 1, 8)
    seqs = groups * _log(rng, 2, 32 // groups)
    rows = rng.choice([1, rng.randint(2, 32), 32])
    hi = rows + _log(rng, 1, 512)
    pre = _log(rng, 16, max(32, min(8192, 400000 // (seqs * hkv))))
    return _case(None, op, seqs=seqs, rows=rows, ragged=rng.random() < 0.5, len_min=rows, len_max=hi,
                 groups=groups, prefix_min=max(1, pre // 2), prefix_max=pre, **kw)


def _sizes(c):
    """Rows and cached positions of each sequence, prefix length and first sequence of
    each group: they follow from the case alone, whatever the seed."""
    r = random.Random(c["mix"])
    rows = [r.randint(1, c["rows"]) if c["ragged"] else c["rows"] for _ in range(c["seqs"])]
    lens = [max(n, r.randint(c["len_min"], c["len_max"])) for n in rows]
    prefix = [r.randint(c["prefix_min"], c["prefix_max"]) for _ in range(c["groups"])]
    cuts = sorted(r.sample(range(1, c["seqs"]), c["groups"] - 1)) if c["groups"] else []
    return rows, lens, prefix, [0] + cuts + [c["seqs"]] if c["groups"] else []


def _segments(c, rows, lens):
    """(start, length) pairs of the keys of each sequence."""
    if not c["pruned"]:
        return [((0, n), (0, 0)) for n in lens]
    out = []
    for m, n in zip(rows, lens):  # left padding, the context up to a window after the block, the last position
        first, end = min(37, n // 4), max(1, n - n // 8)
        out.append(((first, end - first), (n - 1, 1 if n - 1 >= end else 0)))
    return out


def _limits(c, rows, lens):
    """Keys that each row may see under a causal or a block-causal mask; None without a mask."""
    if c["mask"] == "none":
        return None
    b = 1 if c["mask"] == "causal" else 32
    return [min(n, ((n - m + j) // b + 1) * b) for m, n in zip(rows, lens) for j in range(m)]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c, dev = case, "cuda"
    rows, lens, prefix, cuts = _sizes(c)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, ps, D = _TYPES[c["type"]], c["page"], c["D"]
    own_pages = [-(-n // ps) for n in lens]
    pre_pages = [-(-n // ps) for n in prefix]
    pool = sum(own_pages) + sum(pre_pages) + 3

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dt)

    def pages():
        if c["slots_first"]:
            return normal(pool, ps, c["Hkv"], D).transpose(1, 2)
        return normal(pool, c["Hkv"], ps, D)

    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)

    def table(counts, first):
        width = max(counts + [1])
        at = torch.arange(width)[None, :] + (torch.tensor([sum(counts[:i]) for i in range(len(counts))]) + first)[:, None]
        used = torch.arange(width)[None, :] < torch.tensor(counts)[:, None]
        t = order[at.clamp(max=pool - 1).to(dev)]
        return torch.where(used.to(dev), t, torch.full_like(t, -1)).contiguous()

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    n = sum(rows)
    spare = 3  # rows behind the last sequence: a padded batch
    packed = normal(n + spare, c["Hq"] + 2 * c["Hkv"], D)
    s = dict(case=c, rows=rows, lens=lens, n=n, k_pages=pages(), v_pages=pages(), packed=packed,
             row_start=ints([sum(rows[:i]) for i in range(len(rows) + 1)]), table=table(own_pages, 0),
             q=packed[:, :c["Hq"]], k=packed[:, c["Hq"]:c["Hq"] + c["Hkv"]], v=packed[:, c["Hq"] + c["Hkv"]:],
             out=torch.zeros(n + spare, c["Hq"], D, dtype=dt, device=dev), max_rows=max(rows))
    if c["op"] == "append":
        s["pos"] = ints([b - a for a, b in zip(rows, lens)])  # the rows are the sequence's last positions
        s["shift"] = ints([-(i % 5) for i in range(len(rows))])
        s["theta"] = 1e6
        return s
    s["lse"] = torch.zeros(n + spare, c["Hq"], dtype=torch.float32, device=dev) if c["lse"] else None
    s["segs"] = ints(_segments(c, rows, lens))
    lim = _limits(c, rows, lens)
    s["limit"] = None if lim is None else ints(lim + [0] * spare)
    if c["groups"]:
        s["group_start"] = ints(cuts)
        s["prefix_table"] = table(pre_pages, sum(own_pages))
        s["prefix_len"] = ints(prefix)
        s["prefix"], s["cuts"] = prefix, cuts
    return s


# ------------------------------------------------------------------ plain forms
def _row_places(s):
    """Sequence of each row and its place in it."""
    r = torch.arange(s["n"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["row_start"][1:].contiguous(), r, right=True)
    return seq, (r - s["row_start"][seq]).long()


def _plain_append(s):
    c, n = s["case"], s["n"]
    half = c["D"] // 2
    seq, j = _row_places(s)
    p = s["pos"][seq].long() + j
    freq = s["theta"] ** (torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 / c["D"]))
    ang = (p + s["shift"][seq].long()).double()[:, None] * freq
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]

    def turned(x):
        a, b = x[:n, :, :half].float(), x[:n, :, half:].float()
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)

    page, slot = s["table"][seq, p // c["page"]].long(), p % c["page"]
    s["out"][:n] = turned(s["q"])
    s["k_pages"][page, :, slot] = turned(s["k"])
    s["v_pages"][page, :, slot] = s["v"][:n]
    return s["out"], s["k_pages"], s["v_pages"]


def _keys(pages, table):
    """Pages of each list in order: [lists, heads, positions, D] in 32 bits."""
    got = pages[table.clamp(min=0).long()].float()
    return got.permute(0, 2, 1, 3, 4).reshape(got.shape[0], got.shape[2], -1, got.shape[4])


def _plain_attn(s):
    c = s["case"]
    g, D = c["Hq"] // c["Hkv"], c["D"]
    seq, j = _row_places(s)
    m = s["max_rows"]
    at = (s["row_start"][:-1, None] + torch.arange(m, device="cuda")).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float() * D ** -0.5                                       # [seqs, m, Hq, D]
    q = q.reshape(-1, m, c["Hkv"], g, D).permute(0, 2, 1, 3, 4).reshape(-1, c["Hkv"], m * g, D)
    k, v = _keys(s["k_pages"], s["table"]), _keys(s["v_pages"], s["table"])
    pos = torch.arange(k.shape[2], device="cuda")
    a, b = s["segs"][:, :, :1], s["segs"][:, :, 1:]
    seen = ((pos >= a) & (pos < a + b)).any(1)[:, None].expand(-1, m, -1)    # [seqs, m, positions]
    if s["limit"] is not None:
        seen = seen & (pos < s["limit"][at][:, :, None])
    if c["groups"]:
        of = torch.searchsorted(s["group_start"][1:].contiguous(),
                                torch.arange(c["seqs"], device="cuda", dtype=torch.int32), right=True)
        pk, pv = (_keys(x, s["prefix_table"])[of] for x in (s["k_pages"], s["v_pages"]))
        before = torch.arange(pk.shape[2], device="cuda") < s["prefix_len"][of][:, None]
        seen = torch.cat([before[:, None].expand(-1, m, -1), seen], 2)
        k, v = torch.cat([pk, k], 2), torch.cat([pv, v], 2)
    seen = seen[:, None, :, None].expand(-1, 1, -1, g, -1).reshape(c["seqs"], 1, m * g, -1)
    score = (q @ k.transpose(2, 3)).masked_fill_(~seen, -math.inf)
    top = score.amax(3, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = score.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    o = (p @ v) / total.clamp(min=torch.finfo(torch.float32).tiny)
    lse = (top + total.log()).reshape(-1, c["Hkv"], m, g).transpose(1, 2).reshape(-1, m, c["Hq"])
    o = o.reshape(-1, c["Hkv"], m, g, D).transpose(1, 2).reshape(-1, m, c["Hq"], D)
    s["out"][:s["n"]] = o[seq, j].to(s["out"].dtype)
    if s["lse"] is None:
        return (s["out"],)
    s["lse"][:s["n"]] = lse[seq, j]
    return s["out"], s["lse"]


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    c = s["case"]
    if not own:
        return _plain_append(s) if c["op"] == "append" else _plain_attn(s)
    kv = s.get("kv")
    if kv is None:  # a server keeps one for its pool
        from diffusion_decoding_step_b200.paged import PagedKV
        kv = s["kv"] = PagedKV(s["k_pages"], s["v_pages"], n_q_heads=c["Hq"], max_rows=s["out"].shape[0],
                               max_groups=c["groups"])
    if c["op"] == "append":
        kv.append(s["k"], s["v"], s["row_start"], s["table"], s["pos"], q=s["q"], q_out=s["out"],
                  rope_theta=s["theta"], rope_shift=s["shift"])
        return s["out"], s["k_pages"], s["v_pages"]
    if c["op"] == "attn":
        kv.attn(s["q"], s["row_start"], s["table"], s["segs"], row_limit=s["limit"], out=s["out"], lse=s["lse"])
    else:
        kv.shared_prefix_attn(s["q"], s["row_start"], s["table"], s["segs"], s["group_start"], s["prefix_table"],
                              s["prefix_len"], row_limit=s["limit"], out=s["out"], lse=s["lse"])
    return (s["out"],) if s["lse"] is None else (s["out"], s["lse"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    rows, lens, prefix, cuts = _sizes(c)
    n, hq, hkv, D = sum(rows), c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "append":
        return {"bytes": 2 * n * (hq + 2 * hkv) * D * 2, "flops": 3 * n * (hq + hkv) * D}
    lim, seg = _limits(c, rows, lens), _segments(c, rows, lens)
    pairs = keys = at = 0
    for m, sg in zip(rows, seg):
        cut = [sum(max(0, min(a + b, x) - a) for a, b in sg) for x in (lim[at:at + m] if lim else [1 << 40] * m)]
        pairs, keys, at = pairs + sum(cut), keys + max(cut), at + m
    if prefix:
        keys += sum(prefix)
        pairs += sum(p * sum(rows[a:b]) for p, a, b in zip(prefix, cuts, cuts[1:]))
    return {"bytes": 2 * n * hq * D * 2 + 2 * keys * hkv * D * 2 + (4 * n * hq if c["lse"] else 0),
            "flops": 4 * pairs * hq * D}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    ps, D, g = c["page"], c["D"], c["Hq"] // c["Hkv"]
    f = torch.float64
    out = s["out"].to(f)
    starts, table = s["row_start"].tolist(), s["table"].long()
    if c["op"] == "append":
        kp, vp = s["k_pages"].to(f), s["v_pages"].to(f)
        i = torch.arange(D // 2, dtype=f, device="cuda")
        freq = torch.exp(-2.0 * i / D * math.log(s["theta"]))
        for b, (pos, shift) in enumerate(zip(s["pos"].tolist(), s["shift"].tolist())):
            r = torch.arange(starts[b], starts[b + 1], device="cuda")
            p = r - starts[b] + pos
            turn = torch.polar(torch.ones((), dtype=f, device="cuda"), torch.outer((p + shift).to(f), freq))[:, None]

            def rot(x):
                z = torch.complex(x[r, :, :D // 2].to(f), x[r, :, D // 2:].to(f)) * turn
                return torch.cat([z.real, z.imag], -1)

            out[r] = rot(s["q"])
            kp[table[b][p // ps], :, p % ps] = rot(s["k"])
            vp[table[b][p // ps], :, p % ps] = s["v"][r].to(f)
        return out, kp, vp
    lse = None if s["lse"] is None else s["lse"].to(f)
    segs = s["segs"].tolist()

    def listed_keys(pages, t, at):
        return pages[t[at // ps], :, at % ps].to(f).transpose(0, 1)  # [Hkv, keys, D]

    for b in range(c["seqs"]):
        at = torch.cat([torch.arange(a, a + w, device="cuda") for a, w in segs[b]])
        k, v = (listed_keys(x, table[b], at) for x in (s["k_pages"], s["v_pages"]))
        first = 0
        if c["groups"]:
            gi = max(i for i in range(c["groups"]) if s["cuts"][i] <= b)
            first = s["prefix"][gi]
            pt, pa = s["prefix_table"][gi].long(), torch.arange(first, device="cuda")
            k, v = (torch.cat([listed_keys(x, pt, pa), y], 1) for x, y in ((s["k_pages"], k), (s["v_pages"], v)))
        for lo in range(starts[b], starts[b + 1], 256):
            r = torch.arange(lo, min(lo + 256, starts[b + 1]), device="cuda")
            seen = torch.ones(len(r), k.shape[1], dtype=torch.bool, device="cuda")
            if s["limit"] is not None:
                seen[:, first:] = at[None] < s["limit"][r][:, None]
            for h in range(c["Hkv"]):
                q = s["q"][r, h * g:(h + 1) * g].to(f)
                x = torch.einsum("rgd,kd->rgk", q, k[h]) / math.sqrt(D)
                x = torch.where(seen[:, None], x, -math.inf)
                z = torch.logsumexp(x, 2, keepdim=True)
                w = torch.where(torch.isfinite(z), torch.exp(x - z), torch.zeros_like(x))
                out[r, h * g:(h + 1) * g] = torch.einsum("rgk,kd->rgd", w, v[h])
                if lse is not None:
                    lse[r, h * g:(h + 1) * g] = z[:, :, 0]
    return (out,) if lse is None else (out, lse)
