"""Cases of the prompt operators: kv_append_rope and kv_prefill_attn.

``kv_append_rope`` takes the packed query, key and value rows of a step's new tokens (whole
prompts, chunks of prompts, or one token per sequence), rotates queries and keys by their
positions, writes keys and values into the paged cache and keeps the page statistics current.
``kv_prefill_attn`` is causal attention of packed query rows over the paged cache.

A case gives the new tokens of each sequence (``new``) and how many tokens its cache holds
before them (``past``), both as comma-separated numbers; sequences differ in length.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, new, past, dtype="bf16", hq=32, hkv=8, d=128, ps=16, rot=0, inter=False,
          packed=True):
    c = {"op": op, "new": ",".join(map(str, new)), "past": ",".join(map(str, past)),
         "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "ps": ps}
    if op == "append":
        c.update(rot=rot or d, inter=inter)
    c["packed"] = packed          # False: one token per sequence, no offsets are passed
    if name:
        c["name"] = name
    return c


# Lengths of a batch as a server sees it: many short prompts, some long ones, odd sizes.
RAGGED = (1, 37, 512, 129, 2047, 64, 1000, 3, 255, 1531, 777, 4001, 16, 90, 333, 2500)
DECODE_PAST = tuple(1024 + (97 * i * i + 331 * i) % 3001 for i in range(32))


def listed():
    return [
        # A decode step of 32 sequences: latency of the smallest call counts.
        _case("append decode x32", "append", (1,) * 32, DECODE_PAST, packed=False),
        # One whole prompt of an 8B-like model into an empty cache.
        _case("append prompt 8192", "append", (8192,), (0,)),
        # Ragged chunks of prompts that continue in the middle of a page (70B-like heads).
        _case("append ragged 70b ps64", "append", RAGGED,
              tuple((211 * i) % 1500 for i in range(16)), hq=64, ps=64),
        # The fp32 parity configuration with adjacent pairs and half of each head rotated.
        _case("append fp32 partial", "append", (1000, 1, 313), (0, 77, 4000), dtype="fp32",
              hq=8, hkv=2, d=64, rot=32, inter=True),
        # A single new token over a long cache: bound by reading the cache once.
        _case("attn 1 token 32k", "attn", (1,), (32767,), packed=False),
        # Drafted tokens verified by 8 sequences: few rows over middling caches.
        _case("attn 5 drafts x8", "attn", (5,) * 8,
              (4000, 16001, 9000, 30011, 1023, 22222, 12000, 65), ),
        # One chunk of a long prompt: 512 rows over 32K cached tokens.
        _case("attn chunk 512 at 32k", "attn", (512,), (32256,)),
        # One prompt of an 8B-like model.
        _case("attn prompt 8192", "attn", (8192,), (0,)),
        # A server's packed batch of prompts of different lengths.
        _case("attn ragged 8b", "attn", RAGGED, (0,) * 16),
        # Heads of 64 columns without sharing, pages of 32, some prompts continued.
        _case("attn ragged d64", "attn", (700, 1999, 1, 4096), (0, 513, 3000, 0), hq=16, hkv=16,
              d=64, ps=32),
        # The fp32 parity configuration over its 4096 tokens.
        _case("attn fp32 4096", "attn", (4096,), (0,), dtype="fp32", hq=8, hkv=2, d=64),
        # The largest: a 16K prompt with 70B-like heads and pages of 64.
        _case("attn prompt 16384 70b", "attn", (16384,), (0,), hq=64, ps=64),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the same ranges: 1 to 32 sequences, 1 to 16384 new tokens, caches of up
    to 32768 tokens, every page size, head width, group size and type."""
    hkv = rng.choice((1, 2, 8, 16))
    group = rng.choice((1, 2, 4, 8))
    if hkv * group > 64:
        group = 4
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    d, ps = rng.choice((64, 128)), rng.choice((16, 32, 64))
    op = rng.choice(("append", "attn"))
    shape = dict(dtype=dtype, hq=hkv * group, hkv=hkv, d=d, ps=ps)
    if op == "append":
        shape.update(rot=rng.choice((d, d, d // 2)), inter=rng.choice((False, True)))
    batch = _log(rng, 1, 32)
    if rng.random() < 0.3:       # one token per sequence
        past = [_log(rng, 1, 32768 if op == "attn" and dtype == "bf16" else 4096) - 1
                for _ in range(batch)]
        return _case("", op, (1,) * batch, past, packed=rng.choice((False, True)), **shape)
    most = 16384 if dtype == "bf16" else 4096
    total = _log(rng, batch, most)
    cuts = sorted(rng.randrange(total + 1) for _ in range(batch - 1))
    new = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    # the longest prompts start empty, so that no case costs more than the largest listed one
    past = [rng.choice((0, _log(rng, 1, 4096))) if total <= 8192 else 0 for _ in range(batch)]
    return _case("", op, new, past, **shape)


def _lengths(case):
    return ([int(x) for x in case["new"].split(",")], [int(x) for x in case["past"].split(",")])


def _inv_freq(rot):
    return torch.tensor([500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)],
                        dtype=torch.float64)


def prepare(case, seed):
    """The cache as the tokens before left it, and the new rows. For attention the new tokens'
    keys and values are in the cache already; for append its pages are mapped and hold what
    was there before."""
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    new, past = _lengths(case)
    B, T, hq, hkv, d, ps = len(new), sum(new), case["hq"], case["hkv"], case["d"], case["ps"]
    pages = [-(-(n + p) // ps) for n, p in zip(new, past)]
    NP = sum(pages) + 3

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(dt)

    s = {"case": case, "new": new, "past": past}
    s["k_pool"], s["v_pool"] = rand(NP, hkv, ps, d), rand(NP, hkv, ps, d)
    order = torch.randperm(NP, generator=gen, device=dev).to(torch.int32)
    table = torch.full((B, max(max(pages), 1)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["lens"] = torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32, device=dev)
    s["cu"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    # a fused projection's rows: queries, keys and values side by side
    qkv = rand(T, hq + 2 * hkv, d)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "append":
        s["inv_freq"] = _inv_freq(case["rot"])
        s["inv_freq_dev"] = s["inv_freq"].to(dev)
        keys = s["k_pool"].float()                 # statistics of every page as it stands
        s["stats"] = torch.stack([keys.amin(2), keys.amax(2)], dim=2).to(dt).contiguous()
        for b, p in enumerate(past):               # and of a page that ends inside the past
            if p % ps:
                page = table[b, p // ps].long()
                part = s["k_pool"][page, :, :p % ps].float()
                s["stats"][page] = torch.stack([part.amin(1), part.amax(1)], dim=1).to(dt)
    else:
        # trained keys: the first token of a sequence draws much of the attention, and queries
        # are not of unit variance
        mean = s["q"].float().view(T, hkv, hq // hkv, d).mean((0, 2))
        sink = (4.0 * mean / mean.norm(dim=-1, keepdim=True)).to(dt)
        first = torch.tensor([b for b, n in enumerate(pages) if n], device=dev)
        s["k_pool"][table[first, 0].long(), :, 0] = sink
        s["q"] = (1.5 * s["q"]).to(dt)
    if own:
        import sparse_kv_cache_build_gb300 as skv
        s["kv"] = skv.PagedKV(s["k_pool"], s["v_pool"], table, s["lens"])
        if case["op"] == "append":
            s["turns"] = skv.kv_rope_turns(s["inv_freq"], device=dev)
        else:
            n = skv.kv_prefill_attn_workspace_size(s["kv"], hq, T)
            s["workspace"] = torch.empty((n,), dtype=torch.uint8, device=dev)
    return s


def _places(s):
    """Sequence and position of each new token."""
    T = s["q"].shape[0]
    counts = s["cu"][1:].long() - s["cu"][:-1].long()
    seq = torch.repeat_interleave(torch.arange(counts.numel(), device=counts.device), counts,
                                  output_size=T)
    pos = s["lens"].long()[seq] - counts[seq] + torch.arange(T, device=seq.device) - \
        s["cu"].long()[seq]
    return seq, pos


def _rotate(x, cos, sin, rot, inter):
    """Pairs of the first `rot` columns turned by their angle: (i, i + rot/2), or (2i, 2i + 1)."""
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
    u, w = a * cos - b * sin, a * sin + b * cos
    head = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((head, rest), -1)


def _plain_append(s):
    case, dt = s["case"], s["q"].dtype
    seq, pos = _places(s)
    angle = pos.double()[:, None] * s["inv_freq_dev"]            # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(s["q"], cos, sin, case["rot"], case["inter"]).to(dt)
    k = _rotate(s["k"], cos, sin, case["rot"], case["inter"]).to(dt)
    ps = case["ps"]
    page, slot = s["table"][seq, pos // ps].long(), pos % ps
    s["k_pool"][page, :, slot] = k
    s["v_pool"][page, :, slot] = s["v"]
    # a page's first token starts its statistics anew; a spare row takes the other tokens
    NP, hkv, d = s["stats"].shape[0], s["stats"].shape[1], s["stats"].shape[3]
    fresh = torch.where(slot == 0, page, NP)
    for i, inf, kind in ((0, math.inf, "amin"), (1, -math.inf, "amax")):
        rows = torch.zeros((NP + 1, hkv, d), device=q.device)
        rows[:NP] = s["stats"][:, :, i]
        rows.index_fill_(0, fresh, inf)
        rows.index_reduce_(0, page, k.float(), kind)
        s["stats"][:, :, i] = rows[:NP]
    return [q, s["k_pool"], s["v_pool"], s["stats"]]


def _plain_attn(s):
    case, q = s["case"], s["q"]
    T, hq, hkv, d = q.shape[0], case["hq"], case["hkv"], case["d"]
    G = hq // hkv
    out = torch.empty((T, hq, d), dtype=q.dtype, device=q.device)
    lse = torch.empty((T, hq), device=q.device)
    at = 0
    for b, (n, p) in enumerate(zip(s["new"], s["past"])):        # sequences differ in length
        if n == 0:
            continue
        L = n + p
        page = s["table"][b, :-(-L // case["ps"])].long()
        K = s["k_pool"][page].transpose(0, 1).reshape(hkv, -1, d)[:, :L].float()
        V = s["v_pool"][page].transpose(0, 1).reshape(hkv, -1, d)[:, :L].float()
        x = q[at:at + n].float().view(n, hkv, G, d).permute(1, 2, 0, 3).reshape(hkv, G * n, d)
        x = torch.bmm(x, K.transpose(1, 2)).mul_(s["scale"]).view(hkv, G, n, L)
        late = torch.arange(L, device=q.device) > torch.arange(p, L, device=q.device)[:, None]
        x.masked_fill_(late, -math.inf)
        m = x.amax(-1, keepdim=True)
        x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        o = torch.bmm(x.view(hkv, G * n, L), V).view(hkv, G, n, d) / l
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hq, d)
        lse[at:at + n] = (m + l.log()).squeeze(-1).permute(2, 0, 1).reshape(n, hq)
        at += n
    return [out, lse]


def run(state):
    case = state["case"]
    if own:
        import sparse_kv_cache_build_gb300 as skv
        cu = state["cu"] if case["packed"] else None
        if case["op"] == "append":
            q = skv.kv_append_rope(state["kv"], state["q"], state["k"], state["v"],
                                   state["stats"], state["turns"], cu_tokens=cu,
                                   interleaved=case["inter"])
            return [q, state["k_pool"], state["v_pool"], state["stats"]]
        return list(skv.kv_prefill_attn(state["kv"], state["q"], state["scale"], cu_tokens=cu,
                                        workspace=state["workspace"]))
    return _plain_append(state) if case["op"] == "append" else _plain_attn(state)


def work(case):
    new, past = _lengths(case)
    e = 2 if case["dtype"] == "bf16" else 4
    T, hq, hkv, d, ps = sum(new), case["hq"], case["hkv"], case["d"], case["ps"]
    if case["op"] == "append":
        rows = T * (hq + 2 * hkv) * d * e
        touched = sum(-(-(n + p) // ps) - p // ps for n, p in zip(new, past) if n)
        resumed = sum(1 for n, p in zip(new, past) if n and p % ps)
        return {"bytes": 2 * rows + (touched + resumed) * hkv * 2 * d * e,
                "flops": 3 * T * (hq + hkv) * case["rot"]}
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    cached = sum(n + p for n, p in zip(new, past) if n)
    return {"bytes": 2 * cached * hkv * d * e + T * hq * (2 * d * e + 4),
            "flops": 4 * pairs * hq * d}


def exact(case, seed):
    """The same outputs in 64 bits, token block by token block, from the definitions."""
    s = prepare(case, seed)
    new, past = s["new"], s["past"]
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["ps"]
    table = s["table"].cpu().numpy()
    lens = [n + p for n, p in zip(new, past)]
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    if case["op"] == "append":
        return _exact_append(case, s, new, lens, table, kp, vp)
    G, at = hq // hkv, 0
    out = torch.empty((sum(new), hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((sum(new), hq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(new):
        where = torch.arange(lens[b], device="cuda")
        phys = torch.tensor(table[b], device="cuda").long()[where // ps]
        for i in range(0, n, 1024):
            e = min(n, i + 1024)
            last = lens[b] - n + e                 # keys that the block's last row sees
            own_pos = torch.arange(lens[b] - n + i, last, device="cuda")
            hidden = where[None, :last] > own_pos[:, None]
            for g in range(hkv):
                K, V = kp[phys[:last], g, where[:last] % ps], vp[phys[:last], g, where[:last] % ps]
                for h in range(g * G, (g + 1) * G):
                    z = s["q"][at + i:at + e, h].double() @ K.T * s["scale"]
                    z[hidden] = -math.inf
                    top = z.max(1).values
                    w = torch.exp(z - top[:, None])
                    total = w.sum(1)
                    out[at + i:at + e, h] = (w @ V) / total[:, None]
                    lse[at + i:at + e, h] = top + torch.log(total)
        at += n
    return [out, lse]


def _exact_append(case, s, new, lens, table, kp, vp):
    rot, ps = case["rot"], case["ps"]
    half = rot // 2
    low = torch.arange(half) * 2 if case["inter"] else torch.arange(half)
    high = low + 1 if case["inter"] else low + half
    low, high = low.cuda(), high.cuda()
    stats = s["stats"].double()
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    freq = _inv_freq(rot).cuda()
    at = 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        pos = torch.arange(lens[b] - n, lens[b], device="cuda")
        turn = torch.exp(1j * pos.double()[:, None, None] * freq)
        for x in (q, k):
            z = torch.complex(x[at:at + n][..., low], x[at:at + n][..., high]) * turn
            rows = x[at:at + n].clone()
            rows[..., low], rows[..., high] = z.real, z.imag
            x[at:at + n] = rows
        for p in range((lens[b] - n) // ps, -(-lens[b] // ps)):
            P = int(table[b][p])
            first, last = max(p * ps, lens[b] - n), min((p + 1) * ps, lens[b])
            o = at + first - (lens[b] - n)
            rows = k[o:o + last - first].transpose(0, 1)
            kp[P, :, first - p * ps:last - p * ps] = rows
            vp[P, :, first - p * ps:last - p * ps] = v[o:o + last - first].transpose(0, 1)
            mn, mx = rows.min(1).values, rows.max(1).values
            if first > p * ps:                     # the page held tokens before
                mn = torch.minimum(mn, stats[P, :, 0])
                mx = torch.maximum(mx, stats[P, :, 1])
            stats[P, :, 0], stats[P, :, 1] = mn, mx
        at += n
    return [q, kp, vp, stats]
