"""Cases of the operators for drafts, windows and pages over the paged cache.

``kv_tree_attn`` is attention of drafted tokens that form a tree: a row sees the tokens cached
before the drafts and its own ancestors. ``kv_window_attn`` is causal attention within a sliding
window plus a few first tokens. ``kv_compact`` moves a sequence's kept tokens together in place and
brings the page statistics up to date. ``kv_copy_pages`` copies physical pages. ``kv_update_pages``
gives the batch its next page table: rows fork, tokens are dropped, pages go back and new ones come.

A case gives per sequence the rows (``new``) and the tokens cached before them (``past``) as
comma-separated numbers; sequences differ in length.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, new, past, dtype="bf16", hq=32, hkv=8, d=128, ps=16, **more):
    c = {"op": op, "new": ",".join(map(str, new)), "past": ",".join(map(str, past)),
         "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "ps": ps, **more}
    if name:
        c["name"] = name
    return c


# Lengths of a batch as a server sees it: short and long prompts, odd sizes.
RAGGED = (1, 37, 512, 129, 2047, 64, 1000, 3, 255, 1531, 777, 4001, 16, 90, 333, 2500)
SERVED = tuple(700 + (97 * i * i + 331 * i) % 9001 for i in range(32))


def listed():
    return [
        # The smallest verification: one user's eight drafts over a middling cache.
        _case("tree 8 nodes x1", "tree", (8,), (2000,)),
        # A server verifies trees of 26 nodes (70B-like heads, pages of 64).
        _case("tree 26 nodes x16 70b", "tree", (26,) * 16, SERVED[:16], hq=64, ps=64),
        # The fp32 parity configuration.
        _case("tree fp32", "tree", (7, 31, 12, 1), (1000, 4000, 63, 2500), dtype="fp32", hq=8,
              hkv=2, d=64),
        # A decode step of 32 streams that keep four first tokens and the last 1024.
        _case("window decode x32", "window", (1,) * 32, SERVED, window=1024, sinks=4,
              packed=False),
        # A server's packed batch of prompts with a window of 512 tokens, some continued; heads of
        # 64 columns without sharing.
        _case("window ragged d64", "window", RAGGED, tuple((911 * i) % 5003 for i in range(16)),
              hq=16, hkv=16, d=64, ps=32, window=512, sinks=0, packed=True),
        # The largest: a 16K prompt with 70B-like heads, a window of 4096 and 64 sinks.
        _case("window prompt 16384 70b", "window", (16384,), (0,), hq=64, ps=64, window=4096,
              sinks=64, packed=True),
        # Verified trees: a few of each sequence's drafts stay.
        _case("compact accepted x32", "compact", (26,) * 32, SERVED, kept="accept"),
        # An eviction: a long cache keeps an eighth of its tokens.
        _case("compact 32k to 4k", "compact", (32768,), (0,), kept="evict"),
        # Pages a fork has to copy before 16 sequences write to them.
        _case("copy 16 pages", "copy", (16,), (0,)),
        # Sequences that move elsewhere in the pool: 2000 pages of 64 tokens.
        _case("copy 2000 pages", "copy", (2000,), (0,), ps=64),
        # A decode step of 64 streams with a window: pages fall out of it, others are needed.
        _case("pages stream x64", "pages", (1,) * 64, tuple(900 + 517 * i for i in range(64)),
              window=1024, sinks=4, beams=0, stride=4096, pool=65536),
        # A step of 16 requests with 4 beams each: rows fork, partial pages are copied.
        _case("pages beams 16x4", "pages", (1,) * 64, tuple(500 + 37 * (i // 4) for i in range(64)),
              window=0, sinks=0, beams=4, stride=512, pool=8192),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the same ranges: 1 to 64 sequences, trees of 1 to 256 nodes, windows of 1 to
    8192 tokens, caches of up to 32768 tokens, every page size, head width, group size and type."""
    hkv, group = rng.choice((1, 2, 8, 16)), rng.choice((1, 2, 4, 8))
    if hkv * group > 64:
        group = 4
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    shape = dict(dtype=dtype, hq=hkv * group, hkv=hkv, d=rng.choice((64, 128)),
                 ps=rng.choice((16, 32, 64)))
    op = rng.choice(("tree", "window", "compact", "copy", "pages"))
    batch = _log(rng, 1, 32)
    far = 32768 if dtype == "bf16" else 4096
    if op == "tree":
        most = max(1, 1024 // batch)
        new = [_log(rng, 1, min(256, most)) for _ in range(batch)]
        past = [rng.choice((0, _log(rng, 1, far), _log(rng, 1, far))) for _ in range(batch)]
        return _case("", op, new, past, **shape)
    if op == "window":
        window, sinks = _log(rng, 1, 8192), rng.choice((0, 1, 4, _log(rng, 1, 500)))
        if rng.random() < 0.4:       # one token per sequence
            past = [_log(rng, 1, far) - 1 for _ in range(batch)]
            return _case("", op, (1,) * batch, past, window=window, sinks=sinks,
                         packed=rng.choice((False, True)), **shape)
        total = _log(rng, batch, 8192 if dtype == "bf16" else 4096)
        cuts = sorted(rng.randrange(total + 1) for _ in range(batch - 1))
        new = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        past = [rng.choice((0, _log(rng, 1, far))) for _ in range(batch)]
        return _case("", op, new, past, window=window, sinks=sinks, packed=True, **shape)
    if op == "compact":
        if rng.random() < 0.3:
            return _case("", op, (_log(rng, 500, far),), (0,), kept="evict", **shape)
        new = [_log(rng, 1, 256) for _ in range(batch)]
        past = [_log(rng, 1, 4096) - 1 for _ in range(batch)]
        return _case("", op, new, past, kept="accept", **shape)
    if op == "copy":
        big = hkv * shape["ps"] * shape["d"] * (2 if dtype == "bf16" else 4)
        return _case("", op, (_log(rng, 1, max(2, min(4000, (1 << 28) // big))),), (0,), **shape)
    pool = _log(rng, 4096, 262144)
    if rng.random() < 0.5:
        beams = rng.choice((2, 3, 4, 8))
        rows = beams * _log(rng, 1, min(32, pool // (64 * beams)))
        length = [_log(rng, 1, min(8000, 10 * pool // rows)) for _ in range(rows // beams)]
        past = [length[i // beams] for i in range(rows)]
        new = [rng.choice((1, 1, 40)) for _ in range(rows)]
        return _case("", op, new, past, window=0, sinks=0, beams=beams, stride=1024, pool=pool,
                     **shape)
    rows = _log(rng, 1, min(256, pool // 64))
    past = [_log(rng, 1, min(60000, 10 * pool // rows)) for _ in range(rows)]
    new = [rng.choice((0, 1, 1, 1, _log(rng, 2, 200))) for _ in range(rows)]
    return _case("", op, new, past, window=rng.choice((0, _log(rng, 1, 8192))),
                 sinks=rng.choice((0, 4, 100)), beams=0, stride=4096, pool=pool, **shape)


def _lengths(case):
    return ([int(x) for x in case["new"].split(",")], [int(x) for x in case["past"].split(",")])


def _tree(rng, n):
    """Parents of n drafted nodes: most extend a recent branch, some start at the cache's end."""
    parents, depth = [], []
    for i in range(n):
        p = -1 if i == 0 or rng.random() < 0.1 else rng.randrange(max(0, i - 12), i)
        if p >= 0 and depth[p] >= 15:
            p = -1
        parents.append(p)
        depth.append(0 if p < 0 else depth[p] + 1)
    return parents


def _dead(case, p, first):
    """Whether page p holds no token that a row at position `first` or later sees."""
    ps, window = case["ps"], case.get("window", 0)
    return window > 0 and p * ps >= case["sinks"] and (p + 1) * ps <= first - window + 1


def prepare(case, seed):
    """The cache as the steps before left it, and what the step brings."""
    if case["op"] == "pages":
        return _prepare_pages(case, seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    new, past = _lengths(case)
    op, hq, hkv, d, ps = case["op"], case["hq"], case["hkv"], case["d"], case["ps"]
    B, T = len(new), sum(new)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(dt)

    s = {"case": case, "new": new, "past": past, "scale": 1.0 / math.sqrt(d)}
    if op == "copy":
        pages, total = [], 2 * T + 7
    else:
        pages = [-(-(n + p) // ps) for n, p in zip(new, past)]
        total = sum(pages) + 3
    s["k_pool"], s["v_pool"] = rand(total, hkv, ps, d), rand(total, hkv, ps, d)
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    if op in ("copy", "compact"):
        keys = s["k_pool"].float()
        s["stats"] = torch.stack([keys.amin(2), keys.amax(2)], dim=2).to(dt).contiguous()
    if op == "copy":
        s["pairs"] = order[:2 * T].view(T, 2).contiguous()
        s["table"] = order[:1].view(1, 1).contiguous()
        s["lens"] = torch.ones(1, dtype=torch.int32, device=dev)
    else:
        rows = torch.full((B, max(max(pages), 1)), -1, dtype=torch.int32)
        place, at = order.cpu(), 0
        for b, n in enumerate(pages):
            rows[b, :n] = place[at:at + n]
            at += n
            if op == "window":           # pages that fell out of the window were given back
                for p in range(n):
                    if _dead(case, p, past[b]):
                        rows[b, p] = -1
        s["table"] = rows.to(dev)
        s["lens"] = torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32, device=dev)
        s["cu"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    if op in ("tree", "window"):
        # trained keys: the first token of a sequence draws much of the attention, and queries
        # are not of unit variance
        q = torch.randn((T, hq, d), generator=gen, device=dev)
        mean = q.view(T, hkv, hq // hkv, d).mean((0, 2))
        first = [b for b, n in enumerate(pages) if n and s["table"][b, 0] >= 0]
        if first:
            s["k_pool"][s["table"][first, 0].long(), :, 0] = (
                4.0 * mean / mean.norm(dim=-1, keepdim=True)).to(dt)
        s["q"] = (1.5 * q).to(dt)
    if op == "tree":
        s["trees"] = [_tree(rng, n) for n in new]
        s["parents"] = torch.tensor([p for t in s["trees"] for p in t], dtype=torch.int32,
                                    device=dev)
    if op == "compact":
        kept = []
        for n in new:
            if case["kept"] == "evict":
                some = rng.sample(range(n), n // 8)
                kept.append(sorted(set(some) | set(range(min(n, 4))) | set(range(n - n // 64, n))))
            else:
                kept.append(sorted(rng.sample(range(n), min(n, rng.choice((0, 1, 2, 3, 4, 6, 9))))))
        most = max(1, max(map(len, kept)))
        s["kept"] = kept
        s["keep"] = torch.tensor([k + [-1] * (most - len(k)) for k in kept], dtype=torch.int32,
                                 device=dev)
        s["keep_cnt"] = torch.tensor([len(k) for k in kept], dtype=torch.int32, device=dev)
    if own:
        import sparse_kv_cache_build_gb300 as skv
        s["kv"] = skv.PagedKV(s["k_pool"], s["v_pool"], s["table"], s["lens"])
        if op in ("tree", "window"):
            n = skv.kv_prefill_attn_workspace_size(s["kv"], hq, T)
            s["workspace"] = torch.empty((n,), dtype=torch.uint8, device=dev)
    return s


def _prepare_pages(case, seed):
    """Two page tables used in turn, as a fork writes the next batch beside the present one."""
    dev = "cuda"
    rng = random.Random(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    new, past = _lengths(case)
    ps, pool, beams, B = case["ps"], case["pool"], case["beams"], len(new)
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.full((B, case["stride"]), -1, dtype=torch.int32)
    refs = torch.zeros(pool, dtype=torch.int32)
    at = 0
    for b in range(B):
        held = past[b] // ps if beams and b % beams else 0      # full pages shared with beam 0
        if held:
            table[b, :held] = table[b - b % beams, :held]
        n = -(-past[b] // ps)
        for p in range(held, n):
            if not _dead(case, p, max(past[b] - 1, 0)):
                table[b, p] = order[at]
                at += 1
    used = table[table >= 0].long()
    refs += torch.bincount(used, minlength=pool).to(torch.int32)
    refs[order[at:at + 100].long()] += 1                        # pages that another holder keeps
    s = {"case": case, "new": new, "past": past, "table": table.to(dev), "refs": refs.to(dev)}
    s["other"] = torch.full_like(s["table"], -1)
    s["keep"] = torch.tensor(past, dtype=torch.int32, device=dev)
    s["want"] = torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32, device=dev)
    s["lens"] = s["want"].clone()       # the step before was undone: its tokens are dropped
    s["parents"] = None
    if beams:
        s["parents"] = torch.tensor([b - b % beams + rng.randrange(beams) for b in range(B)],
                                    dtype=torch.int32, device=dev)
    if own:
        import sparse_kv_cache_build_gb300 as skv
        kp = torch.empty((pool, 1, ps, 64), dtype=torch.bfloat16, device=dev)
        s["kv"] = skv.PagedKV(kp, kp, s["table"], s["lens"])
        s["kv_other"] = skv.PagedKV(kp, kp, s["other"], s["lens"])
    return s


# ---------------------------------------------------------------------- the plain forms

def _gathered(s, b, idx):
    """Keys and values of sequence b's tokens idx in 32 bits: [Hkv][tokens][D] each."""
    ps = s["case"]["ps"]
    page, slot = s["table"][b].long()[idx // ps], idx % ps
    return (s["k_pool"][page, :, slot].float().transpose(0, 1),
            s["v_pool"][page, :, slot].float().transpose(0, 1))


def _softmax_rows(q, K, V, seen, scale):
    """q [n][Hq][D] over K, V [Hkv][L][D] where `seen` [n][L]: out and lse in 32 bits."""
    n, hq, d = q.shape
    hkv, L = K.shape[0], K.shape[1]
    x = q.float().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    x = torch.bmm(x, K.transpose(1, 2)).mul_(scale).view(hkv, hq // hkv, n, L)
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(hkv, -1, L), V).view(hkv, hq // hkv, n, d) / l
    return (o.permute(2, 0, 1, 3).reshape(n, hq, d),
            (m + l.log()).squeeze(-1).permute(2, 0, 1).reshape(n, hq))


def _ancestors(parents):
    """[n][n]: whether node j is node i or one of its ancestors."""
    n = parents.numel()
    above = torch.eye(n, dtype=torch.bool, device=parents.device)
    up = parents.long()
    for _ in range(max(1, n - 1).bit_length()):
        has = up >= 0
        at = up.clamp(min=0)
        above = above | (above[at] & has[:, None])
        up = torch.where(has, up[at], up)
    return above


def _plain_tree(s):
    q, dev = s["q"], s["q"].device
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)
    at = 0
    for b, (n, p) in enumerate(zip(s["new"], s["past"])):
        K, V = _gathered(s, b, torch.arange(n + p, device=dev))
        seen = torch.ones((n, n + p), dtype=torch.bool, device=dev)
        seen[:, p:] = _ancestors(s["parents"][at:at + n])
        o, l = _softmax_rows(q[at:at + n], K, V, seen, s["scale"])
        out[at:at + n], lse[at:at + n] = o.to(q.dtype), l
        at += n
    return [out, lse]


def _plain_window(s):
    q, dev = s["q"], s["q"].device
    window, sinks = s["case"]["window"], s["case"]["sinks"]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)
    at = 0
    for b, (n, p) in enumerate(zip(s["new"], s["past"])):
        for i in range(0, n, 1024):                  # blocks of rows, so that the scores fit
            e = min(n, i + 1024)
            lo = max(0, p + i - window + 1)          # the first token the block's window holds
            idx = torch.cat((torch.arange(min(sinks, lo), device=dev),
                             torch.arange(lo, p + e, device=dev)))
            K, V = _gathered(s, b, idx)
            pos = torch.arange(p + i, p + e, device=dev)[:, None]
            seen = (idx <= pos) & ((idx > pos - window) | (idx < sinks))
            o, l = _softmax_rows(q[at + i:at + e], K, V, seen, s["scale"])
            out[at + i:at + e], lse[at + i:at + e] = o.to(q.dtype), l
        at += n
    return [out, lse]


def _plain_compact(s):
    ps, dev = s["case"]["ps"], s["table"].device
    lens, table = s["lens"].long(), s["table"].long()
    counts = s["cu"][1:].long() - s["cu"][:-1].long()
    start, cnt = lens - counts, s["keep_cnt"].long()
    i = torch.arange(s["keep"].shape[1], device=dev)
    seq, i = torch.nonzero(i < cnt[:, None], as_tuple=True)
    src, dst = start[seq] + s["keep"].long()[seq, i], start[seq] + i
    sp, dp = table[seq, src // ps], table[seq, dst // ps]
    k, v = s["k_pool"][sp, :, src % ps], s["v_pool"][sp, :, src % ps]
    s["k_pool"][dp, :, dst % ps] = k
    s["v_pool"][dp, :, dst % ps] = v
    # statistics of every page from the first one with candidates to the last kept token
    fresh = start + cnt
    p = torch.arange(table.shape[1], device=dev)
    seq, p = torch.nonzero((p >= (start // ps)[:, None]) & (p * ps < fresh[:, None]), as_tuple=True)
    page = table[seq, p]
    keys = s["k_pool"][page].float()
    gone = (p * ps)[:, None] + torch.arange(ps, device=dev) >= fresh[seq][:, None]
    gone = gone[:, None, :, None]
    s["stats"][page, :, 0] = keys.masked_fill(gone, math.inf).amin(2).to(s["stats"].dtype)
    s["stats"][page, :, 1] = keys.masked_fill(gone, -math.inf).amax(2).to(s["stats"].dtype)
    return [s["k_pool"], s["v_pool"], s["stats"], fresh.to(torch.int32)]


def _plain_copy(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    for x in (s["k_pool"], s["v_pool"], s["stats"]):
        x[dst] = x[src]
    return [s["k_pool"], s["v_pool"], s["stats"]]


def _plain_pages(s, old, out):
    case, ps = s["case"], s["case"]["ps"]
    refs, keep, want = s["refs"], s["keep"].long(), s["want"].long()
    dev, NP = refs.device, refs.numel()
    B, stride = old.shape
    rows = old.long() if s["parents"] is None else old.long()[s["parents"].long()]
    p = torch.arange(stride, device=dev)
    first = (keep + ps - 1) // ps
    held = p < first[:, None]
    if case["window"] > 0:
        held &= (p * ps < case["sinks"]) | ((p + 1) * ps > (keep - case["window"] + 1)[:, None])
    rows = torch.where(held, rows, -1)
    for x, sign in ((rows, 1), (old.long(), -1)):
        counts = torch.bincount(torch.where(x >= 0, x, NP).flatten(), minlength=NP + 1)[:NP]
        refs += sign * counts.to(torch.int32)
    # a partial page that another row holds too is replaced, except for its last holder
    grows = (want > keep) & (keep % ps != 0)
    part = torch.where(grows, rows.gather(1, (first - 1).clamp(min=0)[:, None])[:, 0], NP)
    part = torch.where(part >= 0, part, NP)
    b = torch.arange(B, device=dev)
    growing = torch.bincount(part, minlength=NP + 1)
    last = torch.full((NP + 1,), -1, device=dev).scatter_reduce(0, part, b, "amax")
    only = torch.cat((refs.long(), refs.new_zeros(1).long())) == growing
    fork = (part < NP) & ~(only[part] & (last[part] == b))
    refs -= torch.bincount(torch.where(fork, part, NP), minlength=NP + 1)[:NP].to(torch.int32)
    # the lowest free pages, in the order of the rows
    need = (want + ps - 1) // ps - first + fork.long()
    free = torch.nonzero(refs == 0)[:, 0]
    total = int(need.sum())
    fresh = free[:total]
    refs[fresh] = 1
    seq = torch.repeat_interleave(b, need)
    rank = torch.arange(total, device=dev) - (need.cumsum(0) - need)[seq]
    rows[seq, first[seq] + rank - fork[seq].long()] = fresh
    copies = torch.full((B, 2), -1, dtype=torch.int32, device=dev)
    at = torch.nonzero(fork)[:, 0]
    copies[at, 0] = part[at].to(torch.int32)
    copies[at, 1] = rows[at, first[at] - 1].to(torch.int32)
    out.copy_(rows.to(torch.int32))
    left = torch.tensor([free.numel() - total], dtype=torch.int32, device=dev)
    return [out, refs, copies, left]


def run(state):
    case, op = state["case"], state["case"]["op"]
    if op == "pages":
        old, out = state["table"], state["other"] if case["beams"] else state["table"]
        if case["beams"]:                # the next pass goes the other way
            state["table"], state["other"] = out, old
        if not own:
            return _plain_pages(state, old, out)
        import sparse_kv_cache_build_gb300 as skv
        kv = state["kv"]
        if case["beams"]:
            state["kv"], state["kv_other"] = state["kv_other"], kv
        _, copies, left = skv.kv_update_pages(
            kv, state["refs"], state["want"], keep_lens=state["keep"], parents=state["parents"],
            window=case["window"], sinks=case["sinks"], table=out)
        return [out, state["refs"], copies, left]
    if not own:
        return {"tree": _plain_tree, "window": _plain_window, "compact": _plain_compact,
                "copy": _plain_copy}[op](state)
    import sparse_kv_cache_build_gb300 as skv
    kv = state["kv"]
    if op == "tree":
        return list(skv.kv_tree_attn(kv, state["q"], state["scale"], state["parents"],
                                     cu_tokens=state["cu"], workspace=state["workspace"]))
    if op == "window":
        return list(skv.kv_window_attn(kv, state["q"], state["scale"], case["window"],
                                       case["sinks"], workspace=state["workspace"],
                                       cu_tokens=state["cu"] if case["packed"] else None))
    if op == "compact":
        lens = skv.kv_compact(kv, state["keep"], state["keep_cnt"], state["stats"],
                              cu_tokens=state["cu"])
        return [state["k_pool"], state["v_pool"], state["stats"], lens]
    skv.kv_copy_pages(kv, state["pairs"], state["stats"])
    return [state["k_pool"], state["v_pool"], state["stats"]]


def work(case):
    new, past = _lengths(case)
    e = 2 if case["dtype"] == "bf16" else 4
    T, op, hq, hkv, d, ps = sum(new), case["op"], case["hq"], case["hkv"], case["d"], case["ps"]
    token = 2 * hkv * d * e                              # keys and values of one token
    rows = T * hq * (2 * d * e + 4)
    if op == "tree":
        # a node's ancestors are few beside the cache: a quarter of the square at most
        pairs = sum(n * p + min(n * n // 4 + n, 8 * n) for n, p in zip(new, past))
        return {"bytes": token * (T + sum(past)) + rows, "flops": 4 * pairs * hq * d}
    if op == "window":
        w, k = case["window"], case["sinks"]
        read = pairs = 0
        for n, p in zip(new, past):
            if n == 0:
                continue
            lo = max(0, p - w + 1)
            read += n + p - lo + min(k, lo)
            m = min(max(w + k, p), n + p)                # below m a row sees every token
            pairs += (m - p) * (m + p + 1) // 2 + (n + p - m) * (w + k)
        return {"bytes": token * read + rows, "flops": 4 * pairs * hq * d}
    if op == "compact":
        kept = sum(n // 8 + n // 64 if case["kept"] == "evict" else min(n, 4) for n in new)
        pages = sum(1 + (n // 8 // ps if case["kept"] == "evict" else 0) for n in new)
        return {"bytes": 2 * token * kept + pages * hkv * 2 * d * e, "flops": 2 * kept * hkv * d}
    if op == "copy":
        return {"bytes": 2 * T * (ps * token + hkv * 2 * d * e), "flops": 0}
    # entries of pages in use read and written, and one look at every page's count
    w = case["window"]
    used = sum(-(-min(p, w + case["sinks"] + 2 * ps if w else p) // ps) for p in past)
    return {"bytes": 2 * 4 * used + 4 * case["pool"], "flops": 0}


# ---------------------------------------------------- the definitions, token by token

def _rows64(s, b, at, i, e, hidden):
    """Rows at + i .. at + e of sequence b over its first tokens, `hidden` [rows][tokens]."""
    case, ps = s["case"], s["case"]["ps"]
    G, L = case["hq"] // case["hkv"], hidden.shape[1]
    where = torch.arange(L, device="cuda")
    phys = s["table"][b].long()[where // ps]
    out = torch.empty((e - i, case["hq"], case["d"]), dtype=torch.float64, device="cuda")
    lse = torch.empty((e - i, case["hq"]), dtype=torch.float64, device="cuda")
    some = torch.nonzero(~hidden.all(0))[:, 0]            # tokens that no row sees are not read
    hide = hidden[:, some]
    for g in range(case["hkv"]):
        K = s["k_pool"][phys[some], g, where[some] % ps].double()
        V = s["v_pool"][phys[some], g, where[some] % ps].double()
        for h in range(g * G, (g + 1) * G):
            z = s["q"][at + i:at + e, h].double() @ K.T * s["scale"]
            z[hide] = -math.inf
            top = z.max(1).values
            w = torch.exp(z - top[:, None])
            total = w.sum(1)
            out[:, h] = (w @ V) / total[:, None]
            lse[:, h] = top + torch.log(total)
    return out, lse


def exact(case, seed):
    """The same outputs in 64 bits from the definitions; page tables are whole numbers that the
    plain form's rule fixes, and have no such value."""
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    new, past, ps = s["new"], s["past"], case["ps"]
    if case["op"] in ("tree", "window"):
        outs, lses, at = [], [], 0
        for b, (n, p) in enumerate(zip(new, past)):
            for i in range(0, n, 512):
                e = min(n, i + 512)
                where = torch.arange(p + e, device="cuda")
                pos = torch.arange(p + i, p + e, device="cuda")[:, None]
                if case["op"] == "window":
                    hidden = (where > pos) | ((where <= pos - case["window"]) &
                                              (where >= case["sinks"]))
                else:
                    hide = [[True] * e for _ in range(i, e)]
                    for r in range(i, e):
                        node = r
                        while node >= 0:
                            hide[r - i][node] = False
                            node = s["trees"][b][node]
                    hidden = torch.zeros((e - i, p + e), dtype=torch.bool, device="cuda")
                    hidden[:, p:] = torch.tensor(hide, device="cuda")
                o, l = _rows64(s, b, at, i, e, hidden)
                outs.append(o)
                lses.append(l)
            at += n
        return [torch.cat(outs), torch.cat(lses)]
    k, v, stats = s["k_pool"].double(), s["v_pool"].double(), s["stats"].double()
    if case["op"] == "copy":
        for x in (k, v, stats):
            before = x.clone()
            for a, b in s["pairs"].tolist():
                x[b] = before[a]
        return [k, v, stats]
    table = s["table"].tolist()
    for b, (n, p, kept) in enumerate(zip(new, past, s["kept"])):
        for i, j in enumerate(kept):                      # kept tokens only move forward
            if i != j:
                A, a, C, c = table[b][(p + j) // ps], (p + j) % ps, table[b][(p + i) // ps], \
                    (p + i) % ps
                k[C, :, c], v[C, :, c] = k[A, :, a].clone(), v[A, :, a].clone()
        length = p + len(kept)
        for page in range(p // ps, -(-length // ps)):
            part = k[table[b][page], :, :length - page * ps]
            stats[table[b][page], :, 0], stats[table[b][page], :, 1] = part.amin(1), part.amax(1)
    lens = torch.tensor([p + len(x) for p, x in zip(past, s["kept"])], device="cuda")
    return [k, v, stats, lens]
