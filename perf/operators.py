"""Cases for the operators around drafted tokens and cache eviction: attention of
a tree of drafted tokens over the paged cache, the attention weight every cached
token has received, the choice of the tokens a cache keeps, and the move that
compacts it (which also commits an accepted path of drafted tokens).

`run` computes them in plain torch operations, or, where `own` is set, through
sparse_kv_b200.
"""
import math
import random

import torch

own = False

DEV = "cuda"
D = 128       # head dimension
PAGE = 64     # tokens per page


# ------------------------------------------------------------------ the cases

def _tree(name, B, Hq, Hkv, L, T, ragged=False, tree=True, softcap=0.0, alibi=False, sink=0, recent=0):
    return dict(name=name, op="tree", B=B, Hq=Hq, Hkv=Hkv, L=L, T=T, ragged=ragged, tree=tree,
                softcap=softcap, alibi=alibi, sink=sink, recent=recent)


def _mass(name, B, Hq, Hkv, L, T, **kw):
    return dict(_tree(name, B, Hq, Hkv, L, T, **kw), op="mass")


def _select(name, B, Hkv, L, keep, sink, recent, ragged=False):
    return dict(name=name, op="select", B=B, Hkv=Hkv, L=L, keep=keep, sink=sink, recent=recent, ragged=ragged)


def _compact(name, kind, B, Hkv, L, keep, ragged=False):
    return dict(name=name, op="compact", kind=kind, B=B, Hkv=Hkv, L=L, keep=keep, ragged=ragged)


def listed():
    return [
        # one request, a short context, a small tree of drafts: the time of a call that moves little
        _tree("tree_b1_h8_l4k_t8", 1, 8, 2, 4096, 8),
        # a serving batch of 32-head models over 32k-token caches, 16 drafted tokens each
        _tree("tree_b16_h32_l32k_t16", 16, 32, 8, 32768, 16),
        # 128k-token caches and wide trees: 256 rows for each KV head
        _tree("tree_b4_h32_l128k_t64", 4, 32, 8, 131072, 64),
        # ragged lengths and draft counts in one batch; capped scores and a distance bias
        _tree("tree_b7_h16_l24k_t13_cap_bias", 7, 16, 2, 24001, 13, ragged=True, softcap=30.0, alibi=True),
        # sparse layers of a routed stack: sink + recent window, a chain of drafts
        _tree("tree_b8_h32_l128k_t4_window", 8, 32, 8, 131071, 4, tree=False, sink=64, recent=4096),
        # attention weight after each decoded token of the serving batch
        _mass("mass_b16_h32_l32k_t1", 16, 32, 8, 32768, 1),
        # ragged, capped, after a tree of drafts; odd lengths
        _mass("mass_b5_h32_l9k_t16_cap", 5, 32, 4, 9001, 16, ragged=True, softcap=50.0),
        # one request, 128k tokens, a wide tree
        _mass("mass_b1_h32_l128k_t64", 1, 32, 8, 131072, 64),
        # the kept tokens of one short cache, and of a batch of long ones
        _select("select_b1_l4k", 1, 2, 4096, 1024, 64, 256),
        _select("select_b8_l128k", 8, 8, 131071, 16384, 64, 4096, ragged=True),
        # eviction in place, 32k tokens to 4k
        _compact("evict_b16_l32k_to_4k", "evict", 16, 8, 32768, 4096),
        # the accepted path of 16 drafted tokens, at the end of 32k-token caches
        _compact("commit_b16_l32k_t16", "commit", 16, 8, 32768, 16, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "mass", "mass", "select", "compact"])
    B, Hkv = _log(rng, 1, 16), rng.choice([1, 2, 4, 8])
    # at most the token count of the largest listed cases
    L = _log(rng, 64, min(131072, 16 * 8 * 32768 // (B * Hkv)))
    if op in ("tree", "mass"):
        Hq = Hkv * rng.choice([1, 2, 4, 8])
        most = 4 * 32 * 64 * 131072 if op == "tree" else 32 * 64 * 131072
        T = max(1, min(_log(rng, 1, 64), most // (B * Hq * L), L))
        window = rng.random() < 0.25
        kw = dict(ragged=rng.random() < 0.5, tree=rng.random() < 0.7, alibi=rng.random() < 0.3,
                  softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), sink=64 if window else 0,
                  recent=_log(rng, 16, 4096) if window else 0)
        return {k: v for k, v in (_tree if op == "tree" else _mass)("", B, Hq, Hkv, L, T, **kw).items()
                if k != "name"}
    if op == "select":
        keep = _log(rng, 1, L * 3 // 4)
        sink = rng.randrange(0, min(64, keep // 4) + 1)
        recent = rng.randrange(0, keep // 4 + 1)
        c = _select("", B, Hkv, L, keep, sink, recent, ragged=rng.random() < 0.5)
    else:
        kind = rng.choice(["evict", "copy", "commit"])
        # the cache is read, its kept tokens written: no more tokens than eight 32k caches
        L = min(L, max(64, 8 * 8 * 32768 // (B * Hkv)))
        keep = min(_log(rng, 1, 64), L) if kind == "commit" else _log(rng, 1, L)
        c = _compact("", kind, B, Hkv, L, keep, ragged=rng.random() < 0.5)
    return {k: v for k, v in c.items() if k != "name"}


def _lens(case):
    """Tokens and drafted tokens of every sequence."""
    B, L = case["B"], case["L"]
    T = case.get("T", case["keep"] if case.get("kind") == "commit" else 0)
    if not case["ragged"]:
        return [L] * B, [T] * B
    r = random.Random(L * 131 + B)
    lens = [L] + [max(T, r.randint(max(1, L // 8), L)) for _ in range(B - 1)]
    drafts = [T] + [r.randint(min(1, T), T) for _ in range(B - 1)]
    return lens, drafts


def _seen(case):
    """Cached tokens that some row of a tree case sees, per KV head, and (row, key) pairs over all heads."""
    tokens = pairs = 0
    for n, t in zip(*_lens(case)):
        ctx, k = n - t, n
        if case["sink"] or case["recent"]:
            k = min(n, case["sink"] + case["recent"] + t)
            ctx = k - t
        tokens += k
        pairs += (ctx * t + t * (t + 1) // 2) * case["Hq"]
    return tokens, pairs


def work(case):
    lens, drafts = _lens(case)
    Hkv = case["Hkv"]
    if case["op"] in ("tree", "mass"):
        tokens, pairs = _seen(case)
        rows = sum(drafts) * case["Hq"]
        if case["op"] == "tree":
            return dict(bytes=tokens * Hkv * 512 + rows * (256 + 512 + 4), flops=4 * D * pairs)
        return dict(bytes=tokens * Hkv * 256 + sum(lens) * Hkv * 8 + rows * (256 + 4), flops=2 * D * pairs)
    if case["op"] == "select":
        return dict(bytes=Hkv * (4 * sum(lens) + 4 * sum(min(n, case["keep"]) for n in lens)), flops=0)
    if case["kind"] == "commit":  # an accepted path of half the drafts moves
        moved = sum((t + 1) // 2 for t in drafts)
        return dict(bytes=moved * Hkv * 1024 + case["B"] * 4, flops=0)
    kept = sum(min(n, case["keep"]) for n in lens)
    return dict(bytes=kept * Hkv * (1024 + 4 + 8), flops=0)


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _paged(B, lens, g):
    """A block table over shuffled pages (entries past a sequence's end are -1) and the page count."""
    mb = (max(lens) + PAGE - 1) // PAGE
    nb = torch.tensor([(n + PAGE - 1) // PAGE for n in lens], device=DEV)
    pages = int(sum((n + PAGE - 1) // PAGE for n in lens))
    table = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(mb, device=DEV)[None] < nb[:, None]] = torch.randperm(pages, generator=g, device=DEV).int()
    return table, pages


def _pools(case, g, lens):
    table, pages = _paged(case["B"], lens, g)
    shape = (pages, case["Hkv"], PAGE, D)
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    return k, v, table


def _ancestors(drafts, T, g):
    """Ancestor masks of random trees, one 64-bit word per row: each drafted token hangs below an earlier one."""
    B = len(drafts)
    parent = (torch.rand((B, T), generator=g, device=DEV) * torch.arange(T, device=DEV)).long()
    rows = torch.zeros((B, T), dtype=torch.int64, device=DEV)
    one = torch.ones((B,), dtype=torch.int64, device=DEV)
    for t in range(T):
        above = rows.gather(1, parent[:, t:t + 1])[:, 0] if t else torch.zeros_like(one)
        rows[:, t] = above | (one << t)
    return rows


def prepare(case, seed):
    g = _generator(seed)
    lens, drafts = _lens(case)
    s = dict(case=case, max_len=max(lens), seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    B, Hkv = case["B"], case["Hkv"]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    s["status"] = status
    if case["op"] == "select":
        # accumulated weights: many octaves, and tokens that nothing has looked at
        m = torch.exp2(torch.randn((B, Hkv, case["L"]), generator=g, device=DEV) * 3 - 8)
        m[torch.rand(m.shape, generator=g, device=DEV) < 0.2] = 0
        s["mass"] = m
        s["ids"] = torch.full((B, Hkv, case["keep"]), -1, dtype=torch.int32, device=DEV)
        s["keep_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        return s
    s["k"], s["v"], s["table"] = _pools(case, g, lens)
    if case["op"] == "compact":
        n = s["seq_lens"].long()
        heads = 1 if case["kind"] == "commit" else Hkv
        if case["kind"] == "commit":
            t = torch.tensor(drafts, device=DEV)
            s["first"] = (n - t).int()
            kept = (t + 1) // 2
            span, base = t, n - t
        else:
            s["first"] = None
            kept = torch.clamp(n, max=case["keep"])
            span, base = n, torch.zeros_like(n)
        width = max(1, case["keep"])
        top = int(span.max())
        # a random subset of `kept` positions of [0, span), ascending
        r = torch.rand((B, heads, top), generator=g, device=DEV)
        r = r.masked_fill(torch.arange(top, device=DEV)[None, None] >= span[:, None, None], 2.0)
        order = r.argsort(-1)[..., :width]
        order = order.masked_fill(torch.arange(order.shape[-1], device=DEV) >= kept[:, None, None], 1 << 30)
        ids = order.sort(-1).values
        ids = torch.where(ids < (1 << 30), ids + base[:, None, None], torch.full_like(ids, -1)).int()
        s["ids"] = torch.nn.functional.pad(ids, (0, width - ids.shape[-1]), value=-1).contiguous()
        s["keep_lens"] = kept.int()
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["mass"] = None
        if case["kind"] != "commit":
            s["mass"] = torch.rand((B, Hkv, case["L"]), generator=g, device=DEV)
        if case["kind"] == "copy":  # to pages of another pool
            table, pages = _paged(B, [min(x, case["keep"]) for x in lens], g)
            s["to"] = (torch.zeros((pages, Hkv, PAGE, D), dtype=torch.bfloat16, device=DEV),
                       torch.zeros((pages, Hkv, PAGE, D), dtype=torch.bfloat16, device=DEV), table)
        return s
    T, Hq = case["T"], case["Hq"]
    s["q"] = torch.randn((B, T, Hq, D), generator=g, device=DEV, dtype=torch.bfloat16)
    # a direction that queries share with the first token and one cached token in a hundred: attention
    # sinks and heavy tokens
    u = torch.nn.functional.normalize(torch.randn((Hkv, D), generator=g, device=DEV), dim=-1)
    s["q"] = (s["q"].float() + 4 * u.repeat_interleave(Hq // Hkv, 0)).bfloat16()
    heavy = torch.rand(s["k"].shape[:3], generator=g, device=DEV) < 0.01
    heavy[s["table"][:, 0].long(), :, 0] = True
    s["k"] += (heavy[..., None] * (6 * u)[None, :, None]).bfloat16()
    s["tree_lens"] = torch.tensor(drafts, dtype=torch.int32, device=DEV)
    s["tree"] = _ancestors(drafts, T, g) if case["tree"] else None
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq) if case["alibi"] else None
    s["window"] = (case["sink"], case["recent"]) if case["sink"] or case["recent"] else None
    s["scale"] = 1 / math.sqrt(D)
    if case["op"] == "tree":
        s["out"] = torch.zeros((B, T, Hq, D), device=DEV)
        s["lse"] = torch.zeros((B, T, Hq), device=DEV)
        if own:
            import sparse_kv_b200 as skv
            n = skv.tree_workspace_size(s["q"], s["k"], s["v"], s["table"], s["seq_lens"], s["out"], s["lse"],
                                        **_options(s))
            s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        return s
    s["lse"] = torch.empty((B, T, Hq), device=DEV)
    for b in range(B):  # what the attention call before this one returned
        s["lse"][b] = torch.logsumexp(_scores(s, b, 1)[0], -1).view(Hq, T).t()
    s["weight"] = (torch.rand((B, T), generator=g, device=DEV) < 0.7).float()  # accepted drafts count
    s["weight"][:, 0] = 1
    s["prev"] = torch.rand((B, Hkv, case["L"]), generator=g, device=DEV)
    s["mass"] = torch.zeros((B, Hkv, case["L"]), device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _tokens(pool, table):
    """[n, Hkv, tokens, D] in 32 bits of the sequences in `table`."""
    x = pool[table.long().clamp(min=0)].float()
    n, mb, h = x.shape[:3]
    return x.transpose(1, 2).reshape(n, h, mb * PAGE, D)


def _scores(s, b, n):
    """Scores [n, Hkv, G * T, tokens] of the sequences b .. b + n - 1, -inf where a row does not look."""
    c = s["case"]
    T, Hq, Hkv = c["T"], c["Hq"], c["Hkv"]
    k = _tokens(s["k"], s["table"][b:b + n])
    q = s["q"][b:b + n].float().view(n, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    z = torch.matmul(q.reshape(n, Hkv, -1, D), k.transpose(-1, -2)).view(n, Hkv, Hq // Hkv, T, -1)
    z *= s["scale"]
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    at = torch.arange(z.shape[-1], device=DEV)
    t = torch.arange(T, device=DEV)
    length, drafts = s["seq_lens"][b:b + n].long(), s["tree_lens"][b:b + n].long()
    ctx = (length - drafts)[:, None]
    sees = t[:, None] >= t if s["tree"] is None else (s["tree"][b:b + n, :, None] >> t) & 1 == 1
    sees = sees.expand(n, T, T) & (t < drafts[:, None])[:, None]                    # row, drafted token
    depth = (sees & (t[:, None] != t)).sum(-1)
    j = at - ctx                                                                   # drafted token at a position
    inside = (j >= 0) & (j < drafts[:, None])
    where = j.clamp(0, T - 1)
    look = torch.where(inside[:, None], sees.gather(2, where[:, None].expand(n, T, -1)), (j < 0)[:, None])
    place = torch.where(inside, ctx + depth.gather(1, where), at)                  # position of a key
    row = ctx + depth                                                              # position of a row
    if s["window"]:
        look = look & ((place < c["sink"])[:, None] | (place[:, None] > row[..., None] - c["recent"]))
    if c["alibi"]:
        slope = s["slopes"].view(Hkv, Hq // Hkv)[None, :, :, None, None]
        z = z + slope * (place[:, None] - row[..., None]).float()[:, None, None]
    z = z.masked_fill(~look[:, None, None], -math.inf)
    return z.view(n, Hkv, -1, z.shape[-1]), look


def _plain_tree(s):
    c = s["case"]
    B, T, Hq = c["B"], c["T"], c["Hq"]
    z, look = _scores(s, 0, B)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    v = _tokens(s["v"], s["table"]).masked_fill(~look.any(1)[:, None, :, None], 0.0)
    out = torch.matmul(p, v) / total.clamp(min=1e-30)
    lse = (top + torch.log(total))[..., 0]
    live = (torch.arange(T, device=DEV) < s["tree_lens"][:, None])[..., None]
    out = out.view(B, Hq, T, D).transpose(1, 2)
    return torch.where(live[..., None], out, s["out"]), torch.where(live, lse.view(B, Hq, T).transpose(1, 2), s["lse"])


def _plain_mass(s):
    c = s["case"]
    B, T, Hq, Hkv, L = c["B"], c["T"], c["Hq"], c["Hkv"], c["L"]
    z, _ = _scores(s, 0, B)
    lse = s["lse"].view(B, T, Hkv, -1).permute(0, 2, 3, 1).reshape(B, Hkv, -1, 1)
    live = torch.arange(T, device=DEV) < s["tree_lens"][:, None]
    w = torch.where(live, s["weight"], torch.zeros_like(s["weight"]))[:, None, None].expand(B, Hkv, Hq // Hkv, T)
    p = torch.where(w.reshape(B, Hkv, -1, 1) > 0, torch.exp(z - lse), torch.zeros_like(z))
    new = 0.9 * s["prev"] + (p * w.reshape(B, Hkv, -1, 1)).sum(2)[..., :L]
    return torch.where((torch.arange(L, device=DEV) < s["seq_lens"][:, None])[:, None], new, s["mass"])


def _plain_select(s):
    c = s["case"]
    n, at = s["seq_lens"].long()[:, None, None], torch.arange(c["L"], device=DEV)
    keep = c["keep"]
    fixed = (at < c["sink"]) | (at >= n - c["recent"]) | (n <= keep)
    rank = s["mass"].masked_fill(fixed, math.inf).masked_fill(at >= n, -math.inf)
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    best = best.masked_fill(best >= n, 1 << 30).sort(-1).values
    ids = torch.where(best < (1 << 30), best, torch.full_like(best, -1)).int()
    return ids, torch.clamp(s["seq_lens"], max=keep)


def _plain_compact(s):
    c = s["case"]
    B, Hkv = c["B"], c["Hkv"]
    first = s["first"].long() if s["first"] is not None else torch.zeros(B, dtype=torch.long, device=DEV)
    ids = s["ids"].long().expand(B, Hkv, -1)
    i = torch.arange(ids.shape[-1], device=DEV)
    b, h, i = torch.nonzero((i < s["keep_lens"][:, None])[:, None].expand(ids.shape), as_tuple=True)
    src, dst = ids[b, h, i], first[b] + i
    page = s["table"][b, src // PAGE].long()
    to_k, to_v, to_table = s.get("to", (s["k"], s["v"], s["table"]))
    to_page = to_table[b, dst // PAGE].long()
    for pool, to in ((s["k"], to_k), (s["v"], to_v)):
        to[to_page, h, dst % PAGE] = pool[page, h, src % PAGE]
    if s["mass"] is not None:
        s["mass"][b, h, dst] = s["mass"][b, h, src]
    s["new_lens"].copy_(first + s["keep_lens"])
    return [to_k, to_v, s["new_lens"]] + ([s["mass"]] if s["mass"] is not None else [])


# ------------------------------------------------------------------ one pass

def _options(s):
    return dict(max_seq_len=s["max_len"], scale=s["scale"], tree_mask=s["tree"], tree_lens=s["tree_lens"],
                softcap=s["case"]["softcap"], slopes=s["slopes"], window=s["window"], status=s["status"])


def run(s):
    c = s["case"]
    if not own:
        return {"tree": _plain_tree, "mass": _plain_mass, "select": _plain_select, "compact": _plain_compact}[c["op"]](s)
    import sparse_kv_b200 as skv
    if c["op"] == "tree":
        skv.attn_tree_decode(s["q"], s["k"], s["v"], s["table"], s["seq_lens"], s["out"], s["lse"],
                             workspace=s["workspace"], **_options(s))
        return s["out"], s["lse"]
    if c["op"] == "mass":
        skv.attn_key_mass(s["q"], s["k"], s["table"], s["seq_lens"], s["lse"], s["mass"], row_weight=s["weight"],
                          prev=s["prev"], decay=0.9, **_options(s))
        return s["mass"]
    if c["op"] == "select":
        skv.attn_evict_select(s["mass"], s["seq_lens"], c["keep"], s["ids"], s["keep_lens"], sink=c["sink"],
                              recent=c["recent"], max_seq_len=s["max_len"], status=s["status"])
        return s["ids"], s["keep_lens"]
    skv.attn_compact_cache(s["k"], s["v"], s["table"], s["seq_lens"], s["ids"], s["keep_lens"], s["new_lens"],
                           first=s["first"], dst=s.get("to"), mass=s["mass"], max_seq_len=s["max_len"],
                           status=s["status"])
    to = s.get("to", (s["k"], s["v"]))
    return [to[0], to[1], s["new_lens"]] + ([s["mass"]] if s["mass"] is not None else [])


# ------------------------------------------------------------------ 64 bits, one sequence and KV head at a time

def _rows64(s, b, h):
    """Scores [T, G, L] in 64 bits of one KV head, straight from the definition; -inf where a row does not look."""
    c = s["case"]
    G, L, n = c["Hq"] // c["Hkv"], int(s["seq_lens"][b]), int(s["tree_lens"][b])
    ctx = L - n
    pages = s["table"][b, :(L + PAGE - 1) // PAGE].long()
    k = s["k"][pages, h].reshape(-1, D)[:L].double()
    q = s["q"][b, :n, h * G:(h + 1) * G].double()
    z = torch.einsum("tgd,ld->tgl", q, k) * s["scale"]
    if c["softcap"]:
        z = torch.tanh(z / c["softcap"]) * c["softcap"]
    word = [int(x) for x in s["tree"][b].tolist()] if s["tree"] is not None else [(2 << t) - 1 for t in range(n)]
    seen = [[j for j in range(n) if word[t] >> j & 1] for t in range(n)]
    depth = [sum(j != t for j in seen[t]) for t in range(n)]
    place = torch.arange(L, device=DEV, dtype=torch.float64)
    place[ctx:] = torch.tensor([ctx + d for d in depth], device=DEV, dtype=torch.float64)
    for t in range(n):
        hidden = torch.ones(L, dtype=torch.bool, device=DEV)
        hidden[:ctx] = False
        hidden[[ctx + j for j in seen[t]]] = False
        if s["window"]:
            hidden |= (place >= c["sink"]) & (place <= ctx + depth[t] - c["recent"])
        if c["alibi"]:
            z[t] += s["slopes"][h * G:(h + 1) * G, None].double() * (place - (ctx + depth[t]))
        z[t][:, hidden] = -math.inf
    return z


def exact(case, seed):
    if case["op"] == "select":
        return None
    s = prepare(case, seed)
    B, Hkv = case["B"], case["Hkv"]
    if case["op"] == "compact":
        to_k, to_v, to_table = s.get("to", (s["k"], s["v"], s["table"]))
        to_k, to_v = to_k.clone(), to_v.clone()
        mass = s["mass"].double() if s["mass"] is not None else None
        lens = []
        for b in range(B):
            n = int(s["keep_lens"][b])
            f = int(s["first"][b]) if s["first"] is not None else 0
            lens.append(f + n)
            at = torch.arange(f, f + n, device=DEV)
            page = to_table[b].long()[at // PAGE]
            for h in range(Hkv):
                ids = s["ids"][b, h if s["ids"].shape[1] > 1 else 0, :n].long()
                flat = s["table"][b].long()[ids // PAGE]
                to_k[page, h, at % PAGE] = s["k"][flat, h, ids % PAGE]
                to_v[page, h, at % PAGE] = s["v"][flat, h, ids % PAGE]
                if mass is not None:
                    mass[b, h, f:f + n] = s["mass"][b, h, ids].double()
        return [to_k, to_v, torch.tensor(lens, dtype=torch.int32, device=DEV)] + ([mass] if mass is not None else [])
    G = case["Hq"] // Hkv
    if case["op"] == "tree":
        out, lse = s["out"].double(), s["lse"].double()
    else:
        total = s["mass"].double()
    for b in range(B):
        L, n = int(s["seq_lens"][b]), int(s["tree_lens"][b])
        pages = s["table"][b, :(L + PAGE - 1) // PAGE].long()
        for h in range(Hkv):
            z = _rows64(s, b, h)
            if case["op"] == "tree":
                v = s["v"][pages, h].reshape(-1, D)[:L].double()
                lse[b, :n, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[b, :n, h * G:(h + 1) * G] = torch.einsum("tgl,ld->tgd", torch.softmax(z, -1), v)
            else:
                p = torch.exp(z - s["lse"][b, :n, h * G:(h + 1) * G].double()[..., None])
                p = torch.einsum("tgl,t->l", p, s["weight"][b, :n].double())
                total[b, h, :L] = 0.9 * s["prev"][b, h, :L].double() + p
    return (out, lse) if case["op"] == "tree" else total
